// kvq_pdecode.cuh -- attention of few query rows (a decoded token, drafted
// tokens) over the paged int4 cache.
//
// Mathematics: with the cache rows y = s c (codes c, scales s) in the rotated
// domain, <q, D R^T y> = <R D q, y>, and sum_t p_t D R^T y_t = D R^T sum_t p_t
// y_t: a query is rotated once, the result is rotated back once, and the
// products run on the codes.
//
// Bound: bytes of codes and scales (d/2 + 4 d/g a row, K and V).  What a token
// costs on the SM has to stay below the time its bytes take, so both products
// run on the tensor cores with the cache as the large operand (M = 128 cached
// rows, or 128 coordinates) and exact integers: an int4 code in the high
// nibble of a byte is the signed value 16 c, so eight codes become MMA
// operands by three logic operations.
//   scores   S[t][n] = sum_i 16 c_K[t][i] Q[n][i]     kind::i8, s32
//            Q: each rotated query in 15-bit fixed point, two 7-bit slices
//            (error 1/32512 of its largest coordinate)
//   values   O[i][n] = sum_t 16 c_V[t][i] P[t][n]     kind::i8, s32
//            P: weight times V scale in 32-bit fixed point, four 8-bit
//            slices (error 2^-27 of the largest so far)
// With several scales a row (g < d) the scores of each group accumulate in
// columns of their own and each group of coordinates takes the P that carries
// its scale; O keeps only those blocks.
//
// Online softmax: the reference of a query moves only when a score exceeds it
// by 7 in log2, the fixed point of P when a weight would overflow; either is
// found by the vote in the barrier that P needs anyway.  Weights below half a step
// of P are lost, of a tail of n faint tokens at most n 2^-27 of the largest; hence
// four slices (three, with 7 bits of room: n 2^-17), and what P is made for only 5
// bits below its top.  (With less room more tiles are done twice.  32 sequences of
// 4096 rows, 8 heads, 16 query rows each, d = 128, g = 32: 393 us with 4 bits, 371
// with 5, 357 with 6, 349 with 8; a vote that follows the tail down instead: 209 us
// where the batch of 64 below takes 180.)  O is read back and accumulated in fp32
// after every tile, so it is never rescaled in place.
//
// A tile is 128 smem rows of 128 bytes (two tokens a row at d = 64, half a
// token at d = 256).  A block is a pipeline of roles: four warps expand codes
// (global -> registers a tile ahead -> bytes), four turn scores into weights,
// four accumulate results and prepare the queries of the next item, one issues
// the MMAs, one looks the pages up.  Operands, scores and results are
// double-buffered, so the roles work on neighbouring tiles at once.
//
// Measured: 512 KV heads of 16,384 rows, one query, d = 64, g = 64: 262 us, 2.3
// TB/s, 35% of the copy rate; 64 ragged sequences up to 8192 rows, 8 heads of 4
// queries, d = 128, g = 32: 184 us, 1.9 TB/s, 29%.  No unit is full: the schedulers
// issue in 46% of the clocks (3.9 thousand instructions a tile at d = 64), DRAM and
// the tensor cores are below a third.  Waits are 46% long scoreboard, 17%
// instruction fetch: the roles' latency bounds it.
#pragma once

#include "kvq_sched.cuh"
#include "kvq_tc.cuh"
#include "kvq_wide.cuh"

namespace kvq {

constexpr int kPdThreads = 14 * 32;

constexpr int pow2_at_least(int x) {
  int p = 32;
  while (p < x) p *= 2;
  return p;
}
constexpr int max_of(int a, int b) { return a > b ? a : b; }
constexpr int min_of(int a, int b) { return a < b ? a : b; }

__device__ __forceinline__ float ex2(float x) {  // 2^x
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int D_, int R_, int NG_>
struct Pd {
  static constexpr int D = D_, R = R_, NG = NG_;  // R: query rows of an item
  static constexpr int G = D / NG;
  static constexpr int NCH = D == 256 ? 2 : 1;    // 128-byte columns of a token
  static constexpr int TPR = D == 64 ? 2 : 1;     // tokens of an smem row
  static constexpr int KT = 128 * TPR;            // tokens of a tile
  static constexpr int NQS = max_of(16, 2 * R);   // N of the score MMA
  static constexpr int SBLK = TPR * NG;           // its column blocks
  // bytes of P of a token and group (4 R, to a swizzle width)
  static constexpr int PW = R <= 4 && TPR == 2 ? 16 : (R <= 8 ? 32 : 64);
  static constexpr int NP = TPR * PW;             // N of the value MMA, for a group
  static constexpr int NGM = D == 256 ? max_of(1, NG / 2) : NG;  // P's of a 128-coordinate block
  static constexpr uint32_t PSW = NP == 32 ? kSw32 : (NP == 64 ? kSw64 : kSw128);
  static constexpr int SCOLS = SBLK * NQS, OCOLS = NCH * NGM * NP;
  static constexpr int OBUF = 2 * SCOLS + 2 * OCOLS <= 256 ? 2 : 1;  // two blocks an SM
  static constexpr int TMEM = pow2_at_least(2 * SCOLS + OBUF * OCOLS);
  static_assert(TMEM <= 512, "tensor memory columns");
  static constexpr int PBUF = NG >= 4 ? 1 : 2;    // P's in shared memory
  // shared memory, two of each
  static constexpr int TILE = NCH * 16384;        // expanded K or V
  static constexpr int QB = NCH * NQS * 128;
  static constexpr int PB = NG * 128 * NP;
  static constexpr int OB = TPR * R * D * 4;      // result of an item (one)
  static constexpr int SC = KT * NG * 4;          // scales of K or V
  static constexpr int oK = 0, oV = 2 * TILE, oQ = 4 * TILE, oP = oQ + 2 * QB,
                       oO = oP + PBUF * PB;
  static constexpr int oS = oO + OB;              // scales: K, V of one tile, then the other
  static constexpr int SMEM = oS + 4 * SC + 1024;  // room to align the base
  static constexpr int KP = KT * (D / 32) / 128;  // 16-byte pieces of codes a thread
  static constexpr int SP = (2 * SC / 16 + 127) / 128;  // and of scales
  // Blocks an SM: as many as registers, shared and tensor memory hold (the
  // occupancy calculator answers one for any kernel with tensor memory).
  static constexpr int BLOCKS = R > 8 ? 1 : min_of(2, min_of(512 / TMEM, 233472 / (SMEM + 5120)));
  static_assert(SMEM + 4096 <= 232448, "shared memory");
  static_assert(R % 4 == 0 && R <= 16 && NP >= 32, "rows");
};

// A tile as the page warp writes it down for the others, up to a ring ahead.
struct PdTile {
  int t0, lo, hi;       // first token; the item attends tokens lo .. hi - 1
  int c0, head, row0, rows;
  int starts, ends;     // first, last tile of its item (or of the block's share)
  int whole, last;      // no row's limits lie inside; the item's last tile
  uint32_t have;        // bit i: some of tokens 16 i .. 16 i + 15 are attended, and there
  int64_t row[16];      // cache row of each 16 tokens (0 where they are not)
};
constexpr int kPdRing = 8;

struct PdShared {
  uint64_t dfull[kPdRing], dfree[kPdRing];   // tile described, description read
  uint64_t full[2], pfull[4], qfull[2];      // operands in shared memory: K and V, P, Q
  // (Nobody may fall two phases behind a barrier it waits on.  The accumulation
  // can be two tiles behind the softmax, hence pfull by four.)
  uint64_t sdone[2], odone[2];               // MMAs done: S, or O, ready; operands free
  uint64_t sfree[2], ofree[2];               // S, O read
  PdTile tiles[kPdRing];
  uint32_t tmem;
  int64_t begun;                             // unit at which the first item begins
  float qs[2][16];                           // by item
  int pos[2][16];
  float f[4][16], icw[4][16], m[4][16], l[4][4][16];  // by tile
  float fcur[16], icwcur[16], mcur[16];
  float red[4][16], red2[4][16];
  int64_t scratch[kRunScratch];
};

// smem byte of coordinate i (0..D) of a token, before the 128-byte column is
// taken: eights of coordinates as 0 2 4 6 1 3 5 7 (the order in which a packed
// word comes apart).
__device__ __forceinline__ constexpr int pd_byte(int i) {
  return (i & ~7) | ((i & 1) << 2) | ((i & 7) >> 1);
}
__device__ __forceinline__ constexpr int pd_dim(int b) {
  return (b & ~7) | ((b & 3) << 1) | ((b >> 2) & 1);
}

// Rotates one query row and writes its two slices; returns (in every lane) the
// factor that turns integer sums into log2 scores: NaN for a row that is not finite,
// which integers cannot say.
template <class C, int ROT>
__device__ __forceinline__ float pd_query(const PagedAttnArgs& a, const uint16_t* row, uint8_t* sq,
                                          int r, int lane) {
  using P = Wide<C::D, ROT>;
  WideLane<C::D, ROT> L;
  L.init(a.signs, lane);
  const uint32_t* src = reinterpret_cast<const uint32_t*>(row);
  f2 z[P::C];
#pragma unroll
  for (int j = 0; j < P::C; ++j) {
    const int w = ROT == kRotSRFT ? lane + 32 * j : P::C * lane + j;
    const uint32_t v = __ldg(src + w) ^ L.mask[j];
    const float2 f = a.dtype == kDtF16 ? pair_to_float2<kDtF16>(v) : pair_to_float2<kDtBF16>(v);
    z[j] = mk2(f.x, f.y);
  }
  float Y[P::W];
  wide_rotate_fwd<C::D, ROT>(z, L, Y);
  float top = 0.0f;
  bool finite = true;
#pragma unroll
  for (int w = 0; w < P::W; ++w) {
    top = fmaxf(top, fabsf(Y[w]));
    finite = finite && fabsf(Y[w]) < INFINITY;
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
  finite = __all_sync(kFull, finite);
  const float inv = finite && top > 0.0f ? 16256.0f / top : 0.0f;  // 127 * 128
  const int n0 = r, n1 = C::R + r;                        // columns of the slices
#pragma unroll
  for (int w = 0; w < P::W; ++w) {
    const int v = __float2int_rn(Y[w] * inv);
    const int hi = (v + 64) >> 7, lo = v - hi * 128;
    const int b = pd_byte(L.k2 * P::W + w), col = b >> 7, in = b & 127;
    uint8_t* base = sq + col * C::NQS * 128;
    base[n0 * 128 + (in ^ ((n0 & 7) << 4))] = uint8_t(hi);
    base[n1 * 128 + (in ^ ((n1 & 7) << 4))] = uint8_t(lo);
  }
  if (!finite) return __uint_as_float(0x7FFFFFFFu);
  return top * (1.0f / 16256.0f) * P::KAPPA * a.qscale * (1.0f / 16.0f);
}

// Rotates one result row back and stores it.
template <int D, int ROT>
__device__ __forceinline__ void pd_store(const PagedAttnArgs& a, float (&Y)[D / 32],
                                         const WideLane<D, ROT>& L, uint16_t* row) {
  using P = Wide<D, ROT>;
  f2 z[P::C];
  wide_rotate_inv<D, ROT>(Y, L, z);
  uint32_t* dst = reinterpret_cast<uint32_t*>(row);
#pragma unroll
  for (int j = 0; j < P::C; ++j) {
    const int w = ROT == kRotSRFT ? L.lane + 32 * j : P::C * L.lane + j;
    const uint32_t v = a.dtype == kDtF16 ? float2_to_pair<kDtF16>(lo2(z[j]), hi2(z[j]))
                                         : float2_to_pair<kDtBF16>(lo2(z[j]), hi2(z[j]));
    dst[w] = v ^ L.mask[j];
  }
}

__device__ __forceinline__ uint16_t* out_row(const PagedAttnArgs& a, int c0, int head, int row) {
  const int tok = row / a.n_q;
  return a.out + (int64_t(c0) + tok) * a.out_stride +
         (int64_t(head) * a.n_q + (row - tok * a.n_q)) * a.d;
}

// Partial results in the workspace: per block two slots of R rows (slot 1: of
// an item that began in the block), each m[R], l[R], O[R][D].
template <int D, int R>
constexpr int64_t part_floats() {
  return 2 * R + int64_t(R) * D;
}
template <int D, int R>
__device__ __forceinline__ float* part_slot(const PagedAttnArgs& a, int block, int slot) {
  return a.parts + (int64_t(block) * 2 + slot) * part_floats<D, R>();
}

// Four weights -> slice words (byte k of every weight).
__device__ __forceinline__ void pd_slices(const uint32_t* w, uint32_t& b0, uint32_t& b1,
                                          uint32_t& b2, uint32_t& b3) {
  const uint32_t x = __byte_perm(w[0], w[1], 0x5140), y = __byte_perm(w[2], w[3], 0x5140);
  const uint32_t z = __byte_perm(w[0], w[1], 0x7362), t = __byte_perm(w[2], w[3], 0x7362);
  b0 = __byte_perm(x, y, 0x5410);
  b1 = __byte_perm(x, y, 0x7632);
  b2 = __byte_perm(z, t, 0x5410);
  b3 = __byte_perm(z, t, 0x7632);
}

// As mbar_wait_bounded, for waits that are often long: the hardware may suspend
// the warp for up to 2 us a poll (a role that waits costs few issue slots), and
// the timer is read only after 64 of them.
__device__ __forceinline__ bool mbar_wait_suspended(uint32_t bar, uint32_t parity) {
  uint64_t t0 = 0;
  for (uint32_t it = 0; it < KVQ_WAIT_MAX_POLLS; ++it) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(2000u)
        : "memory");
    if (done) return true;
    if ((it & 63u) == 63u) {
      const uint64_t t = global_timer_ns();
      if (t0 == 0) t0 = t;
      else if (t - t0 > KVQ_WAIT_LIMIT_NS) return false;
    }
  }
  return false;
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool named_or(int id, int threads, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(uint32_t(p)), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

template <int D, int R, int NG>
__global__ void __launch_bounds__(kPdThreads, Pd<D, R, NG>::BLOCKS)
    kvq_paged_decode_kernel(const PagedAttnArgs a, unsigned* status) {
  using C = Pd<D, R, NG>;
  constexpr int KT = C::KT, KP = C::KP;
  extern __shared__ uint8_t smem_raw[];
  __shared__ PdShared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto bar = [](uint64_t& b) { return smem_u32(&b); };
  if (tid == 0) {
    for (int i = 0; i < kPdRing; ++i) {
      mbar_init(bar(sh.dfull[i]), 1);
      mbar_init(bar(sh.dfree[i]), 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(sh.full[i]), 4);
      mbar_init(bar(sh.pfull[2 * i]), 4);
      mbar_init(bar(sh.pfull[2 * i + 1]), 4);
      mbar_init(bar(sh.qfull[i]), 4);
      mbar_init(bar(sh.sdone[i]), 1);
      mbar_init(bar(sh.odone[i]), 1);
      mbar_init(bar(sh.sfree[i]), 4);
      mbar_init(bar(sh.ofree[i]), 4);
    }
    fence_mbar_init();
  }
  pdl_wait();  // no global access before the previous kernel completes
  const Run run = find_run<R, KT, kPdThreads>(a, blockIdx.x, gridDim.x, sh.scratch, status);
  JoinInfo* join = a.join + blockIdx.x;
  if (tid == 0) join->first_block = -1;
  pdl_release();  // the join's blocks wait for this grid's end: let them be placed
  if (run.begin == run.end) return;
  const int n = int(run.end - run.begin);  // tiles
  if (warp == 12) tmem_alloc(smem_u32(&sh.tmem), C::TMEM);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const uint32_t tlane = tmem + (uint32_t(warp & 3) << 21);
  bool ok = true;
  // A wait that runs out is recorded and skipped from then on: every role still
  // takes all its steps, so nobody is left at a barrier.
  auto wait = [&](uint64_t& b, int phase) {
    if (ok) ok = mbar_wait_suspended(smem_u32(&b), uint32_t(phase) & 1u);
  };
  auto arrive = [&](uint64_t& b) {  // one arrival for the warp
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&b));
  };

  if (warp == 13) {
    // ---------------- pages: what each tile is, and where ----------------
    Cursor<R, KT> c;
    c.seek(a, run.seq, run.off);
    if (lane == 0) sh.begun = run.begin - c.tile;
    for (int i = 0; i < n; ++i) {
      PdTile& e = sh.tiles[i % kPdRing];
      if (i >= kPdRing) wait(sh.dfree[i % kPdRing], i / kPdRing - 1);
      const int t0 = (c.first + c.tile) * KT;
      int64_t r = 0;
      bool there = false;
      if (lane < KT / 16) {
        const int64_t t = int64_t(t0) + lane * 16;
        if (t < c.hi && t + 15 >= c.lo) {
          const int64_t page = __ldg(a.page_table + c.seq * a.max_pages + (t >> a.page_shift));
          there = page >= 0 && page < a.n_pages;
          if (there)
            r = ((page * a.n_kv + c.head) << a.page_shift) + (t & ((1 << a.page_shift) - 1));
          else
            flag_bad_index(status);
        }
        e.row[lane] = r;
      }
      const uint32_t have = __ballot_sync(kFull, there);
      if (lane == 0) {
        const int row0 = c.qt * R;
        const int rows = int(min(int64_t(R), int64_t(c.q.n) * a.n_q - row0));
        const int pf = c.q.len - c.q.n + row0 / a.n_q;  // positions of the first and last row
        const int pl = c.q.len - c.q.n + (row0 + rows - 1) / a.n_q;
        e.have = have;
        e.t0 = t0;
        e.lo = c.lo;
        e.hi = c.hi;
        e.c0 = c.q.c0;
        e.head = c.head;
        e.row0 = row0;
        e.rows = rows;
        e.starts = i == 0 || c.tile == 0;
        e.last = c.tile + 1 == c.count;
        e.ends = e.last || i + 1 == n;
        e.whole = t0 + KT - 1 <= pf && (a.window == 0 || t0 > pl - a.window) &&
                  have == (KT == 256 ? 0xFFFFu : 0xFFu);
      }
      arrive(sh.dfull[i % kPdRing]);
      if (i + 1 < n && ++c.tile == c.count) c.next_item(a);
    }
  } else if (warp == 12) {
    // ---------------- MMA issue ----------------
    auto scores = [&](int i, int item) {
      const uint32_t k = sbase + C::oK + (i & 1) * C::TILE;
      const uint32_t q = sbase + C::oQ + (item & 1) * C::QB;
      constexpr uint32_t id = instr_desc(kAccS32, kFmtS8, kFmtS8, false, false, 128, C::NQS);
      tc_fence_after();
#pragma unroll 1
      for (int b = 0; b < C::SBLK; ++b) {
        const int half = b / NG, j = b % NG;
#pragma unroll 1
        for (int x = 0; x < C::G; x += 32) {
          const int byte = j * C::G + x;  // in the token's bytes
          const int abyte = C::TPR == 2 ? half * 64 + byte : byte;
          mma_i8(tmem + (i & 1) * C::SCOLS + b * C::NQS,
                 smem_desc(k + (abyte >> 7) * 16384 + (abyte & 127), 16, 1024, kSw128),
                 smem_desc(q + (byte >> 7) * (C::NQS * 128) + (byte & 127), 16, 1024, kSw128), id,
                 x > 0);
        }
      }
      mma_commit(bar(sh.sdone[i & 1]));
    };
    auto values = [&](int i) {
      const uint32_t v = sbase + C::oV + (i & 1) * C::TILE, p = sbase + C::oP + (i % C::PBUF) * C::PB;
      // one MMA for all groups of a 128-coordinate block
      constexpr uint32_t id = instr_desc(kAccS32, kFmtS8, kFmtU8, true, true, 128, C::NGM * C::NP);
      tc_fence_after();
#pragma unroll 1
      for (int mt = 0; mt < C::NCH; ++mt)
#pragma unroll 1
        for (int x = 0; x < 4; ++x)
          mma_i8(tmem + 2 * C::SCOLS + (i % C::OBUF) * C::OCOLS + mt * C::NGM * C::NP,
                 smem_desc(v + mt * 16384 + x * 4096, 16, 1024, kSw128),
                 smem_desc(p + (NG == 1 ? 0 : mt * C::NGM * 128 * C::NP) + x * 32 * C::NP,
                           128 * C::NP, 8 * C::NP, C::PSW),
                 id, x > 0);
      mma_commit(bar(sh.odone[i & 1]));
    };
    int item = 0;  // of the next tile whose scores are issued
    auto issue_scores = [&](int i) {
      wait(sh.dfull[i % kPdRing], i / kPdRing);
      const bool starts = sh.tiles[i % kPdRing].starts;
      if (i > 0 && starts) ++item;
      if (starts) wait(sh.qfull[item & 1], item >> 1);
      wait(sh.full[i & 1], i >> 1);
      if (i >= 2) wait(sh.sfree[i & 1], (i >> 1) - 1);
      if (lane == 0) scores(i, item);
      __syncwarp();
    };
    issue_scores(0);
    for (int i = 0; i < n; ++i) {
      if (i + 1 < n) issue_scores(i + 1);
      wait(sh.pfull[i & 3], i >> 2);
      if (i >= C::OBUF) wait(sh.ofree[i % C::OBUF], (i / C::OBUF) - 1);
      if (lane == 0) values(i);
      __syncwarp();
    }
  } else if (warp >= 8) {
    // ---------------- expansion: packed codes -> 16 c bytes ----------------
    // Codes and scales are loaded right after the tile before is expanded: the
    // proxy fence at the end of an expansion would wait for loads in flight.
    // What hides their latency is the prefetch into L2 two tiles earlier.
    const int et = tid - 256;
    uint4 kreg[KP], vreg[KP], sreg[C::SP];
    const int piece = (et / (D / 32) & 15) * (D / 2) + et % (D / 32) * 16;  // in 16 tokens' codes
    auto load = [&](int i) {
      const PdTile& e = sh.tiles[i % kPdRing];
#pragma unroll
      for (int k = 0; k < KP; ++k) {
        const int64_t off = e.row[(et + 128 * k) / (D / 2)] * (D / 2) + piece;
        kreg[k] = __ldg(reinterpret_cast<const uint4*>(a.k_packed + off));
        vreg[k] = __ldg(reinterpret_cast<const uint4*>(a.v_packed + off));
      }
#pragma unroll
      for (int k = 0; k < C::SP; ++k) {
        const int p = et + 128 * k, q = p % (C::SC / 16);  // piece of K's, then of V's
        if (2 * C::SC / 16 >= 128 || p < 2 * C::SC / 16)
          sreg[k] = __ldg(reinterpret_cast<const uint4*>(
                              (p < C::SC / 16 ? a.k_scales : a.v_scales) +
                              e.row[q / (4 * NG)] * NG) +
                          q % (4 * NG));
      }
    };
    auto prefetch = [&](int i) {  // a line a thread and step
      const PdTile& e = sh.tiles[i % kPdRing];
      constexpr int LINES = KT * (D / 2) / 128;  // of K, and of V
#pragma unroll
      for (int k = 0; k < 2 * LINES / 128; ++k) {
        const int p = (et + 128 * k) % LINES;
        const uint8_t* base = et + 128 * k < LINES ? a.k_packed : a.v_packed;
        // 256 / D rows a line
        asm volatile("prefetch.global.L2 [%0];" ::"l"(
            base + e.row[p * 256 / D >> 4] * (D / 2) + (p * 128) % (16 * (D / 2))));
      }
    };
    // Where this thread's pieces go: rows 128 / (D / 32) apart for each k, the
    // same column (at d = 64 the other half from the middle on).
    const int r0 = et / (D / 32), col = et % (D / 32) * 32;
    const uint32_t dst0 = uint32_t(col >> 7) * 16384 + uint32_t(r0) * 128 +
                          (((uint32_t(col & 127) >> 4) ^ uint32_t(r0 & 7)) * 16);
    auto expand = [&](const uint4 (&w)[KP], uint32_t tile) {
#pragma unroll
      for (int k = 0; k < KP; ++k) {
        constexpr uint32_t H = 0xF0F0F0F0u;
        const int down = k * (4096 / D) % 128;  // rows
        const bool other = C::TPR == 2 && k * (4096 / D) >= 128;
        const uint32_t at = tile + (other ? dst0 ^ 64u : dst0) + down * 128;
        sts128(at, (w[k].x << 4) & H, w[k].x & H, (w[k].y << 4) & H, w[k].y & H);
        sts128(at ^ 16u, (w[k].z << 4) & H, w[k].z & H, (w[k].w << 4) & H, w[k].w & H);
      }
    };
    wait(sh.dfull[0], 0);
    load(0);
    for (int i = 1; i < min(3, n); ++i) {
      wait(sh.dfull[i], 0);
      prefetch(i);
    }
    for (int i = 0; i < n; ++i) {
      const int buf = i & 1;
      if (i >= 2) wait(sh.odone[buf], (i >> 1) - 1);  // K, V, P and scales are free
      expand(kreg, sbase + C::oK + buf * C::TILE);
      expand(vreg, sbase + C::oV + buf * C::TILE);
#pragma unroll
      for (int k = 0; k < C::SP; ++k)
        if (2 * C::SC / 16 >= 128 || et + 128 * k < 2 * C::SC / 16)
          sts128(sbase + C::oS + buf * 2 * C::SC + uint32_t(et + 128 * k) * 16, sreg[k].x,
                 sreg[k].y, sreg[k].z, sreg[k].w);
      fence_proxy_async_smem();
      arrive(sh.full[buf]);
      if (i + 1 < n) load(i + 1);
      if (i + 3 < n) {
        wait(sh.dfull[(i + 3) % kPdRing], (i + 3) / kPdRing);
        prefetch(i + 3);
      }
    }
  } else if (warp < 4) {
    // ---------------- softmax: a token's scores -> weights ----------------
    const int row = tid;  // smem row; tokens row (and row + 128 at d = 64) of the tile
    constexpr int TPR = C::TPR;
    // The fixed point of P counts in 2^-24 / cw; what it is made for lies in [4, 8) / cw.
    constexpr float kMost = 255.0f;
    float m[R], l[R], cw[R];
    float ks[TPR][NG], vs[TPR][NG];
    bool fresh = true;
    int item = -1;
    for (int i = 0; i < n; ++i) {
      const PdTile& e = sh.tiles[i % kPdRing];
      wait(sh.full[i & 1], i >> 1);  // scales, and the description
      const int rows = e.rows;
      if (e.starts) {
        ++item;
        wait(sh.qfull[item & 1], item >> 1);
#pragma unroll
        for (int r = 0; r < R; ++r) m[r] = -3e38f, l[r] = 0.0f, cw[r] = 1.0f;
        fresh = true;
      }
      const float* qs = sh.qs[item & 1];
      float vmax[TPR];
      bool seen[TPR];
#pragma unroll
      for (int h = 0; h < TPR; ++h) {
        const int tl = row + 128 * h;
        const float* sc = reinterpret_cast<const float*>(smem + C::oS + (i & 1) * 2 * C::SC) + tl * NG;
        seen[h] = e.whole || (e.t0 + tl >= e.lo && e.t0 + tl < e.hi && (e.have >> (tl >> 4) & 1u));
#pragma unroll
        for (int j = 0; j < NG; ++j) {  // rows that no query attends may hold anything
          ks[h][j] = seen[h] ? sc[j] : 0.0f;
          vs[h][j] = seen[h] ? sc[C::SC / 4 + j] : 0.0f;
        }
        vmax[h] = vs[h][0];
        float sum = ks[h][0] + vs[h][0];
#pragma unroll
        for (int j = 1; j < NG; ++j) {
          vmax[h] = fmaxf(vmax[h], vs[h][j]);
          sum += ks[h][j] + vs[h][j];
        }
        // A scale that is not finite makes the token's scores NaN, and with them the
        // sums of those who attend it: integers could not say so.
        ks[h][0] = fmaf(sum, 0.0f, ks[h][0]);
      }
      wait(sh.sdone[i & 1], i >> 1);
      tc_fence_after();
      float s[TPR][R];
#pragma unroll
      for (int h = 0; h < TPR; ++h)
#pragma unroll
        for (int r = 0; r < R; ++r) s[h][r] = 0.0f;
#pragma unroll
      for (int b = 0; b < C::SBLK; ++b) {
        const int h = b / NG, j = b % NG;
        uint32_t x[2 * R];
        tmem_ld<2 * R>(tlane + (i & 1) * C::SCOLS + b * C::NQS, x);
        tmem_wait_ld();
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (r < rows)
            s[h][r] = fmaf(ks[h][j], float(int(x[r]) * 128 + int(x[R + r])), s[h][r]);
      }
      tc_fence_before();
      arrive(sh.sfree[i & 1]);
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r < rows) {
          const float q = qs[r];
#pragma unroll
          for (int h = 0; h < TPR; ++h) s[h][r] *= q;
        }
      if (!e.whole) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int p = sh.pos[item & 1][r];
#pragma unroll
          for (int h = 0; h < TPR; ++h) {
            const int t = e.t0 + row + 128 * h;
            if (!seen[h] || t > p || (a.window > 0 && t <= p - a.window)) s[h][r] = -INFINITY;
          }
        }
      }

      const uint32_t pt = sbase + C::oP + (i % C::PBUF) * C::PB;
      if (i >= C::PBUF)  // P is free
        wait(sh.odone[(i - C::PBUF) & 1], (i - C::PBUF) >> 1);
      auto weights = [&]() {
        bool over = false;
#pragma unroll
        for (int h = 0; h < TPR; ++h) {
          float p[R];
#pragma unroll
          for (int r = 0; r < R; ++r) {
            p[r] = 0.0f;
            if (r < rows) {
              const float x = s[h][r] - m[r];
              p[r] = ex2(x);
              l[r] += p[r];
              over = over || x > 7.0f || p[r] * vmax[h] * cw[r] > kMost;
            }
          }
#pragma unroll
          for (int j = 0; j < NG; ++j) {
            uint32_t w[R], b[R];
#pragma unroll
            for (int r = 0; r < R; ++r)
              w[r] = __float2uint_rn(p[r] * vs[h][j] * (cw[r] * 16777216.0f));
#pragma unroll
            for (int r = 0; r < R / 4; ++r)
              pd_slices(w + 4 * r, b[r], b[R / 4 + r], b[R / 2 + r], b[3 * R / 4 + r]);
            // row of NP bytes, a run of PW for each of its tokens; 16-byte pieces swizzled
            const uint32_t base = pt + uint32_t(j * 128 + row) * C::NP;
            const uint32_t x =
                C::NP == 32 ? (row >> 2) & 1 : (C::NP == 64 ? (row >> 1) & 3 : row & 7);
#pragma unroll
            for (int k = 0; k < R; k += 4)
              sts128(base + ((uint32_t(h * (C::PW / 16) + k / 4) ^ x) * 16), b[k], b[k + 1],
                     b[k + 2], b[k + 3]);
          }
        }
        fence_proxy_async_smem();
        return over;
      };
      float lold[R];
#pragma unroll
      for (int r = 0; r < R; ++r) lold[r] = l[r];
      bool slow = fresh;
      for (;;) {
        if (slow) {  // the tile's maxima -> new references
#pragma unroll
          for (int r = 0; r < R; ++r) {
            l[r] = lold[r];
            float x = -INFINITY;
#pragma unroll
            for (int h = 0; h < TPR; ++h) x = fmaxf(x, s[h][r]);
            if (r >= rows) x = -INFINITY;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
            if (lane == 0) sh.red[warp][r] = x;
          }
          named_sync(1, 128);
          uint32_t moved = 0;
#pragma unroll
          for (int r = 0; r < R; ++r) {
            float mn = m[r];
#pragma unroll
            for (int w = 0; w < 4; ++w) mn = fmaxf(mn, sh.red[w][r]);
            const float f = ex2(m[r] - mn);
            l[r] *= f;
            if (fresh || mn > m[r]) moved |= 1u << r;
            m[r] = mn;
            float x = 0.0f;
#pragma unroll
            for (int h = 0; h < TPR; ++h)
              if (r < rows) x = fmaxf(x, ex2(s[h][r] - mn) * vmax[h]);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
            if (lane == 0) sh.red2[warp][r] = x;
            if (row == 0) sh.fcur[r] = f, sh.mcur[r] = mn;
          }
          named_sync(1, 128);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            float x = 0.0f;
#pragma unroll
            for (int w = 0; w < 4; ++w) x = fmaxf(x, sh.red2[w][r]);
            // the power of two that brings the largest into [4, 8); rows that need no
            // other keep theirs
            if ((moved >> r & 1u) || x * cw[r] > kMost) {
              const int ex = min(max(256 - int(__float_as_uint(x) >> 23), 1), 225);
              cw[r] = __uint_as_float(uint32_t(ex) << 23);
              if (row == 0) sh.icwcur[r] = __uint_as_float(uint32_t(254 - ex) << 23);
            }
          }
        }
        const bool over = weights();
        if (slow || !named_or(1, 128, over)) break;
        slow = true;
      }
      fresh = false;
      __syncwarp();
      if (warp == 0 && lane < R) {  // what the accumulation needs to know of this tile
        sh.f[i & 3][lane] = slow ? sh.fcur[lane] : 1.0f;
        sh.icw[i & 3][lane] = sh.icwcur[lane] * (1.0f / 268435456.0f);
        sh.m[i & 3][lane] = sh.mcur[lane];
      }
      if (e.ends) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float x = l[r];
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) x += __shfl_xor_sync(kFull, x, o);
          if (lane == 0) sh.l[i & 3][warp][r] = x;
        }
      }
      arrive(sh.pfull[i & 3]);
    }
  } else {
    // ---------- accumulation, results, and the queries of the next items ----------
    const int aw = warp - 4, row = tid - 128;  // row: coordinate byte
    const int half = C::TPR == 2 ? row >> 6 : 0, crd = C::TPR == 2 ? row & 63 : row;
    Cursor<R, KT> qc;
    qc.seek(a, run.seq, run.off);
    int64_t next = run.begin - qc.tile + qc.count;  // unit of the item after qc's
    auto prepare = [&](int item) {                  // qc's queries
      const int row0 = qc.qt * R, b = item & 1;
      const int rows = int(min(int64_t(R), int64_t(qc.q.n) * a.n_q - row0));
      for (int r = aw; r < rows; r += 4) {
        const int tok = (row0 + r) / a.n_q;
        const uint16_t* src = a.q + (int64_t(qc.q.c0) + tok) * a.q_stride +
                              (int64_t(qc.head) * a.n_q + (row0 + r - tok * a.n_q)) * D;
        uint8_t* sq = smem + C::oQ + b * C::QB;
        const float qs = a.rot == kRotSRFT ? pd_query<C, kRotSRFT>(a, src, sq, r, lane)
                                           : pd_query<C, kRotSRHT>(a, src, sq, r, lane);
        if (lane == 0) {
          sh.qs[b][r] = qs;
          sh.pos[b][r] = qc.q.len - qc.q.n + tok;
        }
      }
      fence_proxy_async_smem();
      arrive(sh.qfull[b]);
    };
    auto prepare_next = [&](int item) {
      if (next >= run.end) return;
      qc.next_item(a);
      next += qc.count;
      prepare(item);
    };
    prepare(0);
    prepare_next(1);
    int item = 0;
    float acc[C::NCH][R];
    for (int i = 0; i < n; ++i) {
      wait(sh.pfull[i & 3], i >> 2);  // the softmax's words on this tile
      const PdTile& e = sh.tiles[i % kPdRing];
      if (e.starts) {
#pragma unroll
        for (int c = 0; c < C::NCH; ++c)
#pragma unroll
          for (int r = 0; r < R; ++r) acc[c][r] = 0.0f;
      }
      const int rows = e.rows;
      wait(sh.odone[i & 1], i >> 1);
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < C::NCH; ++c) {
        const int blk = D == 256 ? c * C::NGM + crd / (C::G > 128 ? 128 : C::G) : crd / C::G;
        const uint32_t at = tlane + 2 * C::SCOLS + (i % C::OBUF) * C::OCOLS +
                            uint32_t(blk * C::NP + half * C::PW);
        // two slices of every row after the other two (16 rows: to save registers)
        constexpr int RL = R > 8 ? 1 : 2;
        float v[R];
#pragma unroll
        for (int k = 0; k < 4; k += 2 * RL) {
          uint32_t x[2 * RL * R];
          tmem_ld<2 * RL * R>(at + k * R, x);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 2 * RL; j += 2)
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const float two = float(int(x[(j + 1) * R + r]) * 256 + int(x[j * R + r]));
              v[r] = j + k == 0 ? two : fmaf(two, 65536.0f, v[r]);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (r < rows) acc[c][r] = fmaf(v[r], sh.icw[i & 3][r], acc[c][r] * sh.f[i & 3][r]);
      }
      float lsum = 0.0f, mref = 0.0f;
      if (e.ends && lane < R) {  // of query row `lane`
        lsum = sh.l[i & 3][0][lane] + sh.l[i & 3][1][lane] + sh.l[i & 3][2][lane] +
               sh.l[i & 3][3][lane];
        mref = sh.m[i & 3][lane];
      }
      tc_fence_before();
      arrive(sh.ofree[i % C::OBUF]);
      if (!e.ends) {
        arrive(sh.dfree[i % kPdRing]);
        continue;
      }

      // ---- end of the item, or of the block's share of it ----
      const bool began_here = item > 0 || sh.begun == run.begin;
      const bool complete = e.last && began_here;
      float* ob = reinterpret_cast<float*>(smem + C::oO);
      named_sync(2, 128);  // the result before is read
#pragma unroll
      for (int c = 0; c < C::NCH; ++c)
#pragma unroll
        for (int r = 0; r < R; ++r)
          ob[(half * R + r) * D + c * 128 + pd_dim(crd)] = acc[c][r];
      named_sync(2, 128);
      for (int r = aw; r < rows; r += 4) {
        const float ls = __shfl_sync(kFull, lsum, r);
        auto value = [&](int d) {
          float v = ob[r * D + d];
          if constexpr (C::TPR == 2) v += ob[(R + r) * D + d];
          return v;
        };
        if (complete) {
          const float inv = ls != 0.0f ? 1.0f / ls : 0.0f;
          uint16_t* dst = out_row(a, e.c0, e.head, e.row0 + r);
          float Y[D / 32];
          if (a.rot == kRotSRFT) {
            WideLane<D, kRotSRFT> L;
            L.init(a.signs, lane);
#pragma unroll
            for (int w = 0; w < D / 32; ++w)
              Y[w] = value(L.k2 * (D / 32) + w) * inv * Wide<D, kRotSRFT>::KAPPA;
            pd_store<D, kRotSRFT>(a, Y, L, dst);
          } else {
            WideLane<D, kRotSRHT> L;
            L.init(a.signs, lane);
#pragma unroll
            for (int w = 0; w < D / 32; ++w)
              Y[w] = value(L.k2 * (D / 32) + w) * inv * Wide<D, kRotSRHT>::KAPPA;
            pd_store<D, kRotSRHT>(a, Y, L, dst);
          }
        } else {
          float* slot = part_slot<D, R>(a, blockIdx.x, began_here ? 1 : 0);
          const float mr = __shfl_sync(kFull, mref, r);
          if (lane == 0) slot[r] = mr, slot[R + r] = ls;
          for (int d = lane; d < D; d += 32) slot[2 * R + r * D + d] = value(d);
        }
      }
      if (e.last && !began_here && tid == 128) {
        join->c0 = e.c0;
        join->head = e.head;
        join->row0 = e.row0;
        join->rows = rows;
        join->first_block = block_of(sh.begun, run.total, run.blocks);
      }
      arrive(sh.dfree[i % kPdRing]);
      prepare_next(item + 2);
      ++item;
    }
  }
  if (!ok && lane == 0) atomicOr(status, kPagedTimeout);
  tc_fence_before();
  __syncthreads();  // every read of tensor memory is done
  if (warp == 12) tmem_free(tmem, C::TMEM);
}

// Joins the partial results of items that several blocks shared: blockIdx.x the
// one that ended in that block, blockIdx.y a run of RPB rows of it, WPR warps a
// row (each takes every WPR-th part, eight in flight; an item of few rows over a
// long sequence has as many parts as there are blocks).
template <int D, int R, int ROT, int RPB, int WPR>
__global__ void __launch_bounds__(32 * RPB * WPR) kvq_paged_join_kernel(const PagedAttnArgs a) {
  constexpr int W = D / 32;
  __shared__ float s_part[WPR > 1 ? RPB * WPR : 1][D + 2];
  const int b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = blockIdx.y * RPB + warp / WPR, share = warp % WPR;
  WideLane<D, ROT> L;
  L.init(a.signs, lane);  // (signs are no kernel's output)
  pdl_wait();             // the partial results of the kernel before
  const JoinInfo j = a.join[b];
  if (j.first_block < 0 || int(blockIdx.y) * RPB >= j.rows) return;
  const bool there = r < j.rows;
  float Y[W], l = 0.0f, top = -3e38f;
#pragma unroll
  for (int w = 0; w < W; ++w) Y[w] = 0.0f;
  if (there) {
    for (int p = j.first_block + lane; p <= b; p += 32)
      top = fmaxf(top, part_slot<D, R>(a, p, p == j.first_block ? 1 : 0)[r]);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
#pragma unroll 8
    for (int p = j.first_block + share; p <= b; p += WPR) {
      const float* slot = part_slot<D, R>(a, p, p == j.first_block ? 1 : 0);
      const float f = ex2(slot[r] - top);
      l = fmaf(f, slot[R + r], l);
#pragma unroll
      for (int w = 0; w < W; ++w) Y[w] = fmaf(f, slot[2 * R + r * D + L.k2 * W + w], Y[w]);
    }
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int w = 0; w < W; ++w) s_part[warp][L.k2 * W + w] = Y[w];
    if (lane == 0) s_part[warp][D] = l;
    __syncthreads();
    if (share != 0) return;
#pragma unroll
    for (int x = 1; x < WPR; ++x) {
#pragma unroll
      for (int w = 0; w < W; ++w) Y[w] += s_part[warp + x][L.k2 * W + w];
      l += s_part[warp + x][D];
    }
  }
  if (!there) return;
  const float inv = l != 0.0f ? Wide<D, ROT>::KAPPA / l : 0.0f;  // (a NaN stays one)
#pragma unroll
  for (int w = 0; w < W; ++w) Y[w] *= inv;
  pd_store<D, ROT>(a, Y, L, out_row(a, j.c0, j.head, j.row0 + r));
}

}  // namespace kvq
