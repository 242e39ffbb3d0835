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
//            (error 2^-15 of its largest coordinate)
//   values   O[i][n] = sum_t 16 c_V[t][i] P[t][n]     kind::i8, s32
//            P: weight times V scale in 23-bit fixed point, three 8-bit
//            slices (error 2^-17 of the largest so far)
// With several scales a row (g < d) the scores of each group accumulate in
// columns of their own and each group of coordinates takes the P that carries
// its scale; O keeps only those blocks.
//
// Online softmax: the reference of a query moves only when a score exceeds it
// by 7 in log2, the fixed point of P when a weight would overflow; either is
// found by the vote in the barrier that P needs anyway.  O is read back and
// accumulated in fp32 after every tile, so it is never rescaled in place.
//
// A tile is 128 smem rows of 128 bytes (two tokens a row at d = 64, half a
// token at d = 256).  Codes travel global -> registers (a tile's time ahead)
// -> expanded bytes.  Eight warps do, per tile: expand V under the MMA of the
// scores; softmax; expand the next K under the MMA of the values; accumulate.
// A ninth warp issues the MMAs and looks the pages up.  The blocks of an SM
// cover each other's waits.
#pragma once

#include "kvq_sched.cuh"
#include "kvq_tc.cuh"
#include "kvq_wide.cuh"

namespace kvq {

constexpr int kPdThreads = 256;

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
  static constexpr int RQ = D == 64 ? R : R / 2;  // query rows of a thread's scores
  static constexpr int AQ = D == 256 ? R : R / 2;  // query rows of a thread's accumulators
  static constexpr int NQS = 2 * R;               // N of the score MMA
  static constexpr int SBLK = TPR * NG;           // its column blocks
  // bytes of P a thread writes for its token (3 RQ, to a swizzle width)
  static constexpr int PW = RQ == 4 ? 16 : (RQ == 8 ? 32 : 64);
  static constexpr int NP = 2 * PW;               // N of the value MMA
  static constexpr int NGM = D == 256 ? max_of(1, NG / 2) : NG;  // P's of a 128-coordinate block
  static constexpr uint32_t PSW = NP == 32 ? kSw32 : (NP == 64 ? kSw64 : kSw128);
  static constexpr int TMEM = pow2_at_least(max_of(SBLK * NQS, NCH * NGM * NP));
  static_assert(TMEM <= 512, "tensor memory columns");
  // shared memory
  static constexpr int TILE = NCH * 16384;        // expanded K or V
  static constexpr int KP = KT * (D / 32) / kPdThreads;  // 16-byte pieces of codes a thread
  static constexpr int QB = NCH * NQS * 128;
  static constexpr int PB = NG * 128 * NP;
  static constexpr int OB = TPR * R * D * 4;      // result of an item, over P
  static constexpr int oK = 0, oV = oK + TILE, oQ = oV + TILE, oP = oQ + QB;
  static constexpr int SMEM = oP + max_of(PB, OB) + 1024;  // room to align the base
  // Blocks an SM: as many as registers, shared and tensor memory hold (the
  // occupancy calculator answers one for any kernel with tensor memory).
  static constexpr int BLOCKS = min_of(2, min_of(512 / TMEM, 230000 / (SMEM + 4096)));
};

// A tile as the control warp writes it down for the others, up to three tiles
// ahead.
struct PdTile {
  int t0, len;          // first token, cached rows of the sequence
  int c0, head, row0, rows;
  int p0;               // position of the sequence's first new token
  int starts, ends;     // first, last tile of its item
  int pad;
  int64_t row[16];      // cache row of each 16 tokens, -1: not to be read
};

struct PdShared {
  uint64_t sdone, odone;
  PdTile tiles[4];
  uint32_t tmem;
  int fail, began_here;
  int64_t begun;
  float qs[16], m[16], f[16], icw[16];
  int pos[16];
  float red[8][16], red2[8][16];
  int64_t scratch[kPdThreads / 32 + 1 + 4];
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
// factor that turns integer sums into log2 scores.
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
#pragma unroll
  for (int w = 0; w < P::W; ++w) top = fmaxf(top, fabsf(Y[w]));
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
  const float inv = top > 0.0f ? 16256.0f / top : 0.0f;  // 127 * 128
  const int n0 = (r / C::RQ) * 2 * C::RQ + r % C::RQ;     // column of slice 0
#pragma unroll
  for (int w = 0; w < P::W; ++w) {
    const int v = __float2int_rn(Y[w] * inv);
    const int hi = (v + 64) >> 7, lo = v - hi * 128;
    const int b = pd_byte(L.k2 * P::W + w), col = b >> 7, in = b & 127;
    uint8_t* base = sq + col * C::NQS * 128;
    const int n1 = n0 + C::RQ;
    base[n0 * 128 + (in ^ ((n0 & 7) << 4))] = uint8_t(hi);
    base[n1 * 128 + (in ^ ((n1 & 7) << 4))] = uint8_t(lo);
  }
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

// Four 23-bit weights -> slice words (byte k of every weight).
__device__ __forceinline__ void pd_slices(const uint32_t* w, uint32_t& b0, uint32_t& b1,
                                          uint32_t& b2) {
  const uint32_t x = __byte_perm(w[0], w[1], 0x5140), y = __byte_perm(w[2], w[3], 0x5140);
  b0 = __byte_perm(x, y, 0x5410);
  b1 = __byte_perm(x, y, 0x7632);
  b2 = __byte_perm(__byte_perm(w[0], w[1], 0x0062), __byte_perm(w[2], w[3], 0x0062), 0x5410);
}

template <int D, int R, int NG>
__global__ void __launch_bounds__(kPdThreads + 32, Pd<D, R, NG>::BLOCKS)
    kvq_paged_decode_kernel(const PagedAttnArgs a, unsigned* status) {
  using C = Pd<D, R, NG>;
  constexpr int RQ = C::RQ, AQ = C::AQ, KT = C::KT, KP = C::KP;
  extern __shared__ uint8_t smem_raw[];
  __shared__ PdShared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wg = (warp >> 2) & 1;
  const int row = tid & 127;  // smem row, or coordinate byte, of this thread
  const uint32_t sdone = smem_u32(&sh.sdone), odone = smem_u32(&sh.odone);
  if (tid == 0) {
    mbar_init(sdone, 1);
    mbar_init(odone, 1);
    sh.fail = 0;
    fence_mbar_init();
  }
  pdl_wait();  // no global access before the previous kernel completes
  const Run run = find_run<R, KT, kPdThreads + 32>(a, blockIdx.x, gridDim.x, sh.scratch, status);
  JoinInfo* join = a.join + blockIdx.x;
  if (run.begin == run.end) {
    if (tid == 0) join->first_block = -1;
    return;
  }
  const int n_tiles = int(run.end - run.begin);

  if (warp == kPdThreads / 32) {
    // ================= control: tile descriptions and MMA issue =================
    tmem_alloc(smem_u32(&sh.tmem), C::TMEM);
    Cursor<R, KT> c;
    c.seek(a, run.seq, run.off);
    if (lane == 0) {
      join->first_block = -1;
      sh.begun = run.begin - c.tile;  // unit at which the first item begins
      sh.began_here = c.tile == 0;
    }
    auto describe = [&](int i) {  // the cursor's tile as number i
      PdTile& e = sh.tiles[i & 3];
      const int t0 = (c.first + c.tile) * KT;
      if (lane == 0) {
        e.t0 = t0;
        e.len = c.q.len;
        e.c0 = c.q.c0;
        e.head = c.head;
        e.row0 = c.qt * R;
        e.rows = int(min(int64_t(R), int64_t(c.q.n) * a.n_q - int64_t(c.qt) * R));
        e.p0 = c.q.len - c.q.n;
        e.starts = c.tile == 0;
        e.ends = c.tile + 1 == c.count;
      }
      if (lane < KT / 16) {
        const int64_t t = int64_t(t0) + lane * 16;
        int64_t r = -1;
        if (t < c.q.len) {
          const int64_t page = __ldg(a.page_table + c.seq * a.max_pages + (t >> a.page_shift));
          if (page < 0 || page >= a.n_pages)
            flag_bad_index(status);
          else
            r = ((page * a.n_kv + c.head) << a.page_shift) + (t & ((1 << a.page_shift) - 1));
        }
        e.row[lane] = r;
      }
      if (i + 1 < n_tiles && ++c.tile == c.count) c.next_item(a);
    };
    for (int i = 0; i < min(3, n_tiles); ++i) describe(i);
    tc_fence_before();
    __syncthreads();  // descriptions, tensor memory
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    for (int i = 0; i < n_tiles; ++i) {
      __syncthreads();  // A
      if (lane == 0) {
        tc_fence_after();
        constexpr uint32_t id = instr_desc(kAccS32, kFmtS8, kFmtS8, false, false, 128, C::NQS);
#pragma unroll
        for (int b = 0; b < C::SBLK; ++b) {
          const int half = b / NG, j = b % NG;
#pragma unroll
          for (int k = 0; k < C::G; k += 32) {
            const int byte = j * C::G + k;  // in the token's bytes
            const int abyte = C::TPR == 2 ? half * 64 + byte : byte;
            mma_i8(tmem + b * C::NQS,
                   smem_desc(sbase + C::oK + (abyte >> 7) * 16384 + (abyte & 127), 16, 1024, kSw128),
                   smem_desc(sbase + C::oQ + (byte >> 7) * (C::NQS * 128) + (byte & 127), 16, 1024,
                             kSw128),
                   id, k > 0);
          }
        }
        mma_commit(sdone);
      }
      __syncwarp();
      const bool ends = sh.tiles[i & 3].ends || i + 1 == n_tiles;
      if (i + 3 < n_tiles) describe(i + 3);
      if (__syncthreads_or(0)) {  // B
        if (sh.fail) break;
        __syncthreads();
        __syncthreads();
        __syncthreads();
      }
      if (lane == 0) {
        tc_fence_after();
        // one MMA for all groups of a 128-coordinate block
        constexpr uint32_t id =
            instr_desc(kAccS32, kFmtS8, kFmtU8, true, true, 128, C::NGM * C::NP);
#pragma unroll
        for (int mt = 0; mt < C::NCH; ++mt)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_i8(tmem + mt * C::NGM * C::NP,
                   smem_desc(sbase + C::oV + mt * 16384 + k * 4096, 16, 1024, kSw128),
                   smem_desc(sbase + C::oP + (NG == 1 ? 0 : mt * C::NGM * 128 * C::NP) +
                                 k * 32 * C::NP,
                             128 * C::NP, 8 * C::NP, C::PSW),
                   id, k > 0);
        mma_commit(odone);
      }
      __syncwarp();
      if (ends) __syncthreads();  // results of the item
    }
    __syncthreads();  // every read of tensor memory is done
    tmem_free(tmem, C::TMEM);
    return;
  }

  // ========================== the eight other warps ==========================
  __syncthreads();  // descriptions, tensor memory
  tc_fence_after();
  const uint32_t tlane = sh.tmem + (uint32_t(warp & 3) << 21);
  const int tl = C::TPR == 2 ? wg * 128 + row : row;  // token of this thread's scores
  const int q0 = C::TPR == 2 ? 0 : wg * RQ;           // its first query row
  const int half = C::TPR == 2 ? row >> 6 : 0;        // of the accumulators: d = 64 half,
  const int crd = C::TPR == 2 ? row & 63 : row;       // coordinate byte,
  const int a0 = D == 256 ? 0 : wg * AQ;              // first query row

  // Packed codes of a tile in registers: piece tid + 256 k of 16 bytes, each
  // loaded a tile's time before it is expanded.
  uint4 kreg[KP], vreg[KP];
  float ks[NG], vs[NG];
  bool seen;
  auto load_codes = [&](int i, const uint8_t* base, uint4 (&w)[KP]) {
    const PdTile& e = sh.tiles[i & 3];
#pragma unroll
    for (int k = 0; k < KP; ++k) {
      const int p = tid + kPdThreads * k, t = p / (D / 32);
      const int64_t r = e.row[t >> 4];
      w[k] = make_uint4(0, 0, 0, 0);
      if (r >= 0)
        w[k] = __ldg(reinterpret_cast<const uint4*>(base + (r + (t & 15)) * (D / 2)) + p % (D / 32));
    }
  };
  auto load_scales = [&](int i) {
    const PdTile& e = sh.tiles[i & 3];
    const int64_t r = e.row[tl >> 4];
    seen = r >= 0 && e.t0 + tl < e.len;
#pragma unroll
    for (int j = 0; j < NG; ++j) ks[j] = vs[j] = 0.0f;
    if (seen) {
      const float* kp = a.k_scales + (r + (tl & 15)) * NG;
      const float* vp = a.v_scales + (r + (tl & 15)) * NG;
#pragma unroll
      for (int j = 0; j < NG; ++j) ks[j] = __ldg(kp + j), vs[j] = __ldg(vp + j);
    }
  };
  // -> 16 c bytes in a swizzled tile
  auto expand = [&](const uint4 (&w)[KP], uint32_t tile) {
#pragma unroll
    for (int k = 0; k < KP; ++k) {
      const int p = tid + kPdThreads * k, t = p / (D / 32);
      const int r = t & 127;
      const int byte = (t >> 7) * 64 + p % (D / 32) * 32;  // in the row's bytes
      const uint32_t base = tile + uint32_t(byte >> 7) * 16384 + uint32_t(r) * 128;
      const uint32_t c0 = (uint32_t(byte & 127) >> 4) ^ uint32_t(r & 7), c1 = c0 ^ 1u;
      constexpr uint32_t H = 0xF0F0F0F0u;
      sts128(base + c0 * 16, (w[k].x << 4) & H, w[k].x & H, (w[k].y << 4) & H, w[k].y & H);
      sts128(base + c1 * 16, (w[k].z << 4) & H, w[k].z & H, (w[k].w << 4) & H, w[k].w & H);
    }
  };

  float m[RQ], l[RQ], cw[RQ], acc[AQ];
  bool fresh = true;
  auto start_item = [&](const PdTile& e) {
#pragma unroll
    for (int r = 0; r < RQ; ++r) m[r] = -3e38f, l[r] = 0.0f, cw[r] = 1.0f;
#pragma unroll
    for (int r = 0; r < AQ; ++r) acc[r] = 0.0f;
    fresh = true;
    for (int r = warp; r < e.rows; r += kPdThreads / 32) {
      const int tok = (e.row0 + r) / a.n_q;
      const uint16_t* src = a.q + (int64_t(e.c0) + tok) * a.q_stride +
                            (int64_t(e.head) * a.n_q + (e.row0 + r - tok * a.n_q)) * D;
      const float qs = a.rot == kRotSRFT ? pd_query<C, kRotSRFT>(a, src, smem + C::oQ, r, lane)
                                         : pd_query<C, kRotSRHT>(a, src, smem + C::oQ, r, lane);
      if (lane == 0) {
        sh.qs[r] = qs;
        sh.pos[r] = e.p0 + tok;
        sh.m[r] = -3e38f;
      }
    }
  };

  load_codes(0, a.k_packed, kreg);
  load_codes(0, a.v_packed, vreg);
  load_scales(0);
  start_item(sh.tiles[0]);
  expand(kreg, sbase + C::oK);
  if (n_tiles > 1) load_codes(1, a.k_packed, kreg);
  fence_proxy_async_smem();
  bool began_here = sh.began_here, ok = true;

  for (int i = 0; i < n_tiles; ++i) {
    const PdTile& e = sh.tiles[i & 3];
    const uint32_t par = uint32_t(i) & 1u;
    const bool more = i + 1 < n_tiles;
    __syncthreads();  // A: K and the queries are in shared memory, O is read
    expand(vreg, sbase + C::oV);
    if (more) load_codes(i + 1, a.v_packed, vreg);

    // ---- scores of this thread's token ----
    const int nr = min(max(e.rows - q0, 0), RQ);
    const int t = e.t0 + tl;
    const int pf = e.p0 + e.row0 / a.n_q;  // positions of the first and the last row
    const int pl = e.p0 + (e.row0 + e.rows - 1) / a.n_q;
    const bool whole = e.t0 + KT - 1 <= pf && (a.window == 0 || e.t0 > pl - a.window);
    const float vmax = [&] {
      float x = vs[0];
#pragma unroll
      for (int j = 1; j < NG; ++j) x = fmaxf(x, vs[j]);
      return x;
    }();
    ok = mbar_wait_bounded(sdone, par) && ok;
    tc_fence_after();
    float s[RQ];
    {
      uint32_t x[NG][2 * RQ];
#pragma unroll
      for (int j = 0; j < NG; ++j)
        tmem_ld<2 * RQ>(tlane + uint32_t(((C::TPR == 2 ? wg * NG : 0) + j) * C::NQS + q0 * 2), x[j]);
      tmem_wait_ld();
#pragma unroll
      for (int r = 0; r < RQ; ++r)
        if (r < nr) {
          float v = 0.0f;
#pragma unroll
          for (int j = 0; j < NG; ++j)
            v = fmaf(ks[j], float(int(x[j][r]) * 128 + int(x[j][RQ + r])), v);
          s[r] = v * sh.qs[q0 + r];
          if (!seen) s[r] = -INFINITY;
          if (!whole) {
            const int p = sh.pos[q0 + r];
            if (t > p || (a.window > 0 && t <= p - a.window)) s[r] = -INFINITY;
          }
        }
    }

    // ---- weights and their slices ----
    auto weights = [&]() {
      bool over = false;
      float p[RQ];
#pragma unroll
      for (int r = 0; r < RQ; ++r) {
        p[r] = 0.0f;
        if (r < nr) {
          const float x = s[r] - m[r];
          p[r] = ex2(x);
          l[r] += p[r];
          over = over || x > 7.0f || p[r] * vmax * cw[r] > 127.0f;
        }
      }
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        uint32_t w[RQ];
#pragma unroll
        for (int r = 0; r < RQ; ++r)
          w[r] = __float_as_uint(fmaf(p[r] * vs[j], cw[r] * 65536.0f, 8388608.0f));
        constexpr int NB = 3 * RQ / 4;
        uint32_t b[(NB + 3) / 4 * 4];
#pragma unroll
        for (int r = NB; r < (NB + 3) / 4 * 4; ++r) b[r] = 0u;
#pragma unroll
        for (int r = 0; r < RQ / 4; ++r)
          pd_slices(w + 4 * r, b[r], b[RQ / 4 + r], b[RQ / 2 + r]);
        // row of 2 PW bytes, this thread's half of it; 16-byte pieces swizzled
        const uint32_t base = sbase + C::oP + uint32_t(j * 128 + row) * C::NP;
        const uint32_t x = C::NP == 32 ? (row >> 2) & 1 : (C::NP == 64 ? (row >> 1) & 3 : row & 7);
#pragma unroll
        for (int k = 0; k < NB; k += 4)
          sts128(base + ((uint32_t(wg * (C::PW / 16) + k / 4) ^ x) * 16), b[k], b[k + 1], b[k + 2],
                 b[k + 3]);
      }
      fence_proxy_async_smem();  // V's stores too
      return over;
    };
    float lold[RQ];
#pragma unroll
    for (int r = 0; r < RQ; ++r) lold[r] = l[r];
    const bool over = fresh ? true : weights();
    if (!ok) sh.fail = 1;
    tc_fence_before();
    const bool slow = __syncthreads_or(over || !ok);  // B: V and P are in shared memory
    if (slow) {
      if (sh.fail) break;  // uniform: written before the barrier
      // the tile's maxima -> new references; then the weights once more
#pragma unroll
      for (int r = 0; r < RQ; ++r) {
        l[r] = lold[r];
        float x = r < nr ? s[r] : -INFINITY;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
        if (lane == 0) sh.red[warp][r] = x;
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < RQ; ++r) {
        float mn = m[r];
#pragma unroll
        for (int w = 0; w < 4; ++w) mn = fmaxf(mn, sh.red[wg * 4 + w][r]);
        if constexpr (C::TPR == 2) {
#pragma unroll
          for (int w = 0; w < 4; ++w) mn = fmaxf(mn, sh.red[(wg ^ 1) * 4 + w][r]);
        }
        const float f = ex2(m[r] - mn);
        l[r] *= f;
        m[r] = mn;
        float x = r < nr ? ex2(s[r] - mn) * vmax : 0.0f;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
        if (lane == 0) sh.red2[warp][r] = x;
        if (row == 0 && (C::TPR == 1 || wg == 0)) {
          sh.f[q0 + r] = f;
          sh.m[q0 + r] = mn;
        }
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < RQ; ++r) {
        float x = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) x = fmaxf(x, sh.red2[wg * 4 + w][r]);
        if constexpr (C::TPR == 2) {
#pragma unroll
          for (int w = 0; w < 4; ++w) x = fmaxf(x, sh.red2[(wg ^ 1) * 4 + w][r]);
        }
        // the power of two that brings the largest into [1/2, 1)
        const int ex = min(max(253 - int(__float_as_uint(x) >> 23), 1), 237);
        cw[r] = __uint_as_float(uint32_t(ex) << 23);
        if (row == 0 && (C::TPR == 1 || wg == 0))
          sh.icw[q0 + r] = __uint_as_float(uint32_t(254 - ex) << 23);
      }
      weights();
      __syncthreads();
    }
    fresh = false;
    if (more) {
      load_scales(i + 1);
      expand(kreg, sbase + C::oK);
      if (i + 2 < n_tiles) load_codes(i + 2, a.k_packed, kreg);
    }

    // ---- accumulate the tile's O: this thread's coordinate, its query rows ----
    ok = mbar_wait_bounded(odone, par) && ok;
    tc_fence_after();
    // The columns of a query row: segment of P (the byte's half at d = 64, wg at
    // d = 128, both in turn at d = 256), slice, row in the segment.
    constexpr int HN = D == 256 ? 2 : 1, CN = AQ / HN;
    const int blk = D == 256 ? wg * C::NGM + crd / (C::G > 128 ? 128 : C::G) : crd / C::G;
#pragma unroll
    for (int h = 0; h < HN; ++h) {
      const int seg = D == 64 ? half : (D == 128 ? wg : h);
      const uint32_t at =
          tlane + uint32_t(blk * C::NP + seg * C::PW + (D == 64 ? wg * AQ : 0));
      uint32_t x0[CN], x1[CN], x2[CN];
      tmem_ld<CN>(at, x0);
      tmem_ld<CN>(at + RQ, x1);
      tmem_ld<CN>(at + 2 * RQ, x2);
      tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < CN; ++k) {
        const int ai = h * CN + k, r = a0 + ai;
        if (r < e.rows) {
          const float v = fmaf(float(int(x2[k])), 65536.0f, float(int(x1[k]) * 256 + int(x0[k])));
          if (slow) acc[ai] *= sh.f[r];
          acc[ai] = fmaf(v, sh.icw[r] * (1.0f / 1048576.0f), acc[ai]);
        }
      }
    }
    tc_fence_before();

    // ---- end of the item, or of the block's share of it ----
    if (e.ends || !more) {
#pragma unroll
      for (int r = 0; r < RQ; ++r) {
        float x = l[r];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) x += __shfl_xor_sync(kFull, x, o);
        if (lane == 0) sh.red[warp][r] = x;
      }
      const bool complete = e.ends && began_here;
      const int dim = D == 256 ? wg * 128 + pd_dim(row) : pd_dim(crd);
      float* ob = reinterpret_cast<float*>(smem + C::oP);
#pragma unroll
      for (int k = 0; k < AQ; ++k) ob[(half * R + a0 + k) * D + dim] = acc[k];
      __syncthreads();
      for (int r = warp; r < e.rows; r += kPdThreads / 32) {
        float ls = 0.0f;
        const int w0 = C::TPR == 2 ? 0 : (r / RQ) * 4;
        for (int w = 0; w < (C::TPR == 2 ? 8 : 4); ++w) ls += sh.red[w0 + w][r % RQ];
        auto value = [&](int d) {
          float v = ob[r * D + d];
          if constexpr (C::TPR == 2) v += ob[(R + r) * D + d];
          return v;
        };
        if (complete) {
          const float inv = ls > 0.0f ? 1.0f / ls : 0.0f;
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
          if (lane == 0) slot[r] = sh.m[r], slot[R + r] = ls;
          for (int d = lane; d < D; d += 32) slot[2 * R + r * D + d] = value(d);
        }
      }
      if (e.ends && !began_here && tid == 0) {
        join->c0 = e.c0;
        join->head = e.head;
        join->row0 = e.row0;
        join->rows = e.rows;
        join->first_block = block_of(sh.begun, run.total, run.blocks);
      }
      if (more) {
        began_here = true;
        start_item(sh.tiles[(i + 1) & 3]);
      }
    }
    fence_proxy_async_smem();  // K's and the queries' stores
  }
  if (!ok) atomicOr(status, kPagedTimeout);
  pdl_release();
  __syncthreads();  // every read of tensor memory is done
}

// Joins the partial results of items that several blocks shared: block b the
// one that ended in block b, a warp a row.
template <int D, int R, int ROT>
__global__ void __launch_bounds__(256) kvq_paged_join_kernel(const PagedAttnArgs a) {
  pdl_wait();  // the partial results of the kernel before
  const int b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const JoinInfo j = a.join[b];
  if (j.first_block < 0) return;
  WideLane<D, ROT> L;
  L.init(a.signs, lane);
  constexpr int W = D / 32;
  for (int r = warp; r < j.rows; r += 8) {
    float top = -3e38f;
    for (int p = j.first_block + lane; p <= b; p += 32)
      top = fmaxf(top, part_slot<D, R>(a, p, p == j.first_block ? 1 : 0)[r]);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    float Y[W], l = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) Y[w] = 0.0f;
#pragma unroll 4
    for (int p = j.first_block; p <= b; ++p) {
      const float* slot = part_slot<D, R>(a, p, p == j.first_block ? 1 : 0);
      const float f = exp2f(slot[r] - top);
      l = fmaf(f, slot[R + r], l);
#pragma unroll
      for (int w = 0; w < W; ++w) Y[w] = fmaf(f, slot[2 * R + r * D + L.k2 * W + w], Y[w]);
    }
    const float inv = l > 0.0f ? Wide<D, ROT>::KAPPA / l : 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) Y[w] *= inv;
    pd_store<D, ROT>(a, Y, L, out_row(a, j.c0, j.head, j.row0 + r));
  }
}

}  // namespace kvq
