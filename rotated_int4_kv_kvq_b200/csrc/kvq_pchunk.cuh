// kvq_pchunk.cuh -- attention of many query rows (a chunk of a prompt) over the
// paged int4 cache.
//
// Mathematics as in kvq_pdecode.cuh: queries are rotated once, products run on
// the codes in the rotated domain, results are rotated back once.  Here the
// query rows are the large operand and the work is bound by the tensor cores
// (4 d flops a row and key) and by the 2^x of every score.
//
//   S = Q C_K^T      kind::f16, f32 accumulators: Q the rotated queries in fp16
//                    (each row scaled by a power of two, error 2^-11 of a
//                    value: as much as rounding a query to fp16 once), C_K the
//                    codes, exact
//   p = 2^(S s_K[t] c_row - m)      f32; the row's reference m moves only when
//                    its maximum exceeds it by 8, so the accumulators are
//                    rescaled rarely
//   O += P C_V       P = p s_V[t] 2^-v in fp16 (error 2^-11 of a weight, as in
//                    any fp16 product, or 2^-31 of the largest scale where that is
//                    more), v the row's own: the V scales that it has attended so
//                    far stay under 2^(v + 7).  Cached rows that it does not attend
//                    have no say in v: tiles with a mask look for the largest scale
//                    seen.  Scales lie in shared memory over their tile's power of
//                    two; the difference of the exponents joins the reference m.
// With several scales a row (g < d) a row's largest scale is kept apart in f32
// and the codes are multiplied by the ratios s_j / s_max: ratio and product are
// rounded to fp16, 2^-11 each, so a score is off by three times that at most.
//
// That is less than a bf16 result is rounded by, but not less than an fp16 one: with
// scores of a few units fp16 results were 2 to 4 times as far off as their rounding.
// For fp16 activations (TWO) each rounded operand is therefore two: Q and what the
// rounding leaves of it (in tensor memory), P likewise (a slot of S holds both), and
// the ratio's first 8 bits, whose products with codes are exact, and its rest; the
// products of two rests are left out.  2 (g < d: 3) MMAs for one, and tiles of 64
// tokens so that all of it fits.
//
// A block holds 256 query rows (two tiles of 128; one at d = 256, where tensor
// memory holds one): while the tensor cores work for one tile the other one's
// scores become weights.  Roles: four warps of softmax a tile (a thread a row;
// they also rotate their rows in and out), four that turn packed codes into
// fp16 operands (a thread or two a token), one that issues MMAs, one that looks pages
// up.  P overwrites S in tensor memory and is read from there.
//
// Measured: 4096 new tokens over 16,384 rows, 8 KV heads of 4 queries, d = 128,
// bf16: 1.74 ms, 553 TFLOP/s, 34% of the measured tensor rate; the softmax threads'
// chain bounds it: a tile pair takes 8.0 thousand clocks, its products by
// arithmetic 2.0, the 2^x unit is busy for about as long, and the schedulers
// issue in 39% of the clocks.  In two halves: 30 rows of each of 32 sequences of
// 4096 rows and 8 heads take 376 us where one half takes 287 (d = 128, g = 128).
#pragma once

#include "kvq_codec.cuh"
#include "kvq_pdecode.cuh"

namespace kvq {

template <int D_, int NG_, bool TWO_>
struct Pc {
  static constexpr int D = D_, NG = NG_, G = D / NG;
  static constexpr bool TWO = TWO_;             // operands in two halves
  static constexpr bool TWO_KV = TWO && NG > 1; // (codes alone are exact)
  static constexpr int NT = D == 256 ? 1 : 2;   // row tiles of a block
  static constexpr int M = 128 * NT;            // query rows of an item
  static constexpr int KT = TWO ? 64 : 128;     // tokens of a tile
  // K and V operands in shared memory
  static constexpr int KS = D == 256 && (!TWO || TWO_KV) ? 1 : 2;
  static constexpr int NCH = D / 64;            // 128-byte columns of a row
  static constexpr int QCOL = 128 * 128, KCOL = KT * 128;  // bytes of one: of Q, of K or V
  static constexpr int TILE = NCH * QCOL;       // Q tile
  static constexpr int KVH = NCH * KCOL;        // K or V, a half
  static constexpr int KV = TWO_KV ? 2 * KVH : KVH;
  static constexpr int oQ = 0, oK = NT * TILE, oV = oK + KS * KV;
  static constexpr int SMEM = oV + KS * KV + 1024;
  static constexpr int WARPS = NT * 4 + 8;      // whole warpgroups, two warps idle
  static constexpr int THREADS = WARPS * 32;
  // Registers a thread: the softmax threads hold a whole row when they rotate it.
  // 256 x 176 + 256 x 80 is what 512 threads are launched with (at d = 256 the
  // 384 threads have 168 each).
  static constexpr bool SPLIT = NT == 2;
  static constexpr int REGS_MORE = 176, REGS_LESS = 80;
  static constexpr int W_DEQ = NT * 4, W_MMA = W_DEQ + 4, W_PAGE = W_MMA + 1;
  // Tensor memory: S/P slots, the second halves of Q, then O.
  static constexpr uint32_t colQ = 128, colO = 256;
  static_assert(2 * KT + (TWO ? NT * D / 2 : 0) <= 256, "tensor memory");
  static_assert(SMEM + 4096 <= 232448, "shared memory");
};

struct PcTile {
  int t0, lo, hi, c0, head, row0, rows, p0;  // (the item attends tokens lo .. hi - 1)
  int starts, last, ends;
  uint32_t have;
  int64_t row[8];
};
constexpr int kPcRing = 8;

struct PcShared {
  uint64_t dfull[kPcRing], dfree[kPcRing];
  uint64_t kfull[2], kfree[2], vfull[2], vfree[2];
  uint64_t scfull[4];            // scales
  // By slot (a row tile, or tiles in turn: the scores of a tile are issued before
  // the values of the one before, so one barrier could be two phases behind).
  uint64_t qfull[2], sdone[2], pfull[2], odone[2];
  PcTile tiles[kPcRing];
  uint32_t tmem;
  int64_t begun;
  float ks[4][128], vs[4][128];  // by tile: K scales; V scales over 2^vexp, below 2^7
  int vexp[4];
  float wmax[2][4];
  uint32_t sign_in[128], sign_out[128];  // sign masks of a row's words (of each thread of a pair)
  int64_t scratch[kRunScratch];
};

// fp16 pairs of eight codes in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ uint4 codes_to_half(uint32_t w) {
  const uint32_t w8 = w >> 8;
  const __half2 b = __half2half2(__float2half(-1032.0f)), s = __half2half2(__float2half(0.0625f)),
                c = __half2half2(__float2half(-72.0f));
  auto h = [](uint32_t x) { return *reinterpret_cast<__half2*>(&x); };
  auto u = [](__half2 x) { return *reinterpret_cast<uint32_t*>(&x); };
  return make_uint4(u(__hadd2(h((w & 0x000F000Fu) ^ 0x64086408u), b)),
                    u(__hfma2(h((w & 0x00F000F0u) ^ 0x64806480u), s, c)),
                    u(__hadd2(h((w8 & 0x000F000Fu) ^ 0x64086408u), b)),
                    u(__hfma2(h((w8 & 0x00F000F0u) ^ 0x64806480u), s, c)));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
// Column of coordinate i in that order.
__device__ __forceinline__ constexpr int pc_col(int i) {
  return (i & ~7) | ((i & 3) << 1) | ((i >> 2) & 1);
}

// D (+)= A B with A (fp16) in tensor memory.
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(accumulate))
      : "memory");
}
#define KVQ_V4(i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3])
#define KVQ_V16(i) KVQ_V4(i), KVQ_V4(i + 4), KVQ_V4(i + 8), KVQ_V4(i + 12)
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15};" ::KVQ_V16(0),
      "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31};" ::KVQ_V16(0),
      KVQ_V16(16), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Registers of this warpgroup's threads from here on.
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A pair of values as fp16, and what that leaves of them.
template <bool TWO>
__device__ __forceinline__ uint32_t pc_half(float x, float y, uint32_t& rest) {
  const uint32_t h = float2_to_half2_bits(x, y);
  if constexpr (TWO) {
    const float2 f = half2_bits_to_float2(h);
    rest = float2_to_half2_bits(x - f.x, y - f.y);
  }
  return h;
}

// Factor for a row whose largest rotated value is `top`: a power of two that
// brings it into [2^8, 2^9), far from fp16's smallest and largest, with the sign
// of the softmax scale; `back` undoes it and applies the scale.  A row with an
// infinity gets NaN: products of infinities alone could come out as "attends nothing".
__device__ __forceinline__ float pc_scale(float top, float qscale, float& back) {
  const int e = min(max(int(__float_as_uint(top) >> 23), 20), 234);
  back = __uint_as_float(uint32_t(e - 8) << 23) * fabsf(qscale);  // 2^(e - 135)
  if (!(top < INFINITY)) back = __uint_as_float(0x7FFFFFFFu);
  const float mul = __uint_as_float(uint32_t(262 - e) << 23);
  return qscale < 0.0f ? -mul : mul;
}

// d <= 128: a thread rotates its own row, in registers (the two-lane real FFT
// codelets, or a Walsh-Hadamard network), into the Q tile, a second half into the
// columns `rest` of tensor memory (then by whole warps).  Returns the factor from
// the row's products to log2 scores.
template <int D, int ROT, bool TWO>
__device__ __forceinline__ float pc_query_row(const PagedAttnArgs& a, const uint16_t* src,
                                              uint32_t tile, int r, const uint32_t* sign,
                                              uint32_t rest) {
  using C = Cfg<D, ROT, 1>;
  f2 u[C::NW], Y[C::P];
#pragma unroll
  for (int c = 0; c < C::NW / 4; ++c) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + c);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t x = w[j] ^ sign[4 * c + j];
      const float2 f = a.dtype == kDtF16 ? pair_to_float2<kDtF16>(x) : pair_to_float2<kDtBF16>(x);
      u[4 * c + j] = mk2(f.x, f.y);
    }
  }
  rotate_fwd<C>(u, 0, Y);
  const float top = absmax2<C::P>(Y);
  float back;
  const float sg = pc_scale(top, a.qscale, back);
  uint32_t low[16];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {  // columns 0 4 1 5 2 6 3 7 of each eight
    const f2 p = Y[4 * i], q = Y[4 * i + 1], s = Y[4 * i + 2], t = Y[4 * i + 3];
    uint32_t* l = low + 4 * (i & 3);
    sts128(tile + uint32_t(i >> 3) * 16384 + uint32_t(r) * 128 + (uint32_t((i ^ r) & 7) << 4),
           pc_half<TWO>(lo2(p) * sg, lo2(s) * sg, l[0]),
           pc_half<TWO>(hi2(p) * sg, hi2(s) * sg, l[1]),
           pc_half<TWO>(lo2(q) * sg, lo2(t) * sg, l[2]),
           pc_half<TWO>(hi2(q) * sg, hi2(t) * sg, l[3]));
    if constexpr (TWO) {
      if ((i & 3) == 3) tmem_st16(rest + uint32_t(i & ~3) * 4, low);
    }
  }
  return back * C::KAPPA_INV;  // both ways the same
}

// The way back: a row's accumulators (columns 0 4 1 5 2 6 3 7 of each eight) as
// coordinate pairs times `mul`.
template <int D>
__device__ __forceinline__ void pc_row(uint32_t acc, float mul, f2 (&Y)[D / 2]) {
#pragma unroll
  for (int c = 0; c < D; c += 32) {
    uint32_t o[32];
    tmem_ld<32>(acc + c, o);
    tmem_wait_ld();
    const f2 m2 = mk2(mul, mul);
    auto pair = [&](int x, int y) {
      return mul2(mk2(__uint_as_float(o[x]), __uint_as_float(o[y])), m2);
    };
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      f2* y = Y + c / 2 + 4 * g;
      y[0] = pair(8 * g, 8 * g + 2);
      y[1] = pair(8 * g + 4, 8 * g + 6);
      y[2] = pair(8 * g + 1, 8 * g + 3);
      y[3] = pair(8 * g + 5, 8 * g + 7);
    }
  }
}
template <int D, int ROT>
__device__ __forceinline__ void pc_result_row(const PagedAttnArgs& a, f2 (&Y)[D / 2], uint16_t* dst,
                                              const uint32_t* sign) {
  using C = Cfg<D, ROT, 1>;
  f2 x[C::NW];
  if constexpr (ROT == kRotSRHT) {
    fwht<C::P>(Y);
#pragma unroll
    for (int j = 0; j < C::NW; ++j) x[j] = Y[j];
  } else {
    f2 z[C::NW];
    split_lanes_inv<D>(Y, z);
    RFFT2<D / 2>::inv(z, x);
  }
#pragma unroll
  for (int c = 0; c < C::NW / 4; ++c) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const f2 v = x[4 * c + j];
      w[j] = (a.dtype == kDtF16 ? float2_to_pair<kDtF16>(lo2(v), hi2(v))
                                : float2_to_pair<kDtBF16>(lo2(v), hi2(v))) ^
             sign[4 * c + j];
    }
    reinterpret_cast<uint4*>(dst)[c] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// d = 256: a lane pair rotates a row (every lane of the warp takes part; rows
// that are not `there` read nothing).  The factor comes back in both lanes.  The
// second halves reach their rows' lanes of tensor memory through the rows' places
// in the Q tile; r0 is the warp's first row, `half` which 16 of its rows these are.
template <int ROT, bool TWO>
__device__ __forceinline__ float pc_query_pair(const PagedAttnArgs& a, const uint16_t* src,
                                               bool there, uint32_t tile, int r0, int half,
                                               const uint32_t* sign, uint32_t rest) {
  const int lane = threadIdx.x & 31, t = lane & 1, r = r0 + 16 * half + lane / 2;
  using C = Cfg<256, ROT, 2>;
  f2 u[C::NW], Y[C::P];
  const uint32_t* sg = sign + t * C::NW;
  auto word = [&](uint32_t x, int j) {
    x ^= sg[j];
    const float2 f = a.dtype == kDtF16 ? pair_to_float2<kDtF16>(x) : pair_to_float2<kDtBF16>(x);
    u[j] = mk2(f.x, f.y);
  };
  const uint4* p = reinterpret_cast<const uint4*>(src);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  if constexpr (C::PAIR_RFFT) {  // half t of every word of the row, two to a word
    const uint32_t sel = t ? 0x7632u : 0x5410u;
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      const uint4 v = there ? __ldg(p + c) : zero;
      word(__byte_perm(v.x, v.y, sel), 2 * c);
      word(__byte_perm(v.z, v.w, sel), 2 * c + 1);
    }
  } else {
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const uint4 v = there ? __ldg(p + t * 16 + c) : zero;
      word(v.x, 4 * c), word(v.y, 4 * c + 1), word(v.z, 4 * c + 2), word(v.w, 4 * c + 3);
    }
  }
  rotate_fwd<C>(u, t, Y);
  float top = absmax2<C::P>(Y);
  top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
  float back;
  const float mul = pc_scale(top, a.qscale, back);
  auto store = [&](auto low) {  // the halves, or what they leave, into the Q tile
    constexpr bool LOW = decltype(low)::value;
    auto word = [](float x, float y) {
      uint32_t rest = 0;
      const uint32_t h = pc_half<LOW>(x, y, rest);
      return LOW ? rest : h;
    };
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // a quarter of the row: one 128-byte column
      // (thread 1's second half of the Walsh-Hadamard pair is negated)
      const float m = ROT == kRotSRHT && t == 1 && h == 1 ? -mul : mul;
      const uint32_t at = tile + uint32_t(global_y<C>(t, 64 * h) >> 6) * 16384 + uint32_t(r) * 128;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const f2* y = Y + 32 * h + 4 * i;
        sts128(at + (uint32_t((i ^ r) & 7) << 4), word(lo2(y[0]) * m, lo2(y[2]) * m),
               word(hi2(y[0]) * m, hi2(y[2]) * m), word(lo2(y[1]) * m, lo2(y[3]) * m),
               word(hi2(y[1]) * m, hi2(y[3]) * m));
      }
    }
  };
  if constexpr (TWO) {
    store(std::true_type{});
    __syncwarp();
    const int mine = r0 + lane;
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
      uint32_t v[16];
      tmem_ld<16>(rest + 16 * c, v);  // (the other 16 rows')
      tmem_wait_ld();
      if (lane >> 4 == half) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const int piece = 4 * c + p;
          const uint4 x = lds128(tile + uint32_t(piece >> 3) * 16384 + uint32_t(mine) * 128 +
                                 (uint32_t((piece ^ mine) & 7) << 4));
          v[4 * p] = x.x, v[4 * p + 1] = x.y, v[4 * p + 2] = x.z, v[4 * p + 3] = x.w;
        }
      }
      tmem_st16(rest + 16 * c, v);
    }
    tmem_wait_st();  // (the other half reads what is stored here)
    __syncwarp();
  }
  store(std::false_type{});
  return back * C::KAPPA_INV;  // both ways the same
}

template <int D, int NG, bool TWO>
__global__ void __launch_bounds__(Pc<D, NG, TWO>::THREADS, 1)
    kvq_paged_chunk_kernel(const PagedAttnArgs a, unsigned* status) {
  using C = Pc<D, NG, TWO>;
  constexpr int NT = C::NT, M = C::M, KT = C::KT, KS = C::KS;
  extern __shared__ uint8_t smem_raw[];
  __shared__ PcShared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto bar = [](uint64_t& b) { return smem_u32(&b); };
  if (tid == 0) {
    for (int i = 0; i < kPcRing; ++i) {
      mbar_init(bar(sh.dfull[i]), 1);
      mbar_init(bar(sh.dfree[i]), NT * 4 + 1);  // the softmax, and the MMA warp
    }
    for (int i = 0; i < 4; ++i) mbar_init(bar(sh.scfull[i]), 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(sh.kfull[i]), 4);
      mbar_init(bar(sh.vfull[i]), 4);
      mbar_init(bar(sh.kfree[i]), 1);
      mbar_init(bar(sh.vfree[i]), 1);
      mbar_init(bar(sh.qfull[i]), 4);
      mbar_init(bar(sh.pfull[i]), 4);
      mbar_init(bar(sh.sdone[i]), 1);
      mbar_init(bar(sh.odone[i]), 1);
    }
    fence_mbar_init();
  }
  pdl_wait();  // no global access before the previous kernel completes
  if (tid < D / 2) {
    using CF = Cfg<D, kRotSRFT, tpv_of(D)>;
    using CH = Cfg<D, kRotSRHT, tpv_of(D)>;
    const int t = tid / CF::NW, w = tid % CF::NW;
    sh.sign_in[tid] = a.rot == kRotSRFT ? load_mask_word<CF>(a.signs, t, w)
                                        : load_mask_word<CH>(a.signs, t, w);
    sh.sign_out[tid] = a.rot == kRotSRFT ? store_mask_word<CF>(a.signs, t, w)
                                         : store_mask_word<CH>(a.signs, t, w);
  }
  const Run run = find_run<M, KT, C::THREADS>(a, blockIdx.x, gridDim.x, sh.scratch, status);
  JoinInfo* join = a.join + blockIdx.x;
  if (tid == 0) join->first_block = -1;
  pdl_release();  // the join's blocks wait for this grid's end: let them be placed
  if (run.begin == run.end) return;
  const int n = int(run.end - run.begin);  // tiles
  if (warp == C::W_MMA) tmem_alloc(smem_u32(&sh.tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
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

  if (warp >= C::W_DEQ) {
    // (here, before the warps part: all four of a warpgroup have to take the same
    // one of these instructions.  The two warps behind the page warp are idle.)
    if constexpr (C::SPLIT) regs_dec<C::REGS_LESS>();
    if (warp == C::W_PAGE) {
      // ---------------- pages: what each tile is, and where ----------------
      Cursor<M, KT> c;
      c.seek(a, run.seq, run.off);
      if (lane == 0) sh.begun = run.begin - c.tile;
      for (int i = 0; i < n; ++i) {
        PcTile& e = sh.tiles[i % kPcRing];
        if (i >= kPcRing) wait(sh.dfree[i % kPcRing], i / kPcRing - 1);
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
          e.t0 = t0;
          e.lo = c.lo;
          e.hi = c.hi;
          e.c0 = c.q.c0;
          e.head = c.head;
          e.row0 = c.qt * M;
          e.rows = int(min(int64_t(M), int64_t(c.q.n) * a.n_q - int64_t(c.qt) * M));
          e.p0 = c.q.len - c.q.n;
          e.starts = i == 0 || c.tile == 0;
          e.last = c.tile + 1 == c.count;
          e.ends = e.last || i + 1 == n;
          e.have = have;
        }
        arrive(sh.dfull[i % kPcRing]);
        if (i + 1 < n && ++c.tile == c.count) c.next_item(a);
      }
    } else if (warp == C::W_MMA) {
      // ---------------- MMA issue ----------------
      constexpr uint32_t idS = instr_desc(kAccF32, kFmtF16, kFmtF16, false, false, 128, KT);
      constexpr uint32_t idO = instr_desc(kAccF32, kFmtF16, kFmtF16, false, true, 128, D);
      int items[2] = {0, 0}, used[2] = {0, 0};  // of each row tile: items and tiles it took part in
      bool two = false;
      auto scores = [&](int x, int i) {  // row tile x, tile i
        const int slot = NT == 2 ? x : i & 1;
        if (lane == 0) {
          tc_fence_after();
          const uint32_t q = sbase + C::oQ + x * C::TILE, k = sbase + C::oK + (i % KS) * C::KV;
          const uint32_t d = tmem + slot * KT;
#pragma unroll 1
          for (int s = 0; s < D / 16; ++s) {
            const uint64_t dq = smem_desc(q + (s / 4) * C::QCOL + (s % 4) * 32, 16, 1024, kSw128);
            const uint32_t ks = k + (s / 4) * C::KCOL + (s % 4) * 32;
            const uint64_t dk = smem_desc(ks, 16, 1024, kSw128);
            mma_f16(d, dq, dk, idS, s > 0);
            if constexpr (TWO) mma_f16_ts(d, tmem + C::colQ + x * (D / 2) + s * 8, dk, idS, true);
            if constexpr (C::TWO_KV)
              mma_f16(d, dq, smem_desc(ks + C::KVH, 16, 1024, kSw128), idS, true);
          }
          mma_commit(bar(sh.sdone[slot]));
          if (x == NT - 1 || !two) mma_commit(bar(sh.kfree[i % KS]));
        }
        __syncwarp();
      };
      auto values = [&](int x, int i, bool first) {
        const int slot = NT == 2 ? x : i & 1;
        if (lane == 0) {
          tc_fence_after();
          const uint32_t v = sbase + C::oV + (i % KS) * C::KV;
          const uint32_t d = tmem + C::colO + x * 128;
#pragma unroll 1
          for (int s = 0; s < KT / 16; ++s) {
            // (in two halves: 16 columns of each, in turn)
            const uint32_t p = tmem + slot * KT + (TWO ? s / 2 * 32 + s % 2 * 8 : s * 8);
            const uint64_t dv = smem_desc(v + s * 2048, C::KCOL, 1024, kSw128);
            mma_f16_ts(d, p, dv, idO, !first || s > 0);
            if constexpr (TWO) mma_f16_ts(d, p + 16, dv, idO, true);
            if constexpr (C::TWO_KV)
              mma_f16_ts(d, p, smem_desc(v + C::KVH + s * 2048, C::KCOL, 1024, kSw128), idO, true);
          }
          mma_commit(bar(sh.odone[slot]));
          if (x == NT - 1 || !two) mma_commit(bar(sh.vfree[i % KS]));
        }
        __syncwarp();
      };
      for (int i = 0; i < n; ++i) {
        wait(sh.dfull[i % kPcRing], i / kPcRing);
        const bool starts = sh.tiles[i % kPcRing].starts, ends = sh.tiles[i % kPcRing].ends;
        const int rows = sh.tiles[i % kPcRing].rows;
        // (this tile's scores are under way, so the softmax may be through with the
        // description before it is read here)
        arrive(sh.dfree[i % kPcRing]);
        if (starts) {
          two = NT == 2 && rows > 128;
          wait(sh.qfull[0], items[0]++);
          if (two) wait(sh.qfull[1], items[1]++);
          wait(sh.kfull[i % KS], i / KS);
          scores(0, i);
          if (two) scores(1, i);
        }
        // The next scores overwrite columns whose P the values before them read: only
        // products of one accumulator are ordered among themselves, so these wait.
        if constexpr (NT == 2) {
          wait(sh.pfull[0], used[0]);
          wait(sh.vfull[i % KS], i / KS);
          values(0, i, starts);
          if (!ends) {
            wait(sh.kfull[(i + 1) % KS], (i + 1) / KS);
            wait(sh.odone[0], used[0]);
            scores(0, i + 1);
          }
          ++used[0];
          if (two) {
            wait(sh.pfull[1], used[1]);
            values(1, i, starts);
            if (!ends) {
              wait(sh.odone[1], used[1]);
              scores(1, i + 1);
            }
            ++used[1];
          }
        } else {
          if (!ends) {
            wait(sh.kfull[(i + 1) % KS], (i + 1) / KS);
            if (i > 0) wait(sh.odone[(i + 1) & 1], (i - 1) >> 1);
            scores(0, i + 1);
          }
          wait(sh.pfull[i & 1], i >> 1);
          wait(sh.vfull[i % KS], i / KS);
          values(0, i, starts);
        }
      }
    } else if (warp < C::W_MMA) {
      // ---------------- packed codes -> fp16 operands ----------------
      // A thread takes a token, or half of one (and then half of its groups).
      constexpr int TPT = 128 / KT, NP = D / 32 / TPT;  // 16-byte pieces of a thread
      constexpr int NGT = NG > 1 ? NG / TPT : 1;
      const int t = (tid - C::W_DEQ * 32) % KT, part = (tid - C::W_DEQ * 32) / KT;
      uint4 kreg[NP], vreg[NP];
      float ksc[NG], vsc[NG];
      auto load = [&](int i) {
        const PcTile& e = sh.tiles[i % kPcRing];
        const int64_t r = e.row[t >> 4] + (t & 15);
        const uint4* kp = reinterpret_cast<const uint4*>(a.k_packed + r * (D / 2)) + part * NP;
        const uint4* vp = reinterpret_cast<const uint4*>(a.v_packed + r * (D / 2)) + part * NP;
        const bool there =
            (e.have >> (t >> 4) & 1u) && e.t0 + t >= e.lo && e.t0 + t < e.hi;
#pragma unroll
        for (int k = 0; k < NP; ++k) kreg[k] = __ldg(kp + k), vreg[k] = __ldg(vp + k);
#pragma unroll
        for (int j = 0; j < NG; ++j) {  // rows that no query attends may hold anything
          ksc[j] = there ? __ldg(a.k_scales + r * NG + j) : 0.0f;
          vsc[j] = there ? __ldg(a.v_scales + r * NG + j) : 0.0f;
        }
      };
      auto convert = [&](const uint4 (&w)[NP], const float (&sc)[NG], float top, uint32_t tile) {
        const float inv = top >= 0x1p-126f ? 1.0f / top : 0.0f;
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          uint32_t f = 0, fl = 0;
          if constexpr (NG > 1) {
            const int g = k * 32 / C::G;
            const float own = TPT == 2 && part != 0 ? sc[NG - NGT + g] : sc[g];
            const float x = inv > 0.0f ? own * inv : 0.0f;
            // In two halves: 8 bits, so that products with codes are exact, and the rest.
            const float h = TWO ? __uint_as_float(__float_as_uint(x) & 0xFFFF0000u) : x;
            f = float2_to_half2_bits(h, h);
            fl = float2_to_half2_bits(x - h, x - h);
          }
          const uint32_t words[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
          const int kk = part * NP + k;  // piece of the row
          const uint32_t to = tile + uint32_t(kk / 2) * C::KCOL + uint32_t(t) * 128;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 h = codes_to_half(words[j]);
            const uint32_t at = to + (uint32_t(((kk & 1) * 4 + j) ^ (t & 7)) << 4);
            if constexpr (NG > 1)
              sts128(at, hmul2(h.x, f), hmul2(h.y, f), hmul2(h.z, f), hmul2(h.w, f));
            else
              sts128(at, h.x, h.y, h.z, h.w);
            if constexpr (C::TWO_KV)
              sts128(at + C::KVH, hmul2(h.x, fl), hmul2(h.y, fl), hmul2(h.z, fl), hmul2(h.w, fl));
          }
        }
        fence_proxy_async_smem();
      };
      // NaN if one is not finite: the operand is 0 then (another row's P of 0 has to
      // stay one), and who attends the token gets NaN from its scale.
      auto largest = [](const float (&s)[NG]) {
        float x = s[0], sum = s[0];
#pragma unroll
        for (int j = 1; j < NG; ++j) x = fmaxf(x, s[j]), sum += s[j];
        return fmaf(sum, 0.0f, x);
      };
      wait(sh.dfull[0], 0);
      load(0);
      for (int i = 0; i < n; ++i) {
        const float ktop = largest(ksc), vtop = largest(vsc);
        // the V scales of the tile under a power of two
        float x = fmaxf(vtop, 0.0f);  // (of the finite ones)
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
        if (lane == 0) sh.wmax[i & 1][warp - C::W_DEQ] = x;
        named_sync(3, 128);
#pragma unroll
        for (int w = 0; w < 4; ++w) x = fmaxf(x, sh.wmax[i & 1][w]);
        const int vexp = max(int(__float_as_uint(x) >> 23) - 133, -126);
        const float vmul = __uint_as_float(uint32_t(127 - vexp) << 23);
        // ring of four: the softmax of tile i - 4 is behind V's wait of tile i - 1
        if (part == 0) {
          sh.ks[i & 3][t] = ktop;
          sh.vs[i & 3][t] = vtop * vmul;
          if (t == 0) sh.vexp[i & 3] = vexp;
        }
        arrive(sh.scfull[i & 3]);
        // K, then V through the same code (for the instruction cache)
        float top = ktop;
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          if (i >= KS) wait(kv ? sh.vfree[i % KS] : sh.kfree[i % KS], i / KS - 1);
          convert(kreg, ksc, top, sbase + (kv ? C::oV : C::oK) + (i % KS) * C::KV);
          arrive(kv ? sh.vfull[i % KS] : sh.kfull[i % KS]);
#pragma unroll
          for (int k = 0; k < NP; ++k) kreg[k] = vreg[k];
#pragma unroll
          for (int j = 0; j < NG; ++j) ksc[j] = vsc[j];
          top = vtop;
        }
        if (i + 1 < n) {
          wait(sh.dfull[(i + 1) % kPcRing], (i + 1) / kPcRing);
          load(i + 1);
        }
      }
    }
  } else {
    if constexpr (C::SPLIT) regs_inc<C::REGS_MORE>();
    // ---------------- softmax: a thread a query row ----------------
    const int x = NT == 2 ? warp >> 2 : 0, w4 = warp & 3;
    const uint32_t tlane = tmem + (uint32_t(w4) << 21);
    const uint32_t tO = tlane + C::colO + x * 128;
    const uint32_t qtile = sbase + C::oQ + x * C::TILE;
    const uint32_t stage = qtile + w4 * 4096;  // this warp's rows of it, 4 KB of every 16
    float m = 0.0f, l = 0.0f, rowc = 0.0f;
    int used = 0, item = -1, vexp = 0, pos = 0;  // vexp: v of the row
    bool active = false;
    for (int i = 0; i < n; ++i) {
      wait(sh.dfull[i % kPcRing], i / kPcRing);
      const PcTile& e = sh.tiles[i % kPcRing];
      const int rows = e.rows - x * 128;  // of this row tile
      if (e.starts) {
        // ---- this warp's queries ----
        ++item;
        active = rows > 0;
        const int nr = min(max(rows - w4 * 32, 0), 32);
        rowc = 0.0f;
        auto queries = [&](auto rot) {
          constexpr int ROT = decltype(rot)::value;
          auto source = [&](int r) {
            const int g = e.row0 + x * 128 + w4 * 32 + r, tok = g / a.n_q;
            return a.q + (int64_t(e.c0) + tok) * a.q_stride +
                   (int64_t(e.head) * a.n_q + (g - tok * a.n_q)) * D;
          };
          const uint32_t rest = tlane + C::colQ + x * (D / 2);
          if constexpr (D <= 128) {
            if (TWO ? nr > 0 : lane < nr) {  // (the whole warp stores to tensor memory)
              const float f = pc_query_row<D, ROT, TWO>(a, source(min(lane, nr - 1)), qtile,
                                                        w4 * 32 + lane, sh.sign_in, rest);
              if (lane < nr) rowc = f;
            }
          } else {
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {  // rows 0..15, then 16..31
              const int r = 16 * h + lane / 2;
              const float f = pc_query_pair<ROT, TWO>(a, source(min(r, max(nr - 1, 0))), r < nr,
                                                      qtile, w4 * 32, h, sh.sign_in, rest);
              const float g = __shfl_sync(kFull, f, 2 * (lane & 15));
              if (lane >> 4 == h && lane < nr) rowc = g;
            }
          }
        };
        if (a.rot == kRotSRFT)
          queries(std::integral_constant<int, kRotSRFT>{});
        else
          queries(std::integral_constant<int, kRotSRHT>{});
        if constexpr (TWO) {
          tmem_wait_st();
          tc_fence_before();
        }
        fence_proxy_async_smem();
        if (active) arrive(sh.qfull[x]);
        pos = e.p0 + (e.row0 + x * 128 + min(w4 * 32 + lane, max(rows - 1, 0))) / a.n_q;
        m = lane < nr ? -3e38f : 0.0f;  // (what rows that are not there hold moves nothing)
        l = 0.0f;
        vexp = -126;
      }
      if (active) {
        const int slot = NT == 2 ? x : i & 1;
        const uint32_t tS = tlane + slot * KT;
        wait(sh.sdone[slot], NT == 2 ? used : i >> 1);
        wait(sh.scfull[i & 3], i >> 2);
        tc_fence_after();
        // first and last position of the warp's rows decide on masks
        const int pf = __shfl_sync(kFull, pos, 0), pl = __shfl_sync(kFull, pos, 31);
        const bool whole = e.t0 + KT - 1 <= pf && (a.window == 0 || e.t0 > pl - a.window) &&
                           e.have == (1u << (KT / 16)) - 1;
        const int hi = pos - e.t0;                                     // last column seen
        const int lo = a.window > 0 ? pos - a.window + 1 - e.t0 : 0;   // first
        auto seen = [&](int c) {  // bit j: column c + j of 32 is seen
          const int l = max(lo - c, 0), h = min(hi - c, 31);
          const uint32_t there = e.have >> (c >> 4);
          return h < l ? 0u
                       : (0xFFFFFFFFu << l) & (0xFFFFFFFFu >> (31 - h)) &
                             ((there & 1u ? 0xFFFFu : 0u) | (there & 2u ? 0xFFFF0000u : 0u));
        };
        const float4* ks4 = reinterpret_cast<const float4*>(sh.ks[i & 3]);
        const float4* vs4 = reinterpret_cast<const float4*>(sh.vs[i & 3]);
        // ---- the row's maximum, and where a reference moves, the accumulators ----
        const int ve = sh.vexp[i & 3];
        {
          // (All loops over columns are rolled: what the roles run per tile has to
          // stay in the instruction cache.  Unrolled, one pass took 1.6 times as
          // long.)
          float top = -INFINITY, top1 = -INFINITY, vtop = 0.0f;
          auto largest = [&](auto masks) {
            constexpr bool MASK = decltype(masks)::value;
#pragma unroll 1
            for (int c = 0; c < KT; c += 32) {
              uint32_t s[32];
              tmem_ld<32>(tS + c, s);
              const uint32_t sm = MASK ? seen(c) : 0u;
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                const float4 k = ks4[(c + j) / 4];
                f2 u = mul2(mk2(__uint_as_float(s[j]), __uint_as_float(s[j + 1])), mk2(k.x, k.y));
                f2 w = mul2(mk2(__uint_as_float(s[j + 2]), __uint_as_float(s[j + 3])), mk2(k.z, k.w));
                if constexpr (MASK) {
                  u = mk2(sm >> j & 1u ? lo2(u) : -INFINITY, sm >> (j + 1) & 1u ? hi2(u) : -INFINITY);
                  w = mk2(sm >> (j + 2) & 1u ? lo2(w) : -INFINITY,
                          sm >> (j + 3) & 1u ? hi2(w) : -INFINITY);
                  const float4 v = vs4[(c + j) / 4];
                  vtop = max3f(vtop, sm >> j & 1u ? v.x : 0.0f, sm >> (j + 1) & 1u ? v.y : 0.0f);
                  vtop = max3f(vtop, sm >> (j + 2) & 1u ? v.z : 0.0f,
                               sm >> (j + 3) & 1u ? v.w : 0.0f);
                }
                top = max3f(top, lo2(u), hi2(u));
                top1 = max3f(top1, lo2(w), hi2(w));
              }
            }
          };
          if (whole)
            largest(std::false_type{});
          else
            largest(std::true_type{});
          top = fmaxf(top, top1) * rowc;  // (0 for rows that are not there)
          if (!(top > -INFINITY)) top = -3e38f;
          const bool moved = top > m + 8.0f;
          int vn = max(vexp, ve);
          if (!whole)  // (a tile's scales reach down to 2^-100 of its largest)
            vn = vtop > 0.0f ? max(vexp, ve + max(int(__float_as_uint(vtop) >> 23) - 133, -100))
                             : vexp;
          if (__any_sync(kFull, moved || vn != vexp)) {
            const float mn = moved ? top : m;
            const float f = ex2(m - mn);
            const float fo = f * ex2(float(max(vexp - vn, -200)));
            l *= f;
            m = mn;
            vexp = vn;
            if (!e.starts) {
              wait(sh.odone[NT == 2 ? x : (i - 1) & 1], NT == 2 ? used - 1 : (i - 1) >> 1);
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld<32>(tO + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * fo);
                tmem_st32(tO + c, o);
              }
              tmem_wait_st();
            }
          }
        }
        // ---- weights ----
        auto weights = [&](auto masks) {
          constexpr bool MASK = decltype(masks)::value;
          // P = p 2^dv times the scale as it lies there; l takes the 2^dv out again.
          // (From 2^-40 on P is below fp16's smallest: no matter how far.  Upwards the
          // limit is out of reach but for rows that attend none of the tile.)
          const int dv = min(max(ve - vexp, -40), 100);
          const float nm = float(dv) - m;
          const f2 rc2 = mk2(rowc, rowc), nm2 = mk2(nm, nm);
          f2 l2 = mk2(0.0f, 0.0f);
#pragma unroll 1
          for (int c = 0; c < KT; c += 32) {
            uint32_t s[32], p[TWO ? 32 : 16];
            tmem_ld<32>(tS + c, s);
            const uint32_t sm = MASK ? seen(c) : 0u;
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 k = ks4[(c + j) / 4], v = vs4[(c + j) / 4];
#pragma unroll
              for (int b = 0; b < 4; b += 2) {
                const f2 kk = b == 0 ? mk2(k.x, k.y) : mk2(k.z, k.w);
                f2 vv = b == 0 ? mk2(v.x, v.y) : mk2(v.z, v.w);
                const f2 t = mul2(mk2(__uint_as_float(s[j + b]), __uint_as_float(s[j + b + 1])), kk);
                const f2 z = fma2(t, rc2, nm2);
                float z0 = lo2(z), z1 = hi2(z);
                if constexpr (MASK) {
                  // (the scale too: what is hidden may be NaN)
                  const bool s0 = sm >> (j + b) & 1u, s1 = sm >> (j + b + 1) & 1u;
                  z0 = s0 ? z0 : -INFINITY, z1 = s1 ? z1 : -INFINITY;
                  vv = mk2(s0 ? lo2(vv) : 0.0f, s1 ? hi2(vv) : 0.0f);
                }
                const f2 pp = mk2(ex2(z0), ex2(z1));
                l2 = add2(l2, pp);
                const f2 wv = mul2(pp, vv);
                p[(j + b) / 2] = pc_half<TWO>(lo2(wv), hi2(wv), p[(TWO ? 16 : 0) + (j + b) / 2]);
              }
            }
            if constexpr (TWO)  // over columns of S that have been read
              tmem_st32(tS + c, p);
            else
              tmem_st16(tS + c / 2, p);
          }
          l = fmaf(lo2(l2) + hi2(l2), __uint_as_float(uint32_t(127 - dv) << 23), l);
        };
        if (whole)
          weights(std::false_type{});
        else
          weights(std::true_type{});
        tmem_wait_st();
        tc_fence_before();
        arrive(sh.pfull[slot]);
        ++used;
      }
      if (!e.ends) {
        arrive(sh.dfree[i % kPcRing]);
        continue;
      }
      // ---- end of the item, or of the block's share of it ----
      if (active) {
        wait(sh.odone[NT == 2 ? x : i & 1], NT == 2 ? used - 1 : i >> 1);
        tc_fence_after();
        const bool began_here = item > 0 || sh.begun == run.begin;
        const bool complete = e.last && began_here;
        const float unit = ex2(float(vexp));  // of the accumulators
        const int nr = min(max(rows - w4 * 32, 0), 32);
        float* slot = part_slot<D, M>(a, blockIdx.x, began_here ? 1 : 0);
        const int r0 = x * 128 + w4 * 32;  // first row in the item
        if (!complete && lane < nr) slot[r0 + lane] = m, slot[M + r0 + lane] = l;
        const float fin = complete ? (l != 0.0f ? unit / l : 0.0f) : unit;
        if constexpr (D <= 128) {
          f2 Y[D / 2];
          // (the kappa of either rotation's inverse, 1 for a partial result)
          const float kappa = !complete            ? 1.0f
                              : a.rot == kRotSRFT ? Cfg<D, kRotSRFT, 1>::KAPPA_INV
                                                  : Cfg<D, kRotSRHT, 1>::KAPPA_INV;
          pc_row<D>(tO, fin * kappa, Y);
          if (lane < nr) {
            if (!complete) {
              float4* dst = reinterpret_cast<float4*>(slot + 2 * M + (r0 + lane) * D);
#pragma unroll
              for (int j = 0; j < D / 4; ++j)
                dst[j] = make_float4(lo2(Y[2 * j]), hi2(Y[2 * j]), lo2(Y[2 * j + 1]),
                                     hi2(Y[2 * j + 1]));
            } else {
              uint16_t* dst = out_row(a, e.c0, e.head, e.row0 + r0 + lane);
              if (a.rot == kRotSRFT)
                pc_result_row<D, kRotSRFT>(a, Y, dst, sh.sign_out);
              else
                pc_result_row<D, kRotSRHT>(a, Y, dst, sh.sign_out);
            }
          }
        }
        if constexpr (D == 256) {
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {  // rows 0..15, then 16..31, through shared memory
            __syncwarp();
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld<32>(tO + c, o);
              tmem_wait_ld();
              if ((lane >> 4) == h) {
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                  const uint32_t off = uint32_t(lane & 15) * (D * 4) +
                                       ((uint32_t((c + j) / 4) ^ uint32_t(lane & 7)) << 4);
                  sts128(stage + (off >> 12) * 16384 + (off & 4095),
                         __float_as_uint(__uint_as_float(o[j]) * fin),
                         __float_as_uint(__uint_as_float(o[j + 1]) * fin),
                         __float_as_uint(__uint_as_float(o[j + 2]) * fin),
                         __float_as_uint(__uint_as_float(o[j + 3]) * fin));
                }
              }
            }
            __syncwarp();
            auto piece = [&](int r, int c4) {  // four columns of a row
              const uint32_t off = uint32_t(r) * (D * 4) + ((uint32_t(c4) ^ uint32_t(r & 7)) << 4);
              return lds128(stage + (off >> 12) * 16384 + (off & 4095));
            };
            if (complete) {  // a row a lane pair
              auto rows_back = [&](auto rot) {
                constexpr int ROT = decltype(rot)::value;
                using C2 = Cfg<256, ROT, 2>;
                const int r = lane >> 1, t = lane & 1;
                f2 Y[C2::P];
                const f2 kap = mk2(C2::KAPPA_INV, C2::KAPPA_INV);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  const int c0 = global_y<C2>(t, 64 * q) / 4;
#pragma unroll
                  for (int i = 0; i < 8; ++i) {  // columns 0 4 1 5, 2 6 3 7
                    const uint4 v = piece(r, c0 + 2 * i), w = piece(r, c0 + 2 * i + 1);
                    auto pair = [&](uint32_t x, uint32_t y) {
                      return mul2(mk2(__uint_as_float(x), __uint_as_float(y)), kap);
                    };
                    f2* y = Y + 32 * q + 4 * i;
                    y[0] = pair(v.x, v.z), y[1] = pair(w.x, w.z);
                    y[2] = pair(v.y, v.w), y[3] = pair(w.y, w.w);
                  }
                }
                uint32_t xw[C2::NW];
                rotate_inv<C2>(Y, t, xw, 0, a.dtype == kDtBF16);
                if (16 * h + r < nr) {
                  uint4* dst = reinterpret_cast<uint4*>(
                                   out_row(a, e.c0, e.head, e.row0 + r0 + 16 * h + r)) + t * 16;
                  const uint32_t* m = sh.sign_out + t * C2::NW;
#pragma unroll
                  for (int j = 0; j < 16; ++j)
                    dst[j] = make_uint4(xw[4 * j] ^ m[4 * j], xw[4 * j + 1] ^ m[4 * j + 1],
                                        xw[4 * j + 2] ^ m[4 * j + 2], xw[4 * j + 3] ^ m[4 * j + 3]);
                }
              };
              if (a.rot == kRotSRFT)
                rows_back(std::integral_constant<int, kRotSRFT>{});
              else
                rows_back(std::integral_constant<int, kRotSRHT>{});
            } else {
#pragma unroll 1
              for (int r = 0; r < 16 && h * 16 + r < nr; ++r) {
                float* to = slot + 2 * M + (r0 + h * 16 + r) * D;
                for (int d = lane; d < D; d += 32) {
                  const int c = pc_col(d);
                  const uint4 v = piece(r, c >> 2);
                  const uint32_t x = (c & 2) ? ((c & 1) ? v.w : v.z) : ((c & 1) ? v.y : v.x);
                  to[d] = __uint_as_float(x);
                }
              }
            }
          }
        }
        if (e.last && !began_here && tid == 0) {
          join->c0 = e.c0;
          join->head = e.head;
          join->row0 = e.row0;
          join->rows = e.rows;
          join->first_block = block_of(sh.begun, run.total, run.blocks);
        }
        tc_fence_before();
      }
      arrive(sh.dfree[i % kPcRing]);
    }
  }
  if (!ok && lane == 0) atomicOr(status, kPagedTimeout);
  tc_fence_before();
  __syncthreads();  // every use of tensor memory is over
  if (warp == C::W_MMA) tmem_free(tmem, 512);
}

}  // namespace kvq
