// kvq_paged.cuh -- appending new keys and values to the paged int4 cache.
//
// The key's norm and position rotation happen on the way to the forward
// rotation, so a key crosses memory once: 2 d bytes in, d/2 + 4 d/g out (and
// 2 d more where the dequantized rows are wanted).  Two kernels with the same
// results but for rounding: one warp per vector (the layout of kvq_wide.cuh) for
// few rows, where the length of one row's chain is the time, and one thread (d =
// 256: two) per vector (kvq_codec.cuh) for many, where instructions are: the
// warp-wide transform spends most of its own on shuffles.  With norm and rotation,
// d = 128, with dequantized rows and without: 8180 rows 8.5 and 6.5 us (a warp a
// row), 262,144 rows 121 and 98 us (a thread a row; bytes alone would take 24.5, the
// codec's own forward and inverse of as many contiguous rows 18 and 19.  4.7
// thousand instructions a warp and 32 rows, issued in 36% of the clocks: 168
// registers leave 12 warps an SM, too few to hide the chain of each).
#pragma once

#include "kvq_codec.cuh"
#include "kvq_rope.cuh"
#include "kvq_wide.cuh"

namespace kvq {

// The lane's pairs of a row (before the sign flip), as the rotation wants
// them: SRFT word l + 32 j, SRHT word C l + j.
template <int D, int ROT>
__device__ __forceinline__ int wide_word(int lane, int j) {
  return ROT == kRotSRFT ? lane + 32 * j : Wide<D, ROT>::C * lane + j;
}

template <int D, int G, int ROT, int DT>
__global__ void __launch_bounds__(kWideThreads) kvq_append_wide_kernel(const AppendArgs a,
                                                                       unsigned* status) {
  using P = Wide<D, ROT>;
  constexpr int NG = D / G;
  const int lane = threadIdx.x & 31;
  const int64_t gw = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t nw = (int64_t(gridDim.x) * blockDim.x) >> 5;
  pdl_wait();  // no global access before the previous kernel completes
  WideLane<D, ROT> L;
  L.init(a.signs, lane);
  const int per_token = 2 * a.n_heads;  // keys, then values
  for (int64_t it = gw; it < a.n_tokens * per_token; it += nw) {
    const int64_t tok = it / per_token;
    const int r = int(it - tok * per_token);
    const bool key = r < a.n_heads;
    const int head = key ? r : r - a.n_heads;
    const int64_t slot = __ldg(a.slots + tok);
    if (slot < 0) continue;
    if (slot >= a.n_slots) {
      if (lane == 0) flag_bad_index(status);
      continue;
    }
    const float* table = nullptr;
    if (a.rope.cos_sin != nullptr) {  // a token outside the table is skipped whole
      const int64_t pos = __ldg(a.positions + tok);
      if (pos < 0 || pos >= a.rope.n_pos) {
        if (lane == 0) flag_bad_index(status);
        continue;
      }
      if (key) table = a.rope.cos_sin + pos * a.rope.rot_dim;
    }
    const uint32_t* src = reinterpret_cast<const uint32_t*>(
        key ? a.k + tok * a.k_stride + int64_t(head) * D
            : a.v + tok * a.v_stride + int64_t(head) * D);
    f2 z[P::C];
#pragma unroll
    for (int j = 0; j < P::C; ++j) {
      const float2 f = pair_to_float2<DT>(__ldg(src + wide_word<D, ROT>(lane, j)));
      z[j] = mk2(f.x, f.y);
    }
    if (key && (a.k_weight != nullptr || table != nullptr)) {
      float inv = 1.0f;
      if (a.k_weight != nullptr) {
        float sq = 0.0f;
#pragma unroll
        for (int j = 0; j < P::C; ++j)
          sq = fmaf(lo2(z[j]), lo2(z[j]), fmaf(hi2(z[j]), hi2(z[j]), sq));
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) sq += __shfl_xor_sync(kFull, sq, o);
        inv = rsqrtf(sq * (1.0f / D) + a.rope.eps);
      }
      const float2* wt = reinterpret_cast<const float2*>(a.k_weight);
#pragma unroll
      for (int j = 0; j < P::C; ++j) {
        const int w = wide_word<D, ROT>(lane, j);
        float x = lo2(z[j]), y = hi2(z[j]);
        if (wt != nullptr) {
          const float2 f = __ldg(wt + w);
          x = x * inv * f.x;
          y = y * inv * f.y;
        }
        const int hw = a.rope.rot_dim / 4;  // words in half a rotation
        if (table != nullptr && w < 2 * hw) {
          if (a.rope.interleaved) {
            const float c = __ldg(table + w), s = __ldg(table + 2 * hw + w);
            const float nx = fmaf(x, c, -(y * s)), ny = fmaf(x, s, y * c);
            x = nx, y = ny;
          } else {
            const bool low = w < hw;
            const int pw = low ? w + hw : w - hw, tw = low ? w : pw;
            float2 p = pair_to_float2<DT>(__ldg(src + pw));
            if (wt != nullptr) {
              const float2 f = __ldg(wt + pw);
              p.x = p.x * inv * f.x;
              p.y = p.y * inv * f.y;
            }
            const float2 c = __ldg(reinterpret_cast<const float2*>(table) + tw);
            float2 s = __ldg(reinterpret_cast<const float2*>(table) + hw + tw);
            if (low) s.x = -s.x, s.y = -s.y;
            x = fmaf(x, c.x, p.x * s.x);
            y = fmaf(y, c.y, p.y * s.y);
          }
        }
        z[j] = mk2(x, y);
      }
    }
#pragma unroll
    for (int j = 0; j < P::C; ++j)
      z[j] = mk2(__uint_as_float(__float_as_uint(lo2(z[j])) ^ (L.mask[j] << 16)),
                 __uint_as_float(__float_as_uint(hi2(z[j])) ^ (L.mask[j] & 0x80000000u)));
    float Y[P::W];
    wide_rotate_fwd<D, ROT>(z, L, Y);
    const int64_t page = slot >> a.page_shift;
    const int64_t row = ((page * a.n_heads + head) << a.page_shift) + (slot - (page << a.page_shift));
    uint32_t code;
    float s;
    wide_quantize_rotated<D, G, ROT>(Y, (key ? a.k_packed : a.v_packed) + row * (D / 2),
                                     (key ? a.k_scales : a.v_scales) + row * NG, L, code, s);
    uint16_t* hat = key ? a.k_hat : a.v_hat;
    if (hat != nullptr) {
      wide_dequant<D, ROT>(code, s, Y);
      wide_rotate_inv<D, ROT>(Y, L, z);
      uint32_t* dst = reinterpret_cast<uint32_t*>(hat + (tok * a.n_heads + head) * D);
#pragma unroll
      for (int j = 0; j < P::C; ++j)
        dst[wide_word<D, ROT>(lane, j)] = float2_to_pair<DT>(lo2(z[j]), hi2(z[j])) ^ L.mask[j];
    }
  }
  pdl_release();
}

// ------------------------------------------------- many rows: a thread a row ---

constexpr int kAppendWarps = 4;
constexpr int kAppendThreads = 32 * kAppendWarps;
template <int D>
constexpr int append_tile_bytes() {  // a warp's rows in fp32
  return 32 / tpv_of(D) * D * 4;
}

// A warp takes the keys, or the values, of one head of 32 (d = 256: 16)
// consecutive tokens.  First the rows are loaded 16 bytes a lane, normed and
// rotated by position there (the way of kvq_norm_rope_kernel) and left in
// shared memory in fp32; then each thread (pair) takes a row through rotation,
// quantization and, if wanted, back.
template <int D, int G, int ROT>
__global__ void __launch_bounds__(kAppendThreads, 3) kvq_append_tile_kernel(const AppendArgs a,
                                                                            unsigned* status) {
  using C = Cfg<D, ROT, tpv_of(D)>;
  using Gr = Groups<C, G>;
  constexpr int NG = D / G, VPW = C::VPW, LPR = D / 8, RPS = 32 / LPR;
  extern __shared__ __align__(16) uint8_t append_smem[];
  __shared__ uint32_t s_in[2 * 64], s_out[2 * 64];  // sign masks by thread of a pair
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % LPR;
  const uint32_t tile = smem_u32(append_smem) + warp * append_tile_bytes<D>();
  const bool bf16 = a.dtype == kDtBF16;
  pdl_wait();  // no global access before the previous kernel completes
  for (int i = threadIdx.x; i < C::TPV * C::NW; i += kAppendThreads) {
    s_in[i] = load_mask_word<C>(a.signs, i / C::NW, i % C::NW);
    s_out[i] = store_mask_word<C>(a.signs, i / C::NW, i % C::NW);
  }
  __syncthreads();
  auto at = [&](int r, int c) {  // 16-byte piece c of row r
    return tile + uint32_t(r) * (D * 4) + ((uint32_t(c) ^ uint32_t(r & 7)) << 4);
  };
  const int half = a.rope.rot_dim / 2;
  const int64_t per = (a.n_tokens + VPW - 1) / VPW;  // tiles of a head
  const int64_t tiles = per * 2 * a.n_heads;
  for (int64_t it = int64_t(blockIdx.x) * kAppendWarps + warp; it < tiles;
       it += int64_t(gridDim.x) * kAppendWarps) {
    // neighbouring warps take the heads of the same tokens: they share table rows
    const int r = int(it % (2 * a.n_heads));
    const int64_t tok0 = it / (2 * a.n_heads) * VPW;
    const bool key = r < a.n_heads;
    const int head = key ? r : r - a.n_heads;
    // lane j: where token tok0 + j goes, -1 for nowhere, and its position
    int64_t slot = -1;
    int pos = 0;
    if (lane < VPW && tok0 + lane < a.n_tokens) {
      slot = __ldg(a.slots + tok0 + lane);
      if (slot >= a.n_slots) {
        flag_bad_index(status);
        slot = -1;
      }
      if (a.rope.cos_sin != nullptr && slot >= 0) {
        pos = __ldg(a.positions + tok0 + lane);
        if (pos < 0 || pos >= a.rope.n_pos) {
          flag_bad_index(status);
          slot = -1;
          pos = 0;  // the lanes of a skipped row still read the table: its first row
        }
      }
    }
    const uint32_t there = __ballot_sync(kFull, slot >= 0);
    // ---- rows -> fp32 in shared memory ----
    const uint16_t* base = key ? a.k + int64_t(head) * D : a.v + int64_t(head) * D;
    const int64_t stride = key ? a.k_stride : a.v_stride;
    const bool norm = key && a.k_weight != nullptr, rope = key && a.rope.cos_sin != nullptr;
    float wt[8];
    if (norm) {
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const float4 w = __ldg(reinterpret_cast<const float4*>(a.k_weight + 8 * sub + i));
        wt[i] = w.x, wt[i + 1] = w.y, wt[i + 2] = w.z, wt[i + 3] = w.w;
      }
    }
    __syncwarp();  // the rows before have left the tile
    constexpr int U = 8;  // loads in flight
#pragma unroll 1
    for (int s0 = 0; s0 < VPW / RPS; s0 += U) {
      uint4 raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int row = (s0 + u) * RPS + lane / LPR;
        raw[u] = make_uint4(0, 0, 0, 0);
        if (there >> row & 1u)
          raw[u] = __ldg(reinterpret_cast<const uint4*>(base + (tok0 + row) * stride) + sub);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int row = (s0 + u) * RPS + lane / LPR;
        float x[8];
        const uint32_t in[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = bf16 ? pair_to_float2<kDtBF16>(in[i]) : pair_to_float2<kDtF16>(in[i]);
          x[2 * i] = f.x;
          x[2 * i + 1] = f.y;
        }
        if (norm) {
          float sq = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) sq = fmaf(x[i], x[i], sq);
#pragma unroll
          for (int o = 1; o < LPR; o <<= 1) sq += __shfl_xor_sync(kFull, sq, o);
          const float inv = rsqrtf(sq * (1.0f / D) + a.rope.eps);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * wt[i];
        }
        if (rope) {
          const int e = 8 * sub, p = __shfl_sync(kFull, pos, row);
          const float* tab = a.rope.cos_sin + int64_t(p) * a.rope.rot_dim;
          const bool in_rot = e < 2 * half;
          if (a.rope.interleaved) {
            if (in_rot) {
              const float4 c = __ldg(reinterpret_cast<const float4*>(tab + e / 2));
              const float4 s = __ldg(reinterpret_cast<const float4*>(tab + half + e / 2));
              const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float p0 = x[2 * i], p1 = x[2 * i + 1];
                x[2 * i] = fmaf(p0, cs[i], -(p1 * sn[i]));
                x[2 * i + 1] = fmaf(p0, sn[i], p1 * cs[i]);
              }
            }
          } else {
            const bool lo = e < half;
            const int src = in_rot ? (lo ? lane + half / 8 : lane - half / 8) : lane;
            float q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = __shfl_sync(kFull, x[i], src);
            if (in_rot) {
              const int i0 = lo ? e : e - half;
              const float sg = lo ? -1.0f : 1.0f;
#pragma unroll
              for (int i = 0; i < 8; i += 4) {
                const float4 c = __ldg(reinterpret_cast<const float4*>(tab + i0 + i));
                const float4 s = __ldg(reinterpret_cast<const float4*>(tab + half + i0 + i));
                x[i] = fmaf(x[i], c.x, q[i] * (sg * s.x));
                x[i + 1] = fmaf(x[i + 1], c.y, q[i + 1] * (sg * s.y));
                x[i + 2] = fmaf(x[i + 2], c.z, q[i + 2] * (sg * s.z));
                x[i + 3] = fmaf(x[i + 3], c.w, q[i + 3] * (sg * s.w));
              }
            }
          }
        }
        sts128(at(row, 2 * sub), __float_as_uint(x[0]), __float_as_uint(x[1]),
               __float_as_uint(x[2]), __float_as_uint(x[3]));
        sts128(at(row, 2 * sub + 1), __float_as_uint(x[4]), __float_as_uint(x[5]),
               __float_as_uint(x[6]), __float_as_uint(x[7]));
      }
    }
    __syncwarp();
    // the next tile's rows into L2 while this one is worked on
    if (const int64_t nx = it + int64_t(gridDim.x) * kAppendWarps; nx < tiles) {
      const int nr = int(nx % (2 * a.n_heads));
      const bool nk = nr < a.n_heads;
      const int64_t ntok = nx / (2 * a.n_heads) * VPW + lane / C::TPV;
      if (ntok < a.n_tokens) {
        const uint16_t* p = nk ? a.k + ntok * a.k_stride + int64_t(nr) * D
                               : a.v + ntok * a.v_stride + int64_t(nr - a.n_heads) * D;
#pragma unroll
        for (int j = 0; j < D / 64 / C::TPV; ++j)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(p + (lane % C::TPV + j * C::TPV) * 64));
      }
    }
    // ---- a row a thread (pair): rotate, quantize ----
    const int row = lane / C::TPV, t = lane % C::TPV;
    f2 u[C::NW], Y[C::P];
    auto flip = [&](uint32_t x, uint32_t y, int j) {
      const uint32_t m = s_in[t * C::NW + j];
      return mk2(__uint_as_float(x ^ (m << 16)), __uint_as_float(y ^ (m & 0x80000000u)));
    };
#pragma unroll
    for (int c = 0; c < C::NW / 2; ++c) {
      if constexpr (C::PAIR_RFFT) {  // samples 4 j + t, 4 j + 2 + t of the whole row
        const uint4 v0 = lds128(at(row, 2 * c)), v1 = lds128(at(row, 2 * c + 1));
        u[2 * c] = flip(t ? v0.y : v0.x, t ? v0.w : v0.z, 2 * c);
        u[2 * c + 1] = flip(t ? v1.y : v1.x, t ? v1.w : v1.z, 2 * c + 1);
      } else {
        const uint4 v = lds128(at(row, t * (C::NW / 2) + c));
        // (the mask's low half flips by its bit 15; the rest of it is zero)
        u[2 * c] = flip(v.x, v.y, 2 * c);
        u[2 * c + 1] = flip(v.z, v.w, 2 * c + 1);
      }
    }
    rotate_fwd<C>(u, t, Y);
    uint32_t qw[C::NQ];
    float sc[Gr::NL];
    quantize<C, G>(Y, qw, sc, t);
    const int64_t my = __shfl_sync(kFull, slot, row);
    const bool write = my >= 0;
    if (write) {
      const int64_t page = my >> a.page_shift;
      const int64_t dst =
          ((page * a.n_heads + head) << a.page_shift) + (my - (page << a.page_shift));
      uint8_t* codes = (key ? a.k_packed : a.v_packed) + dst * (D / 2);
      float* scales = (key ? a.k_scales : a.v_scales) + dst * NG;
      constexpr int RUN = C::TPV == 1 ? C::NQ : C::NQ / 2;  // words in order
#pragma unroll
      for (int h = 0; h < C::NQ / RUN; ++h) {
        uint4* to = reinterpret_cast<uint4*>(codes + global_y<C>(t, h * (C::E / 2)) / 2);
#pragma unroll
        for (int j = 0; j < RUN; j += 4)
          to[j / 4] = make_uint4(qw[h * RUN + j], qw[h * RUN + j + 1], qw[h * RUN + j + 2],
                                 qw[h * RUN + j + 3]);
      }
#pragma unroll
      for (int g = 0; g < Gr::NL; ++g)
        if (writes_scale<C, G>(t, g)) scales[global_group<C, G>(t, g)] = sc[g];
    }
    // ---- and back ----
    uint16_t* hat = key ? a.k_hat : a.v_hat;
    if (hat != nullptr) {
      dequantize<C, G>(qw, sc, Y);
      uint32_t xw[C::NW];
      rotate_inv<C>(Y, t, xw, 0, bf16);
      __syncwarp();  // both threads of a pair have read their row
#pragma unroll
      for (int c = 0; c < C::NW / 4; ++c) {
        const uint32_t* m = s_out + t * C::NW + 4 * c;
        sts128(at(row, t * (C::NW / 4) + c), xw[4 * c] ^ m[0], xw[4 * c + 1] ^ m[1],
               xw[4 * c + 2] ^ m[2], xw[4 * c + 3] ^ m[3]);
      }
      __syncwarp();
#pragma unroll 4
      for (int s = 0; s < VPW / RPS; ++s) {
        const int rr = s * RPS + lane / LPR;
        const uint4 v = lds128(at(rr, sub));
        if (there >> rr & 1u)
          reinterpret_cast<uint4*>(hat + ((tok0 + rr) * a.n_heads + head) * D)[sub] = v;
      }
    }
  }
  pdl_release();
}

}  // namespace kvq
