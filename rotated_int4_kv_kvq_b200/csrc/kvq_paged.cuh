// kvq_paged.cuh -- appending new keys and values to the paged int4 cache.
//
// One warp per vector (the layout of kvq_wide.cuh).  The key's norm and
// position rotation happen in registers on the way to the forward rotation,
// so a key crosses memory once: 2 d bytes in, d/2 + 4 d/g out.
#pragma once

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

}  // namespace kvq
