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

// ------------------------------------------------- attention, one row a warp ---

// A warp per (token, query head): scores by a shuffle reduction per row.
template <int D, int ROT, int DT>
__global__ void __launch_bounds__(kWideThreads) kvq_paged_attn_simple_kernel(const PagedAttnArgs a,
                                                                             unsigned* status) {
  using P = Wide<D, ROT>;
  const int lane = threadIdx.x & 31;
  const int64_t gw = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  pdl_wait();
  const int heads = a.n_kv * a.n_q;
  const int64_t tok = gw / heads;
  const int h = int(gw - tok * heads), kvh = h / a.n_q;
  if (tok >= a.n_tokens) return;
  int lo = -1;
  int64_t c0 = 0, c1 = 0, len = 0;
  for (int s = 0; s < a.n_seqs; ++s) {
    const int64_t b = __ldg(a.cu_q + s), e = __ldg(a.cu_q + s + 1), n = __ldg(a.kv_len + s);
    if (b < 0 || e < b || e > a.n_tokens || n < 0 || n > (a.max_pages << a.page_shift)) {
      if (lane == 0) flag_bad_index(status);
    } else if (tok >= b && tok < e) {
      lo = s, c0 = b, c1 = e, len = n;
    }
  }
  if (lo < 0) return;  // rows of no sequence
  WideLane<D, ROT> L;
  L.init(a.signs, lane);
  const uint32_t* src = reinterpret_cast<const uint32_t*>(a.q + tok * a.q_stride + int64_t(h) * D);
  f2 z[P::C];
#pragma unroll
  for (int j = 0; j < P::C; ++j) {
    const float2 f = pair_to_float2<DT>(__ldg(src + wide_word<D, ROT>(lane, j)) ^ L.mask[j]);
    z[j] = mk2(f.x, f.y);
  }
  float Q[P::W], acc[P::W];
  wide_rotate_fwd<D, ROT>(z, L, Q);
#pragma unroll
  for (int w = 0; w < P::W; ++w) Q[w] *= P::KAPPA * a.qscale, acc[w] = 0.0f;
  const int64_t p = len - (c1 - c0) + (tok - c0);
  const int64_t t0 = a.window > 0 && p - a.window + 1 > 0 ? p - a.window + 1 : 0;
  const int grp = L.k2 * P::W / a.group, ng = D / a.group;
  float m = -INFINITY, l = 0.0f;
  for (int64_t t = t0; t <= p; ++t) {
    const int64_t page = __ldg(a.page_table + lo * a.max_pages + (t >> a.page_shift));
    if (page < 0 || page >= a.n_pages) {
      if (lane == 0) flag_bad_index(status);
      continue;
    }
    const int64_t row = ((page * a.n_kv + kvh) << a.page_shift) + (t & ((1 << a.page_shift) - 1));
    float Y[P::W];
    wide_dequant<D, ROT>(wide_load_code<D, ROT>(a.k_packed + row * (D / 2), L),
                         __ldg(a.k_scales + row * ng + grp), Y);
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < P::W; ++w) s = fmaf(Q[w], Y[w], s);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) s += __shfl_xor_sync(kFull, s, o);
    s *= 1.0f / P::KAPPA;
    const float mn = fmaxf(m, s), f = exp2f(m - mn), e = exp2f(s - mn);
    wide_dequant<D, ROT>(wide_load_code<D, ROT>(a.v_packed + row * (D / 2), L),
                         __ldg(a.v_scales + row * ng + grp), Y);
    l = fmaf(l, f, e);
    m = mn;
#pragma unroll
    for (int w = 0; w < P::W; ++w) acc[w] = fmaf(acc[w], f, e * Y[w]);
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
  for (int w = 0; w < P::W; ++w) acc[w] *= inv;  // KAPPA is in already
  wide_rotate_inv<D, ROT>(acc, L, z);
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + tok * a.out_stride + int64_t(h) * D);
#pragma unroll
  for (int j = 0; j < P::C; ++j)
    dst[wide_word<D, ROT>(lane, j)] = float2_to_pair<DT>(lo2(z[j]), hi2(z[j])) ^ L.mask[j];
}

}  // namespace kvq
