// kvq_rope.cuh -- norm and position rotation of head rows (queries, keys).
//
// A row of d values is held by d/8 lanes, 8 consecutive values (16 bytes)
// each, so a warp works on 32/(d/8) rows of one token at a time.  The mean of
// squares is a butterfly over those lanes; a rotation partner half a rotation
// away lies in another lane of the same row (one shuffle per value), an
// interleaved one in the same lane.  The table row depends on the token alone:
// a warp keeps its 8 cosines and sines in registers and walks over the
// token's heads, so the table costs 1/heads of its size per row.
//
// Bound: bytes (2 d in, 2 d out per row).  8192 tokens of 32 + 32 heads, d = 64,
// bf16: 23.8 us, 5.7 TB/s, 87% of the measured copy rate.
#pragma once

#include "kvq_device.cuh"
#include "kvq_paged_launch.h"

namespace kvq {

// 16-bit pair -> two floats and back (round to nearest even).
template <int DT>
__device__ __forceinline__ float2 pair_to_float2(uint32_t w) {
  if constexpr (DT == kDtF16) {
    return half2_bits_to_float2(w);
  } else {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
}
template <int DT>
__device__ __forceinline__ uint32_t float2_to_pair(float lo, float hi) {
  if constexpr (DT == kDtF16) {
    return float2_to_half2_bits(lo, hi);
  } else {
    return float2_to_bf162_bits(lo, hi);
  }
}

// Records an index out of range in the status word.
__device__ __forceinline__ void flag_bad_index(unsigned* status) {
  atomicOr(status, kPagedBadIndex);
}

constexpr int kRopeThreads = 128;

template <int D, int DT>
__global__ void __launch_bounds__(kRopeThreads) kvq_norm_rope_kernel(const NormRopeArgs a,
                                                                     unsigned* status) {
  constexpr int LPR = D / 8;       // lanes per row
  constexpr int RPW = 32 / LPR;    // rows of a warp's step
  constexpr int U = 4;             // steps whose loads are in flight together
  const int lane = threadIdx.x & 31, sub = lane % LPR;
  const int64_t w = (int64_t(blockIdx.x) * kRopeThreads + threadIdx.x) >> 5;
  const int64_t tok = w / a.chunks;
  const int row0 = int(w - tok * a.chunks) * a.iters * RPW + lane / LPR;
  pdl_wait();  // no global access before the previous kernel completes
  if (tok >= a.n_tokens) return;

  const int half = a.rope.rot_dim / 2;
  float cs[8], sn[8];
  int src = lane;  // lane of the rotation partner
  int64_t pos = 0;
  if (a.positions != nullptr) {
    pos = __ldg(a.positions + tok);
    if (pos < 0) return;  // padding
  }
  if (a.rope.cos_sin != nullptr) {
    if (pos >= a.rope.n_pos) {
      if (lane == 0) flag_bad_index(status);
      return;
    }
    const float* row = a.rope.cos_sin + pos * a.rope.rot_dim;
    const int e = 8 * sub;
    if (a.rope.interleaved) {  // cs, sn of pair i in slots 2i, 2i + 1
      const bool in = e < 2 * half;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float c = in ? __ldg(row + e / 2 + i) : 1.0f;
        const float s = in ? __ldg(row + half + e / 2 + i) : 0.0f;
        cs[2 * i] = cs[2 * i + 1] = c;
        sn[2 * i] = -s;
        sn[2 * i + 1] = s;
      }
    } else {
      const bool lo = e < half, in = e < 2 * half;
      const int i0 = lo ? e : e - half;
      src = in ? (lo ? lane + half / 8 : lane - half / 8) : lane;
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (in) {
          c = __ldg(reinterpret_cast<const float4*>(row + i0 + i));
          s = __ldg(reinterpret_cast<const float4*>(row + half + i0 + i));
        }
        const float sg = lo ? -1.0f : 1.0f;
        cs[i] = c.x, cs[i + 1] = c.y, cs[i + 2] = c.z, cs[i + 3] = c.w;
        sn[i] = sg * s.x, sn[i + 1] = sg * s.y, sn[i + 2] = sg * s.z, sn[i + 3] = sg * s.w;
      }
    }
  }

  auto work = [&](uint4 raw, int r) {
    const bool key = r >= a.n_heads;
    const float* weight = key ? a.k_weight : a.q_weight;
    float x[8];
    const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = pair_to_float2<DT>(in[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
    if (a.q_weight != nullptr || a.k_weight != nullptr) {  // the same in every lane
      float sq = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sq = fmaf(x[i], x[i], sq);
#pragma unroll
      for (int o = 1; o < LPR; o <<= 1) sq += __shfl_xor_sync(kFull, sq, o);
      if (weight != nullptr) {
        const float inv = rsqrtf(sq * (1.0f / D) + a.rope.eps);
        const float4 w0 = __ldg(reinterpret_cast<const float4*>(weight + 8 * sub));
        const float4 w1 = __ldg(reinterpret_cast<const float4*>(weight + 8 * sub) + 1);
        const float wt[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * wt[i];
      }
    }
    if (a.rope.cos_sin != nullptr) {
      float p[8];
      if (a.rope.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = x[i ^ 1];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = __shfl_sync(kFull, x[i], src);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i], cs[i], p[i] * sn[i]);
    }
    if (r < a.n_rows) {
      uint16_t* dst = key ? a.k_out + tok * a.k_out_stride + int64_t(r - a.n_heads) * D
                          : a.q_out + tok * a.q_out_stride + int64_t(r) * D;
      reinterpret_cast<uint4*>(dst)[sub] =
          make_uint4(float2_to_pair<DT>(x[0], x[1]), float2_to_pair<DT>(x[2], x[3]),
                     float2_to_pair<DT>(x[4], x[5]), float2_to_pair<DT>(x[6], x[7]));
    }
  };
  for (int it = 0; it < a.iters; it += U) {
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = row0 + (it + u) * RPW;
      raw[u] = make_uint4(0, 0, 0, 0);
      if (it + u < a.iters && r < a.n_rows) {
        const bool key = r >= a.n_heads;
        const uint16_t* src_row = key ? a.k + tok * a.k_stride + int64_t(r - a.n_heads) * D
                                      : a.q + tok * a.q_stride + int64_t(r) * D;
        // plain loads: the outputs may be the inputs
        raw[u] = reinterpret_cast<const uint4*>(src_row)[sub];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (it + u < a.iters) work(raw[u], row0 + (it + u) * RPW);
  }
  pdl_release();
}

}  // namespace kvq
