// kvq_paged_launch.h -- internal interface between the C-ABI front end of the
// paged cache (kvq_paged_api.cu) and the per-d translation units
// (kvq_paged_d64.cu, ...).  Not part of the public API.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq_launch.h"

namespace kvq {

constexpr int kDtF16 = 0, kDtBF16 = 1;  // kvq_dtype

// Bits of the paged kernels' status words.
constexpr unsigned kPagedTimeout = 1u, kPagedBadIndex = 2u;

struct RopeTable {
  const float* cos_sin;  // [n_pos][rot_dim], or NULL
  int64_t n_pos;
  int rot_dim;
  int interleaved;
  float eps;
};

struct NormRopeArgs {
  const uint16_t *q, *k;
  uint16_t *q_out, *k_out;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;  // elements per token
  const int32_t* positions;
  const float *q_weight, *k_weight;
  RopeTable rope;
  int64_t n_tokens;
  int n_heads, n_rows;  // query heads; query and key heads
  int iters;            // steps of a warp over a token's heads
  int chunks;           // warps per token
};

struct AppendArgs {
  const uint16_t *k, *v;
  int64_t k_stride, v_stride;
  const int64_t* slots;
  const int32_t* positions;
  const float* k_weight;  // NULL: no norm
  RopeTable rope;
  uint8_t *k_packed, *v_packed;
  float *k_scales, *v_scales;
  const int8_t* signs;
  uint16_t *k_hat, *v_hat;  // NULL: not wanted
  int64_t n_tokens, n_slots;
  int n_heads, page_shift, dtype;
};

struct PagedAttnArgs {
  const uint16_t* q;
  uint16_t* out;
  int64_t q_stride, out_stride;
  const int32_t *cu_q, *kv_len, *page_table;
  const uint8_t *k_packed, *v_packed;
  const float *k_scales, *v_scales;
  const int8_t* signs;
  int64_t n_tokens, n_pages, max_pages;
  int n_seqs, n_kv, n_q, page_shift, d, group, window, dtype, rot;
  float qscale;  // sm_scale * log2(e)
  // workspace, cut up by the launcher
  uint8_t* workspace;
  struct JoinInfo* join;
  float* parts;
};

// Rows of an item of the few-rows kernel for this many rows of a sequence and
// KV head: fewer columns cost less of everything, and 16 do not fit shared
// and tensor memory with 4 or 8 groups of a 256-value row.
constexpr int few_rows_item(int d, int group, int64_t rows) {
  return rows <= 4 ? 4 : (rows <= 8 || (d == 256 && group <= 64) ? 8 : 16);
}
constexpr int64_t kMaxBlocks = 148 * 4;  // of the few-rows kernel
constexpr int64_t kMaxChunkBlocks = 148;  // of the many-rows kernel, one an SM
// Up to this many rows of a sequence and KV head the few-rows kernel runs.
// At 30 rows, many- against few-rows kernel, us: 32 sequences of 4096 rows and 8
// heads, bf16 193 / 421 (d = 64) to 407 / 595 (d = 256), fp16 288 / 421 to 661 / 596;
// one sequence and head, bf16 19.3 / 22.7 (d = 64) to 43.9 / 31.4 (d = 256), fp16 24.2
// / 22.7 to 60.5 / 31.4.  The limit favours large batches.
constexpr int64_t kFewRows = 16;
constexpr int64_t attn_workspace(int d, int64_t rows) {
  const int64_t slots = rows <= kFewRows ? kMaxBlocks * 2 * 16
                                         : kMaxChunkBlocks * 2 * (d == 256 ? 128 : 256);
  return kMaxBlocks * 32 + slots * (int64_t(d) + 2) * 4;
}

// Implemented once per d in the matching translation unit.
template <int D>
cudaError_t launch_norm_rope(int dtype, const NormRopeArgs& a, int sm_count, cudaStream_t stream);
template <int D>
cudaError_t launch_append(int rot, int group, const AppendArgs& a, int sm_count,
                          cudaStream_t stream);
template <int D>
cudaError_t launch_paged_attn(const PagedAttnArgs& a, int max_q_len, int sm_count,
                              cudaStream_t stream);
template <int D>
cudaError_t read_paged_status(uint32_t* value, bool clear);

}  // namespace kvq
