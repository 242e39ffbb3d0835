// kvq_paged_inst.cuh -- host-side launchers of the paged-cache kernels of one
// vector length d.  Included by exactly one translation unit per d
// (kvq_paged_d64.cu, ...).
#pragma once

#include <algorithm>
#include <mutex>
#include <utility>

#include "kvq_paged.cuh"
#include "kvq_pchunk.cuh"
#include "kvq_pdecode.cuh"
#include "kvq_paged_launch.h"

namespace kvq {

// Status word of this translation unit's kernels, one per device context.
// Bit 0: a bounded wait ran out; bit 1: an index out of range was skipped.
static __device__ unsigned g_paged_status;

namespace detail {

// Device address of g_paged_status on the current device (looked up once).
inline cudaError_t paged_status_ptr(unsigned** out) {
  constexpr int kMax = 64;
  static unsigned* ptrs[kMax];
  static std::mutex mu;
  int dev;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMax) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> g(mu);
  if (ptrs[dev] == nullptr) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_paged_status);
    if (e != cudaSuccess) return e;
    ptrs[dev] = static_cast<unsigned*>(p);
  }
  *out = ptrs[dev];
  return cudaSuccess;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_paged_2d(void (*kern)(KArgs...), int64_t grid, int rows, int threads, int smem,
                            cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid), unsigned(rows), 1);
  cfg.blockDim = dim3(unsigned(threads), 1, 1);
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = KVQ_PDL ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_paged(void (*kern)(KArgs...), int64_t grid, int threads, int smem,
                         cudaStream_t stream, Args&&... args) {
  return launch_paged_2d(kern, grid, 1, threads, smem, stream, std::forward<Args>(args)...);
}

// Opts a kernel into its shared memory (once per kernel and device).
template <auto Kern>
cudaError_t paged_setup(int smem) {
  constexpr int kMax = 64;
  static bool done[kMax];
  static std::mutex mu;
  int dev;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMax) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> g(mu);
  if (!done[dev]) {
    e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  return cudaSuccess;
}

// Appending: rows of a call from which a thread (pair) a row beats a warp a row.
// Norm, rotation and dequantized rows, one warp against one thread a row, us:
// d = 64 at 8192 rows 6.2 against 8.5, at 16384 10.4 against 8.8, at 262144 163
// against 60; d = 128 at 16384 13.8 against 16.8, at 32768 24.0 against 18.2, at
// 262144 202 against 124; d = 256 at 8192 12.9 against 19.5, at 16384 22.3
// against 20.9, at 65536 98 against 81.
constexpr int64_t append_tile_rows(int d) { return d == 64 ? 12288 : (d == 128 ? 20480 : 14336); }

template <int D, int G, int ROT>
cudaError_t append_one(const AppendArgs& a, int sm_count, cudaStream_t stream, unsigned* st) {
  const int64_t rows = a.n_tokens * 2 * a.n_heads;
  if (rows >= append_tile_rows(D)) {
    constexpr auto kern = kvq_append_tile_kernel<D, G, ROT>;
    constexpr int smem = kAppendWarps * append_tile_bytes<D>();
    cudaError_t e = paged_setup<kern>(smem);
    if (e != cudaSuccess) return e;
    constexpr int vpw = vpw_of(D);
    const int64_t tiles = (a.n_tokens + vpw - 1) / vpw * 2 * a.n_heads;
    const int64_t grid =
        std::min<int64_t>((tiles + kAppendWarps - 1) / kAppendWarps, int64_t(sm_count) * 3);
    return launch_paged(kern, grid, kAppendThreads, smem, stream, a, st);
  }
  const int64_t grid =
      std::max<int64_t>(1, std::min<int64_t>((rows + 3) / 4, int64_t(sm_count) * 12));
  return a.dtype == kDtF16
             ? launch_paged(kvq_append_wide_kernel<D, G, ROT, kDtF16>, grid, kWideThreads, 0, stream, a, st)
             : launch_paged(kvq_append_wide_kernel<D, G, ROT, kDtBF16>, grid, kWideThreads, 0, stream, a, st);
}

template <int D, int ROT>
cudaError_t append_group(const AppendArgs& a, int group, int sm_count, cudaStream_t stream,
                         unsigned* st) {
  switch (group) {
    case 32: return append_one<D, 32, ROT>(a, sm_count, stream, st);
    case 64: return append_one<D, 64, ROT>(a, sm_count, stream, st);
    case 128:
      if constexpr (D >= 128) return append_one<D, 128, ROT>(a, sm_count, stream, st);
      break;
    case 256:
      if constexpr (D >= 256) return append_one<D, 256, ROT>(a, sm_count, stream, st);
  }
  return cudaErrorInvalidValue;
}

template <int D, int R, int RPB, int WPR>
cudaError_t launch_join(const PagedAttnArgs& a, int64_t grid, cudaStream_t stream) {
  return a.rot == kRotSRFT ? launch_paged_2d(kvq_paged_join_kernel<D, R, kRotSRFT, RPB, WPR>, grid,
                                             R / RPB, 32 * RPB * WPR, 0, stream, a)
                           : launch_paged_2d(kvq_paged_join_kernel<D, R, kRotSRHT, RPB, WPR>, grid,
                                             R / RPB, 32 * RPB * WPR, 0, stream, a);
}

template <int D, int R, int NG>
cudaError_t few_rows(const PagedAttnArgs& args, int sm_count, cudaStream_t stream, unsigned* st) {
  using C = Pd<D, R, NG>;
  constexpr auto kern = kvq_paged_decode_kernel<D, R, NG>;
  cudaError_t e = paged_setup<kern>(C::SMEM);
  if (e != cudaSuccess) return e;
  // no more blocks than can be resident at once, or than there can be units
  const int64_t items = (args.n_tokens * args.n_q + R - 1) / R + args.n_seqs;
  const int64_t tiles = (args.max_pages << args.page_shift) / C::KT + 1;
  int64_t grid = std::min<int64_t>(int64_t(sm_count) * C::BLOCKS, kMaxBlocks);
  if (items * args.n_kv < grid) grid = std::min<int64_t>(grid, items * args.n_kv * std::min<int64_t>(tiles, grid));
  PagedAttnArgs a = args;
  static_assert(sizeof(JoinInfo) <= 32, "workspace");
  a.join = reinterpret_cast<JoinInfo*>(a.workspace);
  a.parts = reinterpret_cast<float*>(a.workspace + kMaxBlocks * 32);
  e = launch_paged(kern, grid, kPdThreads, C::SMEM, stream, a, st);
  if (e != cudaSuccess) return e;
  return launch_join<D, R, 4, 4>(a, grid, stream);
}

template <int D, int NG, bool TWO>
cudaError_t many_rows_one(const PagedAttnArgs& args, int sm_count, cudaStream_t stream, unsigned* st) {
  using C = Pc<D, NG, TWO>;
  constexpr auto kern = kvq_paged_chunk_kernel<D, NG, TWO>;
  cudaError_t e = paged_setup<kern>(C::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t items = (args.n_tokens * args.n_q + C::M - 1) / C::M + args.n_seqs;
  const int64_t tiles = (args.max_pages << args.page_shift) / C::KT + 1;
  int64_t grid = std::min<int64_t>(sm_count, kMaxChunkBlocks);
  if (items * args.n_kv < grid)
    grid = std::min<int64_t>(grid, items * args.n_kv * std::min<int64_t>(tiles, grid));
  PagedAttnArgs a = args;
  a.join = reinterpret_cast<JoinInfo*>(a.workspace);
  a.parts = reinterpret_cast<float*>(a.workspace + kMaxBlocks * 32);
  e = launch_paged(kern, grid, C::THREADS, C::SMEM, stream, a, st);
  if (e != cudaSuccess) return e;
  return launch_join<D, C::M, 8, 1>(a, grid, stream);
}

template <int D, int NG>
cudaError_t many_rows(const PagedAttnArgs& a, int sm_count, cudaStream_t stream, unsigned* st) {
  return a.dtype == kDtF16 ? many_rows_one<D, NG, true>(a, sm_count, stream, st)
                           : many_rows_one<D, NG, false>(a, sm_count, stream, st);
}

template <int D>
cudaError_t many_rows_group(const PagedAttnArgs& a, int sm_count, cudaStream_t stream,
                            unsigned* st) {
  switch (D / a.group) {
    case 1: return many_rows<D, 1>(a, sm_count, stream, st);
    case 2: return many_rows<D, 2>(a, sm_count, stream, st);
    case 4:
      if constexpr (D >= 128) return many_rows<D, 4>(a, sm_count, stream, st);
      break;
    case 8:
      if constexpr (D >= 256) return many_rows<D, 8>(a, sm_count, stream, st);
  }
  return cudaErrorInvalidValue;
}

template <int D, int R>
cudaError_t few_rows_group(const PagedAttnArgs& a, int sm_count, cudaStream_t stream,
                           unsigned* st) {
  switch (D / a.group) {
    case 1: return few_rows<D, R, 1>(a, sm_count, stream, st);
    case 2: return few_rows<D, R, 2>(a, sm_count, stream, st);
    case 4:
      if constexpr (D == 128 || (D == 256 && R <= 8)) return few_rows<D, R, 4>(a, sm_count, stream, st);
      break;
    case 8:
      if constexpr (D >= 256 && R <= 8) return few_rows<D, R, 8>(a, sm_count, stream, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace detail

template <int D>
cudaError_t launch_norm_rope(int dtype, const NormRopeArgs& args, int sm_count,
                             cudaStream_t stream) {
  unsigned* st;
  cudaError_t e = detail::paged_status_ptr(&st);
  if (e != cudaSuccess) return e;
  NormRopeArgs a = args;
  constexpr int RPW = 32 / (D / 8);
  const int steps = (a.n_rows + RPW - 1) / RPW;  // of a warp over one token
  // One warp walks over a token's heads (the table row is loaded once) as
  // long as that leaves 16 warps for every SM; fewer heads a warp otherwise.
  const int64_t want = int64_t(sm_count) * 16;
  a.iters = int(std::min<int64_t>(steps, std::max<int64_t>(1, a.n_tokens * steps / want)));
  a.chunks = (steps + a.iters - 1) / a.iters;
  const int64_t warps = a.n_tokens * a.chunks;
  const int64_t grid = (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  return dtype == kDtF16
             ? detail::launch_paged(kvq_norm_rope_kernel<D, kDtF16>, grid, kRopeThreads, 0, stream, a, st)
             : detail::launch_paged(kvq_norm_rope_kernel<D, kDtBF16>, grid, kRopeThreads, 0, stream, a, st);
}

template <int D>
cudaError_t launch_append(int rot, int group, const AppendArgs& a, int sm_count,
                          cudaStream_t stream) {
  unsigned* st;
  cudaError_t e = detail::paged_status_ptr(&st);
  if (e != cudaSuccess) return e;
  return rot == kRotSRFT ? detail::append_group<D, kRotSRFT>(a, group, sm_count, stream, st)
                         : detail::append_group<D, kRotSRHT>(a, group, sm_count, stream, st);
}

template <int D>
cudaError_t launch_paged_attn(const PagedAttnArgs& a, int max_q_len, int sm_count,
                              cudaStream_t stream) {
  unsigned* st;
  cudaError_t e = detail::paged_status_ptr(&st);
  if (e != cudaSuccess) return e;
  if (int64_t(max_q_len) * a.n_q > kFewRows)
    return detail::many_rows_group<D>(a, sm_count, stream, st);
  const int r = few_rows_item(D, a.group, int64_t(max_q_len) * a.n_q);
  if (r == 4) return detail::few_rows_group<D, 4>(a, sm_count, stream, st);
  return r == 8 ? detail::few_rows_group<D, 8>(a, sm_count, stream, st)
                : detail::few_rows_group<D, 16>(a, sm_count, stream, st);
}

template <int D>
cudaError_t read_paged_status(uint32_t* value, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_paged_status, sizeof(*value));
  const uint32_t zero = 0;
  if (e == cudaSuccess && clear && *value != 0)
    e = cudaMemcpyToSymbol(g_paged_status, &zero, sizeof(zero));
  return e;
}

}  // namespace kvq
