// kvq_sched.cuh -- how attention over the paged cache is divided among blocks.
//
// An item is one tile of up to M query rows (row = token * n_q + query) of a
// sequence and a KV head; it costs as many units as it has tiles of KT cached
// rows to attend (one, for rows that attend nothing: their zeros have to be
// written).  The units of all items, in order of (sequence, head, row tile),
// are cut into equal runs, one a block, so that ragged lengths and few rows
// alike load every SM.  An item that several blocks share leaves a partial
// result of each, and a second kernel joins them.  Lengths live on the device,
// so each block finds its run itself.
#pragma once

#include "kvq_rope.cuh"

namespace kvq {

struct SeqInfo {
  int c0, n, len;  // first token, new tokens, cached rows; n = 0: nothing to do
};

__device__ __forceinline__ SeqInfo load_seq(const PagedAttnArgs& a, int s, unsigned* status) {
  const int b = __ldg(a.cu_q + s), e = __ldg(a.cu_q + s + 1), len = __ldg(a.kv_len + s);
  if (b < 0 || e < b || e > a.n_tokens || len < 0 || len > (a.max_pages << a.page_shift)) {
    if (status != nullptr) flag_bad_index(status);
    return SeqInfo{0, 0, 0};
  }
  return SeqInfo{b, e - b, len};
}

// Row tile qt: the cached rows that some query of it attends, lo .. hi - 1 (none if
// hi <= lo), and their tiles, the first and their number.  What the other rows hold,
// and whether their pages are there, must not matter.  (32-bit arithmetic: rows,
// positions and lengths are below 2^31.)
struct ItemTiles {
  int lo, hi, first, count;
};
template <int M, int KT>
__device__ __forceinline__ ItemTiles item_tiles(const PagedAttnArgs& a, const SeqInfo& q, int qt) {
  const unsigned row = unsigned(qt) * M, rows = unsigned(q.n) * unsigned(a.n_q);
  const unsigned last = min(rows, row + M) - 1;
  const int p0 = q.len - q.n + int(row / unsigned(a.n_q));
  ItemTiles t;
  t.hi = q.len - q.n + int(last / unsigned(a.n_q)) + 1;
  t.lo = a.window > 0 ? max(p0 - a.window + 1, 0) : 0;
  if (t.hi <= t.lo) {
    t.first = 0;
    t.count = 1;
  } else {
    t.first = int(unsigned(t.lo) / KT);
    t.count = int((unsigned(t.hi) + KT - 1) / KT) - t.first;
  }
  return t;
}

template <int M>
__device__ __forceinline__ int row_tiles(const PagedAttnArgs& a, const SeqInfo& q) {
  return int((unsigned(q.n) * unsigned(a.n_q) + M - 1) / M);
}

__device__ __forceinline__ int64_t warp_scan(int64_t x) {  // inclusive, over the lanes
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(kFull, x, o);
    if ((threadIdx.x & 31) >= o) x += up;
  }
  return x;
}

// Units of one head of a sequence, summed by the lanes of a warp (the same
// sequence in all) or by one thread.
template <int M, int KT, bool WARP>
__device__ __forceinline__ int64_t head_units(const PagedAttnArgs& a, const SeqInfo& q) {
  int64_t u = 0;
  const int nqt = row_tiles<M>(a, q);
#pragma unroll 1
  for (int qt = WARP ? threadIdx.x & 31 : 0; qt < nqt; qt += WARP ? 32 : 1) {
    u += item_tiles<M, KT>(a, q, qt).count;
  }
  return WARP ? __shfl_sync(kFull, warp_scan(u), 31) : u;
}

// A place in the order of units.
template <int M, int KT>
struct Cursor {
  SeqInfo q;
  int seq, head, qt, nqt, lo, hi, first, count, tile;

  __device__ __forceinline__ void item(const PagedAttnArgs& a) {
    const ItemTiles t = item_tiles<M, KT>(a, q, qt);
    lo = t.lo, hi = t.hi, first = t.first, count = t.count;
  }
  // To the first unit of the next item; the caller knows that there is one.
  __device__ __forceinline__ void next_item(const PagedAttnArgs& a) {
    tile = 0;
    if (++qt == nqt) {
      qt = 0;
      if (++head == a.n_kv) {
        head = 0;
        do {
          q = load_seq(a, ++seq, nullptr);
        } while (q.n == 0 && seq + 1 < a.n_seqs);
        nqt = row_tiles<M>(a, q);
      }
    }
    item(a);
  }
  // To unit `off` of sequence s; by a whole warp.
  __device__ __forceinline__ void seek(const PagedAttnArgs& a, int s, int64_t off) {
    seq = s;
    q = load_seq(a, s, nullptr);
    nqt = row_tiles<M>(a, q);
    if (nqt == 1) {
      qt = 0;
      item(a);
      head = int(off / count);
      tile = int(off - int64_t(head) * count);
      return;
    }
    const int64_t per_head = head_units<M, KT, true>(a, q);
    head = int(off / per_head);
    off -= head * per_head;
    const int lane = threadIdx.x & 31;
    for (int base = 0;; base += 32) {  // the lanes count 32 row tiles at a time
      const int c = base + lane < nqt ? item_tiles<M, KT>(a, q, base + lane).count : 0;
      const int64_t end = warp_scan(c);
      const uint32_t past = __ballot_sync(kFull, end > off);
      if (past != 0) {
        const int l = __ffs(past) - 1;
        qt = base + l;
        tile = int(off - __shfl_sync(kFull, end - c, l));
        item(a);
        return;
      }
      off -= __shfl_sync(kFull, end, 31);
    }
  }
};

struct Run {
  int64_t total, begin, end;  // units of the call, and of this block
  int blocks;                 // that have units: the first ones, none in between without
  int seq;                    // sequence of unit `begin`
  int64_t off;                // units of that sequence before it
};

constexpr int kFewSeqs = 64;  // up to here a warp counts a sequence, above a thread
constexpr int kRunScratch = kFewSeqs + 4;

// The run of block b of `blocks`; called by all NT threads, `s` scratch.
template <int M, int KT, int NT>
__device__ __forceinline__ Run find_run(const PagedAttnArgs& a, int b, int blocks,
                                        int64_t (&s)[kRunScratch], unsigned* status) {
  static_assert(NT / 32 <= kFewSeqs, "scratch");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned* st = b == 0 ? status : nullptr;
  Run r{0, 0, 0, 0, 0, 0};
  auto cut = [&]() {
    r.blocks = int(min(int64_t(blocks), r.total));
    if (b >= r.blocks) return false;
    r.begin = r.total * b / r.blocks;
    r.end = r.total * (b + 1) / r.blocks;
    return true;
  };
  if (a.n_seqs <= kFewSeqs) {
#pragma unroll 1
    for (int sq = warp; sq < a.n_seqs; sq += NT / 32) {
      const SeqInfo q = load_seq(a, sq, lane == 0 ? st : nullptr);
      const int64_t u = q.n > 0 ? head_units<M, KT, true>(a, q) * a.n_kv : 0;
      if (lane == 0) s[sq] = u;
    }
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < a.n_seqs; ++i) r.total += s[i];
    if (!cut()) return r;
    int64_t before = 0;
#pragma unroll 1
    for (r.seq = 0; before + s[r.seq] <= r.begin; ++r.seq) before += s[r.seq];
    r.off = r.begin - before;
    return r;
  }
  auto scan = [&](int base, int64_t& mine, int64_t& incl) {  // units of seqs base + tid
    const int sq = base + tid;
    mine = 0;
    if (sq < a.n_seqs) {
      const SeqInfo q = load_seq(a, sq, st);
      if (q.n > 0) mine = head_units<M, KT, false>(a, q) * a.n_kv;
    }
    incl = warp_scan(mine);
    __syncthreads();  // the scratch of the call before is read
    if (lane == 31) s[warp] = incl;
    __syncthreads();
    int64_t before = 0;
    for (int w = 0; w < warp; ++w) before += s[w];
    incl += before;
    int64_t all = 0;
    for (int w = 0; w < NT / 32; ++w) all += s[w];
    return all;
  };
  int64_t mine, incl;
  for (int base = 0; base < a.n_seqs; base += NT) r.total += scan(base, mine, incl);
  if (!cut()) return r;
  int64_t before = 0;
  for (int base = 0; base < a.n_seqs; base += NT) {
    // one chunk: the scan above still holds
    const int64_t all = a.n_seqs <= NT ? r.total : scan(base, mine, incl);
    if (r.begin < before + all) {
      const int64_t end = before + incl, start = end - mine;
      if (start <= r.begin && r.begin < end) {
        s[kFewSeqs] = base + tid;
        s[kFewSeqs + 1] = r.begin - start;
      }
      break;
    }
    before += all;
  }
  __syncthreads();
  r.seq = int(s[kFewSeqs]);
  r.off = s[kFewSeqs + 1];
  return r;
}

// The block whose run holds unit u (the inverse of find_run's cuts): the
// largest b with floor(total b / blocks) <= u.
__device__ __forceinline__ int block_of(int64_t u, int64_t total, int blocks) {
  return int(((u + 1) * blocks - 1) / total);
}

// What the second kernel needs to join an item: written by every block, the
// item that ends in the block but began in an earlier one.
struct JoinInfo {
  int first_block;  // block in which it began (its slot 1), or -1: nothing to join
  int c0, head, row0, rows;
};

}  // namespace kvq
