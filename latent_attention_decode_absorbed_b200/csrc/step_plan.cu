// The bookkeeping of a decode step on the GPU: pages, block table, row offsets,
// slot map, positions and ancestor masks from the request lengths, the new row
// counts and the drafted trees.
//
// What it computes.  With L_b cached rows, n_b new rows and h_b held pages of
// sequence b, row offsets s_b = n_0 + ... + n_{b-1} and need_b = ceil((L_b +
// n_b) / 64): pages beyond need_b return to the free list, in sequence and
// table order; then, in the same order, each missing page is taken off the
// list's end.  New row s_b + i goes to slot table[b, (L_b+i) / 64] * 64 +
// (L_b+i) % 64.  Its position is L_b + i, or L_b + depth(i) in a drafted tree,
// and bit k of its mask is set where k is i or an ancestor of i.
//
// How.  One CTA does the state (two passes over the sequences: totals first,
// so that a step that does not fit changes nothing), since a page's place in
// the free list depends on every sequence before it.  A step of few rows has
// them written by the same CTA; one of many (prompts) by a second launch with
// a thread per four rows.  Everything is bound by latency, a handful of
// dependent loads and a block-wide scan: 5.4 us for 64 trees of 16 (from a
// captured graph), 12.7 us for 256 prompts of 1.06 M rows together.
#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kInlineRows = 4096;     // rows that the state's CTA writes itself
constexpr int kSeqsAtOnce = 4;

// rows saturates at kManyRows, so that no sum of counts wraps
struct Sums { unsigned rows; int take, give; };
constexpr unsigned kManyRows = 0x7fffffffu;

__device__ __forceinline__ Sums add(const Sums& a, const Sums& b) {
  return Sums{min(a.rows + b.rows, kManyRows), a.take + b.take, a.give + b.give};
}

__device__ __forceinline__ Sums warp_scan(Sums v) {   // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums u{__shfl_up_sync(0xffffffffu, v.rows, o), __shfl_up_sync(0xffffffffu, v.take, o),
                 __shfl_up_sync(0xffffffffu, v.give, o)};
    if (lane >= o) v = add(v, u);
  }
  return v;
}

// Exclusive prefix of each thread's sums within the CTA, and the CTA's total;
// only the first `live` threads' sums are not zero.  Shuffles bound this (one
// warp's per cycle), so warps without a sum leave the scan out and one warp
// scans the warps' sums.
__device__ __forceinline__ Sums block_scan(const Sums& mine, int live, Sums* warp_sums, Sums& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sums inc{0, 0, 0};
  if (32 * warp < live) inc = warp_scan(mine);
  __syncthreads();                       // the previous use of warp_sums is over
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const Sums w = warp_sums[lane], upto = warp_scan(w);
    warp_sums[lane] = Sums{upto.rows - w.rows, upto.take - w.take, upto.give - w.give};
    if (lane == 31) warp_sums[kWarps] = upto;
  }
  __syncthreads();
  total = warp_sums[kWarps];
  const Sums before = warp_sums[warp];
  return Sums{before.rows + inc.rows - mine.rows, before.take + inc.take - mine.take,
              before.give + inc.give - mine.give};
}

struct SeqPlan { int len, count, held, need; bool bad; };

__device__ __forceinline__ SeqPlan seq_plan(const PlanArgs& a, int b, int32_t* flags) {
  SeqPlan s;
  s.len = a.seq_lens[b];
  s.count = a.new_counts[b];
  s.held = a.held_in[b];
  const int capacity = a.max_pages * 64;        // fits an int (checked on the host)
  s.bad = s.len < 0 || s.count < 0 || s.held < 0 || s.held > a.max_pages;
  if (s.bad) *flags |= MLA_DEVERR_POSITION;
  if (!s.bad && (s.len > capacity || s.count > capacity - s.len || (a.mask && s.count > 64 * a.mask_words))) {
    s.bad = true;
    *flags |= MLA_DEVERR_CAPACITY;
  }
  s.need = s.bad ? 0 : (s.len + s.count + 63) / 64;
  return s;
}
__device__ __forceinline__ Sums sums_of(const SeqPlan& s) {
  if (s.bad) return Sums{0, 0, 0};
  return Sums{(unsigned)s.count, max(s.need - s.held, 0), max(s.held - s.need, 0)};
}

// A row behind the last sequence.
__device__ __forceinline__ void write_padding(const PlanArgs& a, int n) {
  a.slots[n] = -1;
  a.positions[n] = 0;
  if (a.seq_ids) a.seq_ids[n] = -1;
  if (a.mask)
    for (int w = 0; w < a.mask_words; ++w) a.mask[(size_t)n * a.mask_words + w] = 0;
}

// Slot, position and mask of node i of sequence b (new row n), whose page is
// `page`; par: the parents of the sequence's nodes (NULL: a chain).
__device__ __forceinline__ void write_row(const PlanArgs& a, int n, int b, int i, int len, int page,
                                          const int32_t* par) {
  const bool ok = page >= 0 && page < a.num_pages;
  if (!ok) flag_error(a.err, MLA_DEVERR_PAGE);
  a.slots[n] = ok ? page * 64 + ((len + i) & 63) : -1;
  if (a.seq_ids) a.seq_ids[n] = b;
  int depth = i;
  if (par) {
    // up the tree: a parent comes before its children, so the walk ends
    depth = 0;
    uint64_t word = 1ull << (i & 63);
    int w = i >> 6;
    uint64_t* mask = a.mask ? a.mask + (size_t)n * a.mask_words : nullptr;
    if (mask)
      for (int v = w + 1; v < a.mask_words; ++v) mask[v] = 0;
    int at = i;
    while (true) {
      const int up = par[at];
      if (up < 0) break;
      if (up >= at) {                           // not a tree in topological order: taken as a root
        flag_error(a.err, MLA_DEVERR_POSITION);
        break;
      }
      at = up;
      ++depth;
      if ((at >> 6) != w) {
        if (mask) mask[w] = word;
        for (--w; w > (at >> 6); --w)
          if (mask) mask[w] = 0;
        word = 0;
      }
      word |= 1ull << (at & 63);
    }
    if (mask) {
      mask[w] = word;
      for (--w; w >= 0; --w) mask[w] = 0;
    }
  } else if (a.mask) {
    for (int w = 0; w < a.mask_words; ++w) {
      const int k = i + 1 - 64 * w;             // a chain: the nodes 0..i
      a.mask[(size_t)n * a.mask_words + w] = k <= 0 ? 0ull : k >= 64 ? ~0ull : (1ull << k) - 1;
    }
  }
  a.positions[n] = len + depth;
}

// The last sequence that starts at or before row n (start ascends, start[0] <= n).
__device__ __forceinline__ int find_seq(const int* start, int batch, int n) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= n) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// inline_rows: rows this CTA writes itself (at most kInlineRows, and only
// where the batch is one round).  parents of those rows wait in shared memory
// by then, and a new page is read straight from the free list, so that no
// load waits for a store of this kernel.
__global__ void __launch_bounds__(kThreads, 1) plan_kernel(PlanArgs a, int inline_rows) {
  __shared__ Sums warp_sums[kWarps + 1];
  __shared__ int s_take[kThreads], s_give[kThreads], s_held[kThreads], s_need[kThreads], s_len[kThreads];
  __shared__ int s_start[kThreads + 1];
  __shared__ int s_par[kInlineRows];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (a.parents)
    for (int n = tid; n < inline_rows; n += kThreads) s_par[n] = a.parents[n];
  int32_t flags = 0;
  // ---- totals: does the step fit?
  SeqPlan own{0, 0, 0, 0, true};                // this thread's sequence, where the batch is one round
  Sums mine{0, 0, 0};
  const int free_in = *a.free_count_in;
  for (int b = tid; b < a.batch; b += kThreads) {
    own = seq_plan(a, b, &flags);
    mine = add(mine, sums_of(own));
  }
  Sums total;
  const Sums first = block_scan(mine, min(a.batch, kThreads), warp_sums, total);
  if (free_in < 0 || free_in > a.num_pages || (long long)free_in + total.give > a.num_pages)
    flags |= MLA_DEVERR_POSITION;
  else if (total.take > free_in + total.give || total.rows > (unsigned)a.max_rows)
    flags |= MLA_DEVERR_CAPACITY;
  flags = __reduce_or_sync(0xffffffffu, flags);
  if (lane == 0 && flags) flag_error(a.err, flags);
  const bool fits = !__syncthreads_or(flags != 0);
  if (!fits) {
    for (int b = tid; b < a.batch; b += kThreads) {
      a.row_start[b] = 0;
      a.kv_lens[b] = a.seq_lens[b];
      a.held_out[b] = a.held_in[b];
    }
    if (tid == 0) {
      a.row_start[a.batch] = 0;
      *a.free_count_out = free_in;
    }
    for (int n = tid; n < inline_rows; n += kThreads) write_padding(a, n);
    return;
  }
  // ---- state: sequences in rounds of 1024, pages given back before any is taken
  const bool one_round = a.batch <= kThreads;
  const int top = free_in + total.give;
  for (int pass = total.give > 0 ? 0 : 1; pass < 2; ++pass) {     // 0: give back, 1: take
    Sums carry{0, 0, 0};
    for (int base = 0; base < a.batch; base += kThreads) {
      const int b = base + tid;
      int32_t ignored = 0;
      Sums ex = first;
      SeqPlan s = own;
      if (!one_round) {
        s = SeqPlan{0, 0, 0, 0, true};
        if (b < a.batch) s = seq_plan(a, b, &ignored);
        Sums round;
        ex = add(carry, block_scan(sums_of(s), min(a.batch - base, kThreads), warp_sums, round));
        carry = add(carry, round);
      }
      s_take[tid] = ex.take;
      s_give[tid] = ex.give;
      s_held[tid] = s.held;
      s_need[tid] = s.need;
      s_len[tid] = s.len;
      s_start[tid] = (int)ex.rows;
      if (pass == 1 && b < a.batch) {
        a.row_start[b] = (int)ex.rows;
        a.kv_lens[b] = s.len + s.count;
        a.held_out[b] = s.need;                 // may be held_in: this round has read its own
      }
      __syncthreads();
      // a warp per sequence, a lane per page: the first 64 pages of four
      // sequences are loaded before any is stored
      const int seqs = min(kThreads, a.batch - base);
      // the k-th page that sequence q gives back (pass 0) or takes (pass 1)
      auto moves = [&](int q, int k) {
        return q < seqs && k < (pass == 0 ? s_held[q] - s_need[q] : s_need[q] - s_held[q]);
      };
      auto load_page = [&](int q, int k) -> int {
        if (!moves(q, k)) return -1;
        return pass == 0 ? a.block_table[(size_t)(base + q) * a.max_pages + s_need[q] + k]
                         : a.free_pages[top - 1 - (s_take[q] + k)];
      };
      auto store_page = [&](int q, int k, int page) {
        if (!moves(q, k)) return;
        int32_t* row = a.block_table + (size_t)(base + q) * a.max_pages;
        if (pass == 0) {
          a.free_pages[free_in + s_give[q] + k] = page;
          row[s_need[q] + k] = -1;
        } else {
          row[s_held[q] + k] = page;
        }
      };
      for (int q0 = warp; q0 < seqs; q0 += kSeqsAtOnce * kWarps) {
        int page[kSeqsAtOnce][2];
#pragma unroll
        for (int u = 0; u < kSeqsAtOnce; ++u)
#pragma unroll
          for (int t = 0; t < 2; ++t) page[u][t] = load_page(q0 + u * kWarps, lane + 32 * t);
#pragma unroll
        for (int u = 0; u < kSeqsAtOnce; ++u) {
#pragma unroll
          for (int t = 0; t < 2; ++t) store_page(q0 + u * kWarps, lane + 32 * t, page[u][t]);
          const int q = q0 + u * kWarps;
          const int count = q < seqs ? abs(s_need[q] - s_held[q]) : 0;
          for (int k = 64 + lane; k < count; k += 32)
            store_page(q, k, load_page(q, k));
        }
      }
      if (!one_round || pass == 0) __syncthreads();
    }
  }
  if (tid == 0) {
    a.row_start[a.batch] = (int)total.rows;
    *a.free_count_out = top - total.take;
  }
  for (int n = tid; n < inline_rows; n += kThreads) {
    if (n >= (int)total.rows) {
      write_padding(a, n);
      continue;
    }
    const int b = find_seq(s_start, a.batch, n), s0 = s_start[b], i = n - s0, len = s_len[b];
    const int k = (len + i) >> 6, held = s_held[b];
    const int page = k < held ? a.block_table[(size_t)b * a.max_pages + k]
                              : a.free_pages[top - 1 - (s_take[b] + k - held)];
    write_row(a, n, b, i, len, page, a.parents ? s_par + s0 : nullptr);
  }
}

// Many rows: a thread per four consecutive rows.  The CTA counts the sequences
// that start at or before its first row; from there a thread steps on.
constexpr int kRowsPerThread = 4;

__global__ void __launch_bounds__(256) plan_rows_kernel(PlanArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int cta0 = blockIdx.x * blockDim.x * kRowsPerThread;
  const int n0 = cta0 + threadIdx.x * kRowsPerThread;
  const int total = a.row_start[a.batch];
  int b = -1;
  for (int base = 0; base < a.batch; base += blockDim.x) {
    const int q = base + threadIdx.x;
    const int starts = __syncthreads_count(q < a.batch && a.row_start[q] <= cta0);
    b += starts;
    if (starts < (int)blockDim.x) break;
  }
  const int end = min(a.max_rows, n0 + kRowsPerThread);
  if (n0 >= end) return;
  int s0 = 0, s1 = 0, len = 0, k = -1, page = -1;
  auto reach = [&](int n) {                     // the sequence of row n < total
    int next = a.row_start[b + 1];
    while (next <= n) next = a.row_start[++b + 1];
    s0 = a.row_start[b];
    s1 = next;
    len = a.kv_lens[b] - (s1 - s0);
    k = -1;
  };
  if (n0 < total) reach(n0);
  // a prompt's rows: four at once where they lie in one sequence and page
  const int row = len + n0 - s0;
  if (end - n0 == kRowsPerThread && end <= s1 && (row & 63) <= 64 - kRowsPerThread && !a.parents && !a.mask &&
      !a.seq_ids && ((reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.positions)) & 15) == 0) {
    page = a.block_table[(size_t)b * a.max_pages + (row >> 6)];
    const bool ok = page >= 0 && page < a.num_pages;
    if (!ok) flag_error(a.err, MLA_DEVERR_PAGE);
    const int sl = page * 64 + (row & 63);
    *reinterpret_cast<int4*>(a.slots + n0) = ok ? make_int4(sl, sl + 1, sl + 2, sl + 3) : make_int4(-1, -1, -1, -1);
    *reinterpret_cast<int4*>(a.positions + n0) = make_int4(row, row + 1, row + 2, row + 3);
    return;
  }
  for (int n = n0; n < end; ++n) {
    if (n >= total) {
      write_padding(a, n);
      continue;
    }
    if (n >= s1) reach(n);
    const int i = n - s0;
    if ((len + i) >> 6 != k) {
      k = (len + i) >> 6;
      page = a.block_table[(size_t)b * a.max_pages + k];
    }
    write_row(a, n, b, i, len, page, a.parents ? a.parents + s0 : nullptr);
  }
}

}  // namespace

cudaError_t launch_step_plan(const PlanArgs& a, cudaStream_t st) {
  const bool in_one = a.max_rows <= kInlineRows && a.batch <= kThreads;
  cudaError_t e = launch_dependent(plan_kernel, dim3(1), dim3(kThreads), 0, st, a, in_one ? a.max_rows : 0);
  if (e != cudaSuccess || in_one || a.max_rows == 0) return e;
  const unsigned per_cta = 256 * kRowsPerThread;
  return launch_dependent(plan_rows_kernel, dim3(((unsigned)a.max_rows + per_cta - 1) / per_cta), dim3(256), 0, st, a);
}

}  // namespace mla
