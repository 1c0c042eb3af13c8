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
// a thread per row.  Everything is bound by latency: a handful of dependent
// loads and two block-wide scans.
#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kInlineRows = 4096;     // rows that the state's CTA writes itself

struct Sums { long long rows; int take, give; };

__device__ __forceinline__ Sums add(const Sums& a, const Sums& b) {
  return Sums{a.rows + b.rows, a.take + b.take, a.give + b.give};
}

// Exclusive prefix of each thread's sums within the CTA, and the CTA's total.
__device__ __forceinline__ Sums block_scan(const Sums& mine, Sums* warp_sums, Sums& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sums inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    Sums v{__shfl_up_sync(0xffffffffu, inc.rows, o), __shfl_up_sync(0xffffffffu, inc.take, o),
           __shfl_up_sync(0xffffffffu, inc.give, o)};
    if (lane >= o) inc = add(inc, v);
  }
  __syncthreads();                       // the previous use of warp_sums is over
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  Sums before{0, 0, 0};
  total = Sums{0, 0, 0};
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before = add(before, warp_sums[w]);
    total = add(total, warp_sums[w]);
  }
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

// One new row: its sequence by a search in row_start, then slot, position and mask.
__device__ __forceinline__ void write_row(const PlanArgs& a, int n) {
  const int total = a.row_start[a.batch];
  if (n >= total) {                             // rows behind the last sequence
    a.slots[n] = -1;
    a.positions[n] = 0;
    if (a.seq_ids) a.seq_ids[n] = -1;
    if (a.mask)
      for (int w = 0; w < a.mask_words; ++w) a.mask[(size_t)n * a.mask_words + w] = 0;
    return;
  }
  int lo = 0, hi = a.batch - 1;                 // the last sequence that starts at or before n
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.row_start[mid] <= n) lo = mid; else hi = mid - 1;
  }
  const int b = lo, s0 = a.row_start[b], i = n - s0;
  const int len = a.kv_lens[b] - (a.row_start[b + 1] - s0);
  const int row = len + i;
  const int page = a.block_table[(size_t)b * a.max_pages + (row >> 6)];
  const bool ok = page >= 0 && page < a.num_pages;
  if (!ok) flag_error(a.err, MLA_DEVERR_PAGE);
  a.slots[n] = ok ? page * 64 + (row & 63) : -1;
  if (a.seq_ids) a.seq_ids[n] = b;
  int depth = i;
  if (a.parents) {
    // up the tree: parents come before their children, so the walk ends
    depth = 0;
    uint64_t word = 1ull << (i & 63);
    int w = i >> 6;
    uint64_t* mask = a.mask ? a.mask + (size_t)n * a.mask_words : nullptr;
    if (mask)
      for (int v = w + 1; v < a.mask_words; ++v) mask[v] = 0;
    int at = i;
    while (true) {
      const int up = a.parents[s0 + at];
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

__global__ void __launch_bounds__(kThreads, 1) plan_kernel(PlanArgs a, int inline_rows) {
  __shared__ Sums warp_sums[kWarps];
  __shared__ int s_take[kThreads], s_give[kThreads], s_held[kThreads], s_need[kThreads];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t flags = 0;
  // ---- totals: does the step fit?
  Sums mine{0, 0, 0};
  for (int b = tid; b < a.batch; b += kThreads) {
    const SeqPlan s = seq_plan(a, b, &flags);
    mine = add(mine, Sums{s.bad ? 0 : s.count, max(s.need - s.held, 0), s.bad ? 0 : max(s.held - s.need, 0)});
  }
  Sums total;
  const int free_in = *a.free_count_in;
  block_scan(mine, warp_sums, total);
  if (free_in < 0 || free_in > a.num_pages || (long long)free_in + total.give > a.num_pages)
    flags |= MLA_DEVERR_POSITION;
  else if (total.take > free_in + total.give || total.rows > a.max_rows)
    flags |= MLA_DEVERR_CAPACITY;
  flags = __reduce_or_sync(0xffffffffu, flags);
  if (lane == 0 && flags) flag_error(a.err, flags);
  const bool fits = !__syncthreads_or(flags != 0);
  // ---- state: sequences in rounds of 1024, pages given back before any is taken
  const int top = free_in + total.give;
  for (int pass = 0; pass < 2; ++pass) {        // 0: give back and row offsets, 1: take
    Sums carry{0, 0, 0};
    for (int base = 0; base < a.batch; base += kThreads) {
      const int b = base + tid;
      int32_t ignored = 0;
      SeqPlan s{0, 0, 0, 0, true};
      if (b < a.batch && fits) s = seq_plan(a, b, &ignored);
      const Sums v{s.bad ? 0 : s.count, s.bad ? 0 : max(s.need - s.held, 0), s.bad ? 0 : max(s.held - s.need, 0)};
      Sums round;
      const Sums ex = add(carry, block_scan(v, warp_sums, round));
      carry = add(carry, round);
      s_take[tid] = ex.take;
      s_give[tid] = ex.give;
      s_held[tid] = s.bad ? 0 : s.held;
      s_need[tid] = s.bad ? 0 : s.need;
      if (pass == 0 && b < a.batch) {
        a.row_start[b] = (int)ex.rows;
        a.kv_lens[b] = fits ? s.len + s.count : a.seq_lens[b];
      }
      __syncthreads();
      // a warp per sequence, a lane per page
      for (int q = warp; q < kThreads && base + q < a.batch; q += kWarps) {
        int32_t* row = a.block_table + (size_t)(base + q) * a.max_pages;
        const int held = s_held[q], need = s_need[q];
        if (pass == 0) {
          for (int k = need + lane; k < held; k += 32) {
            a.free_pages[free_in + s_give[q] + k - need] = row[k];
            row[k] = -1;
          }
        } else {
          for (int k = held + lane; k < need; k += 32) row[k] = a.free_pages[top - 1 - (s_take[q] + k - held)];
        }
      }
      __syncthreads();
      // held_out may be held_in: a round is written once nothing reads it any more
      if (pass == 1 && b < a.batch) a.held_out[b] = fits ? s.need : a.held_in[b];
    }
  }
  if (tid == 0) {
    a.row_start[a.batch] = fits ? (int)total.rows : 0;
    *a.free_count_out = fits ? top - total.take : free_in;
  }
  __syncthreads();
  for (int n = tid; n < inline_rows; n += kThreads) write_row(a, n);
}

__global__ void __launch_bounds__(256) plan_rows_kernel(PlanArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int n = blockIdx.x * blockDim.x + threadIdx.x;
  if (n < a.max_rows) write_row(a, n);
}

}  // namespace

cudaError_t launch_step_plan(const PlanArgs& a, cudaStream_t st) {
  const bool in_one = a.max_rows <= kInlineRows;
  cudaError_t e = launch_dependent(plan_kernel, dim3(1), dim3(kThreads), 0, st, a, in_one ? a.max_rows : 0);
  if (e != cudaSuccess || in_one) return e;
  return launch_dependent(plan_rows_kernel, dim3((unsigned)((a.max_rows + 255) / 256)), dim3(256), 0, st, a);
}

}  // namespace mla
