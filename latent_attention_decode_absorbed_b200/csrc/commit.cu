// The rows of an accepted path moved to the front of a sequence's drafted rows.
//
// A drafted tree's rows sit behind the sequence's prefix in node order: node k
// at cached row P + k.  Once a path of nodes i_0 < i_1 < ... is accepted, the
// sequence goes on with exactly those rows, so row P + i_j moves to P + j.  The
// key of a row was rotated to its depth's position when it was written, and
// the accepted path's j-th node has depth j, so the rows move as they are.
//
// How.  CTA (sequence, third of the row's nine blocks); a batch of rows is read
// into registers before any of it is written.  Since i_j >= j and the path
// ascends, a batch's targets lie below every later batch's sources, so
// batches in order never overwrite a row that is still to be read.  Bound by
// latency (a few rows per sequence): path, table entries, rows, one after
// another; 2.7 us for 64 sequences, 4.8 for 512 (from a captured graph).
#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kThreads = 128;
constexpr int kParts = 3;         // CTAs per sequence, three blocks of 64 columns each
constexpr int kHold = 4;          // 16-byte pieces a thread holds between reading and writing

__global__ void __launch_bounds__(kThreads) commit_kernel(CommitArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x, part = blockIdx.y, tid = threadIdx.x;
  const int start = a.row_start[b], end = a.row_start[b + 1], kv = a.kv_lens[b], count = a.counts[b];
  // differences only of numbers that are known not to wrap
  bool bad = start < 0 || end < start || end > a.n_rows || kv < end - start;
  const int n = bad ? 0 : end - start;
  const int base = bad ? 0 : kv - n;            // the prefix
  bad |= kv > a.max_pages * 64 || count < 0 || count > n;
  const int32_t* path = a.nodes + start;
  if (!bad)
    for (int j = tid; j < count; j += kThreads) bad |= path[j] < 0 || path[j] >= n || (j && path[j] <= path[j - 1]);
  bad = __syncthreads_or(bad);
  if (bad && tid == 0 && part == 0) flag_error(a.err, MLA_DEVERR_POSITION);
  if (tid == 0 && part == 0 && a.seq_lens) a.seq_lens[b] = bad ? base : base + count;
  if (bad) return;
  const int32_t* table = a.block_table + (size_t)b * a.max_pages;
  // slot of a cached row, -1 for a page outside the pool
  auto slot = [&](int row) -> long long {
    const int pg = table[row >> 6];
    return pg >= 0 && pg < a.num_pages ? (long long)pg * 64 + (row & 63) : -1;
  };
  const int line = 64 * a.elt;                  // bytes of a row in one block
  const int per_row = 3 * line / 16;            // 16-byte pieces of a row in this CTA
  const int batch = kHold * kThreads / per_row; // rows at a time
  uint8_t* pool = static_cast<uint8_t*>(a.cache);
  for (int j0 = 0; j0 < count; j0 += batch) {
    const int rows = min(batch, count - j0);
    uint4 held[kHold];
    uint8_t* to[kHold];
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
      to[k] = nullptr;
      const int piece = tid + k * kThreads;
      const int j = piece / per_row, at = 16 * (piece - j * per_row);
      if (j >= rows) continue;
      const int node = path[j0 + j];
      if (node == j0 + j) continue;             // in its place already
      const long long from = slot(base + node), dst = slot(base + j0 + j);
      if (from < 0 || dst < 0) {
        flag_error(a.err, MLA_DEVERR_PAGE);
        continue;
      }
      const int block = 3 * part + at / line, off = at % line;
      held[k] = *reinterpret_cast<const uint4*>(pool + (((from >> 6) * 9 + block) * 64 + (from & 63)) * line + off);
      to[k] = pool + (((dst >> 6) * 9 + block) * 64 + (dst & 63)) * line + off;
    }
    float sc = 0.f;
    float* sc_to = nullptr;
    if (a.cache_scale && part == 0 && tid < rows && path[j0 + tid] != j0 + tid) {   // batch <= kThreads
      const long long from = slot(base + path[j0 + tid]), dst = slot(base + j0 + tid);
      if (from >= 0 && dst >= 0) {
        sc = a.cache_scale[from];
        sc_to = a.cache_scale + dst;
      }
    }
    __syncthreads();                            // the whole batch is read
#pragma unroll
    for (int k = 0; k < kHold; ++k)
      if (to[k]) *reinterpret_cast<uint4*>(to[k]) = held[k];
    if (sc_to) *sc_to = sc;
    __syncthreads();                            // and written before the next one is read
  }
}

}  // namespace

cudaError_t launch_cache_commit(const CommitArgs& a, cudaStream_t st) {
  return launch_dependent(commit_kernel, dim3((unsigned)a.batch, kParts), dim3(kThreads), 0, st, a);
}

}  // namespace mla
