// Attention of drafted tokens over the paged latent cache, on the tcgen05
// tensor cores: every drafted token (node) of a sequence sees the sequence's
// prefix and those drafted rows whose bit is set in its mask.
//
// What it computes ("DeepSeek-V2: MLA Explained", "MLA Full Formulas" part 3
// with the absorption of "Optimization Note").  For node i of sequence b, head
// h and the rows j that the node sees,
//   z_j = scale * (q_abs[i,h,0:512] . c_j + q_abs[i,h,512:576] . k_j)
//   o_lat[i,h,:] = sum_j e^{z_j - m} c_j / sum_j e^{z_j - m},  lse = m + ln sum_j e^{z_j - m}
//
// How.  All heads of all nodes of a sequence read the same cached rows, so a
// sequence's (node, head) pairs are the rows of one dense problem: they are
// cut into tiles of 128 rows whatever the head count (one node of 128 heads,
// eight nodes of 16), and per tile of 256 cached rows a CTA pair issues
//   S[128 x 256]  = Q[128 x 576] . K[256 x 576]^T,   O[128 x 512] += P[128 x 256] . V[256 x 512]
// exactly as the single-token kernel does for its 128 heads (decode_pair.cu
// explains the operand layouts, the TMEM layout of M = 128 over a pair, the
// ring of stages and the softmax's hand-offs).  The mask costs nothing in the
// prefix: a thread of the softmax owns one row and one 64-row page, and only
// a page that reaches past the prefix builds a 64-bit visibility word.
//
// Work split.  The launch has one persistent CTA pair per SM pair and no
// split count: the tiles (row tile x cached tile) of all sequences form one
// list, a row tile's cached tiles next to each other, and pair p takes the
// p-th equal part of it (or whole row tiles, where those balance).  Each CTA
// finds its part by a scan over the sequences' lengths at its start, so lengths
// stay on the device and a captured graph serves any of them.  A row tile that one pair covers alone is normalised
// and stored as the final result; a row tile that crosses a pair's border
// leaves at most two partials per pair (its first and its last segment) in
// the workspace, which tree_merge_kernel joins.  The partials are thus
// bounded by the number of pairs, not by the lengths or the batch.
//
// What bounds it.  Calls of many row tiles: the shared-memory data path, close
// behind the tensor cores.  Per tile of 256 cached rows a CTA's MMAs take 4357
// cycles and read 3264 x 128 bytes of operands, the copies write 2176 and the
// softmax 256 more: 5700 cycles where one at a time passes.  Measured: 5960 to
// 6010 cycles a tile (a full profile: tensor 45 % of elapsed cycles at 6670 a
// tile, operand reads 44 %, LSU 7 %), 1377 TFLOP/s from L2 in a single call;
// back to back the 1000 W cap takes the clock to ~1.6 GHz.  Calls of few row
// tiles per sequence: HBM (64 x 8 drafts x 16 heads: 117 us of 55).  Calls of a
// few tiles: latency (one token over 4096 rows, 20.5 us: schedule 1.7, query
// and first rows 1.6, scores 2.5, softmax 1.0, values 1.7, epilogue 2.6, exit
// and merge 5.5).
//
// With an e4m3 cache both GEMMs run on kind::f8f6f4 straight from the cache
// codes: the query as two e4m3 terms on a power-of-two scale (split_q_tree
// below: exact for all but tiny components, so the scores are fp32-exact
// products), the softmax weights as an e4m3 and an e5m2 term with the row
// scales folded in, on a reference of their own per (node, head): softmax_q8.cuh.
#include <math.h>

#include <type_traits>

#include "mla_device.cuh"
#include "mla_internal.h"
#include "sm100.cuh"
#include "softmax_q8.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kTile = 256;                // cached rows per pair tile (128 per CTA)
constexpr int kM = 128;                   // (node, head) rows per row tile
constexpr int kHM = 64;                   // of them in one CTA
constexpr int kChunks = 9;                // 576 / 64 column chunks
constexpr int kBox = 8192;                // [64 rows x 64 16-bit values]
constexpr int kBox8 = 4096;               // [64 rows x 64 codes]
constexpr int kQ8Plane = kChunks * kBox8; // one term (hi or lo) of Q, 9 x [64 rows x 64 codes]
constexpr int kQChunk = kHM * 128;        // [64 rows x 64 dims], 16-bit
constexpr int kPChunk = kHM * 128;        // [64 rows x 64 cached rows], 16-bit: P of one page
constexpr int kProducers = 2;             // warps 0, 1: TMA producers
constexpr int kWarpMma = kProducers, kWarpSoft0 = kWarpMma + 1, kSoftWarps = 8;
constexpr int kThreads = 32 * (kWarpSoft0 + kSoftWarps);
constexpr float kRescaleLog2 = 8.0f;      // lazy rescale threshold (log2 units)
// What cutting row tiles costs a call whose pairs are all busy, in tiles of a
// pair: a second segment, the partials and their merge.  128 sequences of one
// row tile of two tiles: 49.6 us cut evenly, 34.5 whole; 60 of sixteen: 93 and
// 86; 4 of up to three, most pairs idle: 17.8 cut and 20.1 whole, hence the
// rule only where there is more than a tile for every pair.
constexpr int kSplitTiles = 3;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;             // S of tile t at kColS + 128 (t & 1)
constexpr uint32_t kColO = 256;           // O: dims 0..255 at 256, dims 256..511 at 384

// offsets inside the misc area
constexpr int kMBars = 0;                 // 64 barriers
constexpr int kMTmem = 64 * 8;
constexpr int kMAbort = kMTmem + 4;
constexpr int kMRedMax = kMTmem + 16;     // float [2 tile parities][4 parts][64 rows]
constexpr int kMRedSum = kMRedMax + 2 * 4 * kHM * 4;    // float [4 parts][64 rows]
constexpr int kMaxPairs = 96;             // bound of the workspace's partials, whatever the GPU's SM count
constexpr int kMaxDealt = 1024;           // sequences whose row tiles can be dealt out (their prefix sums are kept)
constexpr int kMPart = kMRedSum + 4 * kHM * 4;          // int [8]: where this pair's part begins (see there)
constexpr int kMCol = kMPart + 4 * 8;                   // int [96]: tiles of each column
constexpr int kMRt = kMCol + 4 * kMaxPairs;             // uint16 [1024]: row tiles before each sequence
constexpr int kMScale = kMRt + 2 * kMaxDealt;           // 8-bit MMAs: the row scales of the four pages, see softmax_q8.cuh
constexpr int kMScan = kMScale;                         // int2 [16]: per-warp sums of the schedule's scan, before that
constexpr int kMiscBytes = kMScale + q8::kBytes;

template <bool D8>
struct TreeLayout {
  static constexpr int kSlotB = D8 ? 8192 : 16384;       // bytes of one operand stage
  static constexpr int kSlots = D8 ? 14 : 7;
  static constexpr int kOffQ = 0;                        // Q: 9 x 8 KB, K-major SW128 (D8: hi, lo 9 x 4 KB, SW64)
  static constexpr int kOffRing = kOffQ + kChunks * kQChunk;
  static constexpr int kOffP = kOffRing + kSlots * kSlotB;   // P: 4 pages x 8 KB (D8: hi, lo 4 KB each)
  static constexpr int kOffMisc = kOffP + 4 * kPChunk;
  static constexpr int kSmem = kOffMisc + kMiscBytes + 1024;     // + alignment slack
  static constexpr int kBFull = 0;                  // [kSlots] leader: a stage is in both CTAs
  static constexpr int kBEmpty = kSlots;            // [kSlots] both: the MMAs are done with the stage
  static constexpr int kBSFull = 2 * kSlots;        // [2] both: S of a tile is in TMEM
  static constexpr int kBODone = kBSFull + 2;       // both: the value MMAs of a tile are done
  static constexpr int kBPFull = kBODone + 1;       // leader: both CTAs' softmax wrote P (and rescaled O)
  static constexpr int kBQFull = kBPFull + 1;       // leader: both CTAs' Q landed
  static constexpr int kBQFree = kBQFull + 1;       // both: the segment's score MMAs are done with Q
  static constexpr int kBEpiDone = kBQFree + 1;     // leader: both CTAs read O out (TMEM reusable)
  static constexpr int kBSoft = kBEpiDone + 1;      // local: the softmax warps' own barrier
  static constexpr int kBEnd = kBSoft + 1;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static_assert(kBEnd <= 64, "barrier area");
};

// A row tile that crosses its pair's border: where its rows go, and how many
// of the following pairs hold a further part of it (0: nothing to merge).
struct TreeDesc { int row0, rows, follow, pad; };

struct TreeParams {
  int n_heads, batch, n_rows;   // n_rows: nodes of the call (capacity of the row arrays)
  const int32_t* block_table;
  int max_pages, num_pages;
  const int32_t* kv_lens;
  const int32_t* row_start;
  const uint64_t* tree_mask;    // NULL: node i sees the nodes 0..i
  int mask_words;
  float scale_log2;             // softmax_scale * log2(e)
  const float* cache_scale;     // e4m3 cache: per-row dequantisation scale [num_pages * 64]
  const float* q_scale;         // 8-bit MMAs: scale of the two-term query per (node, head)
  float* part_o;                // [2 pairs][128 x 512], in the order of part_at
  float* part_lse;              // [2 pairs][128]
  TreeDesc* desc;               // [pairs]
  void* o_lat;                  // [n_rows, n_heads, 512], bf16 or fp32
  int o_f32;
  float* lse;                   // [n_rows, n_heads] or NULL
  int32_t* err;
  unsigned long long wait_limit;
  int withhold_q;
};

// One sequence's share of the problem; n = 0 (no work) where its numbers are
// not possible ones.
struct SeqInfo { int start, n, L, rt, kt; bool bad, order; };   // order: row_start is out of order here

__device__ __forceinline__ SeqInfo seq_info(const TreeParams& p, int b) {
  SeqInfo s;
  const int r0 = p.row_start[b], r1 = p.row_start[b + 1];
  s.L = p.kv_lens[b];
  s.start = r0;
  s.n = r1 - r0;
  s.order = r0 < 0 || r1 < r0 || r1 > p.n_rows;
  s.bad = s.order || s.L < s.n || s.L > p.max_pages * 64;
  if (s.bad) s.n = 0;
  s.rt = (s.n * p.n_heads + kM - 1) / kM;
  s.kt = s.n > 0 ? (s.L + kTile - 1) / kTile : 0;
  return s;
}

__device__ __forceinline__ uint64_t low_bits(int n) {   // the n lowest bits, n clamped to [0, 64]
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}

// Visibility of the 64 cached rows from `row0` on for one node: bit j set
// where the node sees row row0 + j.  The prefix is rows 0..prefix-1; drafted
// row k (cached row prefix + k) is seen where bit k of the node's mask is
// set, or k <= node without masks.
__device__ __forceinline__ uint64_t visible_rows(int row0, int prefix, int n, int node, const uint64_t* mask,
                                                 int words) {
  const int k0 = row0 - prefix;             // place of the page's first row in the tree
  if (k0 <= -64) return ~0ull;
  uint64_t bits;
  if (!mask) {
    bits = low_bits(node - k0 + 1);
    return bits;                            // rows of the prefix (k < 0) are among them
  }
  if (k0 < 0) {
    bits = (mask[0] << (-k0)) | low_bits(-k0);
  } else {
    const int w = k0 >> 6, sh = k0 & 63;
    bits = w < words ? mask[w] >> sh : 0ull;
    if (sh && w + 1 < words) bits |= mask[w + 1] << (64 - sh);
  }
  return bits & low_bits(n - k0);
}

__device__ __forceinline__ int page_or_minus1(const TreeParams& p, int b, int pidx) {
  const int pg = pidx < p.max_pages ? p.block_table[(size_t)b * p.max_pages + pidx] : -1;
  return pg >= 0 && pg < p.num_pages ? pg : -1;
}

// Partials are stored as the softmax warps read them from TMEM: 32 rows per
// warp, a row per lane, in 4-channel pieces.  Index (in float4, of lane 0) of
// piece `q` (0..31) of the 128 channels 256 ch + 128 (q4 >> 1) of the rows
// 64 rank + 32 (q4 & 1) + (0..31) of a row tile.
__device__ __forceinline__ int part_at(int rank, int ch, int q4, int q) { return (((rank * 2 + ch) * 4 + q4) * 32 + q) * 32; }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// tm_cache: boxes of one [64 rows x 64 columns] block; tm_cache2: boxes of two
// adjacent blocks; tm_q: boxes of 64 (node, head) rows x 64 columns.
template <bool D8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    decode_tree_kernel(const __grid_constant__ CUtensorMap tm_cache, const __grid_constant__ CUtensorMap tm_cache2,
                       const __grid_constant__ CUtensorMap tm_q, const TreeParams p) {
  using L = TreeLayout<D8>;
  constexpr int kSlots = L::kSlots;
  constexpr int kBFull = L::kBFull, kBEmpty = L::kBEmpty, kBSFull = L::kBSFull, kBODone = L::kBODone,
                kBPFull = L::kBPFull, kBQFull = L::kBQFull, kBQFree = L::kBQFree, kBEpiDone = L::kBEpiDone,
                kBSoft = L::kBSoft;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t s_base = smem_u32(smem);
  const uint32_t s_q = s_base + L::kOffQ, s_ring = s_base + L::kOffRing, s_p = s_base + L::kOffP;
  uint8_t* misc = smem + L::kOffMisc;
  uint8_t* s_pbuf = smem + L::kOffP;
  const uint32_t s_misc = s_base + L::kOffMisc;
  auto bar = [&](int i) -> uint32_t { return s_misc + kMBars + 8 * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + kMAbort);
  float* red_max = reinterpret_cast<float*>(misc + kMRedMax);
  float* red_sum = reinterpret_cast<float*>(misc + kMRedSum);
  int2* scan = reinterpret_cast<int2*>(misc + kMScan);
  int* part0 = reinterpret_cast<int*>(misc + kMPart);
  int* col = reinterpret_cast<int*>(misc + kMCol);
  uint16_t* rt_before = reinterpret_cast<uint16_t*>(misc + kMRt);   // at most 64 per pair, see `dealt`

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t lim = p.wait_limit;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;

  // ---- set-up
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(bar(kBFull + i), 1);
      mbar_init(bar(kBEmpty + i), 1);
    }
    mbar_init(bar(kBSFull), 1);
    mbar_init(bar(kBSFull + 1), 1);
    mbar_init(bar(kBODone), 1);
    mbar_init(bar(kBPFull), 2 * kSoftWarps);
    mbar_init(bar(kBQFull), 1);
    mbar_init(bar(kBQFree), 1);
    mbar_init(bar(kBEpiDone), 2 * kSoftWarps);
    mbar_init(bar(kBSoft), kSoftWarps);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == 32 * kWarpMma) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_cache);
    tma_prefetch_desc(&tm_cache2);
  }
  if (warp == 0) tmem_alloc_pair(s_misc + kMTmem, kTmemCols);
  // global memory only after the previous kernel on the stream has completed
  griddep_wait();
  griddep_launch_dependents();

  // ---- this pair's part [g0, g1) of the list of tiles, from a scan over the
  // sequences' tile counts (each thread a run of consecutive sequences).  With
  // more row tiles than pairs the list is dealt out: it runs down `stride`
  // columns, column c holding the row tiles c, c + stride, ... in the order of
  // the sequences.  Pairs next to each other then work on row tiles next to
  // each other, those of one sequence, at about the same time, and its rows
  // come from HBM once.
  int total, g0, g1, used, stride, row_tiles = 0;
  {
    const int per = (p.batch + kThreads - 1) / kThreads;
    const int b_lo = min(p.batch, (int)threadIdx.x * per), b_hi = min(p.batch, b_lo + per);
    int2 sum = make_int2(0, 0);             // tiles (row tiles x cached tiles), row tiles
    bool order = false;
    for (int b = b_lo; b < b_hi; ++b) {
      const SeqInfo q = seq_info(p, b);
      order |= q.order;
      if (q.bad && blockIdx.x == 0) flag_error(p.err, MLA_DEVERR_POSITION);
      sum.x += q.rt * q.kt;
      sum.y += q.rt;
    }
    int2 inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int2 v = make_int2(__shfl_up_sync(0xffffffffu, inc.x, o), __shfl_up_sync(0xffffffffu, inc.y, o));
      if (lane >= o) inc = make_int2(inc.x + v.x, inc.y + v.y);
    }
    if (lane == 31) scan[warp] = inc;
    if (threadIdx.x < kMaxPairs) col[threadIdx.x] = 0;
    // (row offsets out of order: no work at all, since only ascending ones
    // bound the list by the call's rows)
    const bool none = __syncthreads_or(order);
    int2 base = make_int2(inc.x - sum.x, inc.y - sum.y);
    total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const int2 v = scan[w];
      if (w < warp) base = make_int2(base.x + v.x, base.y + v.y);
      total += v.x;
      row_tiles += v.y;
    }
    if (none) total = row_tiles = 0;
    used = min(n_pairs, total);
    g0 = pair < used ? (int)((long long)pair * total / used) : total;
    g1 = pair < used ? (int)((long long)(pair + 1) * total / used) : total;
    // (also with fewer row tiles than pairs, where whole ones may do: see below)
    const int share = used ? (total + used - 1) / used : 0;
    const bool whole = share > 1 && total <= (long long)(share + kSplitTiles) * row_tiles;
    bool dealt = n_pairs > 1 && row_tiles <= 64 * n_pairs && p.batch <= kMaxDealt && (row_tiles > n_pairs || whole);
    stride = dealt ? n_pairs : 1;
    // part0: row tile index, cached tile within it, tiles to the end of its
    // column, its sequence, row tiles before that sequence
    if (dealt) {
      int before = base.y;
      for (int b = b_lo; b < b_hi; ++b) {
        const SeqInfo q = seq_info(p, b);
        rt_before[b] = (uint16_t)before;
        for (int x = 0; x < min(q.rt, stride); ++x)      // q.rt row tiles over consecutive columns
          atomicAdd(col + (before + x) % stride, q.kt * ((q.rt - x + stride - 1) / stride));
        before += q.rt;
      }
      __syncthreads();
      // a column per pair, where the longest is not much longer than an even
      // share: nothing is cut, so nothing is merged
      const int longest = __reduce_max_sync(0xffffffffu, max(max(col[lane], col[lane + 32]), col[lane + 64]));
      if (whole && longest <= share + kSplitTiles) {
        g0 = 0;                                          // (positions matter to cut row tiles only)
        g1 = col[pair];
        if (threadIdx.x == 0) {
          part0[0] = pair;
          part0[1] = 0;
          part0[2] = g1;
        }
      } else if (row_tiles <= n_pairs) {
        dealt = false;
        stride = 1;
      } else if (warp == 0 && g0 < g1) {
        int at = 0, c = 0;                               // tiles before column c
        for (; g0 >= at + col[c]; ++c) at += col[c];
        const int end = at + col[c];
        for (int j0 = 0;; j0 += 32) {                    // a lane per row tile of the column
          const int idx = c + (j0 + lane) * stride;
          int kt = 0;
          if (idx < row_tiles) {
            int lo = 0, hi = p.batch - 1;
            while (lo < hi) {
              const int mid = (lo + hi + 1) >> 1;
              if (rt_before[mid] <= idx) lo = mid; else hi = mid - 1;
            }
            kt = seq_info(p, lo).kt;
          }
          int upto = kt;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
          }
          const uint32_t past = __ballot_sync(0xffffffffu, at + upto > g0);
          if (past) {
            if (lane == __ffs(past) - 1) {
              part0[0] = idx;
              part0[1] = g0 - (at + upto - kt);
              part0[2] = end - g0;
            }
            break;
          }
          at += __shfl_sync(0xffffffffu, upto, 31);
        }
      }
    }
    if (!dealt && g0 < g1 && base.x <= g0 && g0 < base.x + sum.x) {
      int b = b_lo;
      for (;; ++b) {
        const SeqInfo q = seq_info(p, b);
        if (g0 < base.x + q.rt * q.kt) {
          const int rt = (g0 - base.x) / q.kt;
          part0[0] = base.y + rt;
          part0[1] = g0 - base.x - rt * q.kt;
          part0[2] = total - g0;
          part0[3] = b;
          part0[4] = base.y;
          break;
        }
        base = make_int2(base.x + q.rt * q.kt, base.y + q.rt);
      }
    }
    if (leader && threadIdx.x == 0) p.desc[pair].follow = 0;   // a segment below may set it
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(misc + kMTmem);

  // ---- the pair's segments: every role walks the same sequence of them.  A
  // part that begins inside a column (or inside a row tile, where it does not
  // reach the next column) puts that beginning off to its end: so every pair
  // starts at the first cached row of a row tile, the pairs on one sequence
  // read the same rows at about the same time, and they come from L2 (two
  // sequences of 131072 rows with 32 row tiles each: 2.69 -> 2.30 ms a call;
  // 64 sequences of 1024 to 8192 rows with 5 to 16: 970 -> 890 us with the list
  // dealt out, 0.73 GB read from HBM of the 0.52 that a call cannot do without).
  struct Seg { int b, start, n, L, row, k0, nt, kt, g; };
  struct Stretch { int idx, k, left, g, b, rt0; };   // row tile, cached tile, tiles, list position; sequence
  struct Walk { Stretch now, later; };
  // the sequence of row tile w.idx
  auto locate = [&](Stretch& w) -> SeqInfo {
    if (stride > 1) {
      int lo = 0, hi = p.batch - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (rt_before[mid] <= w.idx) lo = mid; else hi = mid - 1;
      }
      w.b = lo;
      w.rt0 = rt_before[lo];
      return seq_info(p, lo);
    }
    SeqInfo q = seq_info(p, w.b);
    while (w.idx >= w.rt0 + q.rt) {
      w.rt0 += q.rt;
      q = seq_info(p, ++w.b);
    }
    return q;
  };
  auto walk_begin = [&]() -> Walk {
    Walk w{{0, 0, 0, 0, 0, 0}, {0, 0, 0, 0, 0, 0}};
    if (g0 >= g1) return w;
    w.now = Stretch{part0[0], part0[1], g1 - g0, g0, part0[3], part0[4]};
    const int to_col = part0[2], len = g1 - g0;
    int off = 0, next = 0;
    if (stride > 1 && to_col < len && (w.now.idx >= stride || w.now.k > 0)) {
      off = to_col;                                // to the next column's first row tile
      next = w.now.idx % stride + 1;
    } else if (w.now.k > 0) {
      const int rest = locate(w.now).kt - w.now.k; // to the column's next row tile
      if (rest < min(len, to_col)) {
        off = rest;
        next = w.now.idx + stride;
      }
    }
    if (off > 0) {
      w.later = w.now;
      w.later.left = off;
      w.now.idx = next;
      w.now.k = 0;
      w.now.left = len - off;
      w.now.g = g0 + off;
    }
    return w;
  };
  auto next_seg = [&](Walk& w, Seg& s) -> bool {
    if (w.now.left == 0) {
      if (w.later.left == 0) return false;
      w.now = w.later;
      w.later.left = 0;
    }
    const SeqInfo q = locate(w.now);
    s.b = w.now.b;
    s.start = q.start;
    s.n = q.n;
    s.L = q.L;
    s.row = (w.now.idx - w.now.rt0) * kM;  // first (node, head) row of the tile within the sequence
    s.k0 = w.now.k;
    s.kt = q.kt;
    s.nt = min(q.kt - s.k0, w.now.left);
    s.g = w.now.g;
    w.now.left -= s.nt;
    w.now.g += s.nt;
    w.now.k = 0;
    const int idx = w.now.idx + stride;
    // past a column's end the next one begins (a stretch of several columns)
    w.now.idx = stride > 1 && idx >= row_tiles ? w.now.idx % stride + 1 : idx;
    return true;
  };

  uint32_t kc = 0;   // ring stages handed out (producer) or consumed (MMA)
  if (warp < kProducers) {
    // ============ TMA producers (both CTAs), in the order the MMA consumes ============
    // S(0), then per tile i: S(i+1), O(i); boxes as in decode_pair.cu.  The
    // stages go to the producers in turn: a stage's wait, expectation and
    // copies take one lane ~430 cycles whatever their size, against 256 that
    // its MMAs take (L2-resident rows: 922 us with one producer, 849 with two;
    // two 131072-row sequences 1840 -> 1700).
    if (lane == 0) {
      const uint64_t pol_keep = policy_evict_last();
      uint32_t uc = 0;
      bool ok = true;
      Walk w = walk_begin();
      Seg s;
      while (ok && next_seg(w, s)) {
        const int32_t* bt = p.block_table + (size_t)s.b * p.max_pages;
        const int pb = 4 * s.k0;      // the segment's first page index
        auto entry = [&](int pidx) -> int { return pidx < p.max_pages ? bt[pidx] : -1; };
        int cur[4], nxt[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          cur[q] = entry(pb + q);
          nxt[q] = entry(pb + 4 + q);
        }
        // the previous segment's score MMAs must be done with Q (both halves)
        if (uc > 0 && warp == 0) ok = mbar_wait<false>(bar(kBQFree), (uc - 1) & 1, abort_flag, lim);
        if (!ok) break;
        // (test hook: the leader leaves the query load of its first segment
        // out, so the MMA issuer's wait for it runs out and the launch aborts)
        if (warp == 0 && !(p.withhold_q && leader && uc == 0)) {
          const int row = s.start * p.n_heads + s.row + (int)rank * kHM;
          const uint32_t q_bar = mapa(bar(kBQFull), 0);
          if (leader) mbar_arrive_expect_tx(bar(kBQFull), 2u * kChunks * kQChunk);
          if constexpr (D8) {
            for (int hl = 0; hl < 2; ++hl)
              for (int c = 0; c < kChunks; ++c)
                tma_load_3d_pair(s_q + hl * kQ8Plane + c * kBox8, &tm_q, 64 * c, row, hl, q_bar);
          } else {
            for (int c = 0; c < kChunks; ++c) tma_load_2d_pair(s_q + c * kQChunk, &tm_q, 64 * c, row, q_bar);
          }
        }
        // rows outside the table or the pool read page 0 (readable; they are masked)
        auto page = [&](int pg) -> int { return pg >= 0 && pg < p.num_pages ? pg : 0; };
        // the next stage: false where it is the other producer's (or the launch
        // aborts).  The slot's previous stage, n - kSlots, may be the other
        // producer's (an odd ring); its release is waited for, and the one
        // before that cannot be outstanding (a parity wait would take the one
        // for the other): this producer's last stage, n - 2, went to a slot
        // freed by stage n - 2 - kSlots, and the MMAs free the slots in order.
        auto take = [&](uint32_t& dst, uint32_t& fb) -> bool {
          const uint32_t my = kc++;
          if ((int)(my % kProducers) != warp || !ok) return false;
          const uint32_t slot = my % kSlots;
          const uint32_t ph = (my / kSlots) & 1u;
          ok = mbar_wait<false>(bar(kBEmpty + slot), ph ^ 1u, abort_flag, lim);
          if (!ok) return false;
          if (leader) mbar_arrive_expect_tx(bar(kBFull + slot), 2u * L::kSlotB);
          dst = s_ring + slot * L::kSlotB;
          fb = mapa(bar(kBFull + slot), 0);
          return true;
        };
        // score stages: column chunk c of this CTA's two pages of the tile
        auto load_s = [&](int pg0, int pg1) {
          for (int c = 0; c < kChunks; ++c) {
            uint32_t dst, fb;
            if (!take(dst, fb)) continue;
            tma_load_2d_pair_hint(dst, &tm_cache, 0, (pg0 * kChunks + c) * 64, fb, pol_keep);
            tma_load_2d_pair_hint(dst + L::kSlotB / 2, &tm_cache, 0, (pg1 * kChunks + c) * 64, fb, pol_keep);
          }
        };
        // value stages: per page of tile j with rows, this CTA's two pairs of dims blocks
        auto load_o = [&](int j, const int (&pg)[4]) {
#pragma unroll
          for (int pg_i = 0; pg_i < 4; ++pg_i) {
            if (kTile * (s.k0 + j) + 64 * pg_i >= s.L) break;
            for (int bb = 0; bb < 2; ++bb) {
              uint32_t dst, fb;
              if (!take(dst, fb)) continue;
              tma_load_2d_pair_hint(dst, &tm_cache2, 0, (pg[pg_i] * kChunks + 4 * bb + 2 * (int)rank) * 64, fb,
                                    pol_keep);
            }
          }
        };
        load_s(page(rank ? cur[2] : cur[0]), page(rank ? cur[3] : cur[1]));
        for (int i = 0; i < s.nt && ok; ++i) {
          int ahead[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) ahead[q] = entry(pb + 4 * (i + 2) + q);
          if (i + 1 < s.nt) load_s(page(rank ? nxt[2] : nxt[0]), page(rank ? nxt[3] : nxt[1]));
          int pg[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) pg[q] = page(cur[q]);
          load_o(i, pg);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            cur[q] = nxt[q];
            nxt[q] = ahead[q];
          }
        }
        ++uc;
      }
    }
  } else if (warp == kWarpMma) {
    // ================= MMA issuer (leader CTA, whole warp, one elected lane) =================
    if (leader) {
      constexpr uint32_t idS = D8 ? idesc_e4m3(kM, 256, false, false) : idesc_f16(kM, 256, false, false);
      constexpr uint32_t idO = D8 ? idesc_e4m3(kM, 256, false, true) : idesc_f16(kM, 256, false, true);
      constexpr uint32_t idO_lo = idesc_e4m3(kM, 256, false, true, true);    // D8: the weights' second term is e5m2
      // Stages are taken in groups (three score chunks, a page's two value
      // boxes), whose barriers are waited for together.  The tensor cores hold
      // little more than one MMA in advance, so whatever stands between a
      // stage's last MMA and the next one's first is a gap (two 131072-row
      // sequences 2.30 -> 2.11 ms a call, e4m3 515 -> 492 us).
      uint32_t slot = 0, ph = 0;
      auto step = [&](uint32_t& sl, uint32_t& q) {
        if (++sl == kSlots) {
          sl = 0;
          q ^= 1u;
        }
      };
      auto ready = [&](auto n, uint32_t (&at)[decltype(n)::value]) -> bool {
        constexpr int N = decltype(n)::value;
        uint32_t q[N];
        bool full = true;
#pragma unroll
        for (int k = 0; k < N; ++k) {
          at[k] = slot;
          q[k] = ph;
          full &= mbar_try_wait<false>(bar(kBFull + slot), ph);
          step(slot, ph);
        }
        if (!__all_sync(0xffffffffu, full)) {
#pragma unroll
          for (int k = 0; k < N; ++k)
            if (!__all_sync(0xffffffffu, mbar_wait<false>(bar(kBFull + at[k]), q[k], abort_flag, lim))) return false;
        }
        tc_fence_after();
        return true;
      };
      uint32_t uc = 0, gt = 0;
      bool ok = true;
      Walk w = walk_begin();
      Seg s;
      while (ok && next_seg(w, s)) {
        ok = __all_sync(0xffffffffu, mbar_wait<false>(bar(kBQFull), uc & 1, abort_flag, lim));
        if (!ok) break;
        tc_fence_after();
        auto issue_s = [&](int i) -> bool {
          const uint32_t sb = (gt + i) & 1u;
          const uint32_t d = tmem + kColS + 128 * sb;
          for (int c0 = 0; c0 < kChunks; c0 += 3) {
            uint32_t at[3];
            if (!ready(std::integral_constant<int, 3>(), at)) return false;
#pragma unroll
            for (int k = 0; k < 3; ++k) {
              const int c = c0 + k;
              const uint32_t a0 = s_ring + at[k] * L::kSlotB;
              if constexpr (D8) {
                const uint64_t qd = smem_desc_sw64(s_q, 16, 512);
                const uint64_t kd = smem_desc_sw64(a0, 16, 512);
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                  for (int hl = 0; hl < 2; ++hl)
                    mma_pair_e4m3_w(d, qd + ((hl * kQ8Plane + c * kBox8 + ks * 32) >> 4), kd + ((ks * 32) >> 4), idS,
                                    (c | ks | hl) != 0);
              } else {
                const uint64_t qd = smem_desc_sw128(s_q, 16, 1024);
                const uint64_t kd = smem_desc_sw128(a0, 16, 1024);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)   // K = 16 per MMA: +32 bytes along the 128-byte lines
                  mma_pair_f16_w(d, qd + ((c * kQChunk + ks * 32) >> 4), kd + ((ks * 32) >> 4), idS, (c | ks) != 0);
              }
              mma_commit_pair_w(bar(kBEmpty + at[k]), 0x3);
            }
          }
          mma_commit_pair_w(bar(kBSFull + sb), 0x3);
          // the segment's last score GEMM: Q may be replaced once it completes
          if (i == s.nt - 1) mma_commit_pair_w(bar(kBQFree), 0x3);
          return true;
        };
        auto issue_o = [&](int j) -> bool {
          const uint32_t t = gt + j;
          if (!__all_sync(0xffffffffu, mbar_wait<false>(bar(kBPFull), t & 1, abort_flag, lim))) return false;
          // the accumulator is overwritten by this segment's first value MMA:
          // the previous segment's epilogue must have read it out
          if (j == 0 && uc > 0 &&
              !__all_sync(0xffffffffu, mbar_wait(bar(kBEpiDone), (uc - 1) & 1, abort_flag, lim)))
            return false;
          tc_fence_after();
          for (int pg_i = 0; pg_i < 4; ++pg_i) {
            if (kTile * (s.k0 + j) + 64 * pg_i >= s.L) break;
            uint32_t at[2];
            if (!ready(std::integral_constant<int, 2>(), at)) return false;
#pragma unroll
            for (int bb = 0; bb < 2; ++bb) {
              const uint32_t b0 = s_ring + at[bb] * L::kSlotB;
              if constexpr (D8) {
                const uint64_t pd = smem_desc_sw64(s_p + pg_i * kPChunk, 16, 512);
                const uint64_t vd = smem_desc_sw64(b0, kBox8, 512);
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                  for (int hl = 0; hl < 2; ++hl)
                    mma_pair_e4m3_w(tmem + kColO + 128 * bb, pd + ((hl * kBox8 + ks * 32) >> 4),
                                    vd + ((ks * 2048) >> 4), hl ? idO_lo : idO, (j | pg_i | ks | hl) != 0);
              } else {
                const uint64_t pd = smem_desc_sw128(s_p + pg_i * kPChunk, 16, 1024);
                const uint64_t vd = smem_desc_sw128(b0, kBox, 1024);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)   // 16 rows per MMA: +32 bytes of P lines, +2 KB of V lines
                  mma_pair_f16_w(tmem + kColO + 128 * bb, pd + ((ks * 32) >> 4), vd + ((ks * 2048) >> 4), idO,
                                 (j | pg_i | ks) != 0);
              }
              mma_commit_pair_w(bar(kBEmpty + at[bb]), 0x3);
            }
          }
          mma_commit_pair_w(bar(kBODone), 0x3);
          return true;
        };
        ok = issue_s(0);
        for (int i = 0; i < s.nt && ok; ++i) {
          if (i + 1 < s.nt) ok = issue_s(i + 1);
          if (ok) ok = issue_o(i);
        }
        gt += s.nt;
        ++uc;
      }
    }
  } else {
    // ================= softmax (both CTAs, warps 3-10) =================
    // Thread (lane quadrant q4, column half ch, lane) owns row hh = 32 (q4 & 1)
    // + lane of this CTA and the 64 tile rows 128 (q4 >> 1) + 64 ch .. +63.
    const int q4 = warp & 3;
    const int half = q4 >> 1;                   // 0: TMEM lanes 0-63, 1: lanes 64-127
    const int hh = 32 * (q4 & 1) + lane;        // row within this CTA
    const int ch = (warp - kWarpSoft0) >> 2;    // score columns [64 ch, 64 ch + 64)
    const uint32_t lane_addr = static_cast<uint32_t>(32 * q4) << 16;
    const int part = 2 * half + ch;             // which of the row's four partial results (= page of the tile)
    uint32_t soft_ph = 0;
    auto soft_sync = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive_local(bar(kBSoft));
      const bool okk = __all_sync(0xffffffffu, mbar_wait<false>(bar(kBSoft), soft_ph & 1, abort_flag, lim));
      ++soft_ph;
      return okk;
    };
    uint32_t gt = 0;
    bool ok = true;
    Walk w = walk_begin();
    Seg s;
    while (ok && next_seg(w, s)) {
      const int seq_rows = s.n * p.n_heads;
      const int my = s.row + kHM * (int)rank + hh;            // this thread's (node, head) row of the sequence
      const int node = min(my, seq_rows - 1) / p.n_heads;     // rows past the end follow the last node
      const size_t grow = (size_t)s.start * p.n_heads + my;   // ... of the whole call
      const int prefix = s.L - s.n;
      const uint64_t* mask = p.tree_mask ? p.tree_mask + (size_t)(s.start + node) * p.mask_words : nullptr;
      float slq = p.scale_log2;
      if constexpr (D8) {
        if (my < seq_rows) slq *= p.q_scale[grow];
      }
      float* page_sc = reinterpret_cast<float*>(misc + kMScale) + part * 64;   // D8: see softmax_q8.cuh
      float m_run = -INFINITY, m_top = -INFINITY, l_acc = 0.f;
      for (int i = 0; i < s.nt; ++i) {
        const uint32_t t = gt + i;
        const uint32_t sb = t & 1u;
        // cached rows of this thread: one page of the sequence
        const int row0 = kTile * (s.k0 + i) + 128 * half + 64 * ch;
        const int nrows = min(max(s.L - row0, 0), 64);
        uint64_t vis = 0;
        float sc_lo = 0.f, sc_hi = 0.f;   // e4m3: the page's dequantisation scales (lane l: rows l, l + 32)
        if (nrows > 0) {
          const int pg = page_or_minus1(p, s.b, row0 >> 6);
          if (pg < 0) {
            flag_error(p.err, MLA_DEVERR_PAGE);
          } else {
            vis = visible_rows(row0, prefix, s.n, node, mask, p.mask_words);
            if constexpr (D8) {
              if (lane < nrows) sc_lo = p.cache_scale[(size_t)pg * 64 + lane];
              if (lane + 32 < nrows) sc_hi = p.cache_scale[(size_t)pg * 64 + 32 + lane];
            }
          }
        }
        float* page_inv = page_sc + (2 + sb) * q8::kPlane;
        if constexpr (D8) q8::put_scales(page_sc, page_inv, lane, sc_lo, sc_hi);
        const bool full = __all_sync(0xffffffffu, vis == ~0ull);
        ok = __all_sync(0xffffffffu, mbar_wait<false>(bar(kBSFull + sb), (t >> 1) & 1, abort_flag, lim));
        if (!ok) break;
        tc_fence_after();
        const uint32_t scol = tmem + lane_addr + kColS + 128 * sb;
        float v[64];
        tmem_ld<32>(scol + 64 * ch, v);
        tmem_ld<32>(scol + 64 * ch + 32, v + 32);
        tmem_wait_ld();
        float mx = -INFINITY;
        if constexpr (D8) {
          q8::scores(v, slq, page_sc);
        } else {
#pragma unroll
          for (int j = 0; j < 64; ++j) v[j] *= slq;
        }
        if (!full) {
          const uint32_t vlo = (uint32_t)vis, vhi = (uint32_t)(vis >> 32);
#pragma unroll
          for (int j = 0; j < 64; ++j)
            if (!((j < 32 ? vlo : vhi) >> (j & 31) & 1u)) v[j] = -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < 64; ++j) mx = fmaxf(mx, v[j]);
        // the four partial maxima of each row, double-buffered by tile parity:
        // a warp writes the next tile's slot only after passing this tile's
        // sync, so no warp can overwrite a slot that another is still reading
        float* rm = red_max + sb * 4 * kHM;
        rm[part * kHM + hh] = mx;
        if (!(ok = soft_sync())) break;
        const float tmax = fmaxf(fmaxf(rm[hh], rm[kHM + hh]), fmaxf(rm[2 * kHM + hh], rm[3 * kHM + hh]));
        float m_new;
        if constexpr (D8) m_new = q8::reference(m_run, tmax, m_top);
        else m_new = tmax > m_run + kRescaleLog2 ? tmax : m_run;
        const bool changed = m_new != m_run;
        // factor for the sums and the accumulator kept so far (0 when nothing was kept)
        const float alpha = (m_run == -INFINITY) ? 0.f : exp2_approx(m_run - m_new);
        m_run = m_new;
        uint32_t pk[32];   // D8: pk[0..15] the hi codes of the 64 rows, pk[16..31] the lo codes
        float sum = 0.f;
        if constexpr (D8) {
          sum = q8::weights(v, m_new, page_inv, pk);
        } else {
          const float msub = m_new == -INFINITY ? 0.f : m_new;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float p0 = exp2_approx(v[2 * j] - msub), p1 = exp2_approx(v[2 * j + 1] - msub);
            sum += p0 + p1;
            pk[j] = pack_bf16(p0, p1);
          }
        }
        l_acc = changed ? fmaf(l_acc, alpha, sum) : l_acc + sum;
        // every phase of o_done is observed in order (a parity wait cannot
        // tell a phase two behind from a completed one); O(i-1) done also
        // frees the P tiles for this tile's probabilities
        if (i >= 1) {
          ok = __all_sync(0xffffffffu, mbar_wait<false>(bar(kBODone), (t - 1) & 1, abort_flag, lim));
          if (!ok) break;
          tc_fence_after();
          if (__any_sync(0xffffffffu, changed)) {
            const float f = changed ? alpha : 1.f;
            const uint32_t oc = tmem + lane_addr + kColO + 128 * ch;
#pragma unroll 1
            for (int c4 = 0; c4 < 4; ++c4) {
              float o[32];
              tmem_ld<32>(oc + 32 * c4, o);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] *= f;
              tmem_st<32>(oc + 32 * c4, o);
            }
          }
        }
        if constexpr (D8) {
#pragma unroll
          for (int hl = 0; hl < 2; ++hl) {
            uint8_t* line = s_pbuf + part * kPChunk + hl * kBox8 + hh * 64;
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<uint4*>(line + ((q ^ ((hh >> 1) & 3)) << 4)) =
                  make_uint4(pk[16 * hl + 4 * q], pk[16 * hl + 4 * q + 1], pk[16 * hl + 4 * q + 2],
                             pk[16 * hl + 4 * q + 3]);
          }
        } else {
          uint8_t* line = s_pbuf + part * kPChunk + hh * 128;
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<uint4*>(line + ((q ^ (hh & 7)) << 4)) =
                make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
        }
        fence_proxy_async_cta();     // read by the tensor core
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_cta(mapa(bar(kBPFull), 0));
      }
      // ---- epilogue: normalise O by the row sums; the final result where the
      // segment covers the whole row tile, else a partial for the merge
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait<false>(bar(kBODone), (gt + s.nt - 1) & 1, abort_flag, lim));
      if (ok) {
        tc_fence_after();
        red_sum[part * kHM + hh] = l_acc;
        ok = soft_sync();
      }
      if (ok) {
        const float lt = red_sum[hh] + red_sum[kHM + hh] + red_sum[2 * kHM + hh] + red_sum[3 * kHM + hh];
        const float inv_l = lt == 0.f ? 0.f : 1.f / lt;        // (a NaN sum, of NaN scores, stays one)
        const bool whole = s.nt == s.kt;
        // a first segment that continues a row tile: slot 2 pair; a last one that leaves its row tile open: 2 pair + 1
        const int slot = 2 * pair + (s.k0 == 0 ? 1 : 0);
        if (part == 0) {
          const float lv = lt == 0.f ? -INFINITY : (m_run - (D8 ? q8::kLog : 0.f) + log2f(lt)) * 0.69314718055994531f;
          if (!whole) p.part_lse[slot * kM + kHM * (int)rank + hh] = lv;
          else if (p.lse && my < seq_rows) p.lse[grow] = lv;
        }
        if (!whole && s.k0 == 0 && leader && part == 0 && hh == 0) {
          // the pair that holds the row tile's last cached tile: pairs q own [q total / used, ...)
          const long long end = (long long)s.g + s.kt;
          const int q_last = (int)((end * used + total - 1) / total) - 1;
          p.desc[pair] = TreeDesc{s.start * p.n_heads + s.row, min(kM, seq_rows - s.row), q_last - pair, 0};
        }
        // this thread's O: dims 256 ch + 128 half + (0..127) of its row, moved
        // through a 4 KB tile of this warp in the P area (idle until the next
        // segment's first probabilities, which these warps write), so that a
        // store instruction covers whole 128-byte lines of four rows
        const uint32_t oc = tmem + lane_addr + kColO + 128 * ch;
        uint8_t* tile = s_pbuf + (warp - kWarpSoft0) * 4096;
        const int rd_row = lane >> 3, rd_q = lane & 7;    // reader: row 4 k + rd_row, 16-byte piece rd_q
        const int row_w = kHM * (int)rank + 32 * (q4 & 1);    // this warp's first row of the tile
        const int dim0 = 256 * ch + 128 * half;
        const int rows_w = min(32, seq_rows - s.row - row_w);   // rows to store (partials: the valid ones too)
        if (whole && !p.o_f32) {
          __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.o_lat) +
                               ((size_t)s.start * p.n_heads + s.row + row_w) * MLA_D_C + dim0 + 8 * rd_q;
#pragma unroll 1
          for (int c2 = 0; c2 < 2; ++c2) {
            float o[64];
            tmem_ld<32>(oc + 64 * c2, o);
            tmem_ld<32>(oc + 64 * c2 + 32, o + 32);
            tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < 8; ++q)
              *reinterpret_cast<uint4*>(tile + lane * 128 + ((q ^ (lane & 7)) << 4)) =
                  make_uint4(pack_bf16(o[8 * q] * inv_l, o[8 * q + 1] * inv_l),
                             pack_bf16(o[8 * q + 2] * inv_l, o[8 * q + 3] * inv_l),
                             pack_bf16(o[8 * q + 4] * inv_l, o[8 * q + 5] * inv_l),
                             pack_bf16(o[8 * q + 6] * inv_l, o[8 * q + 7] * inv_l));
            __syncwarp();
#pragma unroll 4
            for (int k4 = 0; k4 < 8; ++k4) {
              const int j = 4 * k4 + rd_row;
              if (j < rows_w)
                *reinterpret_cast<uint4*>(dst + (size_t)j * MLA_D_C + 64 * c2) =
                    *reinterpret_cast<const uint4*>(tile + j * 128 + ((rd_q ^ (j & 7)) << 4));
            }
            __syncwarp();
          }
        } else if (whole) {
          float* dst = reinterpret_cast<float*>(p.o_lat) + ((size_t)s.start * p.n_heads + s.row + row_w) * MLA_D_C +
                       dim0 + 4 * rd_q;
#pragma unroll 1
          for (int c4 = 0; c4 < 4; ++c4) {
            float o[32];
            tmem_ld<32>(oc + 32 * c4, o);
            tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < 8; ++q)
              *reinterpret_cast<float4*>(tile + lane * 128 + ((q ^ (lane & 7)) << 4)) =
                  make_float4(o[4 * q] * inv_l, o[4 * q + 1] * inv_l, o[4 * q + 2] * inv_l, o[4 * q + 3] * inv_l);
            __syncwarp();
#pragma unroll 4
            for (int k4 = 0; k4 < 8; ++k4) {
              const int j = 4 * k4 + rd_row;
              if (j < rows_w)
                *reinterpret_cast<float4*>(dst + (size_t)j * MLA_D_C + 32 * c4) =
                    *reinterpret_cast<const float4*>(tile + j * 128 + ((rd_q ^ (j & 7)) << 4));
            }
            __syncwarp();
          }
        } else {
          // a partial keeps the order in which the lanes hold it (see part_at): whole lines, nothing to move
          float4* dst = reinterpret_cast<float4*>(p.part_o + (size_t)slot * kM * MLA_D_C) +
                        part_at((int)rank, ch, q4, 0) + lane;
#pragma unroll 1
          for (int c2 = 0; c2 < 2; ++c2) {
            float o[64];
            tmem_ld<32>(oc + 64 * c2, o);
            tmem_ld<32>(oc + 64 * c2 + 32, o + 32);
            tmem_wait_ld();
            if (my < seq_rows)
#pragma unroll
              for (int q = 0; q < 16; ++q)
                dst[32 * (16 * c2 + q)] =
                    make_float4(o[4 * q] * inv_l, o[4 * q + 1] * inv_l, o[4 * q + 2] * inv_l, o[4 * q + 3] * inv_l);
          }
        }
        // this warp's part of O has been read: the pair's next segment may overwrite it
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa(bar(kBEpiDone), 0));
      }
      gt += s.nt;
    }
  }

  // ---- teardown
  __syncwarp();
  if (*abort_flag) {
    if (threadIdx.x == 0) flag_error(p.err, MLA_DEVERR_TIMEOUT);
    // let copies and MMAs already in flight land before the memory is released
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 2000000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

__device__ __forceinline__ void store4(float* dst, float4 v, float f) {
  *reinterpret_cast<float4*>(dst) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
}
__device__ __forceinline__ void store4(__nv_bfloat16* dst, float4 v, float f) {
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(v.x * f, v.y * f), pack_bf16(v.z * f, v.w * f));
}

// Joins the partials of the row tiles that crossed a pair's border: pair p's
// last segment (slot 2 p + 1) and the first segments (slot 2 q) of the pairs
// that follow it.  A warp takes 32 rows of pair p's row tile, a lane each (the
// partials' order), and 8 channels of them; CTA (p, y) has eight of the
// tile's 256 such pieces.  Each partial is read once, and a call of few tiles
// is bound by latency: a descriptor, then kBatch parts' loads at once.  The
// launch takes 16 where a row tile is likely cut into more than four parts
// (16 parts: 25.2 us a call with 8 at a time, 23.1 with 16), else 4, which
// leaves room for more warps (two or three parts: 137 us with 16, 126 with 4).
constexpr int kMergeWarps = 8;
constexpr int kMergePieces = 256;

template <typename OT, int kBatch>
__global__ void __launch_bounds__(32 * kMergeWarps) tree_merge_kernel(const float* __restrict__ part_o,
                                                                      const float* __restrict__ part_lse,
                                                                      const TreeDesc* __restrict__ desc,
                                                                      OT* __restrict__ o_lat,
                                                                      float* __restrict__ lse_out) {
  griddep_wait();
  griddep_launch_dependents();
  const int pair = blockIdx.x;
  const TreeDesc d = desc[pair];
  if (d.follow == 0) return;
  const int lane = threadIdx.x & 31, piece = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
  const int rank = piece >> 7, q4 = (piece >> 5) & 3, ch = (piece >> 4) & 1, q = 2 * (piece & 15);
  const int row = 64 * rank + 32 * (q4 & 1) + lane;      // of the row tile
  if (row - lane >= d.rows) return;
  const int parts = d.follow + 1;
  auto slot = [&](int k) -> size_t { return k == 0 ? 2 * pair + 1 : 2 * (pair + k); };
  const float4* src = reinterpret_cast<const float4*>(part_o) + part_at(rank, ch, q4, q) + lane;
  float mx = -INFINITY, sum = 0.f;
  float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int k0 = 0; k0 < parts; k0 += kBatch) {
    float4 v[kBatch][2];
    float w[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      w[k] = -INFINITY;
      if (k0 + k < parts) {
        const size_t sl = slot(k0 + k);
        w[k] = part_lse[sl * kM + row];
        v[k][0] = src[sl * (kM * MLA_D_C / 4)];
        v[k][1] = src[sl * (kM * MLA_D_C / 4) + 32];
      } else {
        v[k][0] = v[k][1] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    // what was joined so far is scaled to the new maximum
    float top = mx;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) top = fmaxf(top, w[k]);
    if (top == -INFINITY) {                  // nothing seen so far, unless a NaN that the maximum passed over
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (isnan(w[k])) sum = w[k];
      continue;
    }
    const float old = expf(mx - top);
    mx = top;
    sum *= old;
#pragma unroll
    for (int i = 0; i < 2; ++i) acc[i] = make_float4(acc[i].x * old, acc[i].y * old, acc[i].z * old, acc[i].w * old);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float wk = expf(w[k] - mx);
      sum += wk;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        acc[i].x = fmaf(wk, v[k][i].x, acc[i].x);
        acc[i].y = fmaf(wk, v[k][i].y, acc[i].y);
        acc[i].z = fmaf(wk, v[k][i].z, acc[i].z);
        acc[i].w = fmaf(wk, v[k][i].w, acc[i].w);
      }
    }
  }
  if (row >= d.rows) return;
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;
  const size_t out = (size_t)d.row0 + row;
  const int dim = 256 * ch + 128 * (q4 >> 1) + 4 * q;
#pragma unroll
  for (int i = 0; i < 2; ++i) store4(o_lat + out * MLA_D_C + dim + 4 * i, acc[i], inv);
  if (lse_out && dim == 0) lse_out[out] = sum == 0.f ? -INFINITY : mx + logf(sum);
}

// The two-term e4m3 query of the 8-bit form: per (node, head) vector
//   scale = 2^(floor(log2 max|q|) - 7),  y = q / scale,  hi = e4m3(y),  lo = e4m3(y - hi)
// A bf16 value has 8 significant bits and e4m3 has 4: hi takes the upper ones
// and y - hi, at most half a step of hi, is a whole number of at most 8 of
// y's own units, so lo holds it exactly unless it falls below e4m3's smallest
// step 2^-9, i.e. for components under 2^-9 of the largest, whose error is at
// most 2^-17 of the largest.  A power-of-two scale is what makes it exact.
// One warp per vector, as in split_q.cu; planes [2][rows][576].
__global__ void __launch_bounds__(256) split_q_tree_kernel(const __nv_bfloat16* __restrict__ q_abs, int n_vec,
                                                           uint8_t* __restrict__ q8, float* __restrict__ q_scale) {
  griddep_wait();
  griddep_launch_dependents();
  const int vec = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (vec >= n_vec) return;
  const uint32_t* src = reinterpret_cast<const uint32_t*>(q_abs + (size_t)vec * MLA_D_ROW);
  float2 x[9];
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < 9; ++k) {
    const uint32_t w = src[lane + 32 * k];
    x[k] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
    amax = fmaxf(amax, fmaxf(fabsf(x[k].x), fabsf(x[k].y)));
  }
  amax = warp_max(amax);
  // exponent field of amax, kept where scale and 1 / scale are both normal numbers
  const int e = min(max((int)(__float_as_uint(amax) >> 23), 8), 253);
  const float scale = __uint_as_float((uint32_t)(e - 7) << 23);          // 2^(e - 127 - 7)
  const float inv = __uint_as_float((uint32_t)(254 - (e - 7)) << 23);    // its reciprocal
  uint16_t* hi = reinterpret_cast<uint16_t*>(q8 + (size_t)vec * MLA_D_ROW);
  uint16_t* lo = reinterpret_cast<uint16_t*>(q8 + ((size_t)n_vec + vec) * MLA_D_ROW);
#pragma unroll
  for (int k = 0; k < 9; ++k) {
    uint32_t h2, l2;
    split_e4m3x2(x[k].x * inv, x[k].y * inv, h2, l2);
    hi[lane + 32 * k] = (uint16_t)h2;
    lo[lane + 32 * k] = (uint16_t)l2;
  }
  if (lane == 0) q_scale[vec] = scale;
}

// ------------------------------------------------------------------ fp32 cache
// Exact fp32 on the CUDA cores, for small models: CTA = (split of the
// sequence's rows, group of 16 heads, node), four heads per warp, rows staged
// 16 at a time in shared memory while the previous 16 are worked.  Each
// sequence is cut into `splits` equal runs of whole 8-row groups: a call of few
// nodes still fills the GPU, down to one group per CTA, since what bounds it is
// the latency of a CTA's chain of loads, products and reductions (4 nodes x 16
// heads x 260 rows: 10.1 us with the merge).  Many nodes are bound by issue and
// by the reads of the staged rows: a row that a warp reads serves four heads,
// and four rows are worked at a time (8 sequences x 16 nodes x 32 heads x 2064
// rows: 803 us, 22.7 TFLOP/s; two heads per warp, a row at a time and nothing
// staged ahead: 1217 us).  tree_merge_f32_kernel joins the splits.
constexpr int kSimtRows = 16;
constexpr int kSimtGroup = 8;
constexpr int kSimtHeads = 16;
constexpr int kSimtPer = 4;                  // heads per warp
constexpr int kSimtWarps = kSimtHeads / kSimtPer;

// The sequence of node n (-1: n lies outside [row_start[0], row_start[batch]),
// or the sequence's numbers are bad).
__device__ __forceinline__ int seq_of(const TreeParams& p, int n, SeqInfo& s) {
  if (n < p.row_start[0] || n >= p.row_start[p.batch]) return -1;
  int lo = 0, hi = p.batch - 1;             // the last sequence that starts at or before n
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.row_start[mid] <= n) lo = mid; else hi = mid - 1;
  }
  s = seq_info(p, lo);
  return s.bad || n < s.start || n >= s.start + s.n ? -1 : lo;
}

// Sums of sixteen values over the warp: the value of index lane >> 1, on every lane.
__device__ __forceinline__ float warp_sum16(const float (&v)[16]) {
  const int lane = threadIdx.x & 31;
  float a[8], b[4], c[2];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool up = lane & 16;
    a[i] = (up ? v[i + 8] : v[i]) + __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + 8], 16);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool up = lane & 8;
    b[i] = (up ? a[i + 4] : a[i]) + __shfl_xor_sync(0xffffffffu, up ? a[i] : a[i + 4], 8);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool up = lane & 4;
    c[i] = (up ? b[i + 2] : b[i]) + __shfl_xor_sync(0xffffffffu, up ? b[i] : b[i + 2], 4);
  }
  const bool up = lane & 2;
  const float d = (up ? c[1] : c[0]) + __shfl_xor_sync(0xffffffffu, up ? c[0] : c[1], 2);
  return d + __shfl_xor_sync(0xffffffffu, d, 1);
}

// 16 bytes of global memory to shared memory, asynchronously; zeros where !from.
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src, bool from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)),
               "r"(from ? 16 : 0)
               : "memory");
}

__global__ void __launch_bounds__(32 * kSimtWarps, 2) decode_tree_simt_kernel(const float* __restrict__ q_abs,
                                                                              const float* __restrict__ cache,
                                                                              TreeParams p, int splits) {
  extern __shared__ __align__(16) float tiles[];       // [2][kSimtRows][576]
  __shared__ int seen_of[2][kSimtRows];
  __shared__ __align__(16) float score[kSimtWarps][kSimtPer][kSimtRows];   // scores, then weights, of the staged rows
  griddep_wait();
  griddep_launch_dependents();
  const int split = blockIdx.x, n = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h0 = blockIdx.y * kSimtHeads + kSimtPer * warp;
  const int heads = min(max(p.n_heads - h0, 0), kSimtPer);      // of this warp
  const size_t vec = (size_t)n * p.n_heads + h0;
  float q[kSimtPer][18];
#pragma unroll
  for (int e = 0; e < kSimtPer; ++e)
#pragma unroll
    for (int k = 0; k < 18; ++k) q[e][k] = e < heads ? q_abs[(vec + e) * MLA_D_ROW + lane + 32 * k] : 0.f;
  SeqInfo s;
  const int b = seq_of(p, n, s);
  if (b < 0) {
    if (threadIdx.x == 0 && n >= p.row_start[0] && n < p.row_start[p.batch]) flag_error(p.err, MLA_DEVERR_POSITION);
    return;
  }
  const int node = n - s.start, prefix = s.L - s.n;
  const int groups = (s.L + kSimtGroup - 1) / kSimtGroup;
  const int lo = (int)((long long)groups * split / splits) * kSimtGroup;
  const int hi = min((int)((long long)groups * (split + 1) / splits) * kSimtGroup, s.L);
  const uint64_t* mask = p.tree_mask ? p.tree_mask + (size_t)n * p.mask_words : nullptr;
  float m[kSimtPer], l[kSimtPer];
  float o[kSimtPer][16];
#pragma unroll
  for (int e = 0; e < kSimtPer; ++e) {
    m[e] = -INFINITY;
    l[e] = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) o[e][k] = 0.f;
  }
  // stage rows j0 .. j0 + 15: warp w rows w, w + 4, ...; rows that the node
  // does not see (or past the end) as zeros, whatever the cache holds there
  auto stage = [&](int j0, int buf) {
#pragma unroll
    for (int x = 0; x < kSimtRows / kSimtWarps; ++x) {
      const int r = warp + kSimtWarps * x, j = j0 + r;
      int pg = -1;
      bool seen = false;
      if (j < hi) {
        pg = page_or_minus1(p, b, j >> 6);
        if (pg < 0) flag_error(p.err, MLA_DEVERR_PAGE);
        seen = pg >= 0 && (visible_rows(j, prefix, s.n, node, mask, p.mask_words) & 1);
      }
      if (lane == 0) seen_of[buf][r] = seen;
      // a row's piece c (16 bytes): block c / 16 of its page
      const float* src = cache + ((size_t)(seen ? pg : 0) * 9 * 64 + (j & 63)) * 64;
      const uint32_t dst = smem_u32(tiles + (buf * kSimtRows + r) * MLA_D_ROW);
#pragma unroll
      for (int i = 0; i < 5; ++i) {
        const int c = lane + 32 * i;
        if (c < MLA_D_ROW / 4) copy_async16(dst + 16 * c, src + (c >> 4) * 64 * 64 + 4 * (c & 15), seen);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (lo < hi) stage(lo, 0);
  for (int j0 = lo, buf = 0; j0 < hi; j0 += kSimtRows, buf ^= 1) {
    const int cnt4 = (min(kSimtRows, hi - j0) + 3) & ~3;         // rows are worked four at a time
    if (j0 + kSimtRows < hi) {
      stage(j0 + kSimtRows, buf ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    const float* tile = tiles + buf * kSimtRows * MLA_D_ROW;
    if (heads > 0) {
      for (int jj = 0; jj < cnt4; jj += 4) {
        float part[16];                        // [head][row]
#pragma unroll
        for (int x = 0; x < 16; ++x) part[x] = 0.f;
        const float* rows = tile + jj * MLA_D_ROW + lane;
#pragma unroll
        for (int k = 0; k < 18; ++k) {
          float t[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) t[x] = rows[x * MLA_D_ROW + 32 * k];
#pragma unroll
          for (int e = 0; e < kSimtPer; ++e)
#pragma unroll
            for (int x = 0; x < 4; ++x) part[4 * e + x] = fmaf(q[e][k], t[x], part[4 * e + x]);
        }
        const float v = warp_sum16(part);
        if ((lane & 1) == 0) score[warp][lane >> 3][jj + ((lane >> 1) & 3)] = v;
      }
      __syncwarp();
      const bool seen = lane < kSimtRows && seen_of[buf][lane & (kSimtRows - 1)];   // row j0 + lane
#pragma unroll
      for (int e = 0; e < kSimtPer; ++e) {
        const float sc = seen ? score[warp][e][lane & (kSimtRows - 1)] * p.scale_log2 : -INFINITY;   // natural units here, see the launch
        const float mn = fmaxf(m[e], warp_max(sc));
        const float ms = mn == -INFINITY ? 0.f : mn;      // nothing seen so far: every weight is 0
        const float alpha = expf(m[e] - ms), pr = expf(sc - ms);
        if (lane < kSimtRows) score[warp][e][lane] = pr;
        l[e] = l[e] * alpha + warp_sum(pr);
#pragma unroll
        for (int k = 0; k < 16; ++k) o[e][k] *= alpha;
        m[e] = mn;
      }
      __syncwarp();
      for (int jj = 0; jj < cnt4; jj += 4) {
        float4 w[kSimtPer];
#pragma unroll
        for (int e = 0; e < kSimtPer; ++e) w[e] = *reinterpret_cast<const float4*>(&score[warp][e][jj]);
        const float* rows = tile + jj * MLA_D_ROW + lane;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float t0 = rows[32 * k], t1 = rows[MLA_D_ROW + 32 * k], t2 = rows[2 * MLA_D_ROW + 32 * k],
                      t3 = rows[3 * MLA_D_ROW + 32 * k];
#pragma unroll
          for (int e = 0; e < kSimtPer; ++e)
            o[e][k] = fmaf(w[e].w, t3, fmaf(w[e].z, t2, fmaf(w[e].y, t1, fmaf(w[e].x, t0, o[e][k]))));
        }
      }
    }
    __syncthreads();                         // the buffer may be staged again
  }
#pragma unroll
  for (int e = 0; e < kSimtPer; ++e) {
    if (e >= heads) break;
    const size_t base = (vec + e) * splits + split;
    const float inv = l[e] == 0.f ? 0.f : 1.0f / l[e];
#pragma unroll
    for (int k = 0; k < 16; ++k) p.part_o[base * MLA_D_C + lane + 32 * k] = o[e][k] * inv;
    if (lane == 0) p.part_lse[base] = l[e] == 0.f ? -INFINITY : m[e] + logf(l[e]);
  }
}

// CTA = one (node, head) vector; four groups of 128 threads take every fourth
// split, so that all splits' loads are in flight at once.
template <typename OT>
__global__ void __launch_bounds__(512) tree_merge_f32_kernel(TreeParams p, int splits) {
  __shared__ float4 sums[4][128];
  griddep_wait();
  griddep_launch_dependents();
  const size_t vec = blockIdx.x;
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 7, c = threadIdx.x & 127;
  // every load is independent of the others: the row's validity is looked at before the store only
  const float* lp = p.part_lse + vec * splits;
  const float4* op = reinterpret_cast<const float4*>(p.part_o + vec * splits * MLA_D_C) + c;
  float l0 = lane < splits ? lp[lane] : -INFINITY, l1 = lane + 32 < splits ? lp[lane + 32] : -INFINITY;
  float4 v[16];                              // at most 64 splits
#pragma unroll
  for (int k = 0; k < 16; ++k)
    v[k] = grp + 4 * k < splits ? op[(size_t)(grp + 4 * k) * (MLA_D_C / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
  SeqInfo s;
  const bool valid = seq_of(p, (int)(vec / p.n_heads), s) >= 0;
  const float mx = warp_max(fmaxf(l0, l1));
  const float ref = mx == -INFINITY ? 0.f : mx;          // nothing seen: weights e^-inf (a NaN stays one)
  l0 = expf(l0 - ref);
  l1 = expf(l1 - ref);
  const float sum = warp_sum(l0 + l1);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float w = __shfl_sync(0xffffffffu, k < 8 ? l0 : l1, (grp + 4 * k) & 31);
    acc.x = fmaf(w, v[k].x, acc.x);
    acc.y = fmaf(w, v[k].y, acc.y);
    acc.z = fmaf(w, v[k].z, acc.z);
    acc.w = fmaf(w, v[k].w, acc.w);
  }
  sums[grp][c] = acc;
  __syncthreads();
  if (grp || !valid) return;
#pragma unroll
  for (int g = 1; g < 4; ++g) {
    const float4 x = sums[g][c];
    acc.x += x.x;
    acc.y += x.y;
    acc.z += x.z;
    acc.w += x.w;
  }
  store4(reinterpret_cast<OT*>(p.o_lat) + vec * MLA_D_C + 4 * c, acc, sum == 0.f ? 0.f : 1.0f / sum);
  if (p.lse && c == 0) p.lse[vec] = sum == 0.f ? -INFINITY : mx + logf(sum);
}

// ------------------------------------------------------------------ host side
// Splits of the fp32 form: enough CTAs for four per SM of a B200, at most 64.
constexpr int kSimtCtas = 4 * 148, kSimtSplits = 64;
int splits_f32(long long rows, int n_heads) {
  const long long ctas = rows * ((n_heads + kSimtHeads - 1) / kSimtHeads);
  const long long want = (kSimtCtas + ctas - 1) / ctas;
  return (int)(want < kSimtSplits ? want : kSimtSplits);
}

// Partials that a call of `vec` (row, head) pairs may leave: at most kSimtSplits
// per pair, and since splits < kSimtCtas / ctas + 1 and a CTA takes up to
// kSimtHeads pairs, fewer than vec + kSimtHeads * kSimtCtas.  The bound grows
// with vec (vec * splits itself falls where splits drops by one), so that a
// workspace for a larger call holds a smaller one.
size_t partials_f32(size_t vec) {
  const size_t by_splits = vec * kSimtSplits, by_ctas = vec + (size_t)kSimtHeads * kSimtCtas;
  return by_splits < by_ctas ? by_splits : by_ctas;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Workspace: tensor-core forms [partials o][partials lse][descriptors], e4m3 also
// [query planes][query scales]; fp32 [partials o][partials lse].
struct TreeWorkspace { size_t lse, desc, q8, q_scale, bytes; };

TreeWorkspace tree_workspace(int cache_dtype, long long rows, int n_heads) {
  TreeWorkspace w{};
  const size_t vec = (size_t)rows * n_heads;
  if (cache_dtype == MLA_F32) {
    const size_t parts = partials_f32(vec);
    w.lse = up256(parts * MLA_D_C * sizeof(float));
    w.bytes = w.lse + up256(parts * sizeof(float));
    return w;
  }
  w.lse = (size_t)2 * kMaxPairs * kM * MLA_D_C * sizeof(float);
  w.desc = w.lse + up256((size_t)2 * kMaxPairs * kM * sizeof(float));
  w.q8 = w.desc + up256(kMaxPairs * sizeof(TreeDesc));
  w.q_scale = w.q8;
  w.bytes = w.q8;
  if (cache_dtype == MLA_E4M3) {
    w.q_scale = w.q8 + up256(2 * vec * MLA_D_ROW);
    w.bytes = w.q_scale + up256(vec * sizeof(float));
  }
  return w;
}

bool encode(TensorMapEncodeFn enc, CUtensorMap* m, CUtensorMapDataType t, int rank, const void* base,
            const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle sw) {
  const cuuint32_t es[3] = {1, 1, 1};
  return enc(m, t, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool D8>
cudaError_t launch_tc(const TreeArgs& a, TreeParams p, const void* q8, cudaStream_t st) {
  TensorMapEncodeFn enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  CUtensorMap tc, tc2, tq;
  const cuuint64_t elt = D8 ? 1 : 2;
  const CUtensorMapDataType type = D8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUtensorMapSwizzle sw = D8 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  // the page-blocked pool as 2-D [num_pages * 9 * 64 lines x 64 columns]:
  // boxes of one block (64 lines) and of two adjacent blocks
  for (int k = 0; k < 2; ++k) {
    const cuuint64_t dims[2] = {64, (cuuint64_t)a.num_pages * kChunks * 64};
    const cuuint64_t strides[1] = {64 * elt};
    const cuuint32_t box[2] = {64, k == 0 ? 64u : 128u};
    if (!encode(enc, k == 0 ? &tc : &tc2, type, 2, a.cache, dims, strides, box, sw)) return cudaErrorInvalidValue;
  }
  // the queries as [(node, head) rows x 576] (8-bit: two planes of it): boxes
  // of 64 rows x 64 columns, rows past the end read as zeros
  {
    const cuuint64_t vec = (cuuint64_t)a.rows * a.n_heads;
    const cuuint64_t dims[3] = {MLA_D_ROW, vec, 2};
    const cuuint64_t strides[2] = {MLA_D_ROW * elt, vec * MLA_D_ROW};
    const cuuint32_t box[3] = {64, (cuuint32_t)kHM, 1};
    if (!encode(enc, &tq, type, D8 ? 3 : 2, D8 ? q8 : a.q_abs, dims, strides, box, sw)) return cudaErrorInvalidValue;
  }
  const int smem = TreeLayout<D8>::kSmem;
  cudaError_t e = cudaFuncSetAttribute(decode_tree_kernel<D8>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  // no more pairs than tiles there can be
  const long long most = (((long long)a.rows * a.n_heads + kM - 1) / kM + a.batch) *
                         (((long long)a.max_pages * 64 + kTile - 1) / kTile);
  long long pairs = sm_pair_count();
  if (pairs > kMaxPairs) pairs = kMaxPairs;
  if (pairs > most) pairs = most;
  e = launch_dependent(decode_tree_kernel<D8>, dim3((unsigned)(2 * pairs)), dim3(kThreads), smem, st, tc, tc2, tq, p);
  if (e != cudaSuccess || pairs == 1) return e;    // one pair leaves no partials
  const dim3 grid((unsigned)pairs, kMergePieces / kMergeWarps);
  // the parts of a row tile: the pairs over the row tiles there are room for
  const bool many = pairs > 4 * (((long long)a.rows * a.n_heads + kM - 1) / kM);
  auto merge = [&](auto kernel, auto* o) {
    return launch_dependent(kernel, grid, dim3(32 * kMergeWarps), 0, st, p.part_o, p.part_lse, p.desc, o, p.lse);
  };
  if (a.o_dtype == MLA_F32) {
    float* o = static_cast<float*>(p.o_lat);
    return many ? merge(tree_merge_kernel<float, 16>, o) : merge(tree_merge_kernel<float, 4>, o);
  }
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o_lat);
  return many ? merge(tree_merge_kernel<__nv_bfloat16, 16>, o) : merge(tree_merge_kernel<__nv_bfloat16, 4>, o);
}

}  // namespace

size_t decode_tree_workspace_bytes(int cache_dtype, long long rows, int n_heads) {
  return tree_workspace(cache_dtype, rows, n_heads).bytes;
}

cudaError_t launch_decode_tree(const TreeArgs& a, cudaStream_t st) {
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  const TreeWorkspace w = tree_workspace(a.cache_dtype, a.rows, a.n_heads);
  TreeParams p{};
  p.n_heads = a.n_heads;
  p.batch = a.batch;
  p.n_rows = a.rows;
  p.block_table = a.block_table;
  p.max_pages = a.max_pages;
  p.num_pages = a.num_pages;
  p.kv_lens = a.kv_lens;
  p.row_start = a.row_start;
  p.tree_mask = a.tree_mask;
  p.mask_words = a.mask_words;
  p.cache_scale = a.cache_scale;
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_lse = reinterpret_cast<float*>(ws + w.lse);
  p.o_lat = a.o_lat;
  p.o_f32 = a.o_dtype == MLA_F32;
  p.lse = a.lse;
  p.err = a.err;
  if (a.cache_dtype == MLA_F32) {
    p.scale_log2 = a.softmax_scale;    // this form works in natural units
    const long long groups = (long long)a.max_pages * (64 / kSimtGroup);
    int splits = splits_f32(a.rows, a.n_heads);
    if (splits > groups) splits = (int)groups;
    const int smem = 2 * kSimtRows * MLA_D_ROW * (int)sizeof(float);
    cudaError_t e = cudaFuncSetAttribute(decode_tree_simt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)splits, (unsigned)((a.n_heads + kSimtHeads - 1) / kSimtHeads), (unsigned)a.rows);
    e = launch_dependent(decode_tree_simt_kernel, grid, dim3(32 * kSimtWarps), smem, st,
                         static_cast<const float*>(a.q_abs), static_cast<const float*>(a.cache), p, splits);
    if (e != cudaSuccess) return e;
    const dim3 mg((unsigned)((long long)a.rows * a.n_heads));
    if (a.o_dtype == MLA_F32) return launch_dependent(tree_merge_f32_kernel<float>, mg, dim3(512), 0, st, p, splits);
    return launch_dependent(tree_merge_f32_kernel<__nv_bfloat16>, mg, dim3(512), 0, st, p, splits);
  }
  p.scale_log2 = a.softmax_scale * 1.4426950408889634f;
  p.desc = reinterpret_cast<TreeDesc*>(ws + w.desc);
  p.wait_limit = g_wait_limit.load();
  p.withhold_q = g_withhold_q.load();
  if (a.cache_dtype == MLA_BF16) return launch_tc<false>(a, p, nullptr, st);
  uint8_t* q8 = ws + w.q8;
  p.q_scale = reinterpret_cast<float*>(ws + w.q_scale);
  const int n_vec = a.rows * a.n_heads;
  const cudaError_t e =
      launch_dependent(split_q_tree_kernel, dim3((unsigned)(((long long)n_vec + 7) / 8)), dim3(256), 0, st,
                       static_cast<const __nv_bfloat16*>(a.q_abs), n_vec, q8, reinterpret_cast<float*>(ws + w.q_scale));
  if (e != cudaSuccess) return e;
  return launch_tc<true>(a, p, q8, st);
}

}  // namespace mla
