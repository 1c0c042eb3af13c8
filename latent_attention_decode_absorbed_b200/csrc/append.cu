// Paged cache append: one warp writes one token's 576-number cache row (into
// the page-blocked layout: nine contiguous [64 rows x 64 columns] blocks per page).
//
// "KV Compression - DeepSeek-V3", "How it works": the 576-wide wkv_a output is
// split [512, 64]; the latent goes through RMSNorm and the rope part through
// RoPE; the absorb path stores the normalised latent and the rotated key.
// The kernel is memory-bound (2.3 KB in, 1.2 KB out per bf16 token); a warp
// moves a row with 16-byte accesses and reduces sum(c^2) with a fixed
// xor-shuffle tree.
#include "append_row.cuh"

namespace mla {
namespace {

template <typename IN, int CK>  // CK: MLA_F32, MLA_BF16, MLA_E4M3
__global__ void __launch_bounds__(256) append_kernel(AppendArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int warp = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (warp >= a.n_new) return;
  const IN* row = reinterpret_cast<const IN*>(a.kv_a) + (size_t)warp * MLA_D_ROW;
  // latent: lane owns channels [16*lane, 16*lane + 16); rope key: pair `lane`
  float c[16];
  load16(row + 16 * lane, c);
  const float x0 = to_f32(row[MLA_D_C + 2 * lane]);
  const float x1 = to_f32(row[MLA_D_C + 2 * lane + 1]);
  append_row<CK>(a, a.seq_ids[warp], a.positions[warp], c, x0, x1, lane);
}

// The same rows at given slots: a row whose slot is -1 is padding and skipped.
// Prompts bring tens of thousands of rows, and one row is a chain of loads
// (slot and position, then the row and its rope table line), two reductions
// and a store.  So a warp walks rows a grid apart and holds the next row's
// loads in flight while it works on this one's; the gains stay in registers.
// 65536 rows to e4m3 at scattered slots take 31.5 us (3.6 TB/s; one row per
// warp and no look ahead: 76), to bf16 32.0 (4.7 TB/s); 1024 rows 2.2.
template <typename IN>
struct RawRow {
  uint4 v[sizeof(IN)];        // 16 channels
  IN x[2];                    // the rope pair
  int slot, pos;
};
template <typename IN>
__device__ __forceinline__ RawRow<IN> load_raw(const AppendArgs& a, const int32_t* slots, int r, int lane) {
  RawRow<IN> w;
  w.slot = -1;
  w.pos = 0;
  if (r >= a.n_new) return w;
  w.slot = slots[r];
  w.pos = a.positions[r];
  const IN* row = reinterpret_cast<const IN*>(a.kv_a) + (size_t)r * MLA_D_ROW;
  const uint4* src = reinterpret_cast<const uint4*>(row + 16 * lane);
#pragma unroll
  for (int i = 0; i < (int)sizeof(IN); ++i) w.v[i] = __ldcs(src + i);
  if constexpr (sizeof(IN) == 4)
    *reinterpret_cast<float2*>(w.x) = *reinterpret_cast<const float2*>(row + MLA_D_C + 2 * lane);
  else
    *reinterpret_cast<uint32_t*>(w.x) = *reinterpret_cast<const uint32_t*>(row + MLA_D_C + 2 * lane);
  return w;
}

// CTAs per SM: four where 64 registers hold a row, the next one and the gains
// without spilling (65536 rows to bf16: 36.6 us with three, 32.0 with four;
// 6000 rows to e4m3: 4.6 with three, 5.7 with four).
template <typename IN, int CK>
constexpr int kSlotCtas = sizeof(IN) == 2 && CK != MLA_E4M3 ? 4 : 3;

template <typename IN, int CK>
__global__ void __launch_bounds__(256, kSlotCtas<IN, CK>) append_slots_kernel(AppendArgs a, const int32_t* __restrict__ slots) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int stride = (gridDim.x * blockDim.x) >> 5;
  int r = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  RawRow<IN> cur = load_raw<IN>(a, slots, r, lane);
  float g[16];
  load_gain(a, lane, g);
  for (; r < a.n_new; r += stride) {
    const RawRow<IN> next = load_raw<IN>(a, slots, r + stride, lane);
    const int slot = cur.slot, p = cur.pos;
    if (slot != -1) {
      if (slot < 0 || (slot >> 6) >= a.num_pages) {
        if (lane == 0) flag_error(a.err, MLA_DEVERR_PAGE);
      } else if (p < 0 || p >= a.rope_max_pos) {
        if (lane == 0) flag_error(a.err, MLA_DEVERR_POSITION);
      } else {
        const float cs = a.rope_cos[(size_t)p * (MLA_D_R / 2) + lane];
        const float sn = a.rope_sin[(size_t)p * (MLA_D_R / 2) + lane];
        float c[16];
        load16(reinterpret_cast<const IN*>(cur.v), c);
        store_row<CK>(a, (size_t)slot, c, to_f32(cur.x[0]), to_f32(cur.x[1]), g, cs, sn, lane);
      }
    }
    cur = next;
  }
}

template <typename IN, int CK>
cudaError_t launch_slots(const AppendArgs& a, const int32_t* slots, cudaStream_t st) {
  // one row per warp while that fits the GPU, else a grid that fills it
  const long long rows_ctas = ((long long)a.n_new + 7) / 8, most = 2 * sm_pair_count() * kSlotCtas<IN, CK>;
  const long long ctas = rows_ctas < most ? rows_ctas : most;
  return launch_dependent(append_slots_kernel<IN, CK>, dim3((unsigned)ctas), dim3(256), 0, st, a, slots);
}

template <typename IN>
cudaError_t launch_slots_in(const AppendArgs& a, const int32_t* slots, cudaStream_t st) {
  switch (a.cache_dtype) {
    case MLA_F32: return launch_slots<IN, MLA_F32>(a, slots, st);
    case MLA_BF16: return launch_slots<IN, MLA_BF16>(a, slots, st);
    default: return launch_slots<IN, MLA_E4M3>(a, slots, st);
  }
}

template <typename IN>
cudaError_t launch_in(const AppendArgs& a, cudaStream_t st) {
  dim3 block(256);
  dim3 grid((a.n_new + 7) / 8);
  switch (a.cache_dtype) {
    case MLA_F32: return launch_dependent(append_kernel<IN, MLA_F32>, grid, block, 0, st, a);
    case MLA_BF16: return launch_dependent(append_kernel<IN, MLA_BF16>, grid, block, 0, st, a);
    default: return launch_dependent(append_kernel<IN, MLA_E4M3>, grid, block, 0, st, a);
  }
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, cudaStream_t st) {
  if (a.n_new == 0) return cudaSuccess;
  if (a.kv_dtype == MLA_F32) return launch_in<float>(a, st);
  return launch_in<__nv_bfloat16>(a, st);
}

cudaError_t launch_append_slots(const AppendArgs& a, const int32_t* slots, cudaStream_t st) {
  if (a.n_new == 0) return cudaSuccess;
  if (a.kv_dtype == MLA_F32) return launch_slots_in<float>(a, slots, st);
  return launch_slots_in<__nv_bfloat16>(a, slots, st);
}

}  // namespace mla
