// The softmax of the attention on 8-bit MMAs over an e4m3 cache, as the
// kernels that run it share it: a thread owns one (query row, head) and the 64
// cached rows of one page, a CTA's eight softmax warps cover 64 of the former
// and four of the latter, two warps to a page.
//
// The value MMAs multiply cache codes, so a row's weight has to carry its
// scale: with y_j = z_j + log2 sc_j (z_j the score in log2 units) the weight
// operand is x_j = 16 * 2^(y_j - m), m a running reference for the y's of the
// rows that this (query row, head) sees.  The sum of the softmax takes the same
// x_j over sc_j, so O / sum is the result with no factor left.  Weights
// relative to the largest score, times scales relative to the largest one of
// the tile, are no substitute: a row of large scale and no weight, or one that
// a mask hides, pushes the others below e4m3's last step.
//
// x_j is carried as e4m3(x) + e5m2(x - e4m3(x)): 2^-8 of itself down to 2^-6,
// 2^-14 below, so weights to about 2^-21 of the reference count.  m follows a
// tile down as well as up (O and the sum are fp32 and take any factor), so a
// long thin tail behind one strong row is carried on its own reference.  With
// two e4m3 terms and m only rising, weights under 2^-14 of the strongest were
// lost but stayed in the sum: with 0.3 to 0.9 of the mass on the first of 32768
// rows o was off by 0.09 to 3.2 of its norm (now 3e-4 at most; 4096 to 131072
// rows: 7e-4).
//
// A page's scales, their logarithms and reciprocals wait in shared memory.
// Each read is issued four columns before its values are used (128 x 2-6
// drafts x 128 heads over 2048-4096 rows: 458 us a call without that, 425 with
// it; two shuffles per column instead 430).  The shared-memory path is what
// bounds these kernels: of 6806 cycles a tile the MMAs' operands take 3234, the
// copies 1088 and the softmax 2219, 1490 of them these reads (a 16-byte read
// takes four wavefronts though its lanes agree), the tensor cores 4306.
#pragma once

#include "mla_device.cuh"
#include "sm100.cuh"

namespace mla {
namespace q8 {

constexpr float kLog = 4.0f;              // a weight at the reference is carried as 2^4 ...
constexpr float kRaise = 4.8f;            // ... the reference is raised past 4.8 (at most 2^8.8 < 448) ...
constexpr float kLower = 8.0f;            // ... and lowered to a tile whose largest is more than 8 below it, ...
constexpr float kLowest = 32.0f;          // ... to 32 below the largest so far at most
constexpr float kLeastScale = 0x1p-48f;   // smaller row scales (rows below 2e-12) count as this one, which
                                          // keeps the sum finite
constexpr int kPlane = 4 * 64;            // floats of one plane: four pages of 64 rows
constexpr int kBytes = 4 * kPlane * 4;    // planes: scales, logarithms, reciprocals of even and odd tiles

// Lane l writes the scales of rows l and l + 32 of its page (page_sc: the
// page's scales; page_inv: its reciprocals of this tile's parity).  Both warps
// of a page write the same values.  Scales and logarithms are read before a
// tile's barrier among the softmax warps, so the next tile's may be written
// after it; the reciprocals are read behind it and alternate by tile.
__device__ __forceinline__ void put_scales(float* page_sc, float* page_inv, int lane, float sc_lo, float sc_hi) {
  const float a = fmaxf(sc_lo, kLeastScale), c = fmaxf(sc_hi, kLeastScale);
  page_sc[lane] = sc_lo;
  page_sc[lane + 32] = sc_hi;
  page_sc[kPlane + lane] = log2f(a);
  page_sc[kPlane + lane + 32] = log2f(c);
  page_inv[lane] = 1.0f / a;
  page_inv[lane + 32] = 1.0f / c;
  __syncwarp();
}

// Code products to y's; slq: softmax scale * log2 e * the query's scale.
__device__ __forceinline__ void scores(float (&v)[64], float slq, const float* page_sc) {
  const uint32_t at = sm100::smem_u32(page_sc);
  float4 sc_n = sm100::ld_shared_f4(at), lg_n = sm100::ld_shared_f4(at + 4 * kPlane);
#pragma unroll
  for (int j = 0; j < 64; j += 4) {
    const float4 sc = sc_n, lg = lg_n;
    if (j < 60) {
      sc_n = sm100::ld_shared_f4(at + 4 * (j + 4));
      lg_n = sm100::ld_shared_f4(at + 4 * (kPlane + j + 4));
    }
    v[j] = fmaf(v[j] * slq, sc.x, lg.x);
    v[j + 1] = fmaf(v[j + 1] * slq, sc.y, lg.y);
    v[j + 2] = fmaf(v[j + 2] * slq, sc.z, lg.z);
    v[j + 3] = fmaf(v[j + 3] * slq, sc.w, lg.w);
  }
}

// The reference after a tile whose largest y is `tile` (m: before it, top: the largest so far).
__device__ __forceinline__ float reference(float m, float tile, float& top) {
  top = fmaxf(top, tile);
  if (tile > m + kRaise) return tile;
  if (tile < m - kLower && tile > -INFINITY) return fmaxf(tile, top - kLowest);
  return m;
}

// y's to weights on the reference m (-inf: nothing seen so far, every y is
// -inf): their codes (pk[0..15] the first terms of the 64 rows, pk[16..31] the
// second) and their sum, 2^kLog too large.
__device__ __forceinline__ float weights(const float (&v)[64], float m, const float* page_inv, uint32_t (&pk)[32]) {
  const float sub = m == -INFINITY ? 0.f : m - kLog;
  const uint32_t at = sm100::smem_u32(page_inv);
  float4 inv_n = sm100::ld_shared_f4(at);
  float sum = 0.f, sum2 = 0.f;
#pragma unroll
  for (int j = 0; j < 64; j += 4) {
    const float4 inv = inv_n;
    if (j < 60) inv_n = sm100::ld_shared_f4(at + 4 * (j + 4));
    const float x0 = sm100::exp2_approx(v[j] - sub), x1 = sm100::exp2_approx(v[j + 1] - sub);
    const float x2 = sm100::exp2_approx(v[j + 2] - sub), x3 = sm100::exp2_approx(v[j + 3] - sub);
    sum = fmaf(x1, inv.y, fmaf(x0, inv.x, sum));
    sum2 = fmaf(x3, inv.w, fmaf(x2, inv.z, sum2));
    uint32_t h01, l01, h23, l23;
    split_e4m3_e5m2x2(x0, x1, h01, l01);
    split_e4m3_e5m2x2(x2, x3, h23, l23);
    pk[j >> 2] = h01 | h23 << 16;
    pk[16 + (j >> 2)] = l01 | l23 << 16;
  }
  return sum + sum2;
}

}  // namespace q8
}  // namespace mla
