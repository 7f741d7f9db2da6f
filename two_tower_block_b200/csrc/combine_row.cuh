// The log-sum-exp combine of cut units: used by the combine kernel and by the fused tail of the
// default attention kernel.
//
// A cut unit's segments each hold O_s = (sum over its keys of e^{s-m_s} v) / l_s and
// lse_s = m_s + ln l_s.  The joint softmax over all keys of the unit is recovered
// exactly: with M = max_s lse_s and w_s = e^{lse_s - M},
//     out = sum_s w_s O_s / sum_s w_s,     lse = M + ln sum_s w_s.
// One thread does four columns of one row (an item; consecutive items are consecutive rows, as the
// partials lie), with no exchange between threads: it requests kGroup segments' lse values and
// columns before the first use and folds groups online (running maximum, rescaled sums).  A
// warp per row, with shuffled weights, took 2.3 us for the first row; what bounds this is one
// round trip to L2 per group.
#pragma once
#include "problem.h"
#include "sched.cuh"
#include "walker.cuh"

namespace tt {

// Items of a unit; item i is row i % R, columns [4 (i / R), 4 (i / R) + 4).
template <int D>
__device__ __forceinline__ int combine_items(const Problem& p) {
  return p.R * (D / 4);
}

template <int D>
__device__ __forceinline__ void combine_item(const Problem& p, const Unit& x, int c, const SplitRecord& rec, int item) {
  constexpr int kGroup = 8;
  const int nseg = rec.last_range - c + 1;
  const int q = item / p.R, r = item - q * p.R;
  // slot of segment s: 2 c + first_which, 2 (c + 1), 2 (c + 2), ...
  auto slot_of = [&](int s) { return s == 0 ? 2 * c + rec.first_which : 2 * (c + s); };
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -INFINITY, wsum = 0.f;
#pragma unroll 1
  for (int s0 = 0; s0 < nseg; s0 += kGroup) {
    float l[kGroup];
    float4 a[kGroup];
#pragma unroll
    for (int u = 0; u < kGroup; ++u) {
      l[u] = -INFINITY;
      a[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s0 + u < nseg) {
        const int slot = slot_of(s0 + u);
        l[u] = __ldcg(p.part_lse + (size_t)slot * p.R + r);
        a[u] = __ldcg(reinterpret_cast<const float4*>(p.part_o + part_at(p, slot, r, 4 * q, D)));
      }
    }
    float Mn = M;
#pragma unroll
    for (int u = 0; u < kGroup; ++u) Mn = fmaxf(Mn, l[u]);
    // (a row that saw no key in any segment has Mn = -inf: every weight stays 0)
    const float old = M > -INFINITY ? __expf(M - Mn) : 0.f;
    M = Mn;
    acc.x *= old; acc.y *= old; acc.z *= old; acc.w *= old;
    wsum *= old;
#pragma unroll
    for (int u = 0; u < kGroup; ++u) {
      const float w = l[u] > -INFINITY ? __expf(l[u] - Mn) : 0.f;
      wsum += w;
      acc.x = fmaf(w, a[u].x, acc.x);
      acc.y = fmaf(w, a[u].y, acc.y);
      acc.z = fmaf(w, a[u].z, acc.z);
      acc.w = fmaf(w, a[u].w, acc.w);
    }
  }
  const float inv = wsum > 0.f ? 1.f / wsum : 0.f;
  store_out4(p, out_offset(p, x, r, D) + 4 * q, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
  if (q == 0 && p.lse) {
    const int t = r / p.g, j = r - (r / p.g) * p.g;
    p.lse[(size_t)(x.n * p.Hq + x.h * p.g + j) * (p.NB * p.S) + x.b * p.S + t] = M + logf(wsum);
  }
}

}  // namespace tt
