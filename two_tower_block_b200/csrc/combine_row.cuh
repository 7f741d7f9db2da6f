// Rows of the log-sum-exp combine, done by one warp: used by the combine kernel and
// by the fused tail of the default attention kernel.
//
// A cut unit's segments each hold O_s = (sum over its keys of e^{s-m_s} v) / l_s and
// lse_s = m_s + ln l_s.  The joint softmax over all keys of the unit is recovered
// exactly: with M = max_s lse_s and w_s = e^{lse_s - M},
//     out = sum_s w_s O_s / sum_s w_s,     lse = M + ln sum_s w_s.
// The warp requests every lse value and the first kGroup segments' rows before the first
// use, and folds sweeps of 32 segments online (running maximum, rescaled sums).
#pragma once
#include "problem.h"
#include "sched.cuh"
#include "walker.cuh"

namespace tt {

// kRows rows of unit x at a time, r0, r0 + stride, ... (those below r1): their loads are in flight
// together.  kGroup segments' rows are loaded per round: 8 in the separate kernel (more would cost
// occupancy), more in the attention kernel's tail, whose registers are there anyway.
template <int D, int kGroup, int kRows>
__device__ __forceinline__ void combine_rows(const Problem& p, const Unit& x, int c, const SplitRecord& rec, int r0,
                                             int stride, int r1, int lane) {
  constexpr int V = D / 32;  // columns per lane
  const int nseg = rec.last_range - c + 1;
  auto slot_of = [&](int s) { return s == 0 ? 2 * c + rec.first_which : 2 * (c + s); };
  auto load_row = [&](int s, int r, float* a) {
    const float* src = p.part_o + ((size_t)slot_of(s) * p.R + r) * D + lane * V;
    if constexpr (V == 4) {
      const float4 t = __ldcg(reinterpret_cast<const float4*>(src));
      a[0] = t.x; a[1] = t.y; a[2] = t.z; a[3] = t.w;
    } else {
      const float2 t = __ldcg(reinterpret_cast<const float2*>(src));
      a[0] = t.x; a[1] = t.y;
    }
  };
  float acc[kRows][V], M[kRows], wsum[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
#pragma unroll
    for (int v = 0; v < V; ++v) acc[i][v] = 0.f;
    M[i] = -INFINITY;
    wsum[i] = 0.f;
  }
  for (int s0 = 0; s0 < nseg; s0 += 32) {
    const int n = min(32, nseg - s0);
    float lse_lane[kRows], a[kRows][kGroup][V];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = r0 + i * stride;
      lse_lane[i] = lane < n && r < r1 ? __ldcg(p.part_lse + (size_t)slot_of(s0 + lane) * p.R + r) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int u = 0; u < kGroup; ++u)
        if (u < n && r0 + i * stride < r1) load_row(s0 + u, r0 + i * stride, a[i][u]);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = r0 + i * stride;
      if (r >= r1) break;
      float Ms = lse_lane[i];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) Ms = fmaxf(Ms, __shfl_xor_sync(0xffffffffu, Ms, o));
      const float Mn = fmaxf(M[i], Ms);
      const float scale_old = M[i] == -INFINITY ? 0.f : expf(M[i] - Mn);
      wsum[i] *= scale_old;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[i][v] *= scale_old;
      M[i] = Mn;
      // (a row that saw no key in any segment has M = -inf: every weight stays 0)
      const float w_lane = lse_lane[i] > -INFINITY ? expf(lse_lane[i] - Mn) : 0.f;
      float ws = w_lane;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, o);
      wsum[i] += ws;
      for (int k = 0; k < n; k += kGroup) {
        if (k > 0) {
#pragma unroll
          for (int u = 0; u < kGroup; ++u)
            if (k + u < n) load_row(s0 + k + u, r, a[i][u]);
        }
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
          const float w = __shfl_sync(0xffffffffu, w_lane, (k + u) & 31);
          if (k + u < n) {
#pragma unroll
            for (int v = 0; v < V; ++v) acc[i][v] = fmaf(w, a[i][u][v], acc[i][v]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = r0 + i * stride;
    if (r >= r1) break;
    const float inv = wsum[i] > 0.f ? 1.f / wsum[i] : 0.f;
    const int t = r / p.g, j = r - (r / p.g) * p.g;
    const size_t off = out_offset(p, x, r, D) + lane * V;
    if constexpr (V == 4) {
      store_out4(p, off, make_float4(acc[i][0] * inv, acc[i][1] * inv, acc[i][2] * inv, acc[i][3] * inv));
    } else {
      store_out2(p, off, make_float2(acc[i][0] * inv, acc[i][1] * inv));
    }
    if (lane == 0 && p.lse)
      p.lse[(size_t)(x.n * p.Hq + x.h * p.g + j) * (p.NB * p.S) + x.b * p.S + t] = M[i] + logf(wsum[i]);
  }
}

}  // namespace tt
