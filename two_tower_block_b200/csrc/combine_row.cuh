// The log-sum-exp combine of cut units: used by the combine kernel and by the fused tail of the
// default attention kernel.
//
// A cut unit's segments each hold O_s = (sum over its keys of e^{s-m_s} v) / l_s and
// lse_s = (m_s + ln l_s) / ln 2.  The joint softmax over all keys of the unit is recovered
// exactly: with M = max_s lse_s and w_s = 2^{lse_s - M},
//     out = sum_s w_s O_s / sum_s w_s,     lse = (M + log2 sum_s w_s) ln 2.
// (log2 units: the hardware's exponential then takes the difference as it is, within 2 ulp, where one of base e
// would round its product with log2 e first.)
// One thread does eight columns of one row (an item; consecutive items are consecutive rows, as the
// partials lie): it requests kGroup segments' lse values and columns before the first use and folds groups
// online (running maximum, rescaled sums).  A warp per row, with shuffled weights, took 2.3 us for the first
// row; what bounds this is one round trip to L2 per group, and with many rows the partials' traffic (eight
// columns rather than four halve the lse reads and write whole sectors).
// `parts`: neighbouring threads (1, 2 or 4) that share an item, each taking a part of the segments, and join what they have at
// the end.  One where the segments fit a group; four where a few long units are cut into dozens of segments, whose
// groups would follow one another (one sequence of 32768 positions, 74 segments a unit: see kManySegments).
#pragma once
#include "problem.h"
#include "ptx.cuh"
#include "sched.cuh"
#include "walker.cuh"

namespace tt {

// Items of a unit; item i is row i % R, columns [8 (i / R), 8 (i / R) + 8).
template <int D>
__device__ __forceinline__ int combine_items(const Problem& p) {
  return p.R * (D / 8);
}

constexpr int kManySegments = 16;   // from here on several threads may share an item

// kGroup: 8 (16 cost the separate kernel its occupancy: 64 ragged sequences 67 -> 82 us), 4 in the tail of a
// kernel whose launch leaves it 128 registers.  With parts > 1 whole warps call this together; a thread whose
// item is not `there` only takes part in the joining.
template <int D, int kGroup>
__device__ __forceinline__ void combine_item(const Problem& p, const Unit& x, int c, const SplitRecord& rec, int item,
                                             bool there, int parts, int part) {
  const int nseg = there ? rec.last_range - c + 1 : 0;
  const int q = item / p.R, r = item - q * p.R;
  // slot of segment s: 2 c + first_which, 2 (c + 1), 2 (c + 2), ...
  auto slot_of = [&](int s) { return s == 0 ? 2 * c + rec.first_which : 2 * (c + s); };
  float acc[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] = 0.f;
  float M = -INFINITY, wsum = 0.f;
#pragma unroll 1
  for (int s0 = part; s0 < nseg; s0 += parts * kGroup) {
    float l[kGroup];
    float4 a[kGroup][2];
#pragma unroll
    for (int u = 0; u < kGroup; ++u) {
      l[u] = -INFINITY;
      a[u][0] = a[u][1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s0 + parts * u < nseg) {
        const int slot = slot_of(s0 + parts * u);
        l[u] = __ldcg(p.part_lse + (size_t)slot * p.R + r);
        const float* src = p.part_o + part_at(p, slot, r, 8 * q, D);
        a[u][0] = __ldcg(reinterpret_cast<const float4*>(src));
        a[u][1] = __ldcg(reinterpret_cast<const float4*>(src + (size_t)4 * p.R));
      }
    }
    float Mn = M;
#pragma unroll
    for (int u = 0; u < kGroup; ++u) Mn = fmaxf(Mn, l[u]);
    // (a row that saw no key in any segment has Mn = -inf: every weight stays 0)
    const float old = M > -INFINITY ? fast_exp2(M - Mn) : 0.f;
    M = Mn;
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] *= old;
    wsum *= old;
#pragma unroll
    for (int u = 0; u < kGroup; ++u) {
      const float w = l[u] != -INFINITY ? fast_exp2(l[u] - Mn) : 0.f;   // (a NaN segment spoils the row)
      wsum += w;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        acc[4 * h] = fmaf(w, a[u][h].x, acc[4 * h]);
        acc[4 * h + 1] = fmaf(w, a[u][h].y, acc[4 * h + 1]);
        acc[4 * h + 2] = fmaf(w, a[u][h].z, acc[4 * h + 2]);
        acc[4 * h + 3] = fmaf(w, a[u][h].w, acc[4 * h + 3]);
      }
    }
  }
#pragma unroll 1
  for (int o = 1; o < parts; o <<= 1) {
    const float Mn = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float f = M > -INFINITY ? fast_exp2(M - Mn) : 1.f;   // (nothing yet, or only NaN, is kept as it is)
    M = Mn;
    wsum *= f;
    wsum += __shfl_xor_sync(0xffffffffu, wsum, o);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      acc[k] *= f;
      acc[k] += __shfl_xor_sync(0xffffffffu, acc[k], o);
    }
  }
  if (!there || part != 0) return;
  const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] *= inv;
  const size_t off = out_offset(p, x, r, D) + 8 * q;
  if (p.out_bf16) {
    *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) + off) =
        make_uint4(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]), pack_bf16(acc[4], acc[5]),
                   pack_bf16(acc[6], acc[7]));
  } else {
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(acc[k]);
    store_row(reinterpret_cast<uint32_t*>(p.out + off), w, (reinterpret_cast<uintptr_t>(p.out) & 31) == 0);
  }
  if (q == 0 && p.lse) {
    const int t = r / p.g, j = r - (r / p.g) * p.g;
    p.lse[(size_t)(x.n * p.Hq + x.h * p.g + j) * (p.NB * p.S) + x.b * p.S + t] = (M + log2f(wsum)) * kLn2;
  }
}

}  // namespace tt
