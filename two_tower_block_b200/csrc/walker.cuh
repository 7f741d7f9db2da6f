// Device-side walk over one range of the global tile sequence (see sched.cuh).
#pragma once
#include "problem.h"
#include "ptx.cuh"
#include "sched.cuh"

namespace tt {

__device__ __forceinline__ int clamp_len(const Problem& p, int n, bool report) {
  int L = __ldg(p.ctx_lens + n);
  if (L < 0 || L > p.ctx_stride) {
    if (report) raise_error(p.err_word, kErrDeviceArg);
    L = L < 0 ? 0 : p.ctx_stride;
  }
  return L;
}

__device__ __forceinline__ int unit_tiles_k(const Problem& p, int L) {
  return p.blk_tiles + ctx_span(L, p.window, p.sinks, p.win_align, p.key_tile).tiles;
}

__device__ __forceinline__ Unit make_unit(const Problem& p, int u, long long Tu, int cost = 0) {
  Unit x;
  x.u = u;
  x.Tu = Tu;
  x.cost = cost;
  if (p.mode == kDecode) {
    x.n = u / p.Hkv;
    x.h = u - x.n * p.Hkv;
    x.b = 0;
    x.L = clamp_len(p, x.n, false);
  } else {
    int nh = u / p.NB;
    x.b = u - nh * p.NB;
    x.n = nh / p.Hkv;
    x.h = nh - x.n * p.Hkv;
    x.L = p.S * x.b;
  }
  x.ns = x.n * p.NB + x.b;
  const CtxSpan s = ctx_span(x.L, p.window, p.sinks, p.win_align, p.key_tile);
  x.sink_tiles = s.sink_tiles;
  x.wstart = s.wstart;
  x.head = s.head;
  x.tiles = p.blk_tiles + s.tiles;
  return x;
}

__device__ __forceinline__ Unit next_unit(const Problem& p, const Unit& x) {
  return make_unit(p, x.u + 1, x.Tu + x.tiles + x.cost, x.cost);
}
// The boundary table of the call's split, or null for the uniform one.
__device__ __forceinline__ const long long* range_table(const Problem& p) {
  return p.mode == kDecode ? nullptr : p.causal_starts;
}

// Called by one full warp.  Finds the total place count T, this range's
// [start, end) and the first unit with a tile in it (valid only if start < end).
__device__ __forceinline__ void find_range(const Problem& p, int c, long long& T, long long& start,
                                           long long& end, Unit& first) {
  const int lane = threadIdx.x & 31;
  int cost = 0, t = 0;   // t: tiles of a unit of sequence base + lane (sums fit: api.cpp, decode_call)
  if (p.mode == kDecode) {
    int tot = 0, least = INT32_MAX, most = 0;
#pragma unroll 1   // (cold code: short, or its instruction fetches are what a small call waits for)
    for (int base = 0; base < p.B; base += 32) {
      const int n = base + lane;
      t = n < p.B ? unit_tiles_k(p, clamp_len(p, n, c == 0)) : 0;
      tot += __reduce_add_sync(0xffffffffu, t);
      least = min(least, __reduce_min_sync(0xffffffffu, n < p.B ? t : INT32_MAX));
      most = max(most, __reduce_max_sync(0xffffffffu, t));
    }
    T = (long long)p.Hkv * tot;
    const int U = p.B * p.Hkv;
    cost = decode_cost(T, U, p.C, p.unit_cost, least, most);
    T += (long long)U * cost;
    if (whole_units(U, p.C, most, p.whole_tiles)) {
      // short units: range c is unit c
      start = end = T;
      if (c >= U) return;
      const int nc = c / p.Hkv, hc = c - nc * p.Hkv;
      int before = 0;   // tiles of a unit, summed over the sequences before nc
#pragma unroll 1
      for (int base = 0; base < nc; base += 32) {
        const int n = base + lane;
        before += __reduce_add_sync(0xffffffffu, n < nc ? unit_tiles_k(p, clamp_len(p, n, false)) : 0);
      }
      const int tn = unit_tiles_k(p, clamp_len(p, nc, false));
      first = make_unit(p, c, (long long)p.Hkv * before + (long long)hc * tn);
      start = first.Tu;
      end = start + tn;
      return;
    }
  } else {
    T = p.T_causal;
    if (p.whole_tiles > 0) {   // (the host has seen that no unit has more, and that there are no more than C)
      start = end = T;
      if (c >= p.B * p.Hkv * p.NB) return;
      const int nh = c / p.NB;
      first = make_unit(p, c, (long long)nh * p.causal_pref[p.NB] + p.causal_pref[c - nh * p.NB]);
      start = first.Tu;
      end = start + first.tiles;
      return;
    }
  }
  const int Ce = used_ranges(T, p.C);
  if (c >= Ce) {
    start = end = T;
    return;
  }
  const long long* tab = range_table(p);
  start = range_start_tab(tab, T, Ce, c);
  end = range_start_tab(tab, T, Ce, c + 1);
  if (p.mode == kDecode) {
    long long acc = 0;
#pragma unroll 1
    for (int base = 0; base < p.B; base += 32) {
      const int n = base + lane;
      if (p.B > 32) t = n < p.B ? unit_tiles_k(p, clamp_len(p, n, false)) : 0;
      const int mine = n < p.B ? p.Hkv * (t + cost) : 0;
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const int total = __shfl_sync(0xffffffffu, incl, 31);
      if (acc + total > start) {
        const int at = (int)(start - acc);
        const int src = __ffs(__ballot_sync(0xffffffffu, incl > at)) - 1;
        const int pn = __shfl_sync(0xffffffffu, incl - mine, src);
        const int tn = __shfl_sync(0xffffffffu, t, src) + cost;
        const int h = (at - pn) / tn;
        first = make_unit(p, (base + src) * p.Hkv + h, acc + pn + h * tn, cost);
        if (end_tile(first) <= start) first = next_unit(p, first);
        return;
      }
      acc += total;
    }
  } else {
    const long long Tnh = p.causal_pref[p.NB];
    const int nh = (int)(start / Tnh);
    const long long rem = start - (long long)nh * Tnh;
    int lo = 0, hi = p.NB - 1;  // largest b with pref[b] <= rem
    while (lo < hi) {
      int mid = (lo + hi + 1) >> 1;
      if (p.causal_pref[mid] <= rem) lo = mid; else hi = mid - 1;
    }
    first = make_unit(p, nh * p.NB + lo, (long long)nh * Tnh + p.causal_pref[lo]);
  }
}

// Element offset of packed row r of unit x in the final output [.., S, Hq, D].
__device__ __forceinline__ size_t out_offset(const Problem& p, const Unit& x, int r, int D) {
  const int t = r / p.g, j = r - (r / p.g) * p.g;
  return ((size_t)(x.ns * p.S + t) * p.Hq + x.h * p.g + j) * D;
}
constexpr float kLn2 = 0.6931471805599453f;   // the kernels' log-sum-exps are in log2 units, partials' too
// Element offset of columns [col, col + 4) (col a multiple of 4) of packed row r in partial slot `slot`.
// Four columns of consecutive rows lie together: a warp whose lanes hold rows writes 512 bytes at a
// time straight from its registers, and a combining warp reads them so.
__device__ __forceinline__ size_t part_at(const Problem& p, int slot, int r, int col, int D) {
  return (((size_t)slot * (D / 4) + col / 4) * p.R + r) * 4 + (col & 3);
}
// r / g for packed rows r < 256 of a unit (g <= 256): with m = ceil(2^16 / g) the product r m exceeds
// r 2^16 / g by less than 2^8 <= 2^16 / g.
__device__ __forceinline__ uint32_t div_by(int g) { return (65536u + (uint32_t)g - 1u) / (uint32_t)g; }
__device__ __forceinline__ int row_token(int r, uint32_t m) { return (int)(((uint32_t)r * m) >> 16); }

// Four (or two) consecutive final-output values at element offset off: fp32, or bf16 pairs
// rounded to nearest even when the problem asks for a bf16 output.
__device__ __forceinline__ void store_out4(const Problem& p, size_t off, float4 v) {
  if (p.out_bf16) {
    const uint2 u = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
    *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) + off) = u;
  } else {
    *reinterpret_cast<float4*>(p.out + off) = v;
  }
}
__device__ __forceinline__ void store_out2(const Problem& p, size_t off, float2 v) {
  if (p.out_bf16) *reinterpret_cast<uint32_t*>(reinterpret_cast<__nv_bfloat16*>(p.out) + off) = pack_bf16(v.x, v.y);
  else *reinterpret_cast<float2*>(p.out + off) = v;
}

// Keys of unit-local tile i: block keys for i < blk_tiles, context keys after (the sinks'
// tiles first on a windowed layer).
struct TileKeys {
  bool is_blk;
  int first;   // first key index within its source (block position or context position)
  int count;   // keys of the tile that are loaded (>= 1)
  int head;    // of those, the first ones that are not visible (paged windows only)
};
__device__ __forceinline__ TileKeys tile_keys(const Problem& p, const Unit& x, int i) {
  TileKeys k;
  k.head = 0;
  if (i < p.blk_tiles) {
    k.is_blk = true;
    k.first = i * p.key_tile;
    k.count = min(p.S - k.first, p.key_tile);
  } else {
    k.is_blk = false;
    const int j = i - p.blk_tiles - x.sink_tiles;
    if (j < 0) {
      k.first = (i - p.blk_tiles) * p.key_tile;
      k.count = min(p.sinks - k.first, p.key_tile);
    } else {
      k.first = x.wstart + j * p.key_tile;
      k.count = min(x.L - k.first, p.key_tile);
      if (j == 0) k.head = x.head;
    }
  }
  return k;
}

// The unit's inner tiles, whole tiles of visible context keys: those of the window run but its first one where it has a
// head, and its last one.  Most tiles are, and every role asks about every tile: the short answer there is worth
// 160.7 -> 157.8 us on the long decode and 4.71 -> 4.49 ms on the block-causal forward.
struct InnerTiles {
  int lo;
  unsigned num;
  int first;   // position at which unit-local tile 0 would begin if all tiles lay in the window run
};
template <int NK>
__device__ __forceinline__ InnerTiles inner_tiles(const Problem& p, const Unit& x) {
  const int run = p.blk_tiles + x.sink_tiles, lo = run + (x.head > 0 ? 1 : 0);
  return {lo, (unsigned)max(x.tiles - 1 - lo, 0), x.wstart - run * NK};
}
// tile_keys of a problem whose tiles have NK keys.
template <int NK>
__device__ __forceinline__ TileKeys tile_keys(const Problem& p, const Unit& x, const InnerTiles& in, int i) {
  if ((unsigned)(i - in.lo) < in.num) return {false, in.first + i * NK, NK, 0};
  return tile_keys(p, x, i);
}

// Drafted trees: the block rows of tile [first, first + 64) that row t of sequence n sees
// (itself and its ancestors) as a bit mask; `absent` when the row or one of its ancestors is
// not there (such a row sees nothing at all).  Parents come before their children, so the walk
// ends; an entry that breaks this or is below -2 is flagged and its row taken as absent.
__device__ __forceinline__ unsigned long long tree_mask(const Problem& p, int n, int t, int first, bool& absent) {
  const int* par = p.parents + (size_t)n * p.S;
  unsigned long long m = 0ull;
  absent = false;
  int u = t;
  while (u >= 0) {
    if (u >= first && u < first + 64) m |= 1ull << (u - first);
    const int up = __ldg(par + u);
    if (up >= u || up < -2) raise_error(p.err_word, kErrDeviceArg);
    if (up >= u || up < -1) {
      absent = true;
      return 0ull;
    }
    u = up;
  }
  return m;
}

// The same for all rows of sequence n, by one warp in scratch of its own: up[t] becomes kRoot, or
// kAbsent for an absent row, and sees[t] (where given) the mask of row t over block rows
// [first, first + 64).  sees[t] holds the path from t up to, not including, up[t]; joining the path of
// up[t] to it doubles its length, and since parents come before their children, rows 32 at a time
// in order need at most 6 such steps each: 0.3 us where S <= 64, against 2.7 us for a walk up a
// 64-long chain.
constexpr short kRoot = -1, kAbsent = -2;
__device__ __forceinline__ void tree_rows(const Problem& p, int n, int first, int lane, short* up,
                                          unsigned long long* sees) {
  const int* par = p.parents + (size_t)n * p.S;
  __syncwarp();
  for (int t = lane; t < p.S; t += 32) {
    int u = __ldg(par + t);
    if (u >= t || u < kAbsent) {
      raise_error(p.err_word, kErrDeviceArg);
      u = kAbsent;
    }
    up[t] = (short)u;
    if (sees) sees[t] = t >= first && t < first + 64 ? 1ull << (t - first) : 0ull;
  }
  __syncwarp();
  for (int t0 = 0; t0 < p.S; t0 += 32) {
    const int t = t0 + lane;
    int u = t < p.S ? up[t] : kRoot;
    while (__any_sync(0xffffffffu, u >= 0)) {
      unsigned long long m = 0ull;
      int v = u;
      if (u >= 0) {
        if (sees) m = sees[u];
        v = up[u];
      }
      __syncwarp();
      if (u >= 0) {
        if (sees) sees[t] |= m;
        up[t] = (short)v;
      }
      u = v;
      __syncwarp();
    }
  }
}
// The visible keys of a loaded tile without a tree: [head, count).
__device__ __forceinline__ unsigned long long span_mask(int head, int count) {
  const unsigned long long upto = count >= 64 ? ~0ull : (1ull << count) - 1;
  return upto & (~0ull << head);
}

// Pool row (of the [num_pages * Hkv * page_size] rows of k_ctx / v_ctx) holding context
// position pos of (n, h) in a paged cache; -1, reported as a device argument error, when
// the page table names a page outside [0, num_pages).
__device__ __forceinline__ int paged_row(const Problem& p, int n, int h, int pos) {
  const int page = __ldg(p.page_table + (size_t)n * p.pages_per_seq + (pos >> p.page_shift));
  if (page < 0 || page >= p.num_pages) {
    raise_error(p.err_word, kErrDeviceArg);
    return -1;
  }
  return ((page * p.Hkv + h) << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
}

}  // namespace tt
