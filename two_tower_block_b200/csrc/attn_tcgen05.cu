// Block attention on the 5th-generation tensor cores (tcgen05 + TMEM + TMA).
//
// The method (paperfeed.app review of arXiv 2606.26493, "Nemotron-Labs-
// TwoTower", section "The idea: freeze the reader, train the writer"): the S
// noisy block queries of denoiser layer i attend, in one softmax, to the
// frozen context tower's layer-i cache followed by the block's own keys.
//
// One persistent CTA per SM walks its range of key tiles (sched.cuh).  The
// S*g query rows of a unit (all g query heads that share a KV head, for all S
// block tokens) are packed into one or two 128-row tensor-core tiles, so each
// key tile is read from HBM once and feeds up to 256 query rows.
//
// Roles (384 threads):
//   warp 0       TMA producer of Q (each segment) and of the K tiles, into the K half
//                of a ring of shared-memory slots (128-byte swizzle)
//   warp 3       TMA producer of the V tiles, into the V half of the ring; for a
//                tile whose valid rows are not a multiple of 16 it zeroes the V rows
//                the last MMA k-step would otherwise read
//   warp 1       TMEM owner; issues the MMAs of M-tile 0 (one elected lane): S =
//                Q_0 K^T into TMEM, O_0 += P V with P read from TMEM (aliasing its S
//                buffer)
//   warp 2       issues the MMAs of M-tile 1 (when the unit has two)
//   warps 4..7   softmax warpgroup of M-tile 0 (thread = TMEM lane = row)
//   warps 8..11  softmax warpgroup of M-tile 1
// TMEM columns: M-tile m owns S buffers [128m, 128m+128) (NBUF buffers of NK
// keys), O_0 = [256, 256+D), O_1 = [256+D, 256+2D).
//
// Pipeline per M-tile (tile G of the CTA uses S buffer G % NBUF): the MMA
// thread issues PV(j) as soon as P(j) is ready and then S(j+NBUF) into the
// buffer PV(j) has just consumed; with two buffers the softmax of tile j+1
// finds its S ready while the tensor core works on PV(j).
//
// The softmax keeps a running reference maximum per row and rescales O (in
// TMEM) only when a new maximum exceeds it by more than 2^8; the final
// normalisation divides by the sum of the same bf16-rounded weights the PV
// product used, so the result is exact up to rounding.
//
// VIS: tiles in which a row sees only some keys beyond a valid prefix -- a drafted tree's block
// tiles (each row sees itself and its ancestors) and the first tile of a paged window (the load
// starts at a page slice, before the window).  The softmax then selects by a 64-bit mask per row,
// built by every warp for itself (walker.cuh: tree_rows) once per block tile; full tiles run the
// same code as without VIS.  V rows that no row may see are cleared in shared memory, since a
// weight of 0 does not hide an infinity or NaN in them.
//
// MX: the context is e4m3 with a scale byte per 32 elements.  Warp 3 brings its tiles in as they are
// (load_raw_tiles), four more warps (12..15) write them as bf16 into the ring (convert_tiles), and
// warp 0 keeps Q and both of the block's own tiles.
//
// SPLIT (units of at most 128 rows): one M-tile leaves half of the roles idle while the softmax of one tile
// after another bounds the kernel (0.95 us a tile, against 0.75 us that HBM needs for it).  The two
// MMA warps and softmax warpgroups then share the unit's tiles, even ones to the first and
// odd ones to the second, each with its own accumulator; at the end both read both accumulators,
// half of the columns each, and weigh them by e^(m - max) as the combine does.
//
// Every wait is bounded (ptx.cuh: mbar_wait); on a timeout the CTA raises the
// error word, drains what it issued, frees TMEM and returns.
#include <type_traits>

#include "combine_row.cuh"
#include "mx.cuh"
#include "problem.h"
#include "ptx.cuh"
#include "smem_opt_in.h"
#include "tc_common.cuh"
#include "walker.cuh"

namespace tt {
namespace {

constexpr int kMaxRows = 256;
constexpr int kRowBytes = 128;              // one 64-element bf16 row of a swizzled half
constexpr float kRescaleThreshold = 8.0f;   // log2 units
constexpr float kNoKey = -1e30f;            // reference maximum of a row that has seen no key yet

template <int D, int NK, bool VIS = false, bool MX = false, bool SPLIT = false>
struct Cfg {
  static constexpr int kTreeBytes = kMaxRows * (8 + 2);          // what a tree's rows see, and its walk
  static constexpr int kRows = SPLIT ? 128 : kMaxRows;          // rows of Q in shared memory
  static constexpr int kThreads = MX ? 512 : 384;
  static constexpr int kHalves = D / 64;
  static constexpr int kBufs = 128 / NK;                       // S buffers per M-tile
  static constexpr int kSlotBytes = NK * kRowBytes * kHalves;  // one K or V tile
  // the ring: 128 KB, or what fits beside raw tiles
  static constexpr int kStages = (MX ? 64 : 128) * 1024 / kSlotBytes;
  static constexpr int kQBytes = kRows * kRowBytes * kHalves;
  static constexpr int kStageOff = kQBytes;
  static constexpr int kEpiOff = kStageOff + kStages * kSlotBytes;
  static constexpr int kEpiBytes = VIS ? 8 * kTreeBytes : 0;   // trees: scratch of the 8 softmax warps
  static constexpr int kBarOff = kEpiOff + kEpiBytes;
  static constexpr int kBarBytes = 896;
  // MX: the ring of raw tiles: 64 rows of K and of V in e4m3, their scale bytes, a row mask
  static constexpr int kTreeOff = kBarOff + kBarBytes;   // a tree's absent rows, for the V tiles
  static constexpr int kMlOff = kTreeOff + (VIS ? kMaxRows * 2 : 0);   // SPLIT: (maximum, sum) of each row, [2][2][128]
  // MX: word s % kNanSegs is s + 1 if a K row that segment s of the CTA sees holds a NaN.  The converters are
  // at most kStages / 2 + 4 tiles, and so segments, ahead of a softmax warp: the scores of its next two tiles
  // wait for it, and K slots for the scores.
  static constexpr int kNanOff = kMlOff + (SPLIT ? 4 * 128 * 8 : 0);
  static constexpr int kNanSegs = 16;
  static_assert(kStages / 2 + 4 < kNanSegs, "ring of NaN marks");
  static constexpr int kRawOff = kNanOff + (MX ? kNanSegs * 4 : 0);
  static constexpr int kRawScale = 2 * NK * D;                      // byte offsets within a slot
  static constexpr int kScaleBytes = NK * (D / kMxBlock) + 16;
  static constexpr int kRawMask = kRawScale + 2 * kScaleBytes;
  static constexpr int kRawBytes = kRawMask + 16;
  static constexpr int kRaw = MX ? (D == 128 ? 4 : 6) : 0;
  static constexpr int kSmemBytes = kRawOff + kRaw * kRawBytes + 1024;  // + alignment slack
  // Register split: the 128-key variant keeps a full 128-score row per softmax thread (launch: 168
  // per thread = 65536 / 384 rounded down to 8); with converter warps the launch gives 128 and
  // the softmax takes its 176 from the others.
  static constexpr bool kSplitRegs = NK == 128 || MX;
  static constexpr int kCtrlRegs = 80, kConvRegs = 80, kSoftmaxRegs = MX ? 176 : 200;
  static_assert(4 * 32 * (kCtrlRegs + (MX ? kConvRegs : 0)) + 8 * 32 * kSoftmaxRegs <= kThreads * (MX ? 128 : 168),
                "register split");
  static_assert(kStages <= 16 && kRaw <= 6, "ring too deep");
  // SPLIT: a consumer waits for every second tile only, and a barrier's parity tells only one use of a slot
  // from the next, so the use before the one it waits for must be known to be over.  With an even
  // number of slots each of K and V that use was the consumer's own, or one of an earlier segment,
  // all of whose K tiles are consumed when this segment's Q has come, and all V tiles when the
  // accumulators have been read out (which is waited for first).  An odd number would let a wait for a
  // tile pass while the other consumer's tile before it was still on its way.
  static_assert(!SPLIT || kStages / 2 % 2 == 0, "two streams need an even number of slots");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

struct Bars {
  uint64_t q_full, q_empty, tail, drain;
  uint64_t s_full[2][2], p_full[2][2];  // [M-tile][S buffer]
  uint64_t pv_done[2], o_full[2], o_empty[2];
  uint64_t ml_full;         // SPLIT: both warpgroups' (maximum, sum) are in shared memory
  uint64_t kv_full[16], kv_empty[16];
  uint64_t blk_go[16];      // MX: this slot is free for a block tile
  uint64_t raw_full[6], raw_empty[6];  // MX: the ring of raw tiles
};

struct Shared {
  uint32_t tmem_base;
  int abort_flag;
  unsigned arrival;       // the count that this launch's arrivals reach (fused combine)
  long long T, start, end;
  Unit first, last;       // of the range
};
static_assert(sizeof(Bars) + sizeof(Shared) <= 896, "barrier block overflows its shared-memory slot");

// Fused split combine (cooperative launch only: every CTA is resident).  Once its segments and
// partials are written, each CTA adds one to its range's arrival count; every range does so
// exactly once per launch, so all counts of a launch are equal, and one more than this range's before
// it (`k`, read at the start).  For each cut unit with a
// segment in this range (at most two: the unit holding the range's first tile and the one
// holding its last), the CTA waits until every range of that unit has reached the count,
// then combines its share of the unit's items (combine_row.cuh): the i-th of n equal parts for the
// i-th of the unit's n ranges.  No CTA waits for ranges outside its units.  The waits
// are bounded; a CTA that gave up (or whose pipeline aborted) combines nothing and the error
// word says so.
template <int D, int THREADS, int kGroup>
__device__ __forceinline__ void fused_combine(const Problem& p, long long T, long long start, long long end,
                                              const Unit& first, const Unit& last, unsigned k, bool aborted) {
  __shared__ int s_ok;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x;
  __syncthreads();  // every write of this CTA precedes its arrival
  if (tid == 0) red_release_gpu_add(p.arrivals + c, 1u);
  if (start >= end || aborted) return;
  const int Ce = used_ranges(T, p.C);
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const Unit& x = which == 0 ? first : last;
    if (which == 1 && last.u == first.u) break;
    if (first_tile(x) >= start && end_tile(x) <= end) continue;  // whole in this range: not cut
    const long long* tab = range_table(p);
    const int c0 = range_of_tile_tab(tab, T, Ce, first_tile(x)), c1 = range_of_tile_tab(tab, T, Ce, end_tile(x) - 1);
    if (warp == 0) {
      bool ok = true;
      unsigned long long t0 = globaltimer_ns();
      bool anew = false;
      for (int cc = c0 + lane; cc <= c1 && ok; cc += 32) {
        while (ld_acquire_gpu_u32(p.arrivals + cc) < k) {
          if (timer_over(t0, p.wait_limit_ns, anew)) {
            raise_error(p.err_word, kErrTimeout);
            ok = false;
            break;
          }
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      if (lane == 0) s_ok = ok;
    }
    __syncthreads();
    if (!s_ok) return;
    const int n = c1 - c0 + 1, i = c - c0;
    const SplitRecord rec{x.u, c1, first_after(x, range_start_tab(tab, T, Ce, c0)) ? 0 : 1, 0};
    const int items = combine_items<D>(p), share = ceil_div(items, n);
    const int lo = i * share, hi = min(items, lo + share);
    // as many threads an item as there are, where its segments are many; whole warps stay together
    const int sh = n < kManySegments ? 0 : 4 * share <= THREADS ? 2 : 2 * share <= THREADS ? 1 : 0;
    const int warp_items = 32 >> sh;
#pragma unroll 1
    for (int it = lo + (tid >> sh); it < lo + (hi - lo + warp_items - 1) / warp_items * warp_items; it += THREADS >> sh)
      combine_item<D, kGroup>(p, x, c0, rec, min(it, items - 1), it < hi, 1 << sh, tid & ((1 << sh) - 1));
  }
}

// MX: the context tiles of the CTA's range, brought in as they are: K and V rows in e4m3 by untiled bulk
// copies (the rows of a cache or of a page lie one after another), the scale bytes by four-byte
// asynchronous copies, both counted by the slot's barrier.  One warp, which waits for nothing else, so
// that it stays kRaw tiles ahead of the conversion across units.
template <int D, int NK, bool SPLIT>
__device__ __forceinline__ void load_raw_tiles(const Problem& p, const Shared* sh, Bars* bars, uint8_t* smem,
                                               const WaitCtx& wc, int c, int lane) {
  using C = Cfg<D, NK, true, true, SPLIT>;
  const uint8_t* src[2] = {reinterpret_cast<const uint8_t*>(p.k_ctx), reinterpret_cast<const uint8_t*>(p.v_ctx)};
  const uint8_t* scales[2] = {p.k_scale, p.v_scale};
  const long long start = sh->start, end = sh->end;
  const int psh = p.page_table ? min(p.page_shift, 6) : 6;   // rows that lie together: 1 << psh
  uint32_t k = 0;
  bool ok = true;
  Unit x = sh->first;
  for (; ok;) {
    const Segment sg = segment_of(x, start, end, c);
    const InnerTiles inner = inner_tiles<NK>(p, x);
    for (int i = max(sg.lo, p.blk_tiles); i < sg.hi; ++i, ++k) {
      const uint32_t slot = k % C::kRaw;
      ok = mbar_wait_warp(smem_u32(&bars->raw_empty[slot]), ((k / C::kRaw) & 1) ^ 1, wc);
      if (!ok) break;
      uint8_t* dst = smem + C::kRawOff + slot * C::kRawBytes;
      const uint32_t bar = smem_u32(&bars->raw_full[slot]);
      const TileKeys tk = tile_keys<NK>(p, x, inner, i);
      const int mine = min(max(tk.count - (lane << psh), 0), 1 << psh);   // rows of lane's slice
      int row = 0;
      if (mine > 0) {
        const int pos = tk.first + (lane << psh);
        row = p.page_table ? paged_row(p, x.n, x.h, pos) : (x.n * p.Hkv + x.h) * p.ctx_stride + pos;
      }
      const bool there = mine > 0 && row >= 0;   // (a page outside the pool: its rows read as zeros)
      const uint32_t rows = __reduce_add_sync(0xffffffffu, there ? mine : 0);
      const unsigned long long bits = there ? span_mask(0, mine) << (lane << psh) : 0ull;
      const uint32_t m0 = __reduce_or_sync(0xffffffffu, (uint32_t)bits);
      const uint32_t m1 = __reduce_or_sync(0xffffffffu, (uint32_t)(bits >> 32));
      if (lane == 0) {
        *reinterpret_cast<unsigned long long*>(dst + C::kRawMask) =
            (((unsigned long long)m1 << 32) | m0) & span_mask(tk.head, NK);
        mbar_arrive_expect_tx(bar, 2 * rows * D);
      }
      __syncwarp();
      if (there) {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv)
          bulk_load(smem_u32(dst) + (kv * NK + (lane << psh)) * D, src[kv] + (size_t)row * D, mine * D, bar);
      }
      // scale bytes in words of four (sched.cuh: the converters skip the row in front of an odd tile)
      const int odd = mx_odd(D, p.page_table != nullptr, (x.n * p.Hkv + x.h) * p.ctx_stride + tk.first);
#pragma unroll
      for (int e = 0; e < 64; e += 32) {
        const ScaleWord w = scale_word(e + lane, D, p.page_table != nullptr, psh, odd, tk.count);
        const int s = min(w.slice, 31);
        const int row_s = __shfl_sync(0xffffffffu, row, s);
        const bool ok_s = __shfl_sync(0xffffffffu, there, s);
        if (w.bytes > 0 && ok_s) {
          const size_t at = (size_t)scale_word_at(w, D, psh, row_s);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv)
            cp_async_4(smem_u32(dst) + C::kRawScale + kv * C::kScaleBytes + (e + lane) * 4, scales[kv] + at, w.bytes);
        }
      }
      cp_async_mbar_arrive(bar);
    }
    if (!ok || sg.last) break;
    x = next_unit(p, x);
  }
  if (!ok) {
    // copies that may still be landing in shared memory
    int dummy = 0;
    WaitCtx dw{&dummy, nullptr, 2000000ull};
    for (uint32_t j = k > (uint32_t)C::kRaw ? k - C::kRaw : 0; j < k; ++j)
      mbar_wait(smem_u32(&bars->raw_full[j % C::kRaw]), (j / C::kRaw) & 1, dw);
  }
}

// MX: converter warp w of 0..3 turns rows [32 (w & 1), 32 (w & 1) + 32) of every K (w < 2) or V raw tile
// into bf16 in the ring's swizzled slot.  16 bytes at a time become 32; rows that are not visible
// become zeros, so P V meets no other row.  In each quarter of a warp, four lanes work on one
// 64-element half of a row and four on the other half of the next row, which keeps both the
// loads and the swizzled stores free of bank conflicts.
template <int D, int NK, bool SPLIT>
__device__ __forceinline__ void convert_tiles(const Problem& p, const Shared* sh, Bars* bars, uint8_t* smem,
                                              const WaitCtx& wc, int c, int w, int lane) {
  using C = Cfg<D, NK, true, true, SPLIT>;
  constexpr int H = C::kStages / 2, kRowScale = D / kMxBlock;
  const int kv = w >> 1, first_row = 32 * (w & 1);
  const long long start = sh->start, end = sh->end;
  // lane's 16-byte chunk of a row's half: the k4-th, of row r0 + lane / 4
  const int k4 = lane & 3, r4 = lane >> 2;
  uint32_t k = 0, t = 0, seg = 0;   // raw tiles converted, tiles and segments of the CTA passed
  bool ok = true;
  Unit x = sh->first;
  for (; ok;) {
    const Segment sg = segment_of(x, start, end, c);
    const InnerTiles inner = inner_tiles<NK>(p, x);
    for (int i = sg.lo; i < sg.hi; ++i, ++t) {
      const uint32_t stage = kv * H + t % H;
      const bool blk = i < p.blk_tiles;
      // every tile's free slot is waited for here, in order (a barrier's parity tells only one
      // use from the next); a block tile's is handed on to its producer warp, by both converter
      // warps and on a barrier of that slot, so that no barrier runs ahead of one who waits on it
      // (the first use of a slot needs no word)
      ok = mbar_wait_warp(smem_u32(&bars->kv_empty[stage]), ((t / H) & 1) ^ 1, wc);
      if (!ok) break;
      if (blk) {
        if (lane == 0 && t >= (uint32_t)H) mbar_arrive(smem_u32(&bars->blk_go[stage]));
        continue;
      }
      const uint32_t slot = k % C::kRaw;
      ok = mbar_wait_warp(smem_u32(&bars->raw_full[slot]), (k / C::kRaw) & 1, wc);
      if (!ok) break;
      const uint8_t* raw = smem + C::kRawOff + slot * C::kRawBytes;
      const TileKeys tk = tile_keys<NK>(p, x, inner, i);
      const int n = min(max(round16(tk.count) - first_row, 0), 32);   // rows that the MMAs read
      const int odd = mx_odd(D, p.page_table != nullptr, (x.n * p.Hkv + x.h) * p.ctx_stride + tk.first);
      const uint32_t mask = *reinterpret_cast<const uint32_t*>(raw + C::kRawMask + first_row / 8);
      const uint8_t* in = raw + (kv * NK + first_row + r4) * D + k4 * 16;
      const uint8_t* sc = raw + C::kRawScale + kv * C::kScaleBytes + (first_row + r4 + odd) * kRowScale + (k4 >> 1);
      uint8_t* to = smem + C::kStageOff + stage * C::kSlotBytes + (first_row + r4) * kRowBytes;
      // The full rows of most pieces run without selects, and 16 rows at a time with constant offsets from the
      // two halves of a row in lane's order (one half of head_dim 64).  What counts is the number of
      // instructions and the code's length, not a pipe (profiles: the integer pipe is a third busy): the warps of
      // an SM sub-partition run different code, and what is unrolled further is waited for as instruction
      // fetches (a batch of drafted trees: 280 us with 32 rows at a time, 257 with 16, 241 rolled, which cost
      // single tokens a fifth).
      // The look for NaN is two operations a word of four: 16-token blocks over 131072 positions 205 -> 214 us,
      // (at the pairs after conversion, or with a vote of its own: 217 and more).
      const int h0 = C::kHalves == 2 ? r4 & 1 : 0;
      auto chunk_in = [&](int h, int r0) { return in + (h0 ^ h) * 64 + r0 * D; };
      auto chunk_sc = [&](int h, int r0) { return sc + (h0 ^ h) * 2 + r0 * kRowScale; };
      auto chunk_to = [&](int h, int r0, int c2) {
        return reinterpret_cast<uint4*>(to + (h0 ^ h) * (NK * kRowBytes) + (((2 * k4 + c2) ^ r4) << 4) + r0 * kRowBytes);
      };
#pragma unroll 1
      for (int rr = 0; rr < n; rr += 16) {
        constexpr int kChunks = 2 * C::kHalves;   // of lane: rows rr + r4 and rr + 8 + r4
        uint4 b[kChunks];
        uint32_t byte[kChunks], top = 0, nan = 0;
#pragma unroll
        for (int e = 0; e < kChunks; ++e) {
          b[e] = *reinterpret_cast<const uint4*>(chunk_in(e % C::kHalves, rr + e / C::kHalves * 8));
          byte[e] = *chunk_sc(e % C::kHalves, rr + e / C::kHalves * 8);
          top = max(top, byte[e]);
          nan |= mx_nan_bits(b[e].x) | mx_nan_bits(b[e].y) | mx_nan_bits(b[e].z) | mx_nan_bits(b[e].w);
        }
        nan &= kMxNan;
        if (__all_sync(0xffffffffu, ((mask >> rr) & 0xffffu) == 0xffffu && max(top, nan) <= kMxOneFactor)) {
#pragma unroll
          for (int e = 0; e < kChunks; ++e) {
            const int h = e % C::kHalves, r0 = rr + e / C::kHalves * 8;
            const uint32_t f = (byte[e] + 120u) * 0x00800080u;   // mx_factor of a byte up to kMxOneFactor
            const uint2 b0 = mx_to_bf16x4(b[e].x, f), b1 = mx_to_bf16x4(b[e].y, f);
            const uint2 b2 = mx_to_bf16x4(b[e].z, f), b3 = mx_to_bf16x4(b[e].w, f);
            *chunk_to(h, r0, 0) = make_uint4(b0.x, b0.y, b1.x, b1.y);
            *chunk_to(h, r0, 1) = make_uint4(b2.x, b2.y, b3.x, b3.y);
          }
        } else {
#pragma unroll 1
          for (int e = 0; e < kChunks; ++e) {
            const int h = e % C::kHalves, r0 = rr + e / C::kHalves * 8;
            uint4 v = *reinterpret_cast<const uint4*>(chunk_in(h, r0));
            const uint32_t vb = *chunk_sc(h, r0);
            if (!((mask >> (r0 + r4)) & 1u)) v = make_uint4(0, 0, 0, 0);
            // a NaN in K makes NaN of the tile's scores, which the softmax's maximum and rounding pass over: its
            // warps find the mark instead (one in V needs none)
            if (kv == 0 && ((mx_nan_bits(v.x) | mx_nan_bits(v.y) | mx_nan_bits(v.z) | mx_nan_bits(v.w)) & kMxNan))
              reinterpret_cast<volatile uint32_t*>(smem + C::kNanOff)[seg % C::kNanSegs] = seg + 1;
            *chunk_to(h, r0, 0) = mx_to_bf16x8(make_uint2(v.x, v.y), vb);
            *chunk_to(h, r0, 1) = mx_to_bf16x8(make_uint2(v.z, v.w), vb);
          }
        }
      }
      ++k;
      fence_proxy_async_smem();
      __syncwarp();   // every lane has read its raw bytes and written its share of the tile
      if (lane == 0) {
        mbar_arrive(smem_u32(&bars->kv_full[stage]));
        mbar_arrive(smem_u32(&bars->raw_empty[slot]));
      }
    }
    if (!ok || sg.last) break;
    x = next_unit(p, x);
    ++seg;
  }
}

template <int D, int NK, bool VIS, bool MX, bool SPLIT>
__global__ void __launch_bounds__(Cfg<D, NK, VIS, MX, SPLIT>::kThreads, 1)
    attn_tcgen05_kernel(const Problem p, const __grid_constant__ TmaMaps maps) {
  using C = Cfg<D, NK, VIS, MX, SPLIT>;
  constexpr int NBUF = C::kBufs, kThreads = C::kThreads;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t q_s = sbase;
  const uint32_t kv_s = sbase + C::kStageOff;
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kBarOff);
  Shared* sh = reinterpret_cast<Shared*>(smem + C::kBarOff + sizeof(Bars));

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x;
  const int MT = !SPLIT && p.R > 128 ? 2 : 1;
  const int NS = SPLIT ? 2 : MT;        // MMA warps and softmax warpgroups at work
  // a dependent combine launch may be scheduled now; it waits for this grid on the device
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---------------------------------------------------------------- setup --
  {
    // zero Q (rows >= R stay zero for every segment) through the generic proxy; when R
    // fills its M-tiles every row is loaded by TMA and nothing needs clearing
    if (p.R % 128 != 0) {
      uint4* z = reinterpret_cast<uint4*>(smem);
      for (int i = tid; i < C::kQBytes / 16; i += kThreads) z[i] = make_uint4(0, 0, 0, 0);
      fence_proxy_async_smem();
    }
  }
  if (tid == 0) {
    mbar_init(smem_u32(&bars->q_full), 1);
    mbar_init(smem_u32(&bars->q_empty), NS);  // one commit per issuer
    mbar_init(smem_u32(&bars->tail), 1);
    mbar_init(smem_u32(&bars->drain), NS);
    mbar_init(smem_u32(&bars->ml_full), 256);
    for (int m = 0; m < 2; ++m) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(smem_u32(&bars->s_full[m][b]), 1);
        mbar_init(smem_u32(&bars->p_full[m][b]), 128);
      }
      mbar_init(smem_u32(&bars->pv_done[m]), 1);
      mbar_init(smem_u32(&bars->o_full[m]), 1);
      mbar_init(smem_u32(&bars->o_empty[m]), SPLIT ? 256 : 128);
    }
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&bars->kv_full[s]), MX ? 2 : 1);  // MX: the tile's two converter warps
      mbar_init(smem_u32(&bars->kv_empty[s]), MT);
    }
    if (MX)
      for (int s = 0; s < C::kStages; ++s) mbar_init(smem_u32(&bars->blk_go[s]), 2);
    for (int s = 0; s < C::kRaw; ++s) {
      mbar_init(smem_u32(&bars->raw_full[s]), 33);  // the expected bytes, 32 lanes' scale copies
      mbar_init(smem_u32(&bars->raw_empty[s]), 4);  // the converter warps
    }
    sh->abort_flag = 0;
    fence_barrier_init();
  }
  if (MX && tid < C::kNanSegs) reinterpret_cast<uint32_t*>(smem + C::kNanOff)[tid] = 0u;
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k_ctx);
    tma_prefetch_desc(&maps.v_ctx);
    tma_prefetch_desc(&maps.k_blk);
    tma_prefetch_desc(&maps.v_blk);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sh->tmem_base), 512);
    tmem_relinquish();
  }
  // launched as a programmatic dependent of the previous kernel on the stream: everything above
  // (barriers, TMEM, descriptor prefetch) overlaps that kernel's tail; nothing below reads or
  // writes global memory before it has completed
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == 2) {
    long long T = 0, start = 0, end = 0;
    Unit first;
    find_range(p, c, T, start, end, first);
    if (lane == 0) {
      sh->T = T;
      sh->start = start;
      sh->end = end;
      if (start < end) sh->first = first;
      if (p.arrivals != nullptr) sh->arrival = __ldcg(p.arrivals + c) + 1u;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const uint32_t tmem = sh->tmem_base;
  const long long T = sh->T, start = sh->start, end = sh->end;
  const WaitCtx wc{&sh->abort_flag, p.err_word, p.wait_limit_ns, MX};
  const bool have_work = start < end;
  if constexpr (C::kSplitRegs) {
    if (have_work && warp < 4) regs_dec<C::kCtrlRegs>();
    if (have_work && warp >= 12) regs_dec<C::kConvRegs>();
  }

  if (MX && warp == 3 && have_work) {
    if constexpr (MX) load_raw_tiles<D, NK, SPLIT>(p, sh, bars, smem, wc, c, lane);
  } else if ((warp == 0 || warp == 3) && have_work) {
    // =========================================================== producers ==
    // Warp 0 loads Q of each segment and the K tiles, warp 3 the V tiles, each into its own
    // half of the ring: K(t) of the CTA's t-th tile in stage t % H, V(t) in stage H + t % H
    // (H = half the stages).  A K slot frees as soon as both M-tiles' S MMAs have read it, long
    // before P V frees the V slot of the same tile, so K loads run further ahead than they
    // could behind V loads in one ring.
    constexpr int H = C::kStages / 2;
    const int kv = warp == 0 ? 0 : 1;
    uint32_t t = 0, q_it = 0, tail_ph = 0, go_ph = 0;
    bool ok = true;
    Unit x = sh->first;
    for (; ok;) {
      const Segment sg = segment_of(x, start, end, c);
      if (kv == 0) {
        ok = mbar_wait(smem_u32(&bars->q_empty), (q_it & 1) ^ 1, wc);
        if (!ok) break;
        if (lane == 0) {
          const uint32_t bar = smem_u32(&bars->q_full);
          mbar_arrive_expect_tx(bar, (uint32_t)(p.R * kRowBytes * C::kHalves));
          for (int hf = 0; hf < C::kHalves; ++hf)
            tma_load_3d(q_s + hf * (C::kRows * kRowBytes), &maps.q, bar, hf * 64, x.h * p.g, x.ns * p.S);
        }
        ++q_it;
      }
      const int ctx_row0 = (x.n * p.Hkv + x.h) * p.ctx_stride;
      const InnerTiles inner = inner_tiles<NK>(p, x);
      // paged cache: a context tile is loaded in slices of psub rows, one per page (pages of
      // at least NK keys hold whole tiles); slices past the tile's last key are not loaded
      const int psub = p.page_table ? min(1 << p.page_shift, NK) : NK;
      // paged context: lane s looks up the pool row of slice s of a tile (one table read per
      // lane, all in flight together), one tile ahead of the loads that use it
      auto slice_row = [&](int i) -> int {
        const TileKeys tk = tile_keys<NK>(p, x, inner, i);
        if (!p.page_table || tk.is_blk || lane * psub >= tk.count) return 0;
        const int row = paged_row(p, x.n, x.h, tk.first + lane * psub);
        return row < 0 ? (p.num_pages * p.Hkv) << p.page_shift : row;  // a bad page reads as zeros
      };
      int cur_row = MX ? 0 : slice_row(sg.lo);
      const int hi = MX ? min(sg.hi, p.blk_tiles) : sg.hi;   // (MX: context tiles come from the converters)
      auto load_tile = [&](int i, int kv) {
        const TileKeys tk = tile_keys<NK>(p, x, inner, i);
        const int box_rows = tk.is_blk ? min(p.S, NK) : (p.page_table ? ceil_div(tk.count, psub) * psub : NK);
        const uint32_t bytes = (uint32_t)(box_rows * kRowBytes * C::kHalves);
        const int nsl = p.page_table && !tk.is_blk ? box_rows / psub : 0;   // slices of a paged tile
        const int row_i = cur_row;
        if (!MX && i + 1 < sg.hi) cur_row = slice_row(i + 1);
        const int s = kv * H + (int)(t % H);
        if constexpr (MX) {
          if (t >= (uint32_t)H) {
            ok = mbar_wait(smem_u32(&bars->blk_go[s]), (go_ph >> s) & 1, wc);
            go_ph ^= 1u << s;
          }
        } else ok = mbar_wait(smem_u32(&bars->kv_empty[s]), ((t / H) & 1) ^ 1, wc);
        if (!ok) return;
        const uint32_t slot = kv_s + s * C::kSlotBytes;
        const CUtensorMap* m = tk.is_blk ? (kv ? &maps.v_blk : &maps.k_blk) : (kv ? &maps.v_ctx : &maps.k_ctx);
        // V rows [count, round16(count)) are read by the last PV k-step: zero them (with VIS also
        // the rows before a window and the absent rows of a tree).
        unsigned long long zero = 0ull;
        if constexpr (VIS) {
          if (kv == 1) {
            zero = span_mask(0, round16(tk.count)) & ~span_mask(tk.head, tk.count);
          }
        }
        const bool tree = VIS && kv == 1 && tk.is_blk && p.parents;   // which rows are absent: while the loads run
        const bool fix = VIS ? tree || zero != 0ull : kv == 1 && (tk.count & 15) != 0;
        const uint32_t bar = fix ? smem_u32(&bars->tail) : smem_u32(&bars->kv_full[s]);
        if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
        if (nsl > 0) {
          // each slice lands at its row offset in the stage (a multiple of 2 KB: the swizzle
          // pattern stays aligned); issued after the expected byte count is set
          __syncwarp();
          if (lane < nsl)
            for (int hf = 0; hf < C::kHalves; ++hf)
              tma_load_2d(slot + hf * (NK * kRowBytes) + lane * psub * kRowBytes, m, bar, hf * 64, row_i);
        } else if (lane == 0) {
          for (int hf = 0; hf < C::kHalves; ++hf) {
            const uint32_t dst = slot + hf * (NK * kRowBytes);
            if (tk.is_blk) tma_load_3d(dst, m, bar, hf * 64, x.h, x.ns * p.S + tk.first);
            else tma_load_2d(dst, m, bar, hf * 64, ctx_row0 + tk.first);
          }
        }
        if (MX && lane == 0) mbar_arrive(smem_u32(&bars->kv_full[s]));   // for the second converter warp
        if (tree) {
          short* up = reinterpret_cast<short*>(smem + C::kTreeOff);
          if (i == sg.lo) tree_rows(p, x.n, 0, lane, up, nullptr);   // (a segment may begin past tile 0)
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const int t = 32 * w + lane;
            zero |= (unsigned long long)__ballot_sync(0xffffffffu, t < tk.count && up[tk.first + t] == kAbsent)
                    << (32 * w);
          }
        }
        if (fix) {
          ok = mbar_wait(smem_u32(&bars->tail), tail_ph, wc);
          tail_ph ^= 1;
          if (!ok) return;
          const int r0 = VIS ? 0 : tk.count, r1 = round16(tk.count);
          const int n16 = (r1 - r0) * 8 * C::kHalves;  // 16-byte chunks to clear
          for (int e = lane; e < n16; e += 32) {
            const int hf = e / ((r1 - r0) * 8);
            const int rem = e - hf * (r1 - r0) * 8;
            const int row = r0 + rem / 8, ch = rem % 8;
            if (VIS && !((zero >> row) & 1ull)) continue;
            uint4* dst = reinterpret_cast<uint4*>(smem + C::kStageOff + s * C::kSlotBytes +
                                                  hf * (NK * kRowBytes) + row * kRowBytes + ch * 16);
            *dst = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars->kv_full[s]));
        }
      };
      for (int i = sg.lo; i < hi && ok; ++i, ++t) {
        load_tile(i, kv);
        if (MX && ok) load_tile(i, 1);   // (warp 0 brings in both of a block tile)
      }
      if (MX) t += sg.hi - max(sg.lo, hi);
      if (!ok || sg.last) break;
      x = next_unit(p, x);
    }
    if (!ok) {
      // drain: wait (briefly) for loads that may still be landing in shared memory
      int dummy = 0;
      WaitCtx dw{&dummy, nullptr, 2000000ull};
      for (uint32_t j = (t > (uint32_t)H ? t - H : 0); j < t; ++j)
        for (int h = kv; h < (MX ? 2 : kv + 1); ++h) mbar_wait(smem_u32(&bars->kv_full[h * H + j % H]), (j / H) & 1, dw);
      if (q_it) mbar_wait(smem_u32(&bars->q_full), (q_it - 1) & 1, dw);
    }
  } else if ((warp == 1 || (warp == 2 && NS == 2)) && have_work) {
    // ====================================================== MMA issuers ==
    // One warp per M-tile (warp 1: M-tile 0, warp 2: M-tile 1), so an M-tile whose P is not
    // ready never holds back the other's MMAs; the tensor core interleaves the two instruction
    // streams.  The whole warp runs the control flow (waits, tile bookkeeping, descriptors stay
    // warp-uniform) and one elected lane issues each burst of MMAs and its commits.  Each warp
    // commits its own reads of a ring slot and of Q, and those barriers expect one commit per
    // M-tile.
    const int m = warp - 1;
    constexpr int H = C::kStages / 2;   // K tiles in stages [0, H), V tiles in [H, 2H)
    uint32_t tb = 0, q_it = 0, G = 0, seg_cnt = 0;   // tb: the CTA's tile count before this segment
    bool ok = true;
    Unit x = sh->first;
    // descriptors: a start-address offset is added in 16-byte units to the low field
    const uint64_t qdesc = smem_desc_sw128(q_s + (SPLIT ? 0 : m * 128 * kRowBytes), 16, 1024);
    constexpr int kStep = SPLIT ? 2 : 1;   // of a segment's tiles, this warp's are j0, j0 + kStep, ...
    const int j0 = SPLIT ? m : 0;
    const uint64_t kdesc0 = smem_desc_sw128(kv_s, 16, 1024);
    const uint64_t vdesc0 = smem_desc_sw128(kv_s, NK * kRowBytes, 1024);
    const uint32_t idesc_pv = idesc_bf16_f32(128, D, 0, 1);
    const uint32_t idesc_s0 = idesc_bf16_f32(128, 0, 0, 0);
    const uint32_t s_tmem = tmem + m * 128, o_tmem = tmem + 256 + m * D;
    // S = Q K^T of one tile into buffer `buf` (K in ring slot `slot`), then its commits
    auto issue_s = [&](int buf, uint32_t slot, int n_mma) {
      const uint32_t idesc = idesc_s0 | ((uint32_t)(n_mma >> 3) << 17);
      const uint64_t kd = kdesc0 + (uint64_t)((slot * C::kSlotBytes) >> 4);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * (C::kRows * kRowBytes) + (kk & 3) * 32;
          const uint32_t koff = (kk >> 2) * (NK * kRowBytes) + (kk & 3) * 32;
          tc_mma_ss(s_tmem + buf * NK, qdesc + (off >> 4), kd + (koff >> 4), idesc, kk > 0);
        }
        tc_commit(smem_u32(&bars->s_full[m][buf]));
        tc_commit(smem_u32(&bars->kv_empty[slot]));
      }
      __syncwarp();
    };
    // K (kv = 0) or V (kv = 1) of the CTA's tile t
    auto kv_wait = [&](uint32_t t, int kv) {
      return mbar_wait_warp(smem_u32(&bars->kv_full[kv * H + t % H]), (t / H) & 1, wc);
    };
    for (; ok;) {
      const Segment sg = segment_of(x, start, end, c);
      const int n = sg.hi - sg.lo;
      const InnerTiles inner = inner_tiles<NK>(p, x);
      auto keys16 = [&](int j) { return round16(tile_keys<NK>(p, x, inner, sg.lo + j).count); };
      ok = mbar_wait_warp(smem_u32(&bars->q_full), q_it & 1, wc);
      ++q_it;
      if (!ok) break;
      tc_fence_after();
      // prologue: S of the warp's first NBUF tiles
      for (int i = 0, j = j0; i < NBUF && j < n && ok; ++i, j += kStep) {
        ok = kv_wait(tb + j, 0);
        if (!ok) break;
        tc_fence_after();
        issue_s((G + i) % NBUF, (tb + j) % H, keys16(j));
      }
      // (a warp without a tile waits for its accumulator all the same: no phase may be missed)
      if (SPLIT && ok && j0 >= n) ok = mbar_wait_warp(smem_u32(&bars->o_empty[m]), (seg_cnt & 1) ^ 1, wc);
      for (int j = j0; j < n && ok; j += kStep, ++G) {
        const int b = G % NBUF;
        const uint32_t ev = H + (tb + j) % H;  // stage of V of tile j
        // (the accumulator first: SPLIT's V slots of the segment before are all free then)
        if (j == j0) ok = mbar_wait_warp(smem_u32(&bars->o_empty[m]), (seg_cnt & 1) ^ 1, wc);
        if (ok) ok = kv_wait(tb + j, 1);
        if (ok) ok = mbar_wait_warp(smem_u32(&bars->p_full[m][b]), (G / NBUF) & 1, wc);
        if (!ok) break;
        tc_fence_after();
        const int nv = keys16(j);
        const uint64_t vd = vdesc0 + (uint64_t)((ev * C::kSlotBytes) >> 4);
        const uint32_t pa = s_tmem + b * NK;
        if (elect_one()) {
          if (nv == NK) {
#pragma unroll
            for (int kk = 0; kk < NK / 16; ++kk)
              tc_mma_ts(o_tmem, pa + kk * 8, vd + (uint64_t)(kk * 16 * kRowBytes >> 4), idesc_pv,
                        (j > j0 || kk > 0) ? 1u : 0u);
          } else {
            for (int kk = 0; kk < nv / 16; ++kk)
              tc_mma_ts(o_tmem, pa + kk * 8, vd + (uint64_t)(kk * 16 * kRowBytes >> 4), idesc_pv,
                        (j > j0 || kk > 0) ? 1u : 0u);
          }
          tc_commit(smem_u32(&bars->pv_done[m]));
          tc_commit(smem_u32(&bars->kv_empty[ev]));
        }
        __syncwarp();
        const int jn = j + NBUF * kStep;
        if (jn < n) {
          // S of the tile NBUF on into buffer b, after P V(j) has read P(j) from it (in issue order)
          ok = kv_wait(tb + jn, 0);
          if (!ok) break;
          tc_fence_after();
          issue_s(b, (tb + jn) % H, keys16(jn));
        }
      }
      if (!ok) break;
      tb += n;
      if (elect_one()) {
        tc_commit(smem_u32(&bars->o_full[m]));
        tc_commit(smem_u32(&bars->q_empty));
      }
      __syncwarp();
      ++seg_cnt;
      if (sg.last) break;
      x = next_unit(p, x);
    }
    // drain every MMA this warp issued before TMEM can be released
    if (elect_one()) tc_commit(smem_u32(&bars->drain));
    __syncwarp();
    int dummy = 0;
    WaitCtx dw{&dummy, nullptr, 2000000ull};
    mbar_wait(smem_u32(&bars->drain), 0, dw);
    __syncwarp();
  } else if (MX && warp >= 12 && have_work) {
    if constexpr (MX) convert_tiles<D, NK, SPLIT>(p, sh, bars, smem, wc, c, warp - 12, lane);
  } else if (warp >= 4 && have_work) {
    // ========================================================= softmax WGs ==
    if constexpr (C::kSplitRegs) regs_inc<C::kSoftmaxRegs>();
    const int m = (warp - 4) >> 2;
    const int q4 = warp & 3;             // TMEM lane quarter of this warp
    const int row = q4 * 32 + lane;      // row within the M-tile
    const int mr = SPLIT ? 0 : m;        // M-tile of the rows
    const int r = mr * 128 + row;        // packed row of the unit
    const bool rows_here = !SPLIT || q4 * 32 < p.R;    // a warp without rows only keeps the barriers going
    constexpr int kStep = SPLIT ? 2 : 1;
    if (m < NS) {
      const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
      const uint32_t s_base = tmem + lane_off + m * 128;  // + buffer * NK
      const uint32_t o_addr = tmem + lane_off + 256 + m * D;
      uint8_t* scratch = smem + C::kEpiOff + (warp - 4) * C::kTreeBytes;
      unsigned long long* tree_sees = reinterpret_cast<unsigned long long*>(scratch);    // [S <= 256]
      short* tree_up = reinterpret_cast<short*>(tree_sees + kMaxRows);                     // [S]
      const uint32_t gm = div_by(p.g);
      uint32_t G = 0, seg_cnt = 0;
      bool ok = true;
      Unit x = sh->first;
      for (; ok;) {
        const Segment sg = segment_of(x, start, end, c);
        float m_ref = -INFINITY, l = 0.f;
        // a row that a tree leaves out (or whose ancestors are left out) sees nothing
        bool absent = false;
        const int tok = VIS ? row_token(min(r, p.R - 1), gm) : 0;
        if constexpr (VIS) {
          if (p.parents) {
            tree_rows(p, x.n, 0, lane, tree_up, tree_sees);
            absent = tree_up[tok] == kAbsent;
          }
        }
        // One tile of the softmax: its S row in registers, the row maximum in log2 units, the
        // lazy rescale of O, then P (bf16) over the S buffer.  Full tiles and the masked last
        // tile of a unit run separate code: folding them into one path would make every full
        // tile pay for the masking.
        // (VIS: `mask` selects the keys of a tile that is not full; a row may see none of them, so
        // its reference maximum stays finite)
        auto tile = [&](auto full_tag, int count, unsigned long long mask, uint32_t s_addr, bool first) -> bool {
          constexpr bool kFull = decltype(full_tag)::value;
          uint32_t v[NK];
#pragma unroll
          for (int ch = 0; ch < NK / 32; ++ch)
            if (kFull || 32 * ch < count) tmem_ld32(s_addr + 32 * ch, v + 32 * ch);
          tc_wait_ld();
          float mx;
          if constexpr (VIS && !kFull) mx = fmaxf(tile_row_max_masked<NK>(v, mask) * p.scale_log2, kNoKey);
          else mx = tile_row_max<NK, kFull>(v, count) * p.scale_log2;
          if (first) {
            m_ref = mx;  // O is overwritten by the first PV of the segment
          } else {
            const bool need = mx > m_ref + kRescaleThreshold;
            if (__any_sync(0xffffffffu, need)) {
              // O must hold every earlier PV of this segment before it is rescaled
              if (!mbar_wait(smem_u32(&bars->pv_done[m]), (G - 1) & 1, wc)) return false;
              tc_fence_after();
              const float alpha = need ? fast_exp2(m_ref - mx) : 1.f;
              if (need) {
                m_ref = mx;
                l *= alpha;
              }
#pragma unroll 1
              for (int cc = 0; cc < D / 16; ++cc) {
                uint32_t o[16];
                tmem_ld16(o_addr + cc * 16, o);
                tc_wait_ld();
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                tmem_st16(o_addr + cc * 16, o);
              }
            }
          }
          if constexpr (VIS && !kFull) l += tile_exp_store_masked<NK>(v, count, mask, p.scale_log2, m_ref, s_addr);
          else l += tile_exp_store<NK, kFull>(v, count, p.scale_log2, m_ref, s_addr);
          return true;
        };
        const int i0 = sg.lo + (SPLIT ? m : 0);
        const InnerTiles inner = inner_tiles<NK>(p, x);
        for (int i = i0; i < sg.hi; i += kStep, ++G) {
          const TileKeys tk = tile_keys<NK>(p, x, inner, i);
          const int count = tk.count;
          unsigned long long mask = 0ull;
          bool full = count == NK;
          if constexpr (VIS) {
            const bool tree = tk.is_blk && p.parents;
            full = full && tk.head == 0 && !tree;
            if (!full) {
              mask = span_mask(tk.head, count);
              if (tree) {
                if (tk.first > 0) tree_rows(p, x.n, tk.first, lane, tree_up, tree_sees);
                mask &= absent ? 0ull : tree_sees[tok];
              }
            }
          }
          const int b = G % NBUF;
          const uint32_t s_addr = s_base + b * NK;
          ok = mbar_wait(smem_u32(&bars->s_full[m][b]), (G / NBUF) & 1, wc);
          if (!ok) break;
          tc_fence_after();
          // (128-key tiles keep a single masked path: a second copy of their 128-register body
          // would not fit the register budget)
          if (!rows_here)
            ok = true;
          else if constexpr (NK == 128)
            ok = tile(std::false_type{}, count, mask, s_addr, i == i0);
          else
            ok = full ? tile(std::true_type{}, count, mask, s_addr, i == i0)
                      : tile(std::false_type{}, count, mask, s_addr, i == i0);
          if (!ok) break;
          tc_wait_st();
          tc_fence_before();
          mbar_arrive(smem_u32(&bars->p_full[m][b]));
        }
        if (!ok) break;
        // ---- epilogue: O / l to the output (or the segment's partial) ----
        float wa = 1.f, wb = 0.f;             // weights of the accumulators (SPLIT: of both)
        bool has[2] = {true, false};
        if constexpr (SPLIT) {
          float2* ml = reinterpret_cast<float2*>(smem + C::kMlOff) + (seg_cnt & 1) * 256;
          ml[m * 128 + row] = make_float2(m_ref, l);
          mbar_arrive(smem_u32(&bars->ml_full));
          ok = mbar_wait(smem_u32(&bars->ml_full), seg_cnt & 1, wc);
          if (ok) ok = mbar_wait(smem_u32(&bars->o_full[m ^ 1]), seg_cnt & 1, wc);
          if (!ok) break;
          has[1] = sg.hi - sg.lo > 1;
          const float2 a = ml[row], b = has[1] ? ml[128 + row] : make_float2(a.x, 0.f);
          m_ref = fmaxf(a.x, b.x);
          wa = fast_exp2(a.x - m_ref);
          wb = has[1] ? fast_exp2(b.x - m_ref) : 0.f;
          l = wa * a.y + wb * b.y;
        }
        ok = mbar_wait(smem_u32(&bars->o_full[m]), seg_cnt & 1, wc);
        if (!ok) break;
        tc_fence_after();
        if (MX && reinterpret_cast<volatile uint32_t*>(smem + C::kNanOff)[seg_cnt % C::kNanSegs] == seg_cnt + 1)
          l = __int_as_float(0x7FFFFFFF);   // a key of every row is NaN
        const bool none = VIS && (absent || l == 0.f);   // no visible key: 0, lse = -inf
        const float inv = none ? 0.f : 1.f / l;
        wa *= inv;
        wb *= inv;
        // the lane's row of the final output, as an element offset; a lane writes it 32 bytes, whole
        // sectors, at a time.  Staging 32 x 32 blocks in shared memory for stores of 128 bytes a row
        // costs the load-store unit less (a block-causal call with a window of 64: 294 against 320 us),
        // but 0.5 us of every small call and, by its code, 40 us of 900 with a window of 1024.
        size_t row_at;
        {
          const int gr = min(r, p.R - 1), t = row_token(gr, gm);
          row_at = ((size_t)(x.ns * p.S + t) * p.Hq + x.h * p.g + (gr - t * p.g)) * D;
        }
        const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
        float* part = p.part_o + part_at(p, sg.slot, r, 0, D);   // four columns on: 4 R floats further
        constexpr int kChunks = D / 32 / kStep;   // SPLIT: this warpgroup's half of the columns
        const int c_lo = SPLIT ? m * kChunks : 0;
#pragma unroll 1   // (cold code: fetched once, not four times)
        for (int cc = c_lo; cc < c_lo + kChunks; ++cc) {
          uint32_t o[32];
          if constexpr (SPLIT) {
            uint32_t ob[32];
            tmem_ld32(tmem + lane_off + 256 + cc * 32, o);
            tmem_ld32(tmem + lane_off + 256 + D + cc * 32, ob);
            tc_wait_ld();
            // (an accumulator that took no P V holds anything: select, never scale by 0)
#pragma unroll
            for (int k = 0; k < 32; ++k)
              o[k] = __float_as_uint(wa * __uint_as_float(o[k]) + (has[1] ? wb * __uint_as_float(ob[k]) : 0.f));
          } else {
            tmem_ld32(o_addr + cc * 32, o);
            tc_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(wa * __uint_as_float(o[k]));
          }
          if (cc == c_lo + kChunks - 1) {
            // O fully read: the next segment may overwrite it
            tc_fence_before();
            mbar_arrive(smem_u32(&bars->o_empty[m]));
            if constexpr (SPLIT) mbar_arrive(smem_u32(&bars->o_empty[m ^ 1]));
          }
          if (VIS && none) {   // (an absent row's query may be anything: its accumulator too)
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0u;
          }
          if (r < p.R) {
            if (!sg.full) {
#pragma unroll
              for (int q = 0; q < 8; ++q)
                *reinterpret_cast<uint4*>(part + (size_t)(cc * 8 + q) * 4 * p.R) =
                    make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
            } else if (p.out_bf16) {
              uint32_t* to = reinterpret_cast<uint32_t*>(reinterpret_cast<__nv_bfloat16*>(p.out) + row_at + cc * 32);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = pack_bf16(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1]));
#pragma unroll
              for (int q = 0; q < 2; ++q) store_row(to + 8 * q, o + 8 * q, wide);
            } else {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                store_row(reinterpret_cast<uint32_t*>(p.out + row_at + cc * 32 + 8 * q), o + 8 * q, wide);
            }
          }
        }
        if (r < p.R && (!SPLIT || m == 0)) {
          const float lse2 = none ? -INFINITY : m_ref + __log2f(l);   // log2 units
          if (sg.full) {
            if (p.lse) {
              const int t = row_token(r, gm), j = r - t * p.g;
              p.lse[(size_t)(x.n * p.Hq + x.h * p.g + j) * (p.NB * p.S) + x.b * p.S + t] = lse2 * kLn2;
            }
          } else {
            p.part_lse[(size_t)sg.slot * p.R + r] = lse2;
          }
        }
        ++seg_cnt;
        if (sg.last) break;
        x = next_unit(p, x);
      }
    }
  }

  // for the combine: the range's last unit, and the record of the cut unit (if any) that begins in it
  if (tid == 64) {
    SplitRecord rec{-1, -1, 0, 0};
    if (have_work) {
      Unit x = sh->first;
      while (!last_before(x, end)) x = next_unit(p, x);
      sh->last = x;
      rec = record_of(x, T, p.C, start, end, range_table(p));
    }
    if (p.arrivals == nullptr) p.records[c] = rec;
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
  if (p.arrivals != nullptr)
    fused_combine<D, kThreads, C::kSplitRegs ? 4 : 8>(p, T, start, end, sh->first, sh->last, sh->arrival,
                               *(volatile int*)&sh->abort_flag != 0);
}

// The opt-in shared-memory size (first asked for by the plan: not during a graph capture).
template <int D, int NK, bool VIS, bool MX, bool SPLIT>
cudaError_t prepare_as() {
  static std::atomic<unsigned long long> done{0};
  return smem_opt_in(reinterpret_cast<const void*>(&attn_tcgen05_kernel<D, NK, VIS, MX, SPLIT>),
                     Cfg<D, NK, VIS, MX, SPLIT>::kSmemBytes, done);
}
template <int D, bool SPLIT>
cudaError_t prepare64() {
  cudaError_t e = prepare_as<D, 64, false, false, SPLIT>();
  if (e == cudaSuccess) e = prepare_as<D, 64, true, false, SPLIT>();
  if (e == cudaSuccess) e = prepare_as<D, 64, true, true, SPLIT>();
  return e;
}
template <int D>
cudaError_t prepare(int R) {
  const cudaError_t e = R <= 128 ? prepare64<D, true>() : prepare64<D, false>();
  return e != cudaSuccess ? e : prepare_as<D, 128, false, false, false>();
}

template <int D, int NK, bool VIS, bool MX, bool SPLIT>
cudaError_t launch_as(const Problem& p, const TmaMaps& maps, cudaStream_t stream) {
  using C = Cfg<D, NK, VIS, MX, SPLIT>;
  const cudaError_t e = prepare_as<D, NK, VIS, MX, SPLIT>();
  if (e != cudaSuccess) return e;
  // a programmatic dependent of the previous kernel on the stream (its setup overlaps that
  // kernel's tail), and cooperative when the fused combine needs every CTA resident at once
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.C, 1, 1);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeCooperative;
  attrs[1].val.cooperative = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = p.arrivals != nullptr ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, attn_tcgen05_kernel<D, NK, VIS, MX, SPLIT>, p, maps);
}

// Units of at most 128 rows: the two softmax warpgroups share the tiles (64-key tiles only).
template <int D, bool VIS, bool MX>
cudaError_t launch64(const Problem& p, const TmaMaps& maps, cudaStream_t stream) {
  return p.R <= 128 ? launch_as<D, 64, VIS, MX, true>(p, maps, stream) : launch_as<D, 64, VIS, MX, false>(p, maps, stream);
}
template <int D>
cudaError_t launch(const Problem& p, const TmaMaps& maps, cudaStream_t stream) {
  // trees, quantised contexts, and paged windows whose first load may start before the window: 64-key tiles
  const bool vis = p.parents || (p.window > 0 && p.win_align > 1);
  if (p.key_tile == 128) {
    if (vis || p.k_scale) return cudaErrorInvalidValue;
    return launch_as<D, 128, false, false, false>(p, maps, stream);
  }
  if (p.k_scale) return launch64<D, true, true>(p, maps, stream);
  return vis ? launch64<D, true, false>(p, maps, stream) : launch64<D, false, false>(p, maps, stream);
}

}  // namespace

cudaError_t prepare_attn_tcgen05(int D, int R) { return D == 128 ? prepare<128>(R) : prepare<64>(R); }

bool tcgen05_key_tile_supported(int key_tile) { return key_tile == 64 || key_tile == 128; }

cudaError_t launch_attn_tcgen05(const Problem& p, const TmaMaps& maps, cudaStream_t stream) {
  if (!tcgen05_key_tile_supported(p.key_tile)) return cudaErrorInvalidValue;
  // variant 2: head_dim 128 with 128-key tiles on the transposed-PV kernel (attn_tcgen05_pt.cu)
  if (p.D == 128 && p.key_tile == 128 && p.variant == 2) return launch_attn_pt(p, maps, stream);
  return p.D == 128 ? launch<128>(p, maps, stream) : launch<64>(p, maps, stream);
}

}  // namespace tt
