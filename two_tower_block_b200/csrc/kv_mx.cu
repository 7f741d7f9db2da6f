// Writing a microscaled context cache and reading it back (format: mx.cuh).
//
// Write: for every block of 32 elements of a new row, amax is the largest finite magnitude, e the
// least integer with amax <= 448 2^e (not below -127), and each element becomes e4m3(x 2^-e),
// rounded to nearest even.  bf16 keeps its exponent and mantissa in separate bit fields, so e
// comes straight from amax's bits: 448 = 1.75 2^8, hence the exponent of amax minus 8, plus one
// when its mantissa exceeds 1.75's.  The product x 2^-e is exact in fp32; the only rounding is the
// conversion.
//
// Both kernels are bound by HBM: 2 bytes in and 1 + 1/32 out per element for the write, the
// reverse for the read.  A thread holds 16 elements of K and of V (two 16-byte bf16 accesses and one
// 16-byte e4m3 access each), two neighbouring threads one scale block; rows are D contiguous
// elements on both sides, so every access is coalesced whatever the transposition of tokens and
// heads.  A block stays with one (sequence, KV head): no division in the loop.
#include "kv_mx.h"

#include <cuda_bf16.h>

#include "errbits.h"
#include "mx.cuh"

namespace tt {
namespace {

constexpr int kThreads = 256;

// Cache row of position pos of (n, h), or -1 (flagged) when the page table is out of the pool.
__device__ __forceinline__ long long cache_row(const MxRows& m, int n, int h, int pos, unsigned* err_word) {
  if (m.table == nullptr) return ((long long)n * m.Hkv + h) * m.cap + pos;
  const int page = __ldg(m.table + (size_t)n * m.pages_per_seq + (pos >> m.page_shift));
  if (page < 0 || page >= m.num_pages) {
    atomicOr(err_word, kErrDeviceArg);
    return -1;
  }
  return (((long long)page * m.Hkv + h) << m.page_shift) + (pos & ((1 << m.page_shift) - 1));
}

struct Bf16x16 {
  uint4 a, b;
};
__device__ __forceinline__ Bf16x16 load16(const uint4* p) { return {__ldcs(p), __ldcs(p + 1)}; }
// Largest finite magnitude (bit pattern) of this thread's 32-element block, which two threads hold.
__device__ __forceinline__ uint32_t block_amax(const Bf16x16& x) {
  uint32_t a = 0;
  const uint32_t w[8] = {x.a.x, x.a.y, x.a.z, x.a.w, x.b.x, x.b.y, x.b.z, x.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
    a = max(a, lo < 0x7F80u ? lo : 0u);
    a = max(a, hi < 0x7F80u ? hi : 0u);
  }
  return max(a, __shfl_xor_sync(0xffffffffu, a, 1));
}
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  return (uint32_t)max((int)(amax >> 7) - 8 + ((amax & 0x7Fu) > 0x60u ? 1 : 0), 0);
}
// Two bf16 (one word) times `inv` -> two e4m3 (low half); infinities saturate, NaN stays NaN.
__device__ __forceinline__ uint32_t quant2(uint32_t w, float inv) {
  const float lo = __uint_as_float(w << 16) * inv, hi = __uint_as_float(w & 0xFFFF0000u) * inv;
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 quant16(const Bf16x16& x, uint32_t byte) {
  // 2^-(byte - 127): byte 0..247, so the exponent field 254 - byte is a normal number's
  const float inv = __uint_as_float((254u - byte) << 23);
  return make_uint4(quant2(x.a.x, inv) | (quant2(x.a.y, inv) << 16), quant2(x.a.z, inv) | (quant2(x.a.w, inv) << 16),
                    quant2(x.b.x, inv) | (quant2(x.b.y, inv) << 16), quant2(x.b.z, inv) | (quant2(x.b.w, inv) << 16));
}

// Block (x, y): KV head x % Hkv of sequence x / Hkv, and the y-th share of its rows.  Thread: 16
// elements of a row, kThreads / (D / 16) rows at a time.
__global__ void __launch_bounds__(kThreads)
    kv_append_mx_kernel(const uint4* __restrict__ k_new, const uint4* __restrict__ v_new, const MxRows m,
                        int32_t* ctx_lens, const int32_t* __restrict__ counts, int B, int T, int advance,
                        unsigned* ticket, unsigned* err_word) {
  const int n = blockIdx.x / m.Hkv, h = blockIdx.x - n * m.Hkv;
  const int parts = m.D / 16, sh = 31 - __clz(parts);
  const int part = threadIdx.x & (parts - 1), rows = kThreads >> sh;
  auto span = [&](int i, int& L, int& cnt) {   // of sequence i; false: refused and left untouched
    L = ctx_lens[i];
    cnt = counts ? counts[i] : T;
    return L >= 0 && cnt >= 0 && cnt <= T && L <= m.cap - cnt;
  };
  int L, cnt;
  const bool fits = span(n, L, cnt);
  if (!fits && h == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicOr(err_word, kErrDeviceArg);
  const int end = fits ? cnt : 0;
  // whole warps stay in the loop together: two lanes share a scale
  for (long long t0 = (long long)blockIdx.y * rows; t0 < end; t0 += (long long)gridDim.y * rows) {
    const long long t = t0 + (threadIdx.x >> sh);
    const bool in = t < end;
    Bf16x16 kx{}, vx{};
    if (in) {
      const size_t from = ((((size_t)n * T + t) * m.Hkv + h) * parts + part) * 2;
      kx = load16(k_new + from);
      vx = load16(v_new + from);
    }
    const uint32_t kb = scale_byte(block_amax(kx)), vb = scale_byte(block_amax(vx));
    if (!in) continue;
    const long long row = cache_row(m, n, h, L + (int)t, err_word);
    if (row < 0) continue;
    const size_t at = (size_t)row * m.D + part * 16;
    *reinterpret_cast<uint4*>(m.k + at) = quant16(kx, kb);
    *reinterpret_cast<uint4*>(m.v + at) = quant16(vx, vb);
    if ((part & 1) == 0) {
      m.k_scale[at / kMxBlock] = (uint8_t)kb;
      m.v_scale[at / kMxBlock] = (uint8_t)vb;
    }
  }
  if (!advance) return;
  // the last block to arrive moves the lengths: by then every block has read them
  __shared__ bool s_last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicInc(ticket, gridDim.x * gridDim.y - 1) == gridDim.x * gridDim.y - 1;
  }
  __syncthreads();
  if (!s_last) return;
  for (int i = threadIdx.x; i < B; i += kThreads) {
    int Li, ci;
    if (span(i, Li, ci)) ctx_lens[i] = Li + ci;
  }
}

// Two e4m3 (low half of w) times 2^(byte - 127) -> two bf16 (round to nearest even: only scales
// near the bottom of the range reach bf16's subnormals).
__device__ __forceinline__ uint32_t value2(uint32_t w, float s_hi, float s_lo) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
  float a, b;
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h; }" : "=f"(a), "=f"(b) : "r"(h));
  const __nv_bfloat162 r = __floats2bfloat162_rn(a * s_hi * s_lo, b * s_hi * s_lo);
  return *reinterpret_cast<const uint32_t*>(&r);
}
// 16 values of one scale block to 32 bytes of the output.
__device__ __forceinline__ void store16(uint4* to, uint4 w, uint32_t byte) {
  // 2^(byte - 127) as two normal factors (the low end, 2^-127, is subnormal in fp32)
  const int e = (int)byte - 127, h = e >> 1;
  const float f0 = __uint_as_float((uint32_t)(127 + h) << 23), f1 = __uint_as_float((uint32_t)(127 + e - h) << 23);
  __stcs(to, make_uint4(value2(w.x & 0xFFFFu, f0, f1), value2(w.x >> 16, f0, f1), value2(w.y & 0xFFFFu, f0, f1),
                        value2(w.y >> 16, f0, f1)));
  __stcs(to + 1, make_uint4(value2(w.z & 0xFFFFu, f0, f1), value2(w.z >> 16, f0, f1), value2(w.w & 0xFFFFu, f0, f1),
                            value2(w.w >> 16, f0, f1)));
}

// Blocks and threads as in the write.
__global__ void __launch_bounds__(kThreads)
    kv_read_mx_kernel(const MxRows m, const int32_t* __restrict__ ctx_lens, const int32_t* __restrict__ starts, int T,
                      uint4* __restrict__ k_out, uint4* __restrict__ v_out, unsigned* err_word) {
  const int n = blockIdx.x / m.Hkv, h = blockIdx.x - n * m.Hkv;
  const int parts = m.D / 16, sh = 31 - __clz(parts);
  const int part = threadIdx.x & (parts - 1), per = kThreads >> sh;
  int L = ctx_lens[n];
  const int start = starts ? starts[n] : 0;
  if ((L < 0 || L > m.cap || start < 0) && h == 0 && blockIdx.y == 0 && threadIdx.x == 0)
    atomicOr(err_word, kErrDeviceArg);
  if (start < 0) return;
  L = min(max(L, 0), m.cap);
  const int rows = (int)min((long long)T, max(0ll, (long long)L - start));
  for (long long t = (long long)blockIdx.y * per + (threadIdx.x >> sh); t < rows; t += (long long)gridDim.y * per) {
    const long long row = cache_row(m, n, h, start + (int)t, err_word);
    if (row < 0) continue;
    const size_t at = (size_t)row * m.D + part * 16;
    const uint4 kw = __ldcs(reinterpret_cast<const uint4*>(m.k + at));
    const uint4 vw = __ldcs(reinterpret_cast<const uint4*>(m.v + at));
    const uint32_t kb = m.k_scale[at / kMxBlock], vb = m.v_scale[at / kMxBlock];
    const size_t to = ((((size_t)n * m.Hkv + h) * T + t) * parts + part) * 2;
    store16(k_out + to, kw, kb);
    store16(v_out + to, vw, vb);
  }
}

// x: the (sequence, head) pairs (below 2^31, as the plan's rows are).  y: what gives the GPU four waves of full
// SMs over them, at most one block per pass over the rows.
dim3 grid_of(int T, int B, int Hkv, int D, int sms) {
  const long long per = kThreads / (D / 16), pairs = (long long)B * Hkv;
  const long long want = (T + per - 1) / per, most = (sms * 8 * 4 + pairs - 1) / pairs;
  const long long y = want < most ? want : most;
  return dim3((unsigned)pairs, (unsigned)(y > 0 ? y : 1), 1);
}

}  // namespace

cudaError_t launch_kv_append_mx(const void* k_new, const void* v_new, const MxRows& m, int32_t* ctx_lens,
                                const int32_t* counts, int B, int T, int advance, unsigned* ticket,
                                unsigned* err_word, int sms, cudaStream_t stream) {
  const dim3 grid = grid_of(T, B, m.Hkv, m.D, sms);
  kv_append_mx_kernel<<<grid, kThreads, 0, stream>>>(static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new),
                                                     m, ctx_lens, counts, B, T, advance, ticket, err_word);
  return cudaGetLastError();
}

cudaError_t launch_kv_read_mx(const MxRows& m, const int32_t* ctx_lens, const int32_t* starts, int B, int T,
                              void* k_out, void* v_out, unsigned* err_word, int sms, cudaStream_t stream) {
  const dim3 grid = grid_of(T, B, m.Hkv, m.D, sms);
  kv_read_mx_kernel<<<grid, kThreads, 0, stream>>>(m, ctx_lens, starts, T, static_cast<uint4*>(k_out),
                                                   static_cast<uint4*>(v_out), err_word);
  return cudaGetLastError();
}

}  // namespace tt
