// Log-sum-exp combine of the units that a range boundary cut into segments
// (combine_row.cuh: one thread per eight columns of a row), and the bounded-wait self test.
#include "combine_row.cuh"
#include "problem.h"
#include "ptx.cuh"
#include "walker.cuh"

namespace tt {
namespace {

constexpr int kThreads = 128;
constexpr int kFewUnitsSegments = 48;   // segments of a unit from which on combine_few_kernel runs

template <int D>
__global__ void __launch_bounds__(kThreads) combine_kernel(const Problem p) {
  // launched as a programmatic dependent of the attention kernel: wait until its grid has
  // completed and its partials are visible; the next call's attention kernel may be scheduled
  // meanwhile and waits for this grid itself
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x;
  const SplitRecord rec = p.records[c];
  if (rec.unit < 0) return;
  const int item = blockIdx.y * kThreads + threadIdx.x;
  if (item >= combine_items<D>(p)) return;
  combine_item<D, 8>(p, make_unit(p, rec.unit, 0), c, rec, item, true, 1, 0);
}

// Few units of many segments: block (u, y) does the y-th part of unit u, four threads an item.  It looks for
// the unit's record among those of all ranges itself, so that no blocks are launched for ranges without one.
template <int D>
__global__ void __launch_bounds__(kThreads) combine_few_kernel(const Problem p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ int s_range;
  __shared__ SplitRecord s_rec;
  if (threadIdx.x == 0) s_range = -1;
  __syncthreads();
  for (int c = threadIdx.x; c < p.C; c += kThreads) {
    const SplitRecord rec = p.records[c];
    if (rec.unit == (int)blockIdx.x) {
      s_rec = rec;
      s_range = c;
    }
  }
  __syncthreads();
  const int c = s_range;
  if (c < 0) return;
  const int item = blockIdx.y * (kThreads / 4) + threadIdx.x / 4, items = combine_items<D>(p);
  combine_item<D, 8>(p, make_unit(p, blockIdx.x, 0), c, s_rec, min(item, items - 1), item < items, 4, threadIdx.x & 3);
}

// One thread waits on a barrier that nothing arrives at; the bounded wait must
// give up, raise kErrTimeout and return.
__global__ void wait_selftest_kernel(unsigned* err_word, unsigned long long limit_ns) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bar), 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    WaitCtx w{&abort_flag, err_word, limit_ns};
    if (mbar_wait(smem_u32(&bar), 0, w)) atomicOr(err_word, 0x80000000u);  // must not happen
  }
  __syncthreads();
}

// The FMA-pipe exp2 of the softmax (ptx.cuh: exp2_poly2) on n arguments.
__global__ void exp2_selftest_kernel(const float* x, float* y, int n) {
  const int i = (blockIdx.x * blockDim.x + threadIdx.x) * 2;
  if (i + 1 < n) {
    const float2 e = exp2_poly2(make_float2(x[i], x[i + 1]));
    y[i] = e.x;
    y[i + 1] = e.y;
  } else if (i < n) {
    y[i] = exp2_poly2(make_float2(x[i], 0.f)).x;
  }
}

}  // namespace

cudaError_t launch_exp2_selftest(const float* x, float* y, int n, cudaStream_t stream) {
  exp2_selftest_kernel<<<(n + 511) / 512, 256, 0, stream>>>(x, y, n);
  return cudaGetLastError();
}

cudaError_t launch_combine(const Problem& p, cudaStream_t stream) {
  // a programmatic dependent launch: the launch overlaps the attention kernel's tail and the
  // kernel waits for the attention grid on the device
  cudaLaunchConfig_t cfg = {};
  const long long units = (long long)p.B * p.Hkv * p.NB;
  // (looking for the record costs 0.6 us, which few segments do not win back: 2 units of 35 tiles 13.7 -> 14.4 us, of 129
  // 19.3 -> 17.5)
  const bool few = p.C >= kFewUnitsSegments * units && most_unit_tiles(p) >= kFewUnitsSegments;
  const int threads = p.R * (p.D / 8) * (few ? 4 : 1);
  cfg.gridDim = dim3(few ? (unsigned)units : p.C, (threads + kThreads - 1) / kThreads, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.D == 128) return cudaLaunchKernelEx(&cfg, few ? combine_few_kernel<128> : combine_kernel<128>, p);
  return cudaLaunchKernelEx(&cfg, few ? combine_few_kernel<64> : combine_kernel<64>, p);
}

cudaError_t launch_wait_selftest(unsigned* err_word, unsigned long long limit_ns, cudaStream_t stream) {
  wait_selftest_kernel<<<1, 32, 0, stream>>>(err_word, limit_ns);
  return cudaGetLastError();
}

}  // namespace tt
