// A block whose warps wait for barriers that nobody completes (tests/test_gpu_kv_waits.py):
// warp 0 until the limit, warp 1 until warp 0 has aborted, warp 2 for one that is complete.
#include "kv_attend.h"

namespace {
__global__ void waits(int32_t* status, int32_t* result, unsigned long long* ns) {
  __shared__ uint64_t bar[3];
  __shared__ int flag;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 3; ++i) ft::dec::mbar_init(&bar[i], 1);
    ft::dec::mbar_init_fence();
    ft::dec::mbar_arrive(&bar[2]);
    flag = 0;
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5;
  const unsigned long long t0 = ft::dec::global_ns();
  const bool ok = warp == 1 ? [&] {  // no limit of its own would be reached: it begins half a second later
    while (ft::dec::global_ns() - t0 < 500000000ull) __nanosleep(1000);
    return ft::kv::wait_or_abort(&bar[1], 0, status + 1, &flag);
  }() : ft::kv::wait_or_abort(&bar[warp], 0, status, &flag);
  result[threadIdx.x] = ok;
  if ((threadIdx.x & 31) == 0) ns[warp] = ft::dec::global_ns() - t0;
}
}  // namespace

// status [2], result [96], ns [3]: device, zero.
extern "C" int kv_waits(int32_t* status, int32_t* result, unsigned long long* ns) {
  waits<<<1, 96>>>(status, result, ns);
  const cudaError_t e = cudaGetLastError();
  return (int)(e != cudaSuccess ? e : cudaDeviceSynchronize());
}
