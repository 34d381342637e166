// What the kernels of the paged key/value cache share: its addressing, the
// batch's sequences, and the sticky status word.  Internal to libft.
#pragma once

#include <atomic>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "ft_internal.h"

namespace ft {
namespace kv {

constexpr int kMaxSeqs = 4096;
constexpr int kMaxKvHeads = 1024;
constexpr int kMinScaleExp = -110;  // smallest scale 2^-110: code * scale is then a normal bf16 value (or 0)
constexpr int kNanScale = 255;

// Host-side checks shared by the entry points (FT_OK, or set_error's status).
ft_status check_pages(const ft_kv_pages* p);
ft_status check_batch(const ft_kv_pages* p, const ft_kv_batch* b);
ft_status check_rows(const char* name, const void* ptr, int64_t token_stride, int64_t head_stride);
// Device address of the current device's sticky status word.
ft_status status_word(int32_t** out);
int sm_count();  // of the current device
// Raise a kernel's limit of dynamic shared memory, once per device
// (kId: a number of its own for each kernel of one type.  Static: a process may
// load two builds of the library, whose kernels are not the same.)
template <int kId, typename Kernel>
static cudaError_t allow_smem(Kernel* kernel, int bytes) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && (done.load() >> dev & 1))) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev);
  return e;
}
// A launch that may begin while the kernel before it on the stream ends (the kernel waits for its end itself).
template <typename... P, typename... A>
static cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

__device__ __forceinline__ void raise(int32_t* status, int what) { atomicCAS(status, 0, what); }

// A sequence's new tokens and length, held within the batch's bounds.
struct Seq {
  int q0, m, n;  // first row, new tokens, tokens in all
};
__device__ __forceinline__ Seq load_seq(const ft_kv_pages& p, const ft_kv_batch& b, int s, int32_t* status) {
  const int q0 = __ldg(&b.q_start[s]), q1 = __ldg(&b.q_start[s + 1]), n = __ldg(&b.kv_len[s]);
  const int most = (int)(b.table_stride * p.page_tokens);
  Seq r{q0, q1 - q0, n};
  if (q0 < 0 || q1 < q0 || q1 > b.num_tokens || q1 - q0 > b.max_q_len || n < 0 || n > most) {
    raise(status, FT_ERR_INVALID_ARG);
    r = Seq{0, 0, 0};
  }
  return r;
}
// Page of a sequence's token block `i` (which lies within its length), or -1.
__device__ __forceinline__ int load_page(const ft_kv_pages& p, const ft_kv_batch& b, int s, int i, int32_t* status) {
  const int g = __ldg(&b.block_table[s * b.table_stride + i]);
  if ((unsigned)g < (unsigned)p.num_pages) return g;
  raise(status, FT_ERR_INVALID_ARG);
  return -1;
}
// The last s in [0, n) with start[s] <= t (start ascending; 0 if none).
__device__ __forceinline__ int find_seq(const int32_t* start, int n, int t) {
  int lo = 0, hi = n - 1;
  if (hi > 0 && t <= hi) {  // a decode step's place, one row a sequence: its two loads instead of a search's six or twelve in turn
    const int a = __ldg(&start[t]), b = __ldg(&start[t + 1]);
    if (a <= t && (t == hi || t < b)) return t;
  }
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(&start[mid]) <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
// Page row of the batch's new token in row t at head 0 (head h: + h * page_tokens), and the
// token's position; kUnstored: it has a position but no place, kNobodys: it belongs to no sequence.
constexpr int kUnstored = -1, kNobodys = -2;
__device__ __forceinline__ int new_place(const ft_kv_pages& p, const ft_kv_batch& b, int t, int32_t* status, int* pos) {
  const int s = find_seq(b.q_start, b.num_seqs, t);
  const Seq q = load_seq(p, b, s, status);
  *pos = q.n - q.m + (t - q.q0);
  if (t < q.q0) {  // rows before q_start[0]: of no sequence, nor of a position that this would give
    raise(status, FT_ERR_INVALID_ARG);
    return kNobodys;
  }
  if (t - q.q0 >= q.m) return kNobodys;
  if (*pos < 0) return kUnstored;
  const int page = load_page(p, b, s, *pos / p.page_tokens, status);
  if (page < 0) return kUnstored;
  return page * p.num_kv_heads * p.page_tokens + *pos % p.page_tokens;  // rows are below 2^31
}
// 2^(e - 127) of an exponent byte (255: NaN).  Stored bytes are 17..247 or 255.
__device__ __forceinline__ float scale_of(uint32_t e) { return __uint_as_float(e == kNanScale ? 0x7fc00000u : e << 23); }


// Scale exponent of a vector: the smallest k >= -110 with amax <= 448 * 2^k,
// 121 if amax is not finite.  amax = (1 + f) 2^E and 448 = 1.75 * 2^8, so k = E - 8,
// one more if 1 + f > 1.75.
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  if (u >= 0x7f800000u) return 121;
  const int k = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u);
  return max(k, kMinScaleExp);
}
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
// Eight values of a vector whose scale exponent is k, as codes.  (x is overwritten.)
__device__ __forceinline__ uint2 encode8(float* x, int k) {
  const float inv = __uint_as_float((uint32_t)(127 - k) << 23);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] *= inv;
  if (k >= 120) {  // 256 * 2^120 would not be a bf16 value; k = 121: not finite
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = k > 120 ? 0.0f : fminf(fmaxf(x[i], -240.0f), 240.0f);
  }
  return make_uint2(pack_e4m3(x[0], x[1]) | pack_e4m3(x[2], x[3]) << 16,
                    pack_e4m3(x[4], x[5]) | pack_e4m3(x[6], x[7]) << 16);
}
__device__ __forceinline__ uint32_t scale_byte(int k) { return k > 120 ? (uint32_t)kNanScale : (uint32_t)(k + 127); }

}  // namespace kv
}  // namespace ft
