// The paged key/value cache: storing new tokens (ft_kv_append), reading whole
// sequences back (ft_kv_read), the checks of the cache's descriptions and the
// sticky status word of the ft_kv calls.
#include <mutex>

#include "driver_api.h"
#include "kv_common.h"

namespace ft {
namespace kv {

static __device__ int32_t g_kv_status;  // zero at load; set by kernels, read and cleared by ft_kv_status

ft_status status_word(int32_t** out) {
  struct Addr {
    CUcontext ctx = nullptr;
    void* addr = nullptr;
  };
  static std::mutex mu;
  static Addr known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
    return set_error(FT_ERR_CUDA, "cudaGetDevice failed or device ordinal >= 64");
  const CUcontext ctx = current_context();
  std::lock_guard<std::mutex> lk(mu);
  Addr& a = known[dev];
  if (!a.addr || a.ctx != ctx) {  // first call on this device, or in this context
    void* p = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&p, g_kv_status);
    if (e != cudaSuccess || !p) return set_error(FT_ERR_CUDA, "address of the ft_kv status word: %s", cudaGetErrorString(e));
    a.addr = p;
    a.ctx = current_context();
  }
  *out = static_cast<int32_t*>(a.addr);
  return FT_OK;
}

ft_status check_pages(const ft_kv_pages* p) {
  if (!p) return set_error(FT_ERR_INVALID_ARG, "pages is null");
  if (p->kv_dtype != FT_KV_BF16 && p->kv_dtype != FT_KV_FP8E4M3)
    return set_error(FT_ERR_INVALID_ARG, "kv_dtype=%d is not an ft_kv_dtype", p->kv_dtype);
  if (p->head_dim != 64 && p->head_dim != 128)
    return set_error(FT_ERR_UNSUPPORTED, "head_dim=%d is not 64 or 128", p->head_dim);
  if (p->page_tokens < 16 || p->page_tokens > 256 || (p->page_tokens & (p->page_tokens - 1)))
    return set_error(FT_ERR_UNSUPPORTED, "page_tokens=%d is not 16, 32, 64, 128 or 256", p->page_tokens);
  if (p->num_kv_heads < 1 || p->num_kv_heads > kMaxKvHeads)
    return set_error(FT_ERR_INVALID_ARG, "num_kv_heads=%d outside 1..%d", p->num_kv_heads, kMaxKvHeads);
  if (p->num_pages < 1 || p->num_pages > 0x7fffffffLL / (p->num_kv_heads * p->page_tokens))
    return set_error(FT_ERR_INVALID_ARG, "num_pages=%lld: num_pages * num_kv_heads * page_tokens must be 1..2^31-1",
                     (long long)p->num_pages);
  if (!p->k || !p->v || (p->kv_dtype == FT_KV_FP8E4M3 && (!p->k_scale || !p->v_scale)))
    return set_error(FT_ERR_INVALID_ARG, "null page pointer");
  if ((reinterpret_cast<uintptr_t>(p->k) | reinterpret_cast<uintptr_t>(p->v)) & 15)
    return set_error(FT_ERR_INVALID_ARG, "the pages are not 16-byte aligned");
  return FT_OK;
}

ft_status check_batch(const ft_kv_pages* p, const ft_kv_batch* b) {
  if (!b) return set_error(FT_ERR_INVALID_ARG, "batch is null");
  if (b->num_seqs < 0 || b->num_seqs > kMaxSeqs)
    return set_error(FT_ERR_INVALID_ARG, "num_seqs=%d outside 0..%d", b->num_seqs, kMaxSeqs);
  if (b->num_tokens < 0 || (b->num_seqs == 0 && b->num_tokens > 0))
    return set_error(FT_ERR_INVALID_ARG, "num_tokens=%d with num_seqs=%d", b->num_tokens, b->num_seqs);
  if (b->max_q_len < 0 || (b->num_tokens > 0 && b->max_q_len < 1))
    return set_error(FT_ERR_INVALID_ARG, "max_q_len=%d with num_tokens=%d", b->max_q_len, b->num_tokens);
  if (b->num_seqs == 0) return FT_OK;
  if (b->table_stride < 1 || b->table_stride > 0x7fffffffLL / p->page_tokens)
    return set_error(FT_ERR_INVALID_ARG, "table_stride=%lld: table_stride * page_tokens must be 1..2^31-1",
                     (long long)b->table_stride);
  if (!b->q_start || !b->kv_len || !b->block_table) return set_error(FT_ERR_INVALID_ARG, "null batch pointer");
  return FT_OK;
}

ft_status check_rows(const char* name, const void* ptr, int64_t token_stride, int64_t head_stride) {
  if (!ptr) return set_error(FT_ERR_INVALID_ARG, "%s is null", name);
  if ((reinterpret_cast<uintptr_t>(ptr) & 15) || (token_stride & 7) || (head_stride & 7))
    return set_error(FT_ERR_INVALID_ARG, "%s must be 16-byte aligned with strides that are multiples of 8 elements", name);
  return FT_OK;
}

namespace {

// ---------------------------------------------------------------- append

struct AppendArgs {
  ft_kv_pages p;
  ft_kv_batch b;
  const __nv_bfloat16* x[2];  // k, v
  int64_t ts[2], hs[2];
  int32_t* status;
};

// Scale exponent of a vector: the smallest k >= -110 with amax <= 448 * 2^k.
// amax = (1 + f) 2^E and 448 = 1.75 * 2^8, so k = E - 8, one more if 1 + f > 1.75.
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int k = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u);
  return max(k, kMinScaleExp);
}
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// One group of D / 8 lanes per vector (token, k or v, head): a 16-byte load per
// lane, the largest magnitude by shuffles within the group, an 8-byte (fp8) or
// 16-byte (bf16) store.
template <int D, bool kFp8>
__global__ void append_kernel(AppendArgs a) {
  constexpr int kLanes = D / 8;
  const int H = a.p.num_kv_heads;
  const long long g = ((long long)blockIdx.x * blockDim.x + threadIdx.x) / kLanes;
  const int sub = threadIdx.x % kLanes;
  if (g >= 2LL * a.b.num_tokens * H) return;  // whole groups leave together
  const int h = (int)(g % H);
  const long long r = g / H;
  const int which = (int)(r & 1), t = (int)(r >> 1);
  const int s = find_seq(a.b.q_start, a.b.num_seqs, t);
  const Seq q = load_seq(a.p, a.b, s, a.status);
  const int pos = q.n - q.m + (t - q.q0);
  if (t - q.q0 >= q.m || pos < 0) return;
  const int page = load_page(a.p, a.b, s, pos / a.p.page_tokens, a.status);
  if (page < 0) return;
  const uint4 raw = __ldg(reinterpret_cast<const uint4*>(a.x[which] + t * a.ts[which] + h * a.hs[which]) + sub);
  const long long row = ((long long)page * H + h) * a.p.page_tokens + pos % a.p.page_tokens;
  if (!kFp8) {
    reinterpret_cast<uint4*>(static_cast<uint8_t*>(which ? a.p.v : a.p.k) + row * (2 * D))[sub] = raw;
    return;
  }
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  float x[8];
  uint32_t top = 0;  // largest magnitude, as bits: bf16 magnitudes order like integers, NaN above infinity
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    top = max(top, max((w[i] << 16) & 0x7fffffffu, w[i] & 0x7fff0000u));
  }
  const uint32_t mask = (kLanes == 32 ? 0xffffffffu : ((1u << kLanes) - 1u) << ((threadIdx.x & 31) / kLanes * kLanes));
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(mask, top, o));
  uint2 codes = make_uint2(0u, 0u);
  uint32_t e = kNanScale;
  if (top < 0x7f800000u) {
    const int k = scale_exp(__uint_as_float(top));
    e = (uint32_t)(k + 127);
    const float inv = __uint_as_float((uint32_t)(127 - k) << 23);
    const float lim = k == 120 ? 240.0f : 448.0f;  // 256 * 2^120 would not be a bf16 value
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = pack_e4m3(fminf(fmaxf(x[2 * i] * inv, -lim), lim), fminf(fmaxf(x[2 * i + 1] * inv, -lim), lim));
    codes = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
  }
  reinterpret_cast<uint2*>(static_cast<uint8_t*>(which ? a.p.v : a.p.k) + row * D)[sub] = codes;
  if (sub == 0) (which ? a.p.v_scale : a.p.k_scale)[row] = (uint8_t)e;
}

// ---------------------------------------------------------------- read

struct ReadArgs {
  ft_kv_pages p;
  ft_kv_batch b;
  const int32_t* start;
  long long rows;
  __nv_bfloat16* out[2];
  int32_t* status;
};

template <int D, bool kFp8>
__global__ void read_kernel(ReadArgs a) {
  constexpr int kLanes = D / 8;
  const int H = a.p.num_kv_heads;
  const long long g = ((long long)blockIdx.x * blockDim.x + threadIdx.x) / kLanes;
  const int sub = threadIdx.x % kLanes;
  if (g >= 2 * a.rows * H) return;
  const int h = (int)(g % H);
  const long long r2 = g / H;
  const int which = (int)(r2 & 1);
  const long long r = r2 >> 1;
  const int s = find_seq(a.start, a.b.num_seqs, (int)r);
  const int pos = (int)r - __ldg(&a.start[s]);
  const int n = __ldg(&a.b.kv_len[s]);
  uint4 o = make_uint4(0u, 0u, 0u, 0u);
  const bool over = n > a.b.table_stride * a.p.page_tokens;
  if (over) raise(a.status, FT_ERR_INVALID_ARG);
  int page = -1;
  if (!over && pos >= 0 && pos < n) page = load_page(a.p, a.b, s, pos / a.p.page_tokens, a.status);
  if (page >= 0) {
    const long long row = ((long long)page * H + h) * a.p.page_tokens + pos % a.p.page_tokens;
    const uint8_t* src = static_cast<const uint8_t*>(which ? a.p.v : a.p.k);
    if (!kFp8) {
      o = __ldg(reinterpret_cast<const uint4*>(src + row * (2 * D)) + sub);
    } else {
      const uint2 c = __ldg(reinterpret_cast<const uint2*>(src + row * D) + sub);
      const float sc = scale_of(__ldg((which ? a.p.v_scale : a.p.k_scale) + row));
      const uint32_t w[4] = {c.x & 0xffffu, c.x >> 16, c.y & 0xffffu, c.y >> 16};
      uint32_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w[i], __NV_E4M3);
        const float2 f = __half22float2(__half2(hr));
        const __nv_bfloat162 b2 = __floats2bfloat162_rn(f.x * sc, f.y * sc);  // exact: 4 significant bits
        v[i] = *reinterpret_cast<const uint32_t*>(&b2);
      }
      o = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
  reinterpret_cast<uint4*>(a.out[which] + (r * H + h) * D)[sub] = o;
}

template <typename Args>
cudaError_t launch_groups(void (*kernel)(Args), const Args& a, long long groups, int lanes, cudaStream_t s) {
  const long long blocks = (groups * lanes + 255) / 256;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  kernel<<<(unsigned)blocks, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace kv
}  // namespace ft

using namespace ft;
using namespace ft::kv;

extern "C" ft_status ft_kv_append(const ft_kv_pages* pages, const ft_kv_batch* batch, const void* k,
                                  int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
                                  int64_t v_head_stride, void* stream) {
  ft_status st = check_pages(pages);
  if (st == FT_OK) st = check_batch(pages, batch);
  if (st != FT_OK || batch->num_tokens == 0) return st;
  if ((st = check_rows("k", k, k_token_stride, k_head_stride)) != FT_OK) return st;
  if ((st = check_rows("v", v, v_token_stride, v_head_stride)) != FT_OK) return st;
  AppendArgs a{};
  a.p = *pages; a.b = *batch;
  a.x[0] = static_cast<const __nv_bfloat16*>(k); a.x[1] = static_cast<const __nv_bfloat16*>(v);
  a.ts[0] = k_token_stride; a.ts[1] = v_token_stride;
  a.hs[0] = k_head_stride; a.hs[1] = v_head_stride;
  if ((st = status_word(&a.status)) != FT_OK) return st;
  const long long groups = 2LL * batch->num_tokens * pages->num_kv_heads;
  const bool fp8 = pages->kv_dtype == FT_KV_FP8E4M3;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      pages->head_dim == 128 ? launch_groups(fp8 ? append_kernel<128, true> : append_kernel<128, false>, a, groups, 16, s)
                             : launch_groups(fp8 ? append_kernel<64, true> : append_kernel<64, false>, a, groups, 8, s);
  if (e != cudaSuccess) return set_error(FT_ERR_CUDA, "append launch: %s", cudaGetErrorString(e));
  return FT_OK;
}

extern "C" ft_status ft_kv_read(const ft_kv_pages* pages, const ft_kv_batch* batch, const int32_t* kv_start,
                                int64_t num_rows, void* k_out, void* v_out, void* stream) {
  ft_status st = check_pages(pages);
  if (st == FT_OK) st = check_batch(pages, batch);
  if (st != FT_OK) return st;
  if (num_rows < 0 || num_rows > 0x7fffffffLL || (num_rows > 0 && batch->num_seqs == 0))
    return set_error(FT_ERR_INVALID_ARG, "num_rows=%lld with num_seqs=%d", (long long)num_rows, batch->num_seqs);
  if (num_rows == 0) return FT_OK;
  if (!kv_start) return set_error(FT_ERR_INVALID_ARG, "kv_start is null");
  if ((st = check_rows("k_out", k_out, 0, 0)) != FT_OK) return st;
  if ((st = check_rows("v_out", v_out, 0, 0)) != FT_OK) return st;
  ReadArgs a{};
  a.p = *pages; a.b = *batch; a.start = kv_start; a.rows = num_rows;
  a.out[0] = static_cast<__nv_bfloat16*>(k_out); a.out[1] = static_cast<__nv_bfloat16*>(v_out);
  if ((st = status_word(&a.status)) != FT_OK) return st;
  const long long groups = 2LL * num_rows * pages->num_kv_heads;
  const bool fp8 = pages->kv_dtype == FT_KV_FP8E4M3;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      pages->head_dim == 128 ? launch_groups(fp8 ? read_kernel<128, true> : read_kernel<128, false>, a, groups, 16, s)
                             : launch_groups(fp8 ? read_kernel<64, true> : read_kernel<64, false>, a, groups, 8, s);
  if (e != cudaSuccess) return set_error(FT_ERR_CUDA, "read launch: %s", cudaGetErrorString(e));
  return FT_OK;
}

extern "C" ft_status ft_kv_status(void* stream) {
  int32_t* w = nullptr;
  const ft_status st = status_word(&w);
  if (st != FT_OK) return st;
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return set_error(FT_ERR_CUDA, "stream synchronize: %s", cudaGetErrorString(e));
  int32_t word = 0;
  e = cudaMemcpy(&word, w, sizeof word, cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return set_error(FT_ERR_CUDA, "reading the ft_kv status word: %s", cudaGetErrorString(e));
  if (word == FT_OK) return FT_OK;
  const int32_t zero = 0;
  e = cudaMemcpy(w, &zero, sizeof zero, cudaMemcpyHostToDevice);
  if (e != cudaSuccess) return set_error(FT_ERR_CUDA, "clearing the ft_kv status word: %s", cudaGetErrorString(e));
  return set_error((ft_status)word, "an ft_kv call met %s",
                   word == FT_ERR_INVALID_ARG ? "device data out of range (a page, a length or q_start)"
                                              : ft_status_str((ft_status)word));
}
