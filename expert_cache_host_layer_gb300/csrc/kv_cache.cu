// The paged key/value cache: storing new tokens (ft_kv_append), reading whole
// sequences back (ft_kv_read), the checks of the cache's descriptions and the
// sticky status word of the ft_kv calls.
#include <mutex>

#include "driver_api.h"
#include "kv_attend.h"

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

// Both directions move vectors (a token's key or value of one head) between a
// token-major tensor and the pages; they are bound by HBM.  A block takes
// `per` consecutive tokens.  Its first threads look their places up (sequence,
// position, page: a chain of dependent loads that costs more than moving a
// vector, so it is done once per token and not once per vector), and leave the
// rows in shared memory.  Then a group of D / 8 lanes takes a vector at a time,
// kBatch vectors in flight; append has its first batch on the way while the
// places are looked up.  (e4m3, head_dim 128: append of 16,384 tokens x 8 heads
// 21.2 us, 4.8 TB/s, short of the bandwidth for the quantisation's instructions
// and the few vectors of a block; read of 114,865 tokens x 8 heads 112 us, 6.3 TB/s.
// bf16, head_dim 64, 14,292 tokens x 5 heads of 37 sequences: append 7.4 us, 5.0
// TB/s.  One token: 5.2 us, of which the call on the host is 5.)
constexpr int kMoveThreads = 256;
constexpr int kMostTokens = 32;  // of a block
constexpr int kBatch = 2;

struct MoveArgs {
  ft_kv_pages p;
  ft_kv_batch b;
  const int32_t* start;             // read: [num_seqs + 1]
  int rows, per;                    // tokens in all, and of a block
  uint32_t by_h;                    // floor(2^32 / H) + 1, 0 for H = 1: v / H = (v * by_h) >> 32 for v < 2^17, H <= 2^10
  const __nv_bfloat16* x[2];        // append: k, v
  int64_t ts[2], hs[2];
  __nv_bfloat16* out[2];            // read
  int32_t* status;
};

// Page row of token `t` at head 0 (head h: + h * page_tokens), or a negative number.
template <bool kAppend>
__device__ __forceinline__ int place_of(const MoveArgs& a, int t) {
  int pos;
  if (kAppend) return new_place(a.p, a.b, t, a.status, &pos);
  const int s = find_seq(a.start, a.b.num_seqs, t), n = __ldg(&a.b.kv_len[s]);
  pos = t - __ldg(&a.start[s]);
  if (n > a.b.table_stride * a.p.page_tokens) {
    raise(a.status, FT_ERR_INVALID_ARG);
    return -1;
  }
  if (pos < 0 || pos >= n) return -1;
  const int page = load_page(a.p, a.b, s, pos / a.p.page_tokens, a.status);
  if (page < 0) return -1;
  return page * a.p.num_kv_heads * a.p.page_tokens + pos % a.p.page_tokens;  // rows are below 2^31
}

// Eight values of a vector, a lane of its group of kLanes: codes and exponent byte.
template <int kLanes>
__device__ __forceinline__ uint2 quantise(uint4 raw, uint32_t* e) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  // largest magnitude, as bits: bf16 magnitudes order like integers, NaN above infinity
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
  top = max(top & 0xffff0000u, top << 16);
  const int k = scale_exp(__uint_as_float(top));
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  *e = scale_byte(k);
  return encode8(x, k);
}
// Eight codes times their scale: exact, 4 significant bits.
__device__ __forceinline__ uint4 dequantise(uint2 c, float scale) {
  const uint32_t w[4] = {c.x & 0xffffu, c.x >> 16, c.y & 0xffffu, c.y >> 16};
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w[i], __NV_E4M3)));
    const __nv_bfloat162 b2 = __floats2bfloat162_rn(f.x * scale, f.y * scale);
    v[i] = *reinterpret_cast<const uint32_t*>(&b2);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

template <int D, bool kFp8, bool kAppend>
__global__ void __launch_bounds__(kMoveThreads, 8) move_kernel(const __grid_constant__ MoveArgs a) {
  constexpr int kLanes = D / 8, kGroups = kMoveThreads / kLanes;
  __shared__ int s_row[kMostTokens];
  const int H = a.p.num_kv_heads, P = a.p.page_tokens, which = blockIdx.y;  // k or v
  const int t0 = blockIdx.x * a.per, tokens = min(a.per, a.rows - t0), vectors = tokens * H;
  const int sub = threadIdx.x % kLanes;
  uint8_t* pages = static_cast<uint8_t*>(which ? a.p.v : a.p.k);
  uint8_t* scales = which ? a.p.v_scale : a.p.k_scale;
  const int64_t ts = kAppend ? a.ts[which] : (int64_t)H * D, hs = kAppend ? a.hs[which] : D;  // of the token-major side
  uint4* dense = reinterpret_cast<uint4*>(const_cast<__nv_bfloat16*>(kAppend ? a.x[which] : a.out[which]) + t0 * ts) + sub;
  // vector v of the block: token v / H, head v % H
  auto token_of = [&](int v) { return a.by_h ? (int)__umulhi((uint32_t)v, a.by_h) : v; };
  auto dense_at = [&](int v) {
    const int t = token_of(v);
    return dense + (t * ts + (v - t * H) * hs) / 8;
  };
  uint4 x[kBatch];
  dec::pdl_wait_primary();
  int v0 = threadIdx.x / kLanes;
  if (kAppend) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      x[i] = v0 + i * kGroups < vectors ? __ldg(dense_at(v0 + i * kGroups)) : make_uint4(0u, 0u, 0u, 0u);
  }
  if (threadIdx.x < tokens) s_row[threadIdx.x] = place_of<kAppend>(a, t0 + threadIdx.x);
  __syncthreads();
  for (; v0 - threadIdx.x / kLanes < vectors; v0 += kBatch * kGroups) {  // whole warps together
    int row[kBatch];
    uint2 c[kBatch];
    float sc[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int v = v0 + i * kGroups, t = token_of(v);
      row[i] = v < vectors ? s_row[t] : -1;
      if (row[i] < 0) continue;
      row[i] += (v - t * H) * P;
      if (kAppend) continue;
      if (kFp8) {
        c[i] = __ldg(reinterpret_cast<const uint2*>(pages + (long long)row[i] * D) + sub);
        sc[i] = scale_of(__ldg(scales + row[i]));
      } else {
        x[i] = __ldg(reinterpret_cast<const uint4*>(pages + (long long)row[i] * (2 * D)) + sub);
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int v = v0 + i * kGroups;
      if (kAppend) {
        if (kFp8) {
          uint32_t e;
          const uint2 codes = quantise<kLanes>(x[i], &e);
          if (row[i] >= 0) {
            reinterpret_cast<uint2*>(pages + (long long)row[i] * D)[sub] = codes;
            if (sub == 0) scales[row[i]] = (uint8_t)e;
          }
        } else if (row[i] >= 0) {
          reinterpret_cast<uint4*>(pages + (long long)row[i] * (2 * D))[sub] = x[i];
        }
        if (v + kBatch * kGroups < vectors) x[i] = __ldg(dense_at(v + kBatch * kGroups));
      } else if (v < vectors) {
        *dense_at(v) = row[i] < 0 ? make_uint4(0u, 0u, 0u, 0u) : kFp8 ? dequantise(c[i], sc[i]) : x[i];
      }
    }
  }
  dec::pdl_launch_dependents();
}

template <bool kAppend>
ft_status launch_move(MoveArgs& a, const char* name, cudaStream_t s) {
  const ft_status st = status_word(&a.status);
  if (st != FT_OK) return st;
  // one wave of eight blocks an SM, while that leaves a block no more than kMostTokens
  const int blocks = 4 * sm_count();  // for k, and as many for v
  a.per = (int)(((long long)a.rows + blocks - 1) / blocks);
  a.per = a.per > kMostTokens ? kMostTokens : a.per;
  a.by_h = a.p.num_kv_heads == 1 ? 0 : (uint32_t)((1ull << 32) / a.p.num_kv_heads) + 1;
  const dim3 grid((unsigned)(((long long)a.rows + a.per - 1) / a.per), 2);
  const bool fp8 = a.p.kv_dtype == FT_KV_FP8E4M3;
  auto* kernel = a.p.head_dim == 128 ? (fp8 ? move_kernel<128, true, kAppend> : move_kernel<128, false, kAppend>)
                                     : (fp8 ? move_kernel<64, true, kAppend> : move_kernel<64, false, kAppend>);
  const cudaError_t e = launch_dependent(kernel, grid, kMoveThreads, 0, s, a);
  if (e != cudaSuccess) return set_error(FT_ERR_CUDA, "%s launch: %s", name, cudaGetErrorString(e));
  return FT_OK;
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
  if (batch->num_tokens == 1) k_token_stride = v_token_stride = pages->head_dim;  // of single entries: not used
  if (pages->num_kv_heads == 1) k_head_stride = v_head_stride = pages->head_dim;
  if ((st = check_rows("k", k, k_token_stride, k_head_stride)) != FT_OK) return st;
  if ((st = check_rows("v", v, v_token_stride, v_head_stride)) != FT_OK) return st;
  MoveArgs a{};
  a.p = *pages; a.b = *batch; a.rows = batch->num_tokens;
  a.x[0] = static_cast<const __nv_bfloat16*>(k); a.x[1] = static_cast<const __nv_bfloat16*>(v);
  a.ts[0] = k_token_stride; a.ts[1] = v_token_stride;
  a.hs[0] = k_head_stride; a.hs[1] = v_head_stride;
  return launch_move<true>(a, "append", static_cast<cudaStream_t>(stream));
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
  MoveArgs a{};
  a.p = *pages; a.b = *batch; a.start = kv_start; a.rows = (int)num_rows;
  a.out[0] = static_cast<__nv_bfloat16*>(k_out); a.out[1] = static_cast<__nv_bfloat16*>(v_out);
  return launch_move<false>(a, "read", static_cast<cudaStream_t>(stream));
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
