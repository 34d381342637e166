// Attention over the paged key/value cache (ft_kv_attend): the entry point and
// the plain kernel, one warp per row (new token, query head) that walks the
// row's visible tokens with a running maximum and sum.
#include "kv_common.h"

namespace ft {
namespace kv {
namespace {

struct RowArgs {
  ft_kv_pages p;
  ft_kv_batch b;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;
  int64_t qts, qhs, ots, ohs;
  float scale;
  int Hq, causal, window;
  int32_t* status;
};

template <int D, bool kFp8>
__device__ __forceinline__ void load_lane(const uint8_t* base, const uint8_t* scales, long long row, int lane, float* x) {
  constexpr int N = D / 32;
  if (kFp8) {
    const float sc = scale_of(__ldg(scales + row));
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const __nv_fp8x2_storage_t c = __ldg(reinterpret_cast<const uint16_t*>(base + row * D + lane * N + i));
      const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3)));
      x[i] = f.x * sc;
      x[i + 1] = f.y * sc;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(base + row * (2 * D) + (lane * N + i) * 2));
      x[i] = __uint_as_float(w << 16);
      x[i + 1] = __uint_as_float(w & 0xffff0000u);
    }
  }
}

template <int D, bool kFp8>
__global__ void row_kernel(RowArgs a) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31;
  const long long r = (long long)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);
  if (r >= (long long)a.b.num_tokens * a.Hq) return;
  const int t = (int)(r / a.Hq), hq = (int)(r % a.Hq);
  const int H = a.p.num_kv_heads, h = hq / (a.Hq / H), P = a.p.page_tokens;
  const int s = find_seq(a.b.q_start, a.b.num_seqs, t);
  const Seq q = load_seq(a.p, a.b, s, a.status);
  const int pos = q.n - q.m + (t - q.q0);
  const int lo = a.causal && a.window ? max(0, pos - a.window + 1) : 0;
  const int hi = t - q.q0 >= q.m ? 0 : a.causal ? min(q.n, pos + 1) : q.n;
  float x[N], o[N], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = __bfloat162float(a.q[t * a.qts + hq * a.qhs + lane * N + i]);
    o[i] = 0.0f;
  }
  for (int j = lo; j < hi; ++j) {
    const int page = max(0, load_page(a.p, a.b, s, j / P, a.status));
    const long long row = ((long long)page * H + h) * P + j % P;
    float k[N], v[N], d = 0.0f;
    load_lane<D, kFp8>(static_cast<const uint8_t*>(a.p.k), a.p.k_scale, row, lane, k);
    load_lane<D, kFp8>(static_cast<const uint8_t*>(a.p.v), a.p.v_scale, row, lane, v);
#pragma unroll
    for (int i = 0; i < N; ++i) d = fmaf(x[i], k[i], d);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) d += __shfl_xor_sync(0xffffffffu, d, w);
    d *= a.scale;
    const float mn = fmaxf(m, d), base = mn == -INFINITY ? 0.0f : mn;
    const float c = expf(m - base), p = expf(d - base);
    l = l * c + p;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = o[i] * c + p * v[i];
    m = mn;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int i = 0; i < N; ++i) a.out[t * a.ots + hq * a.ohs + lane * N + i] = __float2bfloat16(o[i] * inv);
  if (a.lse && lane == 0) a.lse[r] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace
}  // namespace kv
}  // namespace ft

using namespace ft;
using namespace ft::kv;

extern "C" uint64_t ft_kv_attend_workspace(const ft_kv_pages* pages, const ft_kv_batch* batch, int32_t num_q_heads) {
  if (check_pages(pages) != FT_OK || check_batch(pages, batch) != FT_OK || num_q_heads < 1 ||
      num_q_heads % pages->num_kv_heads)
    return 0;
  return 256;
}

extern "C" ft_status ft_kv_attend(const ft_kv_pages* pages, const ft_kv_batch* batch, int32_t num_q_heads,
                                  const void* q, int64_t q_token_stride, int64_t q_head_stride, void* out,
                                  int64_t out_token_stride, int64_t out_head_stride, float* lse, float scale,
                                  int32_t causal, int32_t window, void* workspace, uint64_t workspace_bytes,
                                  void* stream) {
  ft_status st = check_pages(pages);
  if (st == FT_OK) st = check_batch(pages, batch);
  if (st != FT_OK) return st;
  if (num_q_heads < 1 || num_q_heads % pages->num_kv_heads)
    return set_error(FT_ERR_INVALID_ARG, "num_q_heads=%d is not a multiple of num_kv_heads=%d", num_q_heads,
                     pages->num_kv_heads);
  if (window < 0 || (window > 0 && !causal))
    return set_error(FT_ERR_INVALID_ARG, "window=%d (causal=%d): a window is positive and causal", window, causal);
  if (!(scale == scale)) return set_error(FT_ERR_INVALID_ARG, "scale is NaN");
  if (batch->num_tokens == 0) return FT_OK;
  if ((st = check_rows("q", q, q_token_stride, q_head_stride)) != FT_OK) return st;
  if ((st = check_rows("out", out, out_token_stride, out_head_stride)) != FT_OK) return st;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) ||
      workspace_bytes < ft_kv_attend_workspace(pages, batch, num_q_heads))
    return set_error(FT_ERR_INVALID_ARG, "workspace: %llu bytes at a 256-byte boundary are needed",
                     (unsigned long long)ft_kv_attend_workspace(pages, batch, num_q_heads));
  RowArgs a{};
  a.p = *pages; a.b = *batch;
  a.q = static_cast<const __nv_bfloat16*>(q); a.out = static_cast<__nv_bfloat16*>(out); a.lse = lse;
  a.qts = q_token_stride; a.qhs = q_head_stride; a.ots = out_token_stride; a.ohs = out_head_stride;
  a.scale = scale; a.Hq = num_q_heads; a.causal = causal != 0; a.window = window;
  if ((st = status_word(&a.status)) != FT_OK) return st;
  const long long blocks = ((long long)batch->num_tokens * num_q_heads + 3) / 4;
  if (blocks > 0x7fffffffLL) return set_error(FT_ERR_UNSUPPORTED, "num_tokens * num_q_heads is too large");
  const bool fp8 = pages->kv_dtype == FT_KV_FP8E4M3;
  auto* kernel = pages->head_dim == 128 ? (fp8 ? row_kernel<128, true> : row_kernel<128, false>)
                                        : (fp8 ? row_kernel<64, true> : row_kernel<64, false>);
  kernel<<<(unsigned)blocks, 128, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(FT_ERR_CUDA, "attend launch: %s", cudaGetErrorString(e));
  return FT_OK;
}
