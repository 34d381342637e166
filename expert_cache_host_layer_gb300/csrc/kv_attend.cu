// Attention over the paged key/value cache (ft_kv_attend): the entry point,
// the choice of the kernel, the workspace, and the kernel that joins partial
// sums.
#include <algorithm>
#include <type_traits>

#include "driver_api.h"
#include "kv_attend.h"

namespace ft {
namespace kv {
namespace {

// ---------------------------------------------------------------- partial sums

// Block (c, y) joins rows of the row block that CTA c of chunk_kernel began and
// others went on with: out = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i, in
// the order of the tokens.  kOne: a block per row, its eight warps share the
// parts (few rows of a long sequence, which many CTAs worked on); else a block
// takes kJoinRows rows, a warp kPer of them at once (many rows, a few parts).
constexpr int kJoinThreads = 256, kPer = 4, kJoinRows = 8 * kPer;

template <int D, bool kOne>
__global__ void __launch_bounds__(kJoinThreads) combine_kernel(const __grid_constant__ AttendArgs a) {
  constexpr int N = D / 32, R = kOne ? 1 : kPer;
  using Vec = typename std::conditional<N == 4, float4, float2>::type;
  __shared__ float s_o[kOne ? 8 : 1][D];
  __shared__ float s_l[8];
  dec::pdl_wait_primary();
  const int4 u = __ldcg(&a.desc[blockIdx.x]);  // {s, h, row block, last CTA}
  if (u.x < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Seq q = load_seq(a.p, a.b, u.x, a.status);
  const int c0 = blockIdx.x, parts = u.w - c0 + 1;
  // part i of row r: CTA c0's last slot, then the first slot of each CTA after it
  auto slot = [&](int i, int r) { return (long long)(2 * (c0 + i) + (i == 0)) * kChunkRows + r; };
  int row[R], token[R], head[R];
  float m[R], l[R], acc[R][N];
  bool any = false;
#pragma unroll
  for (int k = 0; k < R; ++k) {
    row[k] = kOne ? blockIdx.y : blockIdx.y * kJoinRows + k * 8 + warp;
    const int rr = row[k] % kSubRows, ti = rr / a.G;
    head[k] = rr - ti * a.G;
    token[k] = (u.z * 2 + row[k] / kSubRows) * a.tps + ti;
    if (ti >= a.tps || token[k] >= q.m) token[k] = -1;
    any |= token[k] >= 0;
    m[k] = -INFINITY;
    l[k] = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) acc[k][i] = 0.0f;
  }
  if (!any) return;  // kOne: all of the block; else whole warps
  for (int i = lane; i < parts; i += 32)
#pragma unroll
    for (int k = 0; k < R; ++k)
      if (token[k] >= 0) m[k] = fmaxf(m[k], __ldcg(&a.part_ml[slot(i, row[k]) * 2]));
#pragma unroll
  for (int k = 0; k < R; ++k)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m[k] = fmaxf(m[k], __shfl_xor_sync(0xffffffffu, m[k], o));
  const int per = kOne ? (parts + 7) / 8 : parts, i0 = kOne ? warp * per : 0, i1 = min(parts, i0 + per);
#pragma unroll 2
  for (int i = i0; i < i1; ++i) {
    float2 ml[R];
    float v[R][N];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      ml[k] = make_float2(-INFINITY, 0.0f);
      if (token[k] < 0) continue;
      ml[k] = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + slot(i, row[k]));
      *reinterpret_cast<Vec*>(v[k]) = __ldcg(reinterpret_cast<const Vec*>(a.part_o + slot(i, row[k]) * D) + lane);
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      if (token[k] < 0) continue;
      const float f = exp2_approx(ml[k].x - (m[k] == -INFINITY ? 0.0f : m[k]));
      l[k] += f * ml[k].y;
#pragma unroll
      for (int n = 0; n < N; ++n) acc[k][n] += f * v[k][n];
    }
  }
  if (kOne) {
#pragma unroll
    for (int i = 0; i < N; ++i) s_o[kOne ? warp : 0][lane * N + i] = acc[0][i];
    if (lane == 0) s_l[warp] = l[0];
    __syncthreads();
    if (warp) return;
    l[0] = 0.0f;
    for (int w = 0; w < 8; ++w) l[0] += s_l[w];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      acc[0][i] = 0.0f;
      for (int w = 0; w < 8; ++w) acc[0][i] += s_o[kOne ? w : 0][lane * N + i];
    }
  }
#pragma unroll
  for (int k = 0; k < R; ++k) {
    if (token[k] < 0) continue;
    const float inv = inverse(l[k]);
    __nv_bfloat16* out = a.out + out_at(a, q, u.y, token[k], head[k]) + lane * N;
#pragma unroll
    for (int i = 0; i < N; i += 2)
      *reinterpret_cast<__nv_bfloat162*>(out + i) = __floats2bfloat162_rn(acc[k][i] * inv, acc[k][i + 1] * inv);
    if (lane == 0) write_lse(a, q, u.y, token[k], head[k], m[k], l[k]);
  }
}

}  // namespace

int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  n = known[dev].load();
  if (n == 0 && cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) known[dev].store(n);
  return n;
}

cudaError_t launch_combine(const AttendArgs& a, int used, cudaStream_t s) {
  const bool one = used <= 64;  // rows enough for a block each without many idle blocks
  const dim3 grid(a.grid, one ? used : (used + kJoinRows - 1) / kJoinRows);
  if (a.p.head_dim == 128)
    return one ? launch_dependent(combine_kernel<128, true>, grid, kJoinThreads, 0, s, a)
               : launch_dependent(combine_kernel<128, false>, grid, kJoinThreads, 0, s, a);
  return one ? launch_dependent(combine_kernel<64, true>, grid, kJoinThreads, 0, s, a)
             : launch_dependent(combine_kernel<64, false>, grid, kJoinThreads, 0, s, a);
}

namespace {
using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                            const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
Encode encoder() {
  static const Encode enc = reinterpret_cast<Encode>(driver_fn("cuTensorMapEncodeTiled"));
  return enc;
}
}  // namespace

bool queries_map(CUtensorMap* m, const AttendArgs& a, int tokens) {
  const Encode enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)a.p.head_dim, (cuuint64_t)a.Hq, (cuuint64_t)a.b.num_tokens};
  const cuuint64_t pitch[2] = {(cuuint64_t)a.qhs * 2, (cuuint64_t)a.qts * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)a.G, (cuuint32_t)tokens};
  const cuuint32_t step[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(a.q), dims, pitch, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool pages_map(CUtensorMap* m, const ft_kv_pages& p, const void* base, int box_rows) {
  const Encode enc = encoder();
  if (!enc) return false;
  const bool fp8 = p.kv_dtype == FT_KV_FP8E4M3;
  const cuuint64_t dims[2] = {(cuuint64_t)p.head_dim, (cuuint64_t)(p.num_pages * p.num_kv_heads * p.page_tokens)};
  const cuuint64_t pitch[1] = {(cuuint64_t)p.head_dim * (fp8 ? 1 : 2)};
  const cuuint32_t box[2] = {fp8 ? (cuuint32_t)p.head_dim : 64u, (cuuint32_t)box_rows};
  const cuuint32_t step[2] = {1, 1};
  return enc(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
             pitch, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
             pitch[0] == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace kv
}  // namespace ft

using namespace ft;
using namespace ft::kv;

namespace {

// Which kernel takes what.  A (sequence, key head) of up to 16 rows is
// token_kernel's, one of more chunk_kernel's: its tiles have 128 rows whether
// they are used or not (a batch of 32 decoding sequences beside a chunk, e4m3:
// 96 us in chunk_kernel alone).  A batch that may hold both gets both, one
// after the other; there token_kernel takes up to 8 rows, its faster form,
// unless a single token has more.
struct Split {
  int small;  // rows of the largest sequence that is token_kernel's
  bool token, chunk;
};
Split split(const ft_kv_batch& b, int G) {
  const long long most = (long long)b.max_q_len * G;
  if (most <= kTokenRows) return {most <= 8 ? 8 : kTokenRows, true, false};
  if ((long long)b.num_seqs * b.max_q_len <= b.num_tokens || G > kTokenRows) return {0, false, true};  // all as long, or no single token fits
  return {G <= 8 ? 8 : kTokenRows, true, true};
}

// The workspace: [counter][desc][token_kernel's part_ml, part_o][chunk_kernel's],
// each 256-byte aligned, the counters in one place for every shape.  The kernels
// have partial sums of their own: they run side by side.
struct Workspace {
  uint64_t desc, ml[2], o[2], bytes;
};
Workspace layout(const ft_kv_pages& p, int grid, const Split& sp) {
  auto up = [](uint64_t x) { return (x + 255) & ~255ull; };
  Workspace w;
  w.desc = up(kMostCtas * sizeof(unsigned));
  w.bytes = up(w.desc + grid * sizeof(int4));
  for (int k = 0; k < 2; ++k) {
    const uint64_t parts = (k ? sp.chunk : sp.token) ? 2ull * grid * (k ? kChunkRows : kTokenRows) : 0;
    w.ml[k] = w.bytes;
    w.o[k] = up(w.ml[k] + parts * 2 * sizeof(float));
    w.bytes = up(w.o[k] + parts * p.head_dim * sizeof(float));
  }
  return w;
}

ft_status check_attend(const ft_kv_pages* pages, const ft_kv_batch* batch, int32_t num_q_heads) {
  ft_status st = check_pages(pages);
  if (st == FT_OK) st = check_batch(pages, batch);
  if (st != FT_OK) return st;
  if (num_q_heads < 1 || num_q_heads % pages->num_kv_heads)
    return set_error(FT_ERR_INVALID_ARG, "num_q_heads=%d is not a multiple of num_kv_heads=%d", num_q_heads,
                     pages->num_kv_heads);
  if (pages->kv_dtype == FT_KV_FP8E4M3 &&
      ((reinterpret_cast<uintptr_t>(pages->k_scale) | reinterpret_cast<uintptr_t>(pages->v_scale)) & 15))
    return set_error(FT_ERR_INVALID_ARG, "the scales are not 16-byte aligned");
  return FT_OK;
}

}  // namespace

extern "C" uint64_t ft_kv_attend_workspace(const ft_kv_pages* pages, const ft_kv_batch* batch, int32_t num_q_heads) {
  if (check_attend(pages, batch, num_q_heads) != FT_OK) return 0;
  const Split sp = split(*batch, num_q_heads / pages->num_kv_heads);
  return layout(*pages, std::min(sm_count(), kMostCtas), sp).bytes;
}

extern "C" ft_status ft_kv_attend(const ft_kv_pages* pages, const ft_kv_batch* batch, int32_t num_q_heads,
                                  const void* q, int64_t q_token_stride, int64_t q_head_stride, void* out,
                                  int64_t out_token_stride, int64_t out_head_stride, float* lse, float scale,
                                  int32_t causal, int32_t window, void* workspace, uint64_t workspace_bytes,
                                  void* stream) {
  ft_status st = check_attend(pages, batch, num_q_heads);
  if (st != FT_OK) return st;
  if (window < 0 || (window > 0 && !causal))
    return set_error(FT_ERR_INVALID_ARG, "window=%d (causal=%d): a window is positive and causal", window, causal);
  if (!(scale == scale)) return set_error(FT_ERR_INVALID_ARG, "scale is NaN");
  if (batch->num_tokens == 0) return FT_OK;
  if ((st = check_rows("q", q, q_token_stride, q_head_stride)) != FT_OK) return st;
  if ((st = check_rows("out", out, out_token_stride, out_head_stride)) != FT_OK) return st;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return set_error(FT_ERR_INVALID_ARG, "workspace is null or not 256-byte aligned");
  const int G = num_q_heads / pages->num_kv_heads;
  const long long rows = (long long)batch->max_q_len * G;  // of a (sequence, key head), at most
  if (rows > 0x7fffffffLL / 2) return set_error(FT_ERR_UNSUPPORTED, "max_q_len * (num_q_heads / num_kv_heads) is too large");
  if (G > kSubRows)
    return set_error(FT_ERR_UNSUPPORTED, "num_q_heads / num_kv_heads = %d is above %d", G, kSubRows);
  if (q_token_stride <= 0 || q_head_stride <= 0)
    return set_error(FT_ERR_INVALID_ARG, "q's strides must be positive");
  const Split sp = split(*batch, G);
  const int grid = std::min(sm_count(), kMostCtas);
  const Workspace ws = layout(*pages, grid, sp);
  if (workspace_bytes < ws.bytes)
    return set_error(FT_ERR_INVALID_ARG, "workspace of %llu bytes: %llu are needed",
                     (unsigned long long)workspace_bytes, (unsigned long long)ws.bytes);
  AttendArgs a{};
  a.p = *pages; a.b = *batch;
  a.q = static_cast<const __nv_bfloat16*>(q); a.out = static_cast<__nv_bfloat16*>(out); a.lse = lse;
  a.qts = q_token_stride; a.qhs = q_head_stride; a.ots = out_token_stride; a.ohs = out_head_stride;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.Hq = num_q_heads; a.G = G; a.tps = kSubRows / G; a.causal = causal != 0; a.window = window; a.grid = grid; a.small = sp.small;
  if ((st = status_word(&a.status)) != FT_OK) return st;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  a.counter = reinterpret_cast<unsigned*>(w);
  a.desc = reinterpret_cast<int4*>(w + ws.desc);
  auto parts = [&](int k) {
    a.part_ml = reinterpret_cast<float*>(w + ws.ml[k]);
    a.part_o = reinterpret_cast<float*>(w + ws.o[k]);
  };
  a.beside = sp.token && sp.chunk;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  parts(0);
  if (sp.token) e = launch_attend_token(a, s);
  parts(1);
  if (e == cudaSuccess && sp.chunk) e = launch_attend_chunk(a, s);
  // (a block's rows are used without a gap only while its first sub-tile holds them all)
  if (e == cudaSuccess && sp.chunk) e = launch_combine(a, batch->max_q_len <= a.tps ? (int)rows : kChunkRows, s);
  if (e != cudaSuccess) return set_error(FT_ERR_CUDA, "attend launch: %s", cudaGetErrorString(e));
  return FT_OK;
}
