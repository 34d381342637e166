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

// What chunk_kernel has left: the row blocks that CTA c began and others went on
// with, and whose other parts were not there when it ended,
//   out = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i,
// in the order of the tokens.  kOne: block (c, r) joins row r, its eight warps
// share the parts (few rows of a long sequence, which many CTAs worked on); else
// block (c, y) joins rows 32 y .. 32 y + 31, a lane a row, a warp an eighth of
// the columns (many rows, a few parts: three are on their way together).  Bound
// by latency: joining every divided block here took 8-12 us of a call, what
// chunk_kernel leaves takes 2-6.
constexpr int kJoinThreads = 256;

template <int D, bool kOne>
__global__ void __launch_bounds__(kJoinThreads) combine_kernel(const __grid_constant__ AttendArgs a) {
  dec::pdl_wait_primary();
  const int c0 = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.y == 0 && threadIdx.x < 8) a.arrived[c0 * 8 + threadIdx.x] = 0u;
  const int row = kOne ? (int)blockIdx.y : (int)blockIdx.y * 32 + lane;
  const int4 u = __ldcg(&a.desc[c0 * 8 + (row >> 5)]);  // {s, h, row block, last CTA}
  if (u.x < 0) return;
  const Seq q = load_seq(a.p, a.b, u.x, a.status);
  const int parts = u.w - c0 + 1, in_sub = row % kSubRows, ti = in_sub / a.G, head = in_sub - ti * a.G;
  const int token = (u.z * 2 + row / kSubRows) * a.tps + ti;
  const bool mine = ti < a.tps && token < q.m;
  // part i: CTA c0's last slot, then the first slot of each CTA after it
  auto slot = [&](int i) { return 2LL * (c0 + i) + (i == 0); };
  auto ml = [&](int i) { return __ldcg(reinterpret_cast<const float2*>(a.part_ml) + slot(i) * kChunkRows + row); };
  if constexpr (kOne) {
    constexpr int N = D / 32;  // columns of a lane in the end; here lanes 0 .. D / 4 - 1 have four each
    __shared__ float s_o[8][D];
    __shared__ float s_l[8];
    if (!mine) return;  // all of the block
    float m = -INFINITY, l = 0.0f;
    for (int i = lane; i < parts; i += 32) m = fmaxf(m, ml(i).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float base = m == -INFINITY ? 0.0f : m;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int i = warp; i < parts; i += 8) {
      const float2 x = ml(i);
      const float f = exp2_approx(x.x - base);
      l = join(l, f, x.y);
      if (lane < D / 4) {
        const float4 y = __ldcg(part_at<D>(a, slot(i), row, lane * 4));
        acc.x = join(acc.x, f, y.x);
        acc.y = join(acc.y, f, y.y);
        acc.z = join(acc.z, f, y.z);
        acc.w = join(acc.w, f, y.w);
      }
    }
    if (lane < D / 4) *reinterpret_cast<float4*>(&s_o[warp][lane * 4]) = acc;
    if (lane == 0) s_l[warp] = l;
    __syncthreads();
    if (warp) return;
    l = 0.0f;
    for (int w = 0; w < 8; ++w) l += s_l[w];
    float o[N] = {};
    for (int w = 0; w < 8; ++w)
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] += s_o[w][lane * N + i];
    const float inv = inverse(l);
    __nv_bfloat16* out = a.out + out_at(a, q, u.y, token, head) + lane * N;
#pragma unroll
    for (int i = 0; i < N; i += 2)
      *reinterpret_cast<__nv_bfloat162*>(out + i) = __floats2bfloat162_rn(o[i] * inv, o[i + 1] * inv);
    if (lane == 0) write_lse(a, q, u.y, token, head, m, l);
  } else {
    constexpr int N = D / 8, kAhead = 3;  // columns of a warp; parts that are on their way together
    if (!mine) return;
    float2 x[kAhead];
    float4 y[kAhead][N / 4];
    auto load = [&](int i0) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (i0 + j < parts) {
          x[j] = ml(i0 + j);
#pragma unroll
          for (int k = 0; k < N / 4; ++k) y[j][k] = __ldcg(part_at<D>(a, slot(i0 + j), row, warp * N + 4 * k));
        }
    };
    load(0);
    float m = -INFINITY, l = 0.0f, o[N] = {};
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (j < parts) m = fmaxf(m, x[j].x);
    for (int i = kAhead; i < parts; ++i) m = fmaxf(m, ml(i).x);
    const float base = m == -INFINITY ? 0.0f : m;
    for (int i0 = 0; i0 < parts; i0 += kAhead) {
      if (i0) load(i0);
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (i0 + j < parts) {
          const float f = exp2_approx(x[j].x - base);
          l = join(l, f, x[j].y);
#pragma unroll
          for (int k = 0; k < N / 4; ++k) {
            o[4 * k] = join(o[4 * k], f, y[j][k].x);
            o[4 * k + 1] = join(o[4 * k + 1], f, y[j][k].y);
            o[4 * k + 2] = join(o[4 * k + 2], f, y[j][k].z);
            o[4 * k + 3] = join(o[4 * k + 3], f, y[j][k].w);
          }
        }
    }
    const float inv = inverse(l);
    __nv_bfloat162* out = reinterpret_cast<__nv_bfloat162*>(a.out + out_at(a, q, u.y, token, head) + warp * N);
#pragma unroll
    for (int k = 0; k < N / 2; ++k) out[k] = __floats2bfloat162_rn(o[2 * k] * inv, o[2 * k + 1] * inv);
    if (warp == 0) write_lse(a, q, u.y, token, head, m, l);
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
  const dim3 grid(a.grid, one ? used : (used + 31) / 32);
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
// token_kernel's, one of more chunk_kernel's, whose tiles have 128 rows whether
// they are used or not.  (token_kernel / chunk_kernel: 64 bf16 sequences of
// 301-8000 tokens, 4 rows each, 101.9 / 118 us; eight of e4m3 with 8 rows, 30 / 54;
// twenty with 16 rows, 29 / 35.)  A batch that may hold both gets both, side by
// side (a chunk of 1000 tokens and 32 decoding sequences, e4m3: 74.5 us, in
// chunk_kernel alone 93); there token_kernel takes up to 8 rows, its faster
// form, unless a single token has more.
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

// The workspace: [counter][arrived][desc][token_kernel's part_ml, part_o][chunk_kernel's],
// each 256-byte aligned, the counters in one place for every shape.  The kernels
// have partial sums of their own: they run side by side.  (Its size goes by
// max_q_len and the heads alone, not by the sequences of one step.)
struct Workspace {
  uint64_t arrived, desc, ml[2], o[2], bytes;
};
Workspace layout(const ft_kv_pages& p, int grid, const Split& sp) {
  auto up = [](uint64_t x) { return (x + 255) & ~255ull; };
  Workspace w;
  w.arrived = up(kMostCtas * sizeof(unsigned));
  w.desc = up(w.arrived + 8 * kMostCtas * sizeof(unsigned));
  static_assert(9 * kMostCtas * sizeof(unsigned) + 2 * 256 <= FT_KV_WORKSPACE_ZERO, "the counters are zeroed");
  w.bytes = up(w.desc + 8 * grid * sizeof(int4));
  for (int k = 0; k < 2; ++k) {
    const uint64_t parts = k == 0 || sp.chunk ? 2ull * grid * (k ? kChunkRows : kTokenRows) : 0;
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

// What the kernels do not take.
ft_status check_sizes(const ft_kv_batch* batch, int G) {
  if ((long long)batch->max_q_len * G > 0x7fffffffLL / 2)
    return set_error(FT_ERR_UNSUPPORTED, "max_q_len * (num_q_heads / num_kv_heads) is too large");
  if (G > kSubRows) return set_error(FT_ERR_UNSUPPORTED, "num_q_heads / num_kv_heads = %d is above %d", G, kSubRows);
  return FT_OK;
}

}  // namespace

extern "C" uint64_t ft_kv_attend_workspace(const ft_kv_pages* pages, const ft_kv_batch* batch, int32_t num_q_heads) {
  if (check_attend(pages, batch, num_q_heads) != FT_OK) return 0;
  const int G = num_q_heads / pages->num_kv_heads;
  if (check_sizes(batch, G) != FT_OK) return 0;
  const Split sp = split(*batch, G);
  return layout(*pages, std::min(sm_count(), kMostCtas), sp).bytes;
}

extern "C" uint64_t ft_stream_capture(void* stream) {
  cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
  unsigned long long id = 0;
  if (cudaStreamGetCaptureInfo(static_cast<cudaStream_t>(stream), &st, &id) != cudaSuccess) {
    cudaGetLastError();  // (the legacy stream beside another's capture, or no device: not capturing)
    return 0;
  }
  return st == cudaStreamCaptureStatusNone ? 0 : id;
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
  if (batch->num_tokens == 1) q_token_stride = out_token_stride = pages->head_dim;  // of single entries: not used
  if (num_q_heads == 1) q_head_stride = out_head_stride = pages->head_dim;
  if ((st = check_rows("q", q, q_token_stride, q_head_stride)) != FT_OK) return st;
  if ((st = check_rows("out", out, out_token_stride, out_head_stride)) != FT_OK) return st;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return set_error(FT_ERR_INVALID_ARG, "workspace is null or not 256-byte aligned");
  const int G = num_q_heads / pages->num_kv_heads;
  if ((st = check_sizes(batch, G)) != FT_OK) return st;
  const long long rows = (long long)batch->max_q_len * G;  // of a (sequence, key head), at most
  if (q_token_stride <= 0 || q_head_stride <= 0 || out_token_stride <= 0 || out_head_stride <= 0)
    return set_error(FT_ERR_INVALID_ARG, "q's and out's strides must be positive");
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
  a.arrived = reinterpret_cast<unsigned*>(w + ws.arrived);
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
