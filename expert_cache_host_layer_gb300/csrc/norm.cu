// The residual's addition and the root-mean-square norm of the sum
// (ft_add_norm), in bf16, fp32, or e4m3 with fp32 scales.
//
//   r = x + delta,  total = r rounded to x's type,  y = r w / sqrt(mean r^2 + eps)
//   e4m3: s_g = max |y| / 448 over group g of channels,  codes = y / s_g
//
// Every value is read and written once, so HBM bounds the large calls and the
// chain load -> reduction -> store the small ones.  A row's values stay in the
// registers of its threads between the two halves: r is formed in fp32 and the
// norm takes it unrounded (the stored total is its one rounding).  The
// quotient y / s_g does not need the row's norm: r w times 448 / max |r w| is
// the same number with fewer roundings, and the row's mean square and the
// largest |r w| come out of one reduction.
//
// Measured: 16,384 rows of 2048, bf16 plus fp32 to bf16, 48.7 us, 6.9 TB/s (a copy
// runs at 6.8); 4099 x 1800, fp32 plus bf16 to e4m3 by groups of 128, 14.9 us, 5.5
// TB/s, of which 2 are a launch's; one row 1.6 us in a graph, 4.7 with the call on
// the host.  Rows below 256 channels leave lanes without a vector, and the loads
// few: 327,680 rows of 128, bf16, 84 us, 2.0 TB/s, of 256 43, 3.9.
#include "kv_common.h"
#include "decode_common.h"

namespace ft {
namespace {

constexpr int kMostThreads = 512;  // of a row: 128 registers a thread
constexpr int kMostHidden = kMostThreads * 4 * 8;
constexpr float kLeastMean = 0x1p-126f;  // the least mean r^2 + eps: its inverse root is a finite number, and zeros times that are zeros
constexpr float kLeast = 0x1p-100f;  // the least max |r w| that a scale is made of: 448 / it is a finite number

struct NormArgs {
  const void* x;
  const void* delta;
  const void* w;
  void* total;
  void* out;
  float* scales;
  int64_t xs, ds, ts, os, rows;  // strides in elements
  int hidden, w_dtype, out_dtype, group, groups;
  float eps;
};

// Eight consecutive values: one 16-byte load of bf16, two of fp32.
template <int T> struct Raw { uint4 v[T == FT_F32 ? 2 : 1]; };
template <int T>
__device__ __forceinline__ void fetch(Raw<T>& r, const void* base, int64_t at) {  // at: of the first, a multiple of 8
  const uint4* p = static_cast<const uint4*>(base) + (T == FT_F32 ? at / 4 : at / 8);
  r.v[0] = p[0];
  if (T == FT_F32) r.v[T == FT_F32 ? 1 : 0] = p[1];
}
template <int T>
__device__ __forceinline__ void values(const Raw<T>& r, float* v) {
  if (T == FT_F32) {
    dec::decode_chunk<FT_W_F32>(r.v[0], v);
    dec::decode_chunk<FT_W_F32>(r.v[T == FT_F32 ? 1 : 0], v + 4);
  } else {
    dec::decode_chunk<FT_W_BF16>(r.v[0], v);
  }
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ void put_f32(void* base, int64_t at, const float* v) {
  float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
  p[0] = make_float4(v[0], v[1], v[2], v[3]);
  p[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void put_bf16(void* base, int64_t at, const float* v) {
  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + at) =
      make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
// max(a, |b|), NaN if either is.
__device__ __forceinline__ float max_abs(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(fabsf(b)));
  return m;
}
// 448 / m for m in [2^-100, 2^128), rounded but for an ulp at times: a quotient and its remainder, 2^-16 aside from both
// so that the reciprocal is a normal number.  (An IEEE division here costs as much as the rest of a group's work.)
__device__ __forceinline__ float over(float m) {
  const float d = m * 0x1p-16f;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  const float q = 448.0f * 0x1p-16f * r;
  return fmaf(fmaf(-d, q, 448.0f * 0x1p-16f), r, q);
}

// A row to a group of `per_row` threads (a power of two, 32 or more), thread t
// of which holds vectors t, t + per_row, .. of eight values, kVecs of them.
template <int X, int D, int kVecs>  // types of x and delta (-1: none)
__global__ void __launch_bounds__(kMostThreads) norm_kernel(const __grid_constant__ NormArgs a, int per_row) {
  __shared__ float s_sum[kMostThreads / 32];
  __shared__ float s_top[kMostThreads / 32];
  const int t = threadIdx.x & (per_row - 1), in_block = threadIdx.x / per_row;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / per_row) + in_block;
  const bool by_row = a.out_dtype == FT_FP8E4M3 && a.group == 0;
  bool ok[kVecs];
#pragma unroll
  for (int j = 0; j < kVecs; ++j) ok[j] = row < a.rows && (j * per_row + t) * 8 < a.hidden;
  dec::pdl_wait_primary();
  Raw<X> x[kVecs];
  Raw<D < 0 ? FT_BF16 : D> d[kVecs];
  Raw<FT_F32> w[kVecs];
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int i = (j * per_row + t) * 8;
    if (!ok[j]) continue;
    fetch<X>(x[j], a.x, row * a.xs + i);
    if (D >= 0) fetch<D < 0 ? FT_BF16 : D>(d[j], a.delta, row * a.ds + i);
  }
  const bool w32 = a.w_dtype == FT_F32;
  if (a.w && w32) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const uint4* p = static_cast<const uint4*>(a.w) + (j * per_row + t) * 2;
      if (ok[j]) {
        w[j].v[0] = __ldg(p);
        w[j].v[1] = __ldg(p + 1);
      }
    }
  } else if (a.w) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
      if (ok[j]) w[j].v[0] = __ldg(static_cast<const uint4*>(a.w) + j * per_row + t);
  }
  float r[kVecs][8];
  float sum = 0.0f, top = 0.0f;  // top: largest |r w| of a row
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
#pragma unroll
    for (int e = 0; e < 8; ++e) r[j][e] = 0.0f;
    if (!ok[j]) continue;
    values<X>(x[j], r[j]);
    if (D >= 0) {
      float add[8];
      values<D < 0 ? FT_BF16 : D>(d[j], add);
#pragma unroll
      for (int e = 0; e < 8; ++e) r[j][e] += add[e];
      if (a.total) {
        const int64_t at = row * a.ts + (j * per_row + t) * 8;
        if (X == FT_F32) put_f32(a.total, at, r[j]);
        else put_bf16(a.total, at, r[j]);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(r[j][e], r[j][e], sum);
  }
  if (a.w && w32) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      if (!ok[j]) continue;
      float m[8];
      values<FT_F32>(w[j], m);
#pragma unroll
      for (int e = 0; e < 8; ++e) r[j][e] *= m[e];
    }
  } else if (a.w) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      if (!ok[j]) continue;
      float m[8];
      dec::decode_chunk<FT_W_BF16>(w[j].v[0], m);
#pragma unroll
      for (int e = 0; e < 8; ++e) r[j][e] *= m[e];
    }
  }
  auto warp_top = [](float m) { return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m))); };  // (NaN above infinity)
  if (by_row) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max_abs(top, r[j][e]);
    top = warp_top(top);
  }
  sum = dec::warp_sum(sum);
  if (per_row > 32) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = per_row >> 5, first = in_block * warps;
    if (lane == 0) {
      s_sum[warp] = sum;
      s_top[warp] = top;
    }
    __syncthreads();
    sum = dec::warp_sum(lane < warps ? s_sum[first + lane] : 0.0f);
    if (by_row) top = warp_top(lane < warps ? s_top[first + lane] : 0.0f);
  }
  const float norm = __frsqrt_rn(max_abs(kLeastMean, sum / (float)a.hidden + a.eps));
  if (a.out_dtype != FT_FP8E4M3) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      if (!ok[j]) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) r[j][e] *= norm;
      const int64_t at = row * a.os + (j * per_row + t) * 8;
      if (a.out_dtype == FT_F32) put_f32(a.out, at, r[j]);
      else put_bf16(a.out, at, r[j]);
    }
  } else {
    const int log_group = __ffs(a.group) - 1;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int i = (j * per_row + t) * 8;
      if (!by_row) {  // a group is 4, 8 or 16 lanes; lanes past the row hold zeros
        top = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max_abs(top, r[j][e]);
        for (int o = a.group / 16; o > 0; o >>= 1) top = max_abs(top, __shfl_xor_sync(0xffffffffu, top, o));
      }
      if (!ok[j]) continue;
      const float most = top == top ? fmaxf(top, kLeast) : top, inv = over(most);
#pragma unroll
      for (int e = 0; e < 8; ++e) r[j][e] *= inv;
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + row * a.os + i) =
          make_uint2(kv::pack_e4m3(r[j][0], r[j][1]) | kv::pack_e4m3(r[j][2], r[j][3]) << 16,
                     kv::pack_e4m3(r[j][4], r[j][5]) | kv::pack_e4m3(r[j][6], r[j][7]) << 16);
      if (by_row) {
        if (i == 0) a.scales[row] = most * norm * (1.0f / 448.0f);
      } else if ((i & (a.group - 1)) == 0) {
        a.scales[row * a.groups + (i >> log_group)] = most * norm * (1.0f / 448.0f);
      }
    }
  }
  dec::pdl_launch_dependents();
}

template <int X, int D>
cudaError_t launch(const NormArgs& a, cudaStream_t s) {
  // Few rows: as many threads to a row as it has vectors, for the shortest chain (one row of 4096 2.0 us, with two vectors a
  // thread 2.1).  Many: two vectors to a thread (4099 x 1800 14.9 us; one 15.7, four 17.7: fewer warps fit).
  const int vecs = a.hidden / 8;
  int per_row = 32;
  const bool many = a.rows >= 4 * kv::sm_count();
  while (per_row < kMostThreads && per_row * (many ? 2 : 1) < vecs) per_row *= 2;
  const int each = (vecs + per_row - 1) / per_row;
  const int threads = per_row < 128 && a.rows > 1 ? 128 : per_row;
  const int64_t blocks = (a.rows + threads / per_row - 1) / (threads / per_row);  // below 2^31, as rows are
  auto* kernel = each <= 1 ? norm_kernel<X, D, 1> : each <= 2 ? norm_kernel<X, D, 2> : norm_kernel<X, D, 4>;
  return kv::launch_dependent(kernel, dim3((unsigned)blocks), threads, 0, s, a, per_row);
}

ft_status check_matrix(const char* name, const void* p, int64_t stride, int64_t rows, int hidden) {
  if (!p) return set_error(FT_ERR_INVALID_ARG, "%s is null", name);
  if ((reinterpret_cast<uintptr_t>(p) & 15) || (stride & 7))
    return set_error(FT_ERR_INVALID_ARG, "%s must be 16-byte aligned with a row stride that is a multiple of 8 elements", name);
  if (rows > 1 && stride < hidden)
    return set_error(FT_ERR_INVALID_ARG, "%s: row stride %lld is below hidden=%d", name, (long long)stride, hidden);
  return FT_OK;
}

// An output in an input's place: every element has to be where the thread that writes it has read it.
ft_status check_place(const char* name, const void* p, int dtype, int64_t stride, const char* input, const void* q, int of_dtype,
                      int64_t of_stride) {
  if (p != q || (dtype == of_dtype && stride == of_stride)) return FT_OK;
  return set_error(FT_ERR_INVALID_ARG, "%s may be %s itself only with its type and row stride", name, input);
}

}  // namespace
}  // namespace ft

using namespace ft;

extern "C" ft_status ft_add_norm(const ft_norm* norm, const ft_norm_args* args, void* stream) {
  if (!norm || !args) return set_error(FT_ERR_INVALID_ARG, "norm or args is null");
  const ft_norm_args& g = *args;
  const int H = norm->hidden;
  if (H < 8 || H > kMostHidden || H % 8)
    return set_error(FT_ERR_UNSUPPORTED, "hidden=%d is not a multiple of 8 in 8..%d", H, kMostHidden);
  if (!(norm->eps >= 0.0f) || norm->eps > 3.0e38f) return set_error(FT_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (g.num_rows < 0 || g.num_rows > 0x7fffffffLL)
    return set_error(FT_ERR_INVALID_ARG, "num_rows=%lld outside 0..2^31-1", (long long)g.num_rows);
  if (norm->weight && norm->weight_dtype != FT_F32 && norm->weight_dtype != FT_BF16)
    return set_error(FT_ERR_INVALID_ARG, "weight_dtype=%d is not FT_F32 or FT_BF16", norm->weight_dtype);
  if (reinterpret_cast<uintptr_t>(norm->weight) & 15) return set_error(FT_ERR_INVALID_ARG, "weight is not 16-byte aligned");
  if (g.x_dtype != FT_F32 && g.x_dtype != FT_BF16)
    return set_error(FT_ERR_INVALID_ARG, "x_dtype=%d is not FT_F32 or FT_BF16", g.x_dtype);
  if (g.delta && g.delta_dtype != FT_F32 && g.delta_dtype != FT_BF16)
    return set_error(FT_ERR_INVALID_ARG, "delta_dtype=%d is not FT_F32 or FT_BF16", g.delta_dtype);
  if (g.total && !g.delta) return set_error(FT_ERR_INVALID_ARG, "total goes with delta");
  if (g.out_dtype != FT_F32 && g.out_dtype != FT_BF16 && g.out_dtype != FT_FP8E4M3)
    return set_error(FT_ERR_INVALID_ARG, "out_dtype=%d is not FT_F32, FT_BF16 or FT_FP8E4M3", g.out_dtype);
  const bool fp8 = g.out_dtype == FT_FP8E4M3;
  if (fp8 && norm->group != 0 && norm->group != 32 && norm->group != 64 && norm->group != 128)
    return set_error(FT_ERR_UNSUPPORTED, "group=%d is not 0, 32, 64 or 128", norm->group);
  if (g.num_rows == 0) return FT_OK;
  NormArgs a{};
  a.x = g.x; a.delta = g.delta; a.w = norm->weight; a.total = g.total; a.out = g.out; a.scales = g.scales;
  a.xs = g.x_stride; a.ds = g.delta_stride; a.ts = g.total_stride; a.os = g.out_stride; a.rows = g.num_rows;
  if (a.rows == 1) a.xs = a.ds = a.ts = a.os = H;  // of a single row: not used
  ft_status st = check_matrix("x", a.x, a.xs, a.rows, H);
  if (st == FT_OK && a.delta) st = check_matrix("delta", a.delta, a.ds, a.rows, H);
  if (st == FT_OK && a.total) st = check_matrix("total", a.total, a.ts, a.rows, H);
  if (st == FT_OK) st = check_matrix("out", a.out, a.os, a.rows, H);
  if (st == FT_OK && a.total) st = check_place("total", a.total, g.x_dtype, a.ts, "x", a.x, g.x_dtype, a.xs);
  if (st == FT_OK && a.total) st = check_place("total", a.total, g.x_dtype, a.ts, "delta", a.delta, g.delta_dtype, a.ds);
  if (st == FT_OK) st = check_place("out", a.out, g.out_dtype, a.os, "x", a.x, g.x_dtype, a.xs);
  if (st == FT_OK && a.delta) st = check_place("out", a.out, g.out_dtype, a.os, "delta", a.delta, g.delta_dtype, a.ds);
  if (st != FT_OK) return st;
  if (a.total == a.out) return set_error(FT_ERR_INVALID_ARG, "total and out are one matrix");
  if (fp8 && (!a.scales || (reinterpret_cast<uintptr_t>(a.scales) & 3)))
    return set_error(FT_ERR_INVALID_ARG, "an e4m3 output needs scales, 4-byte aligned");
  a.hidden = H; a.w_dtype = norm->weight_dtype; a.out_dtype = g.out_dtype; a.eps = norm->eps;
  a.group = norm->group;
  a.groups = norm->group ? (H + norm->group - 1) / norm->group : 1;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int d = a.delta ? g.delta_dtype : -1;
  const cudaError_t e = g.x_dtype == FT_F32
      ? (d < 0 ? launch<FT_F32, -1>(a, s) : d == FT_F32 ? launch<FT_F32, FT_F32>(a, s) : launch<FT_F32, FT_BF16>(a, s))
      : (d < 0 ? launch<FT_BF16, -1>(a, s) : d == FT_F32 ? launch<FT_BF16, FT_F32>(a, s) : launch<FT_BF16, FT_BF16>(a, s));
  if (e != cudaSuccess) return set_error(FT_ERR_CUDA, "add_norm launch: %s", cudaGetErrorString(e));
  return FT_OK;
}
