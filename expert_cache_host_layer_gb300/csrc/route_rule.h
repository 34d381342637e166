// A token's experts and gates by a routing rule (ft_router), one warp to a
// token: what ft_route's kernel and route_classify's first phase share.
// Internal to libft.
//
//   s = softmax(l) or 1 / (1 + e^-l),  v = s + bias for the choice
//   groups: by their best v, or the sum of their best two; the top_groups best take part
//   the k best v, ties to the lowest expert;  w = s, renormalised over the picks or not, times scale
//
// The choice is that of exact arithmetic.  Without a bias v orders as the logit
// does, and logits are compared as they are.  With one, fp32 values of v are
// good to `err`: whatever lies within 2 err of another candidate (or, for sums
// of a group, of the border between taking part and not) is compared again in
// fp64, for which few rows in a thousand have cause.
//
// What bounds it: a row's E logits are read once, but k selections over them
// are instructions (issue slots on a chunk, their latency for one token).  So
// the warp does not select k times over E: its lanes' k-th largest maximum,
// from k warp-wide integer maxima (redux) over one value a lane, bounds the
// k-th largest value from below; the few values above that bound (9 of 256 for
// k = 8) go to a list in shared memory, and each finds its rank by comparing
// itself with the others.
#pragma once

#include <cfloat>

#include <cuda_bf16.h>

#include "ft_internal.h"

namespace ft {
namespace rule {

constexpr int kMostGroups = 32;

// Lanes of a group: the largest power of two that fits 32 / groups; expert i of
// a group is the lane's value q with i = (q / V) * lanes * V + sub * V + q % V,
// V = min(4, PL) (vector loads).
__host__ __device__ __forceinline__ int group_lanes(int groups) {
  int n = 32;
  while (n * groups > 32) n >>= 1;
  return n;
}
// Values a lane needs room for (1, 2, 4, .. 32), or 0 if 32 are not enough.
inline int values_per_lane(int E, int groups) {
  const int size = E / groups, lanes = group_lanes(groups);
  for (int pl = 1; pl <= 32; pl *= 2) {
    const int block = lanes * (pl < 4 ? pl : 4);
    if ((size + block - 1) / block * (pl < 4 ? pl : 4) <= pl) return pl;
  }
  return 0;
}
// Shared memory of a warp: the list's (value, expert) pairs, their fp64 values where a bias is given, the picks.
__host__ __device__ __forceinline__ int warp_bytes(int E, bool scored) {
  return (E + 1) / 2 * 2 * (scored ? 16 : 8) + kMaxTopK * 4;
}

// Floats as unsigned integers of the same order; 0 is below all of them.
__device__ __forceinline__ uint32_t order(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 is +0
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
// A logit as it counts: NaN as -inf, +inf as the largest number.
__device__ __forceinline__ float clean(float l) { return l != l ? -INFINITY : fminf(l, FLT_MAX); }
__device__ __forceinline__ float logit(const float* row, int e) { return clean(row[e]); }
__device__ __forceinline__ float logit(const __nv_bfloat16* row, int e) { return clean(__bfloat162float(row[e])); }
__device__ __forceinline__ void logits4(const float* row, int e, float* l) {
  const float4 v = *reinterpret_cast<const float4*>(row + e);
  l[0] = v.x; l[1] = v.y; l[2] = v.z; l[3] = v.w;
}
__device__ __forceinline__ void logits4(const __nv_bfloat16* row, int e, float* l) {
  const uint2 v = *reinterpret_cast<const uint2*>(row + e);
  l[0] = __uint_as_float(v.x << 16); l[1] = __uint_as_float(v.x & 0xffff0000u);
  l[2] = __uint_as_float(v.y << 16); l[3] = __uint_as_float(v.y & 0xffff0000u);
}

// Scores in fp64, for the comparisons that fp32 does not decide.
struct Exact {
  int softmax;
  const float* bias;
  double top, inv;  // softmax: largest logit, 1 / sum of e^(l - top)
  __device__ double value(float l, int e) const {
    const double s = softmax ? exp((double)l - top) * inv : 1.0 / (1.0 + exp(-(double)l));
    if (!bias) return s;
    const double v = s + (double)__ldg(&bias[e]);
    return v != v ? -INFINITY : fmin(v, (double)FLT_MAX);
  }
};
template <typename T>
__device__ __noinline__ Exact make_exact(const Rule r, const T* row, float top) {
  Exact x{r.softmax, r.bias, (double)top, 1.0};
  if (r.softmax) {
    double z = 0.0;
    for (int e = threadIdx.x & 31; e < r.E; e += 32) z += exp((double)logit(row, e) - (double)top);
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    x.inv = z > 0.0 ? 1.0 / z : 0.0;
  }
  return x;
}
// Whether the lane's group takes part, in fp64.
template <typename T>
__device__ __noinline__ bool exact_groups(const Rule r, const T* row, float top, int group, int sub) {
  const Exact x = make_exact(r, row, top);
  double a = -INFINITY, b = -INFINITY;
  if (group < r.groups)
    for (int i = sub; i < r.size; i += r.lanes) {
      const int e = group * r.size + i;
      const double v = x.value(logit(row, e), e);
      b = fmax(b, fmin(a, v));
      a = fmax(a, v);
    }
  for (int o = r.lanes / 2; o > 0; o >>= 1) {
    const double oa = __shfl_xor_sync(0xffffffffu, a, o), ob = __shfl_xor_sync(0xffffffffu, b, o);
    b = fmax(fmin(a, oa), fmax(b, ob));
    a = fmax(a, oa);
  }
  const double mine = r.group_top == 2 ? a + b : a;
  int above = 0;
  for (int g = 0; g < r.groups; ++g) {
    const double of = __shfl_sync(0xffffffffu, mine, g * r.lanes);
    above += of > mine || (of == mine && g < group);
  }
  return above < r.top_groups;
}
// The list's ranks in fp64; picks: the k best.
template <typename T>
__device__ __noinline__ void exact_ranks(const Rule r, const T* row, float top, const int2* list, double* keys, int n, int* picks) {
  const Exact x = make_exact(r, row, top);
  const int lane = threadIdx.x & 31;
  for (int i = lane; i < n; i += 32) keys[i] = x.value(logit(row, list[i].y), list[i].y);
  __syncwarp();
  for (int i = lane; i < n; i += 32) {
    const double v = keys[i];
    const int e = list[i].y;
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += keys[j] > v || (keys[j] == v && list[j].y < e);
    if (rank < r.k) picks[rank] = e;
  }
}

// The row's picks in order: expert and gate of pick j to lane j < k.  `shared`:
// warp_bytes of the warp's own, 16-byte aligned.
template <int PL, typename T>
__device__ __forceinline__ void route_row(const Rule& r, const T* row, unsigned char* shared, int* expert, float* gate) {
  constexpr int V = PL < 4 ? PL : 4;
  const int lane = threadIdx.x & 31, group = lane / r.lanes, sub = lane & (r.lanes - 1);
  const bool scored = r.bias != nullptr;
  int2* list = reinterpret_cast<int2*>(shared);
  double* keys = reinterpret_cast<double*>(shared + (r.E + 1) / 2 * 16);
  int* picks = reinterpret_cast<int*>(shared + (r.E + 1) / 2 * 2 * (scored ? 16 : 8));
  auto in_group = [&](int q) { return (q / V) * r.lanes * V + sub * V + q % V; };

  float v[PL];
  bool ok[PL];
#pragma unroll
  for (int q = 0; q < PL; ++q) ok[q] = group < r.groups && in_group(q) < r.size;
  if (V == 4 && r.vectors) {
#pragma unroll
    for (int q = 0; q < PL; q += 4)
      if (ok[q]) logits4(row, group * r.size + in_group(q), &v[q]);
  } else {
#pragma unroll
    for (int q = 0; q < PL; ++q)
      if (ok[q]) v[q] = logit(row, group * r.size + in_group(q));
  }
#pragma unroll
  for (int q = 0; q < PL; ++q) v[q] = ok[q] ? clean(v[q]) : -INFINITY;

  // scores: `largest` of the row's, for the error bound
  float top = 0.0f, inv_z = 1.0f, largest = 1.0f;
  if (r.softmax) {
    float m = v[0];
#pragma unroll
    for (int q = 1; q < PL; ++q) m = fmaxf(m, v[q]);
    top = fmaxf(value(__reduce_max_sync(0xffffffffu, order(m))), -FLT_MAX);
    if (scored || !r.renormalise) {
      float z = 0.0f;
#pragma unroll
      for (int q = 0; q < PL; ++q) z += expf(v[q] - top);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
      inv_z = z > 0.0f ? 1.0f / z : 0.0f;
      largest = inv_z;
    }
  }
  auto score = [&](float l) { return r.softmax ? __expf(l - top) * inv_z : __fdividef(1.0f, 1.0f + __expf(-l)); };
  if (scored) {
#pragma unroll
    for (int q = 0; q < PL; ++q) {
      if (!ok[q]) continue;
      const float c = score(v[q]) + __ldg(&r.bias[group * r.size + in_group(q)]);
      v[q] = clean(c);
    }
  }
  // fp32's error of a score (__expf: 2 ulp and its argument's rounding, sums and quotient the rest), and of the sum with the bias
  const float err_score = r.softmax ? largest * 0x1p-18f : 0x1p-20f;

  bool part = group < r.groups;
  if (r.groups > 1 && r.top_groups < r.groups) {
    float a = -INFINITY, b = -INFINITY;
#pragma unroll
    for (int q = 0; q < PL; ++q) {
      b = fmaxf(b, fminf(a, v[q]));
      a = fmaxf(a, v[q]);
    }
    for (int o = r.lanes / 2; o > 0; o >>= 1) {
      const float oa = __shfl_xor_sync(0xffffffffu, a, o), ob = __shfl_xor_sync(0xffffffffu, b, o);
      b = fmaxf(fminf(a, oa), fmaxf(b, ob));
      a = fmaxf(a, oa);
    }
    float mine = a;
    if (r.group_top == 2) mine = scored ? a + b : score(a) + score(b);
    int above = 0;
    for (int g = 0; g < r.groups; ++g) {
      const float of = __shfl_sync(0xffffffffu, mine, g * r.lanes);
      above += of > mine || (of == mine && g < group);
    }
    const bool in = part && above < r.top_groups;
    const bool mine_is_a_sum = r.group_top == 2;
    if (scored || mine_is_a_sum) {  // the border between the groups that take part and the others
      const float worst = value(~__reduce_max_sync(0xffffffffu, in ? ~order(mine) : 0u));
      const float best = value(__reduce_max_sync(0xffffffffu, part && !in ? order(mine) : 0u));
      const float size = part ? (scored ? fabsf(a) : 1.0f) + (scored && mine_is_a_sum ? fabsf(b) : 1.0f) : 0.0f;
      const float err = 2.0f * err_score + 0x1p-22f * value(__reduce_max_sync(0xffffffffu, order(size)));
      if (worst - best > 2.0f * err) {
        part = in;
      } else {
        const bool in_exactly = exact_groups(r, row, top, group, sub);
        part = part && in_exactly;
      }
    } else {
      part = in;
    }
  }

  // a bound below the k-th largest value: the k-th largest of the lanes' maxima
  uint32_t u[PL], most = 0;
#pragma unroll
  for (int q = 0; q < PL; ++q) {
    u[q] = part && ok[q] ? order(v[q]) : 0u;
    most = max(most, u[q]);
  }
  uint32_t cut = 0, first = 0;
  for (int j = 0; j < r.k; ++j) {
    cut = __reduce_max_sync(0xffffffffu, most);
    if (j == 0) first = cut;
    if (most == cut) most = 0;
  }
  float near = -1.0f;  // values so close to each other are not told apart
  if (cut == 0) {      // fewer lanes than picks have any
    cut = 1;
    uint32_t size = 0;
#pragma unroll
    for (int q = 0; q < PL; ++q) size = max(size, u[q] ? __float_as_uint(value(u[q])) & 0x7fffffffu : 0u);
    if (scored) near = 2.0f * err_score + 0x1p-21f * __uint_as_float(__reduce_max_sync(0xffffffffu, size));
  } else if (scored) {
    near = 2.0f * err_score + 0x1p-21f * fmaxf(fabsf(value(first)), fabsf(value(cut)));
    cut = order(value(cut) - near);
  }
  int n = 0;
#pragma unroll
  for (int q = 0; q < PL; ++q) {
    const unsigned m = __ballot_sync(0xffffffffu, u[q] >= cut);
    if (u[q] >= cut)
      list[n + __popc(m & ((1u << lane) - 1u))] = make_int2(__float_as_int(value(u[q])), group * r.size + in_group(q));
    n += __popc(m);
  }
  __syncwarp();
  bool close = false;
  for (int i = lane; i < n; i += 32) {
    const int2 own = list[i];
    const float x = __int_as_float(own.x);
    int rank = 0;
    for (int j = 0; j < n; ++j) {
      const int2 o = list[j];
      const float y = __int_as_float(o.x);
      rank += y > x || (y == x && o.y < own.y);
      close |= fabsf(y - x) <= near && o.y != own.y;
    }
    if (rank < r.k) picks[rank] = own.y;
  }
  if (__any_sync(0xffffffffu, close)) exact_ranks(r, row, top, list, keys, n, picks);
  __syncwarp();

  // gates
  const int e = lane < r.k ? picks[lane] : 0;
  const float l = lane < r.k ? logit(row, e) : -INFINITY;
  float w = 0.0f;
  if (!r.renormalise) {
    w = r.softmax ? expf(l - top) * inv_z : 1.0f / (1.0f + expf(-l));
  } else {
    // Factors that all picks share cancel, and with them what might underflow: the softmax's denominator, and e^m of
    // sigmoids whose largest is small (e^l / (1 + e^l) = e^m e^(l - m) / (1 + e^l)).
    const float m = fmaxf(value(__reduce_max_sync(0xffffffffu, order(l))), -FLT_MAX);
    if (r.softmax) w = expf(l - m);
    else w = m < 0.0f ? expf(l - m) / (1.0f + expf(l)) : 1.0f / (1.0f + expf(-l));
  }
  if (r.renormalise) {
    float sum = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    w = sum > 0.0f ? w / sum : 0.0f;
  }
  *expert = e;
  *gate = w * r.scale;
  __syncwarp();  // the next row's list
}

}  // namespace rule

// Checks of a router for E experts and top_k picks (FT_OK, or set_error's status).
ft_status check_router(const ft_router* r, int num_experts, int top_k);
// A checked router as kernels take it; bias: of the layer.
rule::Rule make_rule(const ft_router& r, int num_experts, int top_k, const float* bias, bool aligned_rows);

}  // namespace ft
