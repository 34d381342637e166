// A token's experts and gates by a routing rule (ft_router), one warp to a
// token: what ft_route's kernel and route_classify's first phase share.
// Internal to libft.
//
//   s = softmax(l) or 1 / (1 + e^-l),  v = s + bias for the choice
//   groups: by their best v, or the sum of their best two; the top_groups best take part
//   the k best v, ties to the lowest expert;  w = s, renormalised over the picks or not, times scale
//
// Without a bias v orders as the logit does, and logits are compared as they are.
// With one (and where a group counts by two) fp32 values of v are good to a known
// error: a pick that has another candidate within twice that (or a group that
// takes part, one that does not within its own bound) sends the row to a
// comparison in fp64, for which few rows in a thousand have cause.  There a score
// is good to 2^-45 of itself, and its sum with the bias to fp64; values that are
// the same even so are in the order of their logits, which is right where the
// biases are equal (scores next to 1, or lost beside a large bias).  Sums of two
// that are the same are groups in the order of their numbers.
//
// What bounds it: a row's E logits are read once, but k selections over them
// are a chain of dependent instructions, whose latency shows for one token and
// also on a chunk (16 warps an SM leave half of the issue slots empty).  So
// the warp does not select k times over E: its lanes' k-th largest maximum,
// from k warp-wide integer maxima (redux) over one value a lane, bounds the
// k-th largest value from below; the few values above that bound (9 of 256 for
// k = 8) go to a list in shared memory, and each finds its rank by counting the
// others above it.  Values that a lane does not have (a ragged group, or a group
// that takes no part) are NaN, which no comparison holds for.
//
// Measured, 256 experts, k = 8, sigmoid scores, a bias, 4 of 8 groups: one token 3.4
// us in a graph (5.1 with the call on the host), 16,384 tokens 15.9 us (one row a
// warp 20.7; with fp64's own exponentials for close values and IEEE quotients for
// all 31.4), of which 2 are rows that fp64 decides; plain softmax 10.1 us.
#pragma once

#include <cfloat>

#include <cuda_bf16.h>

#include "float_pair.h"
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
// Shared memory of a warp: the list's values (padded to fours with NaN) and experts, fp64 values where a bias is given, the
// picks.
__host__ __device__ __forceinline__ int list_room(int E) { return (E + 3) / 4 * 4 + 4; }
__host__ __device__ __forceinline__ int warp_bytes(int E, bool scored) { return list_room(E) * (scored ? 16 : 8) + kMaxTopK * 4; }

// Floats as unsigned integers of the same order; 0 is below all of them.
__device__ __forceinline__ uint32_t order(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 is +0
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ long long order(double x) {  // (signed: fp64 comparisons are slow here)
  const long long u = __double_as_longlong(x + 0.0);
  return u ^ (u >> 63 & 0x7fffffffffffffffll);
}
// A number as it counts: NaN as -inf (fmaxf gives the other operand), +inf as the largest number.
__device__ __forceinline__ float clean(float l) { return fminf(fmaxf(l, -INFINITY), FLT_MAX); }
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;
template <int PL>
__device__ __forceinline__ constexpr float softmax_error() { return PL <= 8 ? 0x1p-19f : 0x1p-18f; }  // (see route_row)
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

// Scores in fp64 for the comparisons that fp32 does not decide (by pairs of floats as far as those reach: fp64 is slow here).
struct Exact {
  int softmax;
  const float* bias;
  float top;
  FloatPair inv;  // softmax: 1 / sum of e^(l - top)
  __device__ double value(float l, int e) const {
    double s;
    if (softmax) {
      const FloatPair x = two_sum(l, -top);
      s = x.h >= -60.0f ? wide(exp_pair(x) * inv) : exp((double)l - (double)top) * wide(inv);
    } else {
      s = fabsf(l) <= 60.0f ? wide(sigmoid_pair(l)) : 1.0 / (1.0 + exp(-(double)l));
    }
    if (!bias) return s;
    const double v = __dadd_rn(s, (double)__ldg(&bias[e]));  // (not contracted: the same number wherever it is formed)
    return v != v ? -INFINITY : fmin(v, (double)FLT_MAX);
  }
};
template <typename T>
__device__ __noinline__ Exact make_exact(const Rule r, const T* row, float top) {
  Exact x{r.softmax, r.bias, top, {1.0f, 0.0f}};
  if (r.softmax) {
    FloatPair z{0.0f, 0.0f};
    for (int e = threadIdx.x & 31; e < r.E; e += 32) {
      const FloatPair d = two_sum(logit(row, e), -top);
      if (d.h >= -60.0f) z = z + exp_pair(d);  // (what is left out is below 2^-76 of the sum)
    }
    for (int o = 16; o > 0; o >>= 1) z = z + FloatPair{__shfl_xor_sync(0xffffffffu, z.h, o), __shfl_xor_sync(0xffffffffu, z.l, o)};
    x.inv = z.h > 0.0f ? inverse(z) : FloatPair{0.0f, 0.0f};
  }
  return x;
}
// Whether the lane's group takes part, in fp64 (of logits where those decide: without a bias, by a group's best).  least: a
// bound below the fp32 values that may count, as the caller has them.
template <typename T>
__device__ __noinline__ bool exact_groups(const Rule r, const T* row, float top, float inv_z, int group, int sub, float least) {
  const Exact x = make_exact(r, row, top);
  const bool logits = !r.bias && r.group_top == 1;
  double a = -INFINITY, b = -INFINITY;
  int i = group < r.groups ? sub : r.size;
  for (;;) {
    float l = 0.0f;
    for (; i < r.size; i += r.lanes) {  // the lane's next value that may count
      l = logit(row, group * r.size + i);
      const float s = logits ? l : r.softmax ? exp2_approx((l - top) * kLog2e) * inv_z : rcp_approx(1.0f + exp2_approx(-l * kLog2e));
      if ((r.bias ? s + clean(__ldg(&r.bias[group * r.size + i])) : s) >= least) break;
    }
    if (!__any_sync(0xffffffffu, i < r.size)) break;
    if (i < r.size) {
      const double v = logits ? (double)l : x.value(l, group * r.size + i);
      b = fmax(b, fmin(a, v));
      a = fmax(a, v);
      i += r.lanes;
    }
  }
  for (int o = r.lanes / 2; o > 0; o >>= 1) {
    const double oa = __shfl_xor_sync(0xffffffffu, a, o), ob = __shfl_xor_sync(0xffffffffu, b, o);
    b = fmax(fmin(a, oa), fmax(b, ob));
    a = fmax(a, oa);
  }
  const long long mine = order(r.group_top == 2 ? a + b : a);
  int above = 0, same = 0;  // same: of the groups before this one
  for (int g = 0; g < r.groups; ++g) {
    const long long of = __shfl_sync(0xffffffffu, mine, g * r.lanes);
    above += of > mine;
    same += of == mine && g < group;
  }
  if (!logits && r.group_top == 1 && __any_sync(0xffffffffu, same && a > -INFINITY)) {  // by their best's logit, largest first
    float by = -INFINITY;
    for (int i = group < r.groups ? sub : r.size; i < r.size; i += r.lanes) {
      const float l = logit(row, group * r.size + i);
      if (l > by && x.value(l, group * r.size + i) == a) by = l;
    }
    for (int o = r.lanes / 2; o > 0; o >>= 1) by = fmaxf(by, __shfl_xor_sync(0xffffffffu, by, o));
    if (a == -INFINITY) by = 0.0f;  // (nothing to go by)
    same = 0;
    for (int g = 0; g < r.groups; ++g) {
      const long long of = __shfl_sync(0xffffffffu, mine, g * r.lanes);
      const float key = __shfl_sync(0xffffffffu, by, g * r.lanes);
      same += of == mine && (key > by || (key == by && g < group));
    }
  }
  above += same;
  return group < r.groups && above < r.top_groups;
}
// The list's ranks in fp64; keys: room for n of them.
template <typename T, typename I>
__device__ __noinline__ void exact_ranks(const Rule r, const T* row, float top, const I* experts, long long* keys, int n, int* picks) {
  const int lane = threadIdx.x & 31;
  const Exact x = make_exact(r, row, top);
  for (int i = lane; i < n; i += 32) keys[i] = order(x.value(logit(row, experts[i]), experts[i]));
  __syncwarp();
  for (int i = lane; i < n; i += 32) {
    const long long v = keys[i];
    const int e = experts[i];
    int rank = 0, same = 0;
    for (int j = 0; j < n; ++j) {
      rank += keys[j] > v;
      same += keys[j] == v;
    }
    if (same > 1 && rank < r.k) {  // others than itself: by their logits, largest first (without a value by their numbers)
      const bool none = v == order(-(double)INFINITY);
      const float l = logit(row, e);
      for (int j = 0; j < n; ++j) {
        if (keys[j] != v) continue;
        const float of = none ? l : logit(row, experts[j]);
        rank += of > l || (of == l && experts[j] < e);
      }
    }
    if (rank < r.k) picks[rank] = e;
  }
  __syncwarp();
}
// bf16 logits, many of which are equal, as keys that order like (value, lower expert first): their 16 bits in order (one more
// than that takes negative ones, whose low bits are ones, and FLT_MAX, which stands for infinity, to whole steps).
__device__ __forceinline__ uint32_t rank_key(float l, int e) { return ((order(l) + 1u) & 0xffff0000u) | (0xffffu - (uint32_t)e); }
__device__ __forceinline__ int count_above(uint32_t x, const float* keys, int n) {
  int above = 0;
#pragma unroll 1
  for (int j = 0; j < n; j += 4) {
    const uint4 y = *reinterpret_cast<const uint4*>(keys + j);
    above += (y.x > x) + (y.y > x) + (y.z > x) + (y.w > x);
  }
  return above;
}
// The rank of (x, e) among a list's values, equal ones by expert.
template <typename I>
__device__ __forceinline__ int rank_of(float x, int e, const float* values, const I* experts, int n) {
  int rank = 0;
#pragma unroll 1
  for (int j = 0; j < n; ++j) rank += values[j] > x || (values[j] == x && experts[j] < e);
  return rank;
}

// What a lane keeps for every row: its experts' bias (0 without one; NaN: it has no such expert), and where they are.
template <int PL>
struct Lane {
  static constexpr int V = PL < 4 ? PL : 4;
  float add[PL];
  uint32_t own;            // bit q: it has value q (known before the bias is: the row's loads need not wait for that)
  int group, sub, expert;  // expert: of value 0
  __device__ __forceinline__ explicit Lane(const Rule& r) {
    const int lane = threadIdx.x & 31;
    group = lane / r.lanes;
    sub = lane & (r.lanes - 1);
    expert = group * r.size + sub * V;
    own = 0;
#pragma unroll
    for (int q = 0; q < PL; ++q)
      if (group < r.groups && sub * V + step(r, q) < r.size) own |= 1u << q;
#pragma unroll
    for (int q = 0; q < PL; ++q) add[q] = !has(q) ? NAN : r.bias ? clean(__ldg(&r.bias[expert + step(r, q)])) : 0.0f;
  }
  static __device__ __forceinline__ int step(const Rule& r, int q) { return (q / V) * r.lanes * V + q % V; }
  __device__ __forceinline__ bool has(int q) const { return own >> q & 1u; }
};

// The row's picks in order: expert and gate of pick j to lane j < k.  `shared`:
// warp_bytes of the warp's own, 16-byte aligned.
template <int PL, typename T>
__device__ __forceinline__ void route_row(const Rule& r, const Lane<PL>& own, const T* row, unsigned char* shared, int* expert,
                                          float* gate) {
  constexpr int V = Lane<PL>::V;
  const int lane = threadIdx.x & 31, room = list_room(r.E);
  const bool scored = r.bias != nullptr, by_key = sizeof(T) == 2 && !scored;
  float* values = reinterpret_cast<float*>(shared);
  int* experts = reinterpret_cast<int*>(values + room);
  long long* keys = reinterpret_cast<long long*>(experts + room);
  int* picks = scored ? reinterpret_cast<int*>(keys + room) : experts + room;

  float v[PL];
#pragma unroll
  for (int q = 0; q < PL; ++q) v[q] = NAN;
  if (V == 4 && r.vectors) {
#pragma unroll
    for (int q = 0; q < PL; q += 4)
      if (own.has(q)) logits4(row, own.expert + own.step(r, q), &v[q]);
  } else {
#pragma unroll
    for (int q = 0; q < PL; ++q)
      if (own.has(q)) v[q] = logit(row, own.expert + own.step(r, q));
  }
#pragma unroll
  for (int q = 0; q < PL; ++q) v[q] = clean(v[q]);  // (-inf where there is none, for now)

  float top = 0.0f, inv_z = 1.0f, largest = 1.0f;  // largest: of the row's scores, for the error bound
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
  // With u = 2^-24: exp2 (4 u) of a rounded argument (1.5 u |l|, at most 0.23 of it left in s (1 - s)), 1 + e (u) and rcp
  // (2 u) come to less than 2^-21.5 of a sigmoid.  Of a softmax's largest score: 5 u for the same, 4 u for expf, ln E u for
  // its arguments and PL + 5 u for the sum in the denominator, 2 u for its inverse: 30 u for 8 values a lane, 55 u for 32.
  auto score = [&](float l) {
    return r.softmax ? exp2_approx((l - top) * kLog2e) * inv_z : rcp_approx(1.0f + exp2_approx(-l * kLog2e));
  };
  const float err_score = r.softmax ? largest * softmax_error<PL>() : 0x1p-21f;
  if (scored) {
    if (r.softmax) {
#pragma unroll
      for (int q = 0; q < PL; ++q) v[q] = exp2_approx((v[q] - top) * kLog2e) * inv_z;
    } else {
#pragma unroll
      for (int q = 0; q < PL; ++q) v[q] = rcp_approx(1.0f + exp2_approx(-v[q] * kLog2e));
    }
  }
#pragma unroll
  for (int q = 0; q < PL; ++q) v[q] += own.add[q];

  bool part = own.group < r.groups;
  if (r.top_groups < r.groups) {
    float a = -INFINITY, b = -INFINITY;
    if (r.group_top == 1) {
#pragma unroll
      for (int q = 0; q < PL; ++q) a = fmaxf(a, v[q]);
      for (int o = r.lanes / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    } else {
#pragma unroll
      for (int q = 0; q < PL; ++q) {
        const float c = fmaxf(v[q], -INFINITY);
        b = fmaxf(b, fminf(a, c));
        a = fmaxf(a, c);
      }
      for (int o = r.lanes / 2; o > 0; o >>= 1) {
        const float oa = __shfl_xor_sync(0xffffffffu, a, o), ob = __shfl_xor_sync(0xffffffffu, b, o);
        b = fmaxf(fminf(a, oa), fmaxf(b, ob));
        a = fmaxf(a, oa);
      }
    }
    if (r.group_top == 2 && !scored) {
      a = score(a);
      b = score(b);
    }
    const float mine = r.group_top == 1 ? a : a + b;
    // the top_groups largest (fewer rounds than groups; more groups than that if some are equal)
    uint32_t left = part ? order(mine) : 0u;
    bool in = false;
#pragma unroll 1
    for (int j = 0; j < r.top_groups; ++j) {
      const uint32_t m = __reduce_max_sync(0xffffffffu, left);
      if (left == m && m != 0u) {
        in = true;
        left = 0u;
      }
    }
    bool sure = __popc(__ballot_sync(0xffffffffu, in && own.sub == 0)) == r.top_groups;
    if (scored || r.group_top == 2) {
      const float err = r.group_top == 1 ? err_score + 0x1p-23f * fabsf(a) : 2.0f * err_score + 0x1p-22f * (fabsf(a) + fabsf(b));
      const uint32_t worst = __reduce_min_sync(0xffffffffu, in ? order(mine - err) : 0xffffffffu);
      const uint32_t best = __reduce_max_sync(0xffffffffu, part && !in ? order(mine == -INFINITY ? mine : mine + err) : 0u);
      sure = sure && worst > best;
    }
    part = in;
    if (!sure) {  // (for logits the bound is their own value)
      const float off = scored || r.group_top == 2 ? 4.0f * err_score + 0x1p-21f * (fabsf(a) + (r.group_top == 2 ? fabsf(b) : 0.0f)) : 0.0f;
      part = exact_groups(r, row, top, inv_z, own.group, own.sub, (r.group_top == 1 ? a : b) - off);
    }
  }

  // a bound below the k-th largest value: the k-th largest of the lanes' maxima
  float m = v[0];
#pragma unroll
  for (int q = 1; q < PL; ++q) m = fmaxf(m, v[q]);
  uint32_t most = part && m == m ? order(m) : 0u;
  const uint32_t first = __reduce_max_sync(0xffffffffu, most);
  uint32_t last = first;
#pragma unroll 2
  for (int j = 1; j < r.k; ++j) {
    if (most == last) most = 0u;
    last = __reduce_max_sync(0xffffffffu, most);
  }
  float cut = -INFINITY, near = 0.0f;  // near: values so close to each other are not told apart
  if (last != 0u) {
    cut = value(last);
    if (scored) {
      near = 2.0f * err_score + 0x1p-22f * fmaxf(fabsf(value(first)), fabsf(cut));
      cut -= near;
    }
  } else if (scored) {  // fewer lanes than picks have any value: all of them are candidates
    float size = 0.0f;
#pragma unroll
    for (int q = 0; q < PL; ++q) size = fmaxf(size, fabsf(v[q]));
    near = 2.0f * err_score + 0x1p-22f * value(__reduce_max_sync(0xffffffffu, order(size)));
  }
  if (!part) cut = NAN;
  int n = 0;
#pragma unroll
  for (int q = 0; q < PL; ++q) {
    const bool in = v[q] >= cut;
    const unsigned who = __ballot_sync(0xffffffffu, in);
    if (in) {
      const int at = n + __popc(who & ((1u << lane) - 1u));
      const int e = own.expert + own.step(r, q);
      values[at] = by_key ? __uint_as_float(rank_key(v[q], e)) : v[q];
      experts[at] = e;
    }
    n += __popc(who);
  }
  if (lane < 4) values[n + lane] = by_key ? 0.0f : NAN;
  __syncwarp();
  bool unsure = false;
  for (int i = lane; i < n; i += 32) {
    if (by_key) {
      const int above = count_above(__float_as_uint(values[i]), values, n);
      if (above < r.k) picks[above] = experts[i];
      continue;
    }
    const float x = values[i], lo = x - near, hi = x + near;
    int above = 0, not_below = 0;
#pragma unroll 1
    for (int j = 0; j < n; j += 4) {
      const float4 y = *reinterpret_cast<const float4*>(values + j);
      above += (y.x > hi) + (y.y > hi) + (y.z > hi) + (y.w > hi);
      not_below += (y.x >= lo) + (y.y >= lo) + (y.z >= lo) + (y.w >= lo);
    }
    if (above < r.k) {
      picks[above] = experts[i];
      unsure |= not_below - above != 1;  // another one beside itself
    }
  }
  if (__any_sync(0xffffffffu, unsure)) {
    if (scored) {
      exact_ranks(r, row, top, experts, keys, n, picks);
    } else {
      __syncwarp();  // equal logits have all been stored to one place: their own ones come after that
      for (int i = lane; i < n; i += 32) {
        const int rank = rank_of(values[i], experts[i], values, experts, n);
        if (rank < r.k) picks[rank] = experts[i];
      }
    }
  }
  __syncwarp();

  // gates
  const int e = lane < r.k ? picks[lane] : 0;
  const float l = lane < r.k ? logit(row, e) : -INFINITY;
  float w = 0.0f;
  // (__fdividef: 2 ulp, as the exponential; 0 for a denominator above 2^126.)
  if (!r.renormalise) {
    w = r.softmax ? expf(l - top) * inv_z : __fdividef(1.0f, 1.0f + expf(-l));
  } else {
    // Factors that all picks share cancel, and with them what might underflow: the softmax's denominator, and e^m of
    // sigmoids whose largest is small (e^l / (1 + e^l) = e^m e^(l - m) / (1 + e^l)).
    const float m = fmaxf(value(__reduce_max_sync(0xffffffffu, order(l))), -FLT_MAX);
    if (r.softmax) w = expf(l - m);
    else if (m < 0.0f) w = __fdividef(expf(l - m), 1.0f + expf(l));
    else w = __fdividef(1.0f, 1.0f + expf(-l));
    float sum = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    w = sum > 0.0f ? w / sum : 0.0f;
  }
  *expert = e;
  *gate = w * r.scale;
  __syncwarp();  // the next row's list
}


// ---------------------------------------------------------------- four rows to a warp

// The same for four consecutive rows at a time, for top_k and groups up to
// eight and up to eight values a lane: what a single row leaves most lanes idle
// for (the groups' order, the list's ranks, the gates) is done by eight lanes a
// row for all four, and the rest has four rows' instructions to interleave.
constexpr int kFew = 8;
template <int PL>
struct FourLists {  // room for every value: many may be equal
  float values[4][32 * PL + 4];
  long long keys[32 * PL];
  int picks[4][kFew];
  uint16_t experts[4][32 * PL];
};
template <typename X>
__device__ __forceinline__ X pick4(const X (&x)[4], int j) {
  return j == 0 ? x[0] : j == 1 ? x[1] : j == 2 ? x[2] : x[3];
}

// Rows t0 .. t0 + 3 of T, to idx and w.
template <int PL, typename T>
__device__ __forceinline__ void route_four(const Rule& r, const Lane<PL>& own, const T* logits, int64_t stride, int t0, int rows,
                                           unsigned char* shared, int32_t* idx, float* w) {
  constexpr int V = Lane<PL>::V;
  const int lane = threadIdx.x & 31, mine_of = lane >> 3, at8 = lane & 7;  // the row and place of the lane where eight lanes have a row
  const unsigned below = (1u << lane) - 1u;
  const bool scored = r.bias != nullptr, by_key = sizeof(T) == 2 && !scored;
  FourLists<PL>& list = *reinterpret_cast<FourLists<PL>*>(shared);

  float v[4][PL];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const T* row = logits + (int64_t)min(t0 + j, rows - 1) * stride;
#pragma unroll
    for (int q = 0; q < PL; ++q) v[j][q] = NAN;
    if (V == 4 && r.vectors) {
#pragma unroll
      for (int q = 0; q < PL; q += 4)
        if (own.has(q)) logits4(row, own.expert + own.step(r, q), &v[j][q]);
    } else {
#pragma unroll
      for (int q = 0; q < PL; ++q)
        if (own.has(q)) v[j][q] = logit(row, own.expert + own.step(r, q));
    }
  }
  float top[4], inv_z[4], err_score[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int q = 0; q < PL; ++q) v[j][q] = clean(v[j][q]);
    top[j] = 0.0f;
    inv_z[j] = 1.0f;
    err_score[j] = 0x1p-21f;
    if (r.softmax) {
      float m = v[j][0];
#pragma unroll
      for (int q = 1; q < PL; ++q) m = fmaxf(m, v[j][q]);
      top[j] = fmaxf(value(__reduce_max_sync(0xffffffffu, order(m))), -FLT_MAX);
      if (scored || !r.renormalise) {
        float z = 0.0f;
#pragma unroll
        for (int q = 0; q < PL; ++q) z += expf(v[j][q] - top[j]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        inv_z[j] = z > 0.0f ? 1.0f / z : 0.0f;
      }
      err_score[j] = inv_z[j] * softmax_error<PL>();
    }
  }
  auto score = [&](float l, float t, float z) {
    return r.softmax ? exp2_approx((l - t) * kLog2e) * z : rcp_approx(1.0f + exp2_approx(-l * kLog2e));
  };
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (scored) {
      if (r.softmax) {
#pragma unroll
        for (int q = 0; q < PL; ++q) v[j][q] = exp2_approx((v[j][q] - top[j]) * kLog2e) * inv_z[j];
      } else {
#pragma unroll
        for (int q = 0; q < PL; ++q) v[j][q] = rcp_approx(1.0f + exp2_approx(-v[j][q] * kLog2e));
      }
    }
#pragma unroll
    for (int q = 0; q < PL; ++q) v[j][q] += own.add[q];
  }

  unsigned parts = 0xffffffffu;  // bit 8 j + g: group g of row j takes part
  if (r.top_groups < r.groups) {
    float of[4], err[4], least[4];  // a group's score, its bound, and the least of its values in it
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a = -INFINITY, b = -INFINITY;
      if (r.group_top == 1) {
#pragma unroll
        for (int q = 0; q < PL; ++q) a = fmaxf(a, v[j][q]);
        for (int o = r.lanes / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        of[j] = least[j] = a;
        err[j] = scored ? err_score[j] + 0x1p-23f * fabsf(a) : 0.0f;
      } else {
#pragma unroll
        for (int q = 0; q < PL; ++q) {
          const float c = fmaxf(v[j][q], -INFINITY);
          b = fmaxf(b, fminf(a, c));
          a = fmaxf(a, c);
        }
        for (int o = r.lanes / 2; o > 0; o >>= 1) {
          const float oa = __shfl_xor_sync(0xffffffffu, a, o), ob = __shfl_xor_sync(0xffffffffu, b, o);
          b = fmaxf(fminf(a, oa), fmaxf(b, ob));
          a = fmaxf(a, oa);
        }
        if (!scored) {
          a = score(a, top[j], inv_z[j]);
          b = score(b, top[j], inv_z[j]);
        }
        of[j] = a + b;
        least[j] = b;
        err[j] = 2.0f * err_score[j] + 0x1p-22f * (fabsf(a) + fabsf(b));
      }
    }
    // lane 8 j + g: group g of row j
    float x = NAN, e = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float xj = __shfl_sync(0xffffffffu, of[j], (at8 * r.lanes) & 31), ej = __shfl_sync(0xffffffffu, err[j], (at8 * r.lanes) & 31);
      if (mine_of == j && at8 < r.groups) {
        x = xj;
        e = ej;
      }
    }
    int above = 0;
#pragma unroll
    for (int d = 1; d < 8; ++d) {
      const float y = __shfl_xor_sync(0xffffffffu, x, d);
      above += y > x || (y == x && (at8 ^ d) < at8);
    }
    const bool in = at8 < r.groups && above < r.top_groups;
    parts = __ballot_sync(0xffffffffu, in);
    if (scored || r.group_top == 2) {  // the border: a sum that may not be told from another's
      float worst = in ? x - e : INFINITY, best = !in && x > -INFINITY ? x + e : -INFINITY;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) {
        worst = fminf(worst, __shfl_xor_sync(0xffffffffu, worst, o));
        best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
      }
      const unsigned unsure = __ballot_sync(0xffffffffu, !(worst > best));  // (eight lanes alike)
      if (unsure) {
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
          if (!(unsure >> (8 * j) & 1u)) continue;
          const T* row = logits + (int64_t)min(t0 + j, rows - 1) * stride;
          const float t = pick4(top, j), z = pick4(inv_z, j), off = 2.0f * pick4(err, j);
          const bool mine = exact_groups(r, row, t, z, own.group, own.sub, pick4(least, j) - off);
          unsigned bits = 0;
          for (int g = 0; g < r.groups; ++g) bits |= (__ballot_sync(0xffffffffu, mine && own.group == g) != 0u) << g;
          parts = (parts & ~(0xffu << (8 * j))) | bits << (8 * j);
        }
      }
    }
  }

  // the bound, and the list of what is above it
  float cut[4], near[4];
  uint32_t most[4], first[4], last[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float m = v[j][0];
#pragma unroll
    for (int q = 1; q < PL; ++q) m = fmaxf(m, v[j][q]);
    const bool part = own.group < r.groups && (parts >> (8 * j + (own.group & 7)) & 1u);
    most[j] = part && m == m ? order(m) : 0u;
    first[j] = last[j] = __reduce_max_sync(0xffffffffu, most[j]);
    cut[j] = part ? 0.0f : NAN;
  }
#pragma unroll 1
  for (int i = 1; i < r.k; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (most[j] == last[j]) most[j] = 0u;
      last[j] = __reduce_max_sync(0xffffffffu, most[j]);
    }
  }
  int n[4];
  unsigned left[4];  // the lane's values that go to the list
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float least = -INFINITY;
    near[j] = 0.0f;
    if (last[j] != 0u) {
      least = value(last[j]);
      if (scored) {
        near[j] = 2.0f * err_score[j] + 0x1p-22f * fmaxf(fabsf(value(first[j])), fabsf(least));
        least -= near[j];
      }
    } else if (scored) {
      float size = 0.0f;
#pragma unroll
      for (int q = 0; q < PL; ++q) size = fmaxf(size, fabsf(v[j][q]));
      near[j] = 2.0f * err_score[j] + 0x1p-22f * value(__reduce_max_sync(0xffffffffu, order(size)));
    }
    cut[j] += least;  // NaN in groups that take no part
    left[j] = 0;
#pragma unroll
    for (int q = 0; q < PL; ++q)
      if (v[j][q] >= cut[j]) left[j] |= 1u << q;
    n[j] = 0;
  }
  for (;;) {  // of each row a value of each lane that has one left
    unsigned who[4], any = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) any |= who[j] = __ballot_sync(0xffffffffu, left[j] != 0u);
    if (!any) break;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (left[j]) {
        const int q = __ffs(left[j]) - 1, at = n[j] + __popc(who[j] & below);
        left[j] &= left[j] - 1;
        list.experts[j][at] = (uint16_t)(own.expert + own.step(r, q));
      }
      n[j] += __popc(who[j]);
    }
  }
  __syncwarp();

  // eight lanes a row from here
  const int t = min(t0 + mine_of, rows - 1), count = pick4(n, mine_of);
  const T* row = logits + (int64_t)t * stride;
  const float row_top = pick4(top, mine_of), row_z = pick4(inv_z, mine_of), apart = pick4(near, mine_of);
  float* values = list.values[mine_of];
  const uint16_t* experts = list.experts[mine_of];
  int* picks = list.picks[mine_of];
  auto listed = [&](float l, int e) {
    return scored ? score(l, row_top, row_z) + clean(__ldg(&r.bias[e])) : by_key ? __uint_as_float(rank_key(l, e)) : l;
  };
  for (int i = at8; i < count; i += 16) {  // two of a lane's at a time
    const int e = experts[i], f = experts[min(i + 8, count - 1)];
    const float l = logit(row, e), m = logit(row, f);
    values[i] = listed(l, e);
    if (i + 8 < count) values[i + 8] = listed(m, f);
  }
  if (at8 < 4) values[count + at8] = by_key ? 0.0f : NAN;
  __syncwarp();
  bool unsure = false;
  for (int i = at8; i < count; i += 16) {
    const float x[2] = {values[i], values[min(i + 8, count - 1)]};
    int above[2] = {0, 0};
    if (by_key) {
      const uint32_t a = __float_as_uint(x[0]), b = __float_as_uint(x[1]);
#pragma unroll 1
      for (int c = 0; c < count; c += 4) {
        const uint4 y = *reinterpret_cast<const uint4*>(values + c);
        above[0] += (y.x > a) + (y.y > a) + (y.z > a) + (y.w > a);
        above[1] += (y.x > b) + (y.y > b) + (y.z > b) + (y.w > b);
      }
    } else {
      const float lo[2] = {x[0] - apart, x[1] - apart}, hi[2] = {x[0] + apart, x[1] + apart};
      int not_below[2] = {0, 0};
#pragma unroll 1
      for (int c = 0; c < count; c += 4) {
        const float4 y = *reinterpret_cast<const float4*>(values + c);
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          above[d] += (y.x > hi[d]) + (y.y > hi[d]) + (y.z > hi[d]) + (y.w > hi[d]);
          not_below[d] += (y.x >= lo[d]) + (y.y >= lo[d]) + (y.z >= lo[d]) + (y.w >= lo[d]);
        }
      }
#pragma unroll
      for (int d = 0; d < 2; ++d)
        if (i + 8 * d < count && above[d] < r.k && not_below[d] - above[d] != 1) {  // another one beside itself
          if (scored) unsure = true;
          else above[d] = rank_of(x[d], experts[i + 8 * d], values, experts, count);  // equal logits
        }
    }
#pragma unroll
    for (int d = 0; d < 2; ++d)
      if (i + 8 * d < count && above[d] < r.k) picks[above[d]] = experts[i + 8 * d];
  }
  const unsigned undecided = __ballot_sync(0xffffffffu, unsure);
  if (undecided) {
#pragma unroll 1
    for (int j = 0; j < 4; ++j)
      if (undecided >> (8 * j) & 0xffu)
        exact_ranks(r, logits + (int64_t)min(t0 + j, rows - 1) * stride, pick4(top, j), list.experts[j], list.keys,
                    pick4(n, j), list.picks[j]);
  }
  __syncwarp();
  const int e = at8 < r.k ? picks[at8] : 0;
  const float l = at8 < r.k ? logit(row, e) : -INFINITY;
  float g = 0.0f;
  if (!r.renormalise) {
    g = r.softmax ? expf(l - row_top) * row_z : __fdividef(1.0f, 1.0f + expf(-l));
  } else {  // (as in route_row)
    float m = l;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    m = fmaxf(m, -FLT_MAX);
    if (r.softmax) g = expf(l - m);
    else g = m < 0.0f ? __fdividef(expf(l - m), 1.0f + expf(l)) : __fdividef(1.0f, 1.0f + expf(-l));
    float sum = g;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    g = sum > 0.0f ? g / sum : 0.0f;
  }
  if (at8 < r.k && t0 + mine_of < rows) {
    idx[(int64_t)t * r.k + at8] = e;
    w[(int64_t)t * r.k + at8] = g * r.scale;
  }
  __syncwarp();  // the next rows' lists
}

}  // namespace rule

// Checks of a router for E experts and top_k picks (FT_OK, or set_error's status).
ft_status check_router(const ft_router* r, int num_experts, int top_k);
// A checked router as kernels take it; bias: of the layer.
rule::Rule make_rule(const ft_router& r, int num_experts, int top_k, const float* bias, bool aligned_rows);

}  // namespace ft
