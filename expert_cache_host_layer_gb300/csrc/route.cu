// ft_route: experts and gates of a batch's tokens by a routing rule
// (route_rule.h has the rule and how a warp follows it).
#include <algorithm>

#include "decode_common.h"
#include "kv_common.h"
#include "route_rule.h"

namespace ft {
namespace {

constexpr int kWarps = 4;
constexpr int kMostRows = 1 << 30;
// From here on four rows go to a warp: 16,384 rows of 256 experts 15.9 us against 20.7, 8192 11.1 against 11.4 (plain softmax
// 6.2 against 8.2), 4096 10.1 against 8.5: below, every row has a warp of its own at once, and its chain is shorter.  (At the
// border itself, one row a warp against four: 256 experts 10.7 and 10.8 us, 128 6.5 and 6.2, 64 4.8 and 4.1.)
constexpr int kManyRows = 6144;

struct RouteBatch {
  rule::Rule r;
  const void* logits;
  int64_t stride;
  int T;
  int32_t* idx;
  float* w;
};

template <int PL, typename T, bool kFour>
__global__ void __launch_bounds__(kWarps * 32, kFour ? 4 : PL <= 8 ? 8 : PL == 16 ? 5 : 3) route_kernel(const __grid_constant__ RouteBatch a) {
  extern __shared__ __align__(16) unsigned char shared[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool scored = a.r.bias != nullptr;
  unsigned char* list = shared + warp * (kFour ? (int)sizeof(rule::FourLists<PL>) : rule::warp_bytes(a.r.E, scored));
  dec::pdl_wait_primary();
  const rule::Lane<PL> own(a.r);
  const T* logits = static_cast<const T*>(a.logits);
  const int t = (kFour ? 4 : 1) * (blockIdx.x * kWarps + warp);
  if (t < a.T) {
    if constexpr (kFour) {
      rule::route_four<PL>(a.r, own, logits, a.stride, t, a.T, list, a.idx, a.w);
    } else {
      int e;
      float w;
      rule::route_row<PL>(a.r, own, logits + t * a.stride, list, &e, &w);
      if (lane < a.r.k) {
        a.idx[(int64_t)t * a.r.k + lane] = e;
        a.w[(int64_t)t * a.r.k + lane] = w;
      }
    }
  }
  dec::pdl_launch_dependents();
}

template <int PL, typename T, bool kFour>
cudaError_t launch(const RouteBatch& a, cudaStream_t s) {
  const bool scored = a.r.bias != nullptr;
  const int bytes = kWarps * (kFour ? (int)sizeof(rule::FourLists<PL>) : rule::warp_bytes(a.r.E, scored));
  const cudaError_t e = kv::allow_smem<4 * PL + 2 * kFour + (sizeof(T) == 2)>(route_kernel<PL, T, kFour>,
                                                                              kWarps * rule::warp_bytes(kMaxExperts, true));
  if (e != cudaSuccess) return e;
  const int rows = kWarps * (kFour ? 4 : 1);
  const int blocks = (a.T + rows - 1) / rows;
  return kv::launch_dependent(route_kernel<PL, T, kFour>, dim3(blocks), kWarps * 32, bytes, s, a);
}
template <int PL, typename T>
cudaError_t launch(const RouteBatch& a, cudaStream_t s) {
  if constexpr (PL <= 8)
    if (a.T >= kManyRows && a.r.k <= rule::kFew && a.r.groups <= rule::kFew) return launch<PL, T, true>(a, s);
  return launch<PL, T, false>(a, s);
}
template <typename T>
cudaError_t launch(const RouteBatch& a, cudaStream_t s) {
  switch (rule::values_per_lane(a.r.E, a.r.groups)) {
    case 1: return launch<1, T>(a, s);
    case 2: return launch<2, T>(a, s);
    case 4: return launch<4, T>(a, s);
    case 8: return launch<8, T>(a, s);
    case 16: return launch<16, T>(a, s);
    default: return launch<32, T>(a, s);
  }
}

}  // namespace

ft_status check_router(const ft_router* r, int E, int k) {
  if (!r) return set_error(FT_ERR_INVALID_ARG, "router is null");
  if (E < 1 || E > kMaxExperts) return set_error(FT_ERR_INVALID_ARG, "num_experts=%d outside 1..%d", E, kMaxExperts);
  if (k < 1 || k > kMaxTopK || k > E) return set_error(FT_ERR_INVALID_ARG, "top_k=%d outside 1..min(num_experts, %d)", k, kMaxTopK);
  if (r->score != FT_SCORE_SOFTMAX && r->score != FT_SCORE_SIGMOID)
    return set_error(FT_ERR_INVALID_ARG, "score=%d is not an ft_score", r->score);
  if (r->num_groups < 1 || r->num_groups > rule::kMostGroups || E % r->num_groups)
    return set_error(FT_ERR_INVALID_ARG, "num_groups=%d is not a divisor of num_experts=%d in 1..%d", r->num_groups, E, rule::kMostGroups);
  if (r->top_groups < 1 || r->top_groups > r->num_groups)
    return set_error(FT_ERR_INVALID_ARG, "top_groups=%d outside 1..num_groups=%d", r->top_groups, r->num_groups);
  const int size = E / r->num_groups;
  if (r->group_top < 1 || r->group_top > 2 || (r->num_groups > 1 && r->group_top > size))
    return set_error(FT_ERR_INVALID_ARG, "group_top=%d is not 1 or 2 experts of a group's %d", r->group_top, size);
  if (k > r->top_groups * size)
    return set_error(FT_ERR_INVALID_ARG, "top_k=%d is beyond the %d experts of %d groups", k, r->top_groups * size, r->top_groups);
  if (rule::values_per_lane(E, r->num_groups) == 0)
    return set_error(FT_ERR_UNSUPPORTED, "num_experts=%d in %d groups: at most %d", E, r->num_groups,
                     32 * rule::group_lanes(r->num_groups) * r->num_groups);
  if (!(r->scale >= -3.0e38f && r->scale <= 3.0e38f)) return set_error(FT_ERR_INVALID_ARG, "the router's scale must be finite");
  if (reinterpret_cast<uintptr_t>(r->bias) & 3) return set_error(FT_ERR_INVALID_ARG, "bias is not 4-byte aligned");
  return FT_OK;
}

rule::Rule make_rule(const ft_router& r, int E, int k, const float* bias, bool aligned_rows) {
  rule::Rule x{};
  x.softmax = r.score == FT_SCORE_SOFTMAX;
  x.groups = r.num_groups; x.top_groups = r.top_groups; x.group_top = r.num_groups > 1 ? r.group_top : 1;
  x.renormalise = r.renormalise != 0; x.scale = r.scale; x.bias = bias;
  x.E = E; x.k = k; x.size = E / r.num_groups; x.lanes = rule::group_lanes(r.num_groups);
  x.vectors = aligned_rows && x.size % 4 == 0;
  return x;
}

}  // namespace ft

using namespace ft;

extern "C" ft_status ft_route(const ft_router* router, const ft_route_args* args, void* stream) {
  if (!args) return set_error(FT_ERR_INVALID_ARG, "args is null");
  const ft_route_args& g = *args;
  const ft_status st = check_router(router, g.num_experts, g.top_k);
  if (st != FT_OK) return st;
  if (g.num_tokens < 0 || g.num_tokens > kMostRows)
    return set_error(FT_ERR_INVALID_ARG, "num_tokens=%d outside 0..%d", g.num_tokens, kMostRows);
  if (g.logits_dtype != FT_F32 && g.logits_dtype != FT_BF16)
    return set_error(FT_ERR_INVALID_ARG, "logits_dtype=%d is not FT_F32 or FT_BF16", g.logits_dtype);
  if (g.num_tokens == 0) return FT_OK;
  const int size = g.logits_dtype == FT_F32 ? 4 : 2;
  const uintptr_t logits = reinterpret_cast<uintptr_t>(g.logits), outs = reinterpret_cast<uintptr_t>(g.topk_idx) | reinterpret_cast<uintptr_t>(g.topk_w);
  if (!g.logits || !g.topk_idx || !g.topk_w) return set_error(FT_ERR_INVALID_ARG, "null logits, topk_idx or topk_w");
  if ((logits & (size - 1)) || (outs & 3))
    return set_error(FT_ERR_INVALID_ARG, "logits, topk_idx or topk_w is not aligned to its elements");
  const int64_t stride = g.num_tokens == 1 ? g.num_experts : g.logits_stride;  // (of a single row it is not used)
  if (stride < g.num_experts)
    return set_error(FT_ERR_INVALID_ARG, "logits_stride=%lld is below num_experts=%d", (long long)stride, g.num_experts);
  RouteBatch a{};
  const bool aligned = logits % (4 * size) == 0 && (g.num_tokens == 1 || stride % 4 == 0);
  a.r = make_rule(*router, g.num_experts, g.top_k, router->bias, aligned);
  a.logits = g.logits; a.stride = stride; a.T = g.num_tokens; a.idx = g.topk_idx; a.w = g.topk_w;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = size == 4 ? launch<float>(a, s) : launch<__nv_bfloat16>(a, s);
  if (e != cudaSuccess) return set_error(FT_ERR_CUDA, "route launch: %s", cudaGetErrorString(e));
  return FT_OK;
}
