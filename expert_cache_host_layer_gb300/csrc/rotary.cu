// Rotary positions: ft_rotate, and ft_kv_append_rotary, which rotates a
// batch's new queries, and its new keys on their way into the pages.
//
// Pair i of a head's first rot_dim values is turned by position * f_i:
//   (a, b) -> scale * (a cos - b sin, b cos + a sin)
// At position 10^6 an fp32 product position * f_i would leave few bits of the
// turn's fraction, so the frequencies come as 64-bit fixed-point fractions of a
// turn: position * turns_i mod 2^64 is the turn's fraction, exactly.  The
// nearest quarter turn comes off in integers too, and the rest, at most an
// eighth of a turn, becomes a float of 24 bits for sincospif.
//
// Values are read and written once: HBM bounds a chunk, the chain of loads
// (q_start -> kv_len -> page; position -> sine) a decode step.  A block takes
// `per` consecutive tokens.  Its threads look the places up and form each
// (token, pair)'s sine and cosine once, for all heads, in shared memory.  Then
// head_dim / 16 lanes have a head each, of one of `step` tokens, and go through
// the block's tokens: which head it is, whether it is turned and stored, and
// where, is the same for all of them.  A lane has 16 values of a head: both
// halves of eight pairs (8c.. and rot_dim / 2 + 8c.. where the halves lie apart,
// 16c.. where pairs are interleaved), so that a pair never leaves its thread,
// whatever rot_dim is.
//
// Measured (head_dim 128, 16 query and 4 key heads): 16,384 tokens into the e4m3
// cache 32.9 us, 5.6 TB/s (with the head worked out for every vector, 42: 260
// instructions a warp and vector instead of 200); 8191 tokens x 24 heads of 96, a
// third of each turned, 14.3 us, 5.3 TB/s; one token 2.6 us in a graph.  The
// start (places, sines) is 3 to 4 us of each, and most of a chunk of few heads:
// 16,384 tokens x 1, 3 and 4 heads 5.7, 7.7 and 9.9 us, their bytes 1.2, 3.7 and 5.0.
#include <algorithm>

#include "decode_common.h"
#include "kv_common.h"

namespace ft {
namespace kv {
namespace {

constexpr int kMostThreads = 384;  // three such blocks an SM: 56 registers a thread (64: 34.6 us where these took 33.7, 48: 39.9)
constexpr int kThreads = 256;      // of a block, if its heads leave a choice
constexpr int kMostTokens = 32;    // of a block
constexpr int kTrigFloats = 4096;  // of a block: tokens x rot_dim
constexpr int kMostHeads = 8192;
constexpr int kMostDim = 512;

struct RotArgs {
  ft_rotary r;
  ft_kv_pages p;              // append
  ft_kv_batch b;
  const int32_t* positions;   // rotate
  const __nv_bfloat16* x[3];  // q, k, v
  int64_t ts[3], hs[3];
  __nv_bfloat16* out;         // of q
  int64_t ots, ohs;
  int rows, per;              // tokens in all, and of a block
  int Hq, heads, units;       // heads of q, of q, k and v, and lanes to a head
  int pass, step;             // heads and tokens that a block's threads have at a time
  int32_t* status;
};

__device__ __forceinline__ uint4 pack8(const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// scale * (cos, sin) of a 64-bit fraction of a turn.
__device__ __forceinline__ float2 turn(uint64_t fraction, float scale) {
  const uint32_t f = (uint32_t)(fraction >> 32), quarter = (f + 0x20000000u) >> 30;
  const int32_t rest = (int32_t)(f - (quarter << 30));  // of a turn of 2^32, within +-2^29
  float s, c;
  sincospif((float)rest * 0x1p-31f, &s, &c);
  s *= scale;
  c *= scale;
  const float x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;  // cos(t + pi / 2) = -sin t, sin(t + pi / 2) = cos t
  return make_float2(quarter == 1 || quarter == 2 ? -x : x, quarter & 2 ? -y : y);
}

constexpr int kNone = 0, kBf16 = 1, kFp8 = 2;  // the cache

template <int kCache, bool kInterleaved>
__global__ void __launch_bounds__(kMostThreads, 3) rotary_kernel(const __grid_constant__ RotArgs a) {
  __shared__ float4 s_trig[kTrigFloats / 4];  // [token][cos 0..3, cos 4..7, sin 0..3, sin 4..7 of a lane's pairs][lane]
  __shared__ int s_pos[kMostTokens], s_row[kMostTokens];
  const int half = a.r.rot_dim / 2, lanes = a.r.rot_dim / 16;  // lanes: of a head, those with pairs
  const int t0 = blockIdx.x * a.per, tokens = min(a.per, a.rows - t0);
  const int wide = a.pass * a.units, first = threadIdx.x / wide, in_pass = threadIdx.x - first * wide;
  const int head = in_pass / a.units, c = in_pass - head * a.units;
  const int Hk = kCache == kNone ? 0 : a.p.num_kv_heads;
  dec::pdl_wait_primary();

  for (int h0 = 0; h0 < a.heads; h0 += a.pass) {  // (one time, but for more heads than a block has threads for)
    const int h = h0 + head;
    const bool mine = first < a.step && h < a.heads, query = kCache == kNone || h < a.Hq, key = !query && h < a.Hq + Hk;
    const bool turned = c < lanes && (query || key);
    const bool apart = !kInterleaved && turned;
    const int e0 = apart ? 8 * c : 16 * c, to1 = apart ? half : 8;  // the lane's first vector, and from there to the second
    const int of = query ? h : key ? h - a.Hq : h - a.Hq - Hk;
    const int64_t ts = query ? a.ts[0] : key ? a.ts[1] : a.ts[2], hs = query ? a.hs[0] : key ? a.hs[1] : a.hs[2];
    const __nv_bfloat16* src = (query ? a.x[0] : key ? a.x[1] : a.x[2]) + ((int64_t)t0 + first) * ts + of * hs + e0;
    __nv_bfloat16* out = a.out + ((int64_t)t0 + first) * a.ots + of * a.ohs + e0;
    const bool stores = kCache == kFp8 && __any_sync(0xffffffffu, mine && !query);  // of the warp's heads
    uint4 next[2];
    auto load = [&](int t) {
      if (!mine || t >= tokens) return;
      next[0] = *reinterpret_cast<const uint4*>(src);
      next[1] = *reinterpret_cast<const uint4*>(src + to1);
      src += a.step * ts;
    };
    load(first);
    if (h0 == 0) {  // the tokens' places, and their pairs' sines and cosines
      if (threadIdx.x < tokens) {
        int pos, row = 0;
        if (kCache == kNone) pos = __ldg(&a.positions[t0 + threadIdx.x]);
        else row = new_place(a.p, a.b, t0 + threadIdx.x, a.status, &pos);
        s_pos[threadIdx.x] = pos;
        s_row[threadIdx.x] = row;
      }
      __syncthreads();
      for (int i = threadIdx.x; i < tokens * half; i += blockDim.x) {
        const int t = i / half, pair = i - t * half;
        const float2 cs = turn((uint64_t)(int64_t)s_pos[t] * __ldg(&a.r.turns[pair]), a.r.scale);
        float* to = reinterpret_cast<float*>(s_trig) + ((t * 4 + (pair >> 2 & 1)) * lanes + (pair >> 3)) * 4 + (pair & 3);
        to[0] = cs.x;
        to[8 * lanes] = cs.y;
      }
      __syncthreads();
    }
    for (int t = first; t - first < tokens; t += a.step, out += a.step * a.ots) {  // the whole block together
      const bool live = mine && t < tokens;
      float y[2][8];
      dec::decode_chunk<FT_W_BF16>(next[0], y[0]);
      dec::decode_chunk<FT_W_BF16>(next[1], y[1]);
      load(t + a.step);
      if (live && turned) {
        const float4* at = s_trig + t * 4 * lanes + c;
        float cs[8], sn[8];
        *reinterpret_cast<float4*>(cs) = at[0];
        *reinterpret_cast<float4*>(cs + 4) = at[lanes];
        *reinterpret_cast<float4*>(sn) = at[2 * lanes];
        *reinterpret_cast<float4*>(sn + 4) = at[3 * lanes];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float& p = kInterleaved ? y[e / 4][2 * (e % 4)] : y[0][e];
          float& q = kInterleaved ? y[e / 4][2 * (e % 4) + 1] : y[1][e];
          const float u = fmaf(p, cs[e], -(q * sn[e])), w = fmaf(q, cs[e], p * sn[e]);
          p = u;
          q = w;
        }
      }
      uint32_t bits = 0;
      if (stores) {  // largest magnitude of the head's vector (as bits: NaN above infinity), over its lanes
#pragma unroll
        for (int e = 0; e < 16; ++e) bits = max(bits, __float_as_uint(y[e / 8][e % 8]) & 0x7fffffffu);
        for (int o = a.units / 2; o > 0; o >>= 1) bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, o));
      }
      if (!live) continue;
      const int row = s_row[t];
      if (query) {
        if (row == kNobodys) continue;
        *reinterpret_cast<uint4*>(out) = pack8(y[0]);
        *reinterpret_cast<uint4*>(out + to1) = pack8(y[1]);
      } else if (row >= 0) {
        const int64_t at = (int64_t)(row + of * a.p.page_tokens);  // rows are below 2^31
        void* pages = key ? a.p.k : a.p.v;
        if (kCache == kFp8) {
          const int k = scale_exp(__uint_as_float(bits));
          uint8_t* dst = static_cast<uint8_t*>(pages) + at * a.p.head_dim + e0;
          *reinterpret_cast<uint2*>(dst) = encode8(y[0], k);
          *reinterpret_cast<uint2*>(dst + to1) = encode8(y[1], k);
          if (c == 0) (key ? a.p.k_scale : a.p.v_scale)[at] = (uint8_t)scale_byte(k);
        } else {
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(pages) + at * a.p.head_dim + e0;
          *reinterpret_cast<uint4*>(dst) = pack8(y[0]);
          *reinterpret_cast<uint4*>(dst + to1) = pack8(y[1]);
        }
      }
    }
  }
  dec::pdl_launch_dependents();
}

ft_status check_rotary(const ft_rotary* r, int head_dim) {
  if (!r) return set_error(FT_ERR_INVALID_ARG, "rotary is null");
  if (r->rot_dim < 16 || r->rot_dim % 16 || r->rot_dim > head_dim)
    return set_error(FT_ERR_UNSUPPORTED, "rot_dim=%d is not a multiple of 16 in 16..head_dim=%d", r->rot_dim, head_dim);
  if (!(r->scale >= -3.0e38f && r->scale <= 3.0e38f)) return set_error(FT_ERR_INVALID_ARG, "the rotary's scale must be finite");
  if (!r->turns || (reinterpret_cast<uintptr_t>(r->turns) & 7))
    return set_error(FT_ERR_INVALID_ARG, "turns is null or not 8-byte aligned");
  return FT_OK;
}

// An output: with positive strides, and where it is its input, with that one's (each value is written where it was read).
ft_status check_out(const char* name, const RotArgs& a) {
  const ft_status st = check_rows(name, a.out, a.ots, a.ohs);
  if (st != FT_OK) return st;
  if (a.ots <= 0 || a.ohs <= 0) return set_error(FT_ERR_INVALID_ARG, "%s's strides must be positive", name);
  if (a.out == a.x[0] && (a.ots != a.ts[0] || a.ohs != a.hs[0]))
    return set_error(FT_ERR_INVALID_ARG, "%s may be its input itself only with its strides", name);
  return FT_OK;
}

ft_status launch(RotArgs& a, const char* name, int cache, cudaStream_t s) {
  a.heads = a.Hq + (cache == kNone ? 0 : 2 * a.p.num_kv_heads);
  const int fit = kMostThreads / a.units, passes = (a.heads + fit - 1) / fit;
  a.pass = (a.heads + passes - 1) / passes;
  const int wide = a.pass * a.units;  // threads of a token
  const int most = std::min(kMostTokens, kTrigFloats / a.r.rot_dim);
  a.step = std::min({std::max(1, kThreads / wide), a.rows, most});
  const int threads = (wide * a.step + 31) / 32 * 32;
  // One wave of blocks while they go through less than 18 tokens in turn (8191 x 24 heads in one 14.3 us, in two 14.5; 16,384
  // x 3 heads in one 7.7, in two 7.9, three 9.0), then as many waves as leave them nine: other blocks' loads fill a block's
  // start (16,384 x 24 heads in one 33.6 us, in two 32.9, three 32.8, four 33.2).
  const int wave = 3 * kMostThreads / threads * sm_count();
  if (wave == 0) return set_error(FT_ERR_CUDA, "%s: no CUDA device", name);
  auto tokens_each = [&](long long blocks) { return (int)((a.rows + blocks - 1) / blocks); };
  a.per = std::min(most, tokens_each((long long)wave * std::max(1, tokens_each(wave) / a.step / 9)));
  if (a.per > a.step) a.per = std::min(most, (a.per + a.step - 1) / a.step * a.step);
  const dim3 grid((unsigned)(((long long)a.rows + a.per - 1) / a.per));
  const bool pairs = a.r.interleaved != 0;
  auto* kernel = cache == kFp8 ? (pairs ? rotary_kernel<kFp8, true> : rotary_kernel<kFp8, false>)
                 : cache == kBf16 ? (pairs ? rotary_kernel<kBf16, true> : rotary_kernel<kBf16, false>)
                                  : (pairs ? rotary_kernel<kNone, true> : rotary_kernel<kNone, false>);
  const cudaError_t e = launch_dependent(kernel, grid, threads, 0, s, a);
  if (e != cudaSuccess) return set_error(FT_ERR_CUDA, "%s launch: %s", name, cudaGetErrorString(e));
  return FT_OK;
}

}  // namespace
}  // namespace kv
}  // namespace ft

using namespace ft;
using namespace ft::kv;

extern "C" ft_status ft_rotate(const ft_rotary* rotary, const ft_rotate_args* args, void* stream) {
  if (!args) return set_error(FT_ERR_INVALID_ARG, "args is null");
  const ft_rotate_args& g = *args;
  if (g.head_dim < 16 || g.head_dim % 16 || g.head_dim > kMostDim)
    return set_error(FT_ERR_UNSUPPORTED, "head_dim=%d is not a multiple of 16 in 16..%d", g.head_dim, kMostDim);
  ft_status st = check_rotary(rotary, g.head_dim);
  if (st != FT_OK) return st;
  if (g.num_heads < 1 || g.num_heads > kMostHeads)
    return set_error(FT_ERR_INVALID_ARG, "num_heads=%d outside 1..%d", g.num_heads, kMostHeads);
  if (g.num_tokens < 0) return set_error(FT_ERR_INVALID_ARG, "num_tokens=%d", g.num_tokens);
  if (g.num_tokens == 0) return FT_OK;
  if (!g.positions) return set_error(FT_ERR_INVALID_ARG, "positions is null");
  RotArgs a{};
  a.r = *rotary; a.positions = g.positions;
  a.x[0] = static_cast<const __nv_bfloat16*>(g.x); a.ts[0] = g.x_token_stride; a.hs[0] = g.x_head_stride;
  a.out = static_cast<__nv_bfloat16*>(g.out); a.ots = g.out_token_stride; a.ohs = g.out_head_stride;
  if (g.num_tokens == 1) a.ts[0] = a.ots = g.head_dim;  // of single entries: not used
  if (g.num_heads == 1) a.hs[0] = a.ohs = g.head_dim;
  if ((st = check_rows("x", a.x[0], a.ts[0], a.hs[0])) != FT_OK) return st;
  if ((st = check_out("out", a)) != FT_OK) return st;
  a.rows = g.num_tokens; a.Hq = g.num_heads; a.units = g.head_dim / 16;
  return launch(a, "rotate", kNone, static_cast<cudaStream_t>(stream));
}

extern "C" ft_status ft_kv_append_rotary(const ft_kv_pages* pages, const ft_kv_batch* batch, const ft_rotary* rotary,
                                         const ft_append_args* args, void* stream) {
  if (!args) return set_error(FT_ERR_INVALID_ARG, "args is null");
  const ft_append_args& g = *args;
  ft_status st = check_pages(pages);
  if (st == FT_OK) st = check_batch(pages, batch);
  if (st == FT_OK) st = check_rotary(rotary, pages->head_dim);
  if (st != FT_OK) return st;
  if (g.num_q_heads < 0 || g.num_q_heads > kMostHeads)
    return set_error(FT_ERR_INVALID_ARG, "num_q_heads=%d outside 0..%d", g.num_q_heads, kMostHeads);
  if (batch->num_tokens == 0) return FT_OK;
  const int D = pages->head_dim;
  RotArgs a{};
  a.r = *rotary; a.p = *pages; a.b = *batch;
  a.x[0] = static_cast<const __nv_bfloat16*>(g.q); a.ts[0] = g.q_token_stride; a.hs[0] = g.q_head_stride;
  a.x[1] = static_cast<const __nv_bfloat16*>(g.k); a.ts[1] = g.k_token_stride; a.hs[1] = g.k_head_stride;
  a.x[2] = static_cast<const __nv_bfloat16*>(g.v); a.ts[2] = g.v_token_stride; a.hs[2] = g.v_head_stride;
  a.out = static_cast<__nv_bfloat16*>(g.q_out); a.ots = g.q_out_token_stride; a.ohs = g.q_out_head_stride;
  if (batch->num_tokens == 1) a.ts[0] = a.ts[1] = a.ts[2] = a.ots = D;  // of single entries: not used
  if (pages->num_kv_heads == 1) a.hs[1] = a.hs[2] = D;
  if (g.num_q_heads == 1) a.hs[0] = a.ohs = D;
  if ((st = check_rows("k", a.x[1], a.ts[1], a.hs[1])) != FT_OK) return st;
  if ((st = check_rows("v", a.x[2], a.ts[2], a.hs[2])) != FT_OK) return st;
  if (g.num_q_heads > 0) {
    if ((st = check_rows("q", a.x[0], a.ts[0], a.hs[0])) != FT_OK) return st;
    if ((st = check_out("q_out", a)) != FT_OK) return st;
    if (a.out == a.x[1] || a.out == a.x[2]) return set_error(FT_ERR_INVALID_ARG, "q_out is k or v");
  }
  a.rows = batch->num_tokens; a.Hq = g.num_q_heads; a.units = D / 16;
  if ((st = status_word(&a.status)) != FT_OK) return st;
  return launch(a, "append_rotary", pages->kv_dtype == FT_KV_FP8E4M3 ? kFp8 : kBf16, static_cast<cudaStream_t>(stream));
}
