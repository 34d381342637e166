// What the attention kernels over the paged cache share: the call's arguments,
// visibility, the even cut of the work over the CTAs, partial sums and the
// launch helpers.  Internal to libft.
#pragma once

#include <cuda.h>

#include "decode_common.h"
#include "kv_common.h"

namespace ft {
namespace kv {

constexpr int kTokenRows = 16;    // most rows of a (sequence, key head) in token_kernel
constexpr int kMostCtas = 160;    // of a main kernel's grid, one per SM
constexpr int kTokenTile = 64;    // tokens per tile of its ring
constexpr int kChunkRows = 256;   // rows of a block in chunk_kernel: two sub-tiles of 128
constexpr int kSubRows = 128;

struct AttendArgs {
  ft_kv_pages p;
  ft_kv_batch b;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;             // or null
  int64_t qts, qhs, ots, ohs;
  float scale_log2;       // scale * log2(e)
  int Hq, G, causal, window;
  int tps;                // chunk_kernel: new tokens of a sub-tile of 128 rows, 128 / G
  int small;              // sequences of up to so many rows a head are token_kernel's, the others chunk_kernel's
  int grid;               // CTAs of the main kernel
  bool beside;            // token_kernel and chunk_kernel both run
  int32_t* status;
  // workspace
  unsigned* counter;      // [grid] token_kernel: parts done of what CTA c begins and does not end; 0 between calls
  unsigned* arrived;      // [grid][8] chunk_kernel: parts that others have done of 32 rows of what CTA c begins and does
                          // not end; 0 between calls
  int4* desc;             // [grid][8] chunk_kernel: the (sequence, head, row block) whose 32 rows CTA c begins and leaves for
                          // combine_kernel: {s, h, row block, last CTA}; s = -1: none
  float* part_o;          // [2 grid][rows][D] unnormalised sums: slot 2c of what CTA c finds begun, 2c + 1 of what it
                          // begins and leaves (chunk_kernel: see part_at)
  float* part_ml;         // [2 grid][rows][2] running maximum (log2 domain) and sum
};

__device__ __forceinline__ float exp2_approx(float x) {  // relative error 2^-22, 2^-inf = 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A box of a 2-D map at column c0, row c1.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
          "r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(dec::smem_addr(bar))
      : "memory");
}

// chunk_kernel's partial sums: where columns d .. d + 3 of a row are.  32 rows lie
// side by side, so that a thread per row writes and reads whole lines.
template <int D>
__device__ __forceinline__ float4* part_at(const AttendArgs& a, long long slot, int row, int d) {
  return reinterpret_cast<float4*>(a.part_o) + ((slot * kChunkRows + (row & ~31)) * (D / 4) + d * 8 + (row & 31));
}
// x + f y, rounded twice: whoever joins partial sums gives the same.
__device__ __forceinline__ float join(float x, float f, float y) { return __fadd_rn(x, __fmul_rn(f, y)); }

// Tokens [lo, hi) that new token i of a sequence sees; lo and hi grow with i.
struct Span {
  int lo, hi;
};
__device__ __forceinline__ Span visible(const AttendArgs& a, const Seq& q, int i) {
  const int pos = q.n - q.m + i;
  Span v;
  v.hi = a.causal ? max(0, pos + 1) : q.n & ~(pos >> 31);
  v.lo = a.window ? min(v.hi, max(0, pos - a.window + 1)) : 0;
  return v;
}

// Sequence s as token_kernel (or chunk_kernel) sees it: without new tokens if it is the other's.
template <bool kToken>
__device__ __forceinline__ Seq own_seq(const AttendArgs& a, int s) {
  Seq q = load_seq(a.p, a.b, s, a.status);
  if ((q.m * a.G <= a.small) != kToken) q.m = 0;
  return q;
}

// Whole warp: wait for phase `parity` of a barrier; false if the CTA has
// aborted or the wait ran out (which aborts the CTA).
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, int32_t* status,
                                              volatile int* abort_flag) {
  bool ok = dec::mbar_try_wait(bar, parity);
  if (!ok) {
    const unsigned long long t0 = dec::global_ns();
    for (;;) {
      for (int i = 0; i < 64 && !ok; ++i) ok = dec::mbar_try_wait(bar, parity);
      if (ok || *abort_flag) break;
      if (dec::global_ns() - t0 > dec::kWaitLimitNs) {
        raise(status, FT_ERR_TIMEOUT);
        *abort_flag = 1;
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// The work laid end to end over the sequences, and the part of it that is
// this CTA's: items [w0, w1) of `total`, sequence s's items beginning at `base`.
struct Range {
  long long w0, w1, base, total;
  int s, n;  // first sequence; CTAs that have work
};
// x / y, x >= 0, y > 0: in 32 bits where they do (64 take some 100 instructions).
__device__ __forceinline__ long long quotient(long long x, long long y) {
  if (((x | y) >> 32) == 0) return (long long)((uint32_t)x / (uint32_t)y);
  return x / y;
}
// CTA of item w.
__device__ __forceinline__ int cta_of(long long w, long long total, int n) {
  return (int)quotient((w + 1) * n - 1, total);
}

// Every thread of the CTA: exclusive prefix sums of count(s) over the
// sequences into pre[0 .. S], and this CTA's even share of the total.
template <typename Count>
__device__ __forceinline__ Range cut(const AttendArgs& a, long long* pre, long long* scan, Count count) {
  const int S = a.b.num_seqs, T = blockDim.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (S + T - 1) / T, s0 = min(S, (int)threadIdx.x * per), s1 = min(S, s0 + per);
  long long mine = 0;
  for (int k = 0; k < per; ++k) {  // whole warps together: count() may use them; count(S) = 0
    const int s = s0 + k < s1 ? s0 + k : S;
    if (s < S) pre[s] = mine;
    mine += count(s);
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  long long before = incl - mine, total = 0;
  for (int w = 0; w < T / 32; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  for (int s = s0; s < s1; ++s) pre[s] += before;
  __syncthreads();
  Range r;
  r.total = total;
  r.n = (int)min((long long)gridDim.x, total);
  r.w0 = r.w1 = r.base = 0;
  r.s = 0;
  if ((int)blockIdx.x < r.n) {
    r.w0 = quotient(blockIdx.x * total, r.n);
    r.w1 = quotient((blockIdx.x + 1) * total, r.n);
    int lo = 0, hi = S - 1;  // the last sequence that begins at or before w0 (ones without work begin where the next does)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= r.w0) lo = mid;
      else hi = mid - 1;
    }
    r.s = lo;
    r.base = pre[lo];
  }
  return r;
}

// ---------------------------------------------------------------- token_kernel's items: tiles of a (sequence, head)

// A (sequence, head)'s fixed cost (its rows of q, joining the warps and the
// parts, all of it latency), in tiles: 8 of 32 KB, 12 of the smaller ones.
// (e4m3, head_dim 128, 4 / 8 / 12 / 20: eight sequences of 2000-32500 tokens 31.5 /
// 30.7 / 29.6 / 29.0 us, twenty of 200-6500 22.7 / 20.5 / 20.1 / 21.4; bf16,
// twenty 25.7 / 24.7 / 24.0 / 23.7, 64 of 301-8000 100.9 / 101.3 / 102.0 / 103.6.)
__device__ __forceinline__ int pair_items(const AttendArgs& a) {
  return a.p.head_dim == 128 && a.p.kv_dtype == FT_KV_BF16 ? 8 : 12;
}

__device__ __forceinline__ Span token_tiles(const AttendArgs& a, const Seq& q, Span* seen) {
  seen->lo = visible(a, q, 0).lo;
  seen->hi = visible(a, q, max(0, q.m - 1)).hi;
  Span t;
  t.lo = seen->lo / kTokenTile;
  t.hi = q.m == 0 ? t.lo : max(t.lo + 1, (seen->hi + kTokenTile - 1) / kTokenTile);  // rows that see nothing: one tile
  return t;
}
// Items of one head of a sequence: its tiles, after the fixed cost.
__device__ __forceinline__ int token_items(const AttendArgs& a, const Span& t) {
  return t.hi > t.lo ? t.hi - t.lo + pair_items(a) : 0;
}
__device__ __forceinline__ Range token_range(const AttendArgs& a, long long* pre, long long* scan) {
  return cut(a, pre, scan, [&](int s) {
    if (s == a.b.num_seqs) return 0LL;
    Span seen;
    return (long long)token_items(a, token_tiles(a, own_seq<true>(a, s), &seen)) * a.p.num_kv_heads;
  });
}
// The parts of (sequence, head)s in a CTA's range, one after the other.
struct TokenWalk {
  long long w, end, base, total;
  int n;
  int s, h;      // this one
  Seq q;
  int lo, hi;    // tokens that some row sees
  int t0, t1;    // tiles of it that are this CTA's
  bool begins, ends;
  Span tiles;
  int loaded;
  __device__ __forceinline__ TokenWalk(const AttendArgs&, const Range& r)
      : w(r.w0), end(r.w1), base(r.base), total(r.total), n(r.n), s(r.s), loaded(-1) {}
  __device__ __forceinline__ bool next(const AttendArgs& a) {
    for (;;) {
      if (w >= end) return false;
      if (loaded != s) {
        q = own_seq<true>(a, s);
        Span seen;
        tiles = token_tiles(a, q, &seen);
        lo = seen.lo;
        hi = seen.hi;
        loaded = s;
      }
      const int items = token_items(a, tiles);
      const long long all = (long long)items * a.p.num_kv_heads;
      if (w - base >= all) {
        base += all;
        ++s;
        continue;
      }
      h = (int)quotient(w - base, items);
      const int rel = (int)(w - base - (long long)h * items), cnt = (int)min((long long)(items - rel), end - w);
      w += cnt;
      t0 = tiles.lo + max(0, rel - pair_items(a));
      t1 = tiles.lo + max(0, rel + cnt - pair_items(a));
      if (t0 == t1) continue;  // only of the fixed cost
      begins = t0 == tiles.lo;
      ends = t1 == tiles.hi;
      return true;
    }
  }
  // first and last CTA of this (sequence, head)
  __device__ __forceinline__ int first_cta(const AttendArgs& a) const {
    return cta_of(base + (long long)h * token_items(a, tiles) + pair_items(a), total, n);
  }
  __device__ __forceinline__ int last_cta(const AttendArgs& a) const {
    return cta_of(base + (long long)(h + 1) * token_items(a, tiles) - 1, total, n);
  }
};

// ---------------------------------------------------------------- results

// Query head g of the group of key head h, new token i of the sequence.
__device__ __forceinline__ long long out_at(const AttendArgs& a, const Seq& q, int h, int i, int g) {
  return (long long)(q.q0 + i) * a.ots + (long long)(h * a.G + g) * a.ohs;
}
__device__ __forceinline__ void write_lse(const AttendArgs& a, const Seq& q, int h, int i, int g, float m, float l) {
  if (a.lse)
    a.lse[(long long)(q.q0 + i) * a.Hq + h * a.G + g] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}
// 1 / l; 0 for a row without weight (it sees nothing, or only scores of -inf).
__device__ __forceinline__ float inverse(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }

// ---------------------------------------------------------------- host

cudaError_t launch_attend_token(const AttendArgs& a, cudaStream_t s);
cudaError_t launch_attend_chunk(const AttendArgs& a, cudaStream_t s);
// Joins the partial sums of chunk_kernel's row blocks that a cut divided;
// `used`: rows of a block that any sequence has.
cudaError_t launch_combine(const AttendArgs& a, int used, cudaStream_t s);
// Pages of k or v as rows of head_dim, boxes of box_rows rows x 128 bytes (or the whole row, if shorter), swizzled.
bool pages_map(CUtensorMap* m, const ft_kv_pages& p, const void* base, int box_rows);
// q as [token][head][64 of head_dim], boxes of `tokens` x G heads x 128 bytes, swizzled.
bool queries_map(CUtensorMap* m, const AttendArgs& a, int tokens);

}  // namespace kv
}  // namespace ft
