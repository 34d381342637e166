// Attention of a few rows over long sequences: every (sequence, key head) of
// the batch has at most 16 rows (new tokens x query heads of the group), as in
// decoding.  The work is reading K and V once: memory-bound.
//
//   out = sum_j w_j v_j / sum_j w_j,   w_j = 2^(x_j - m),  x_j = scale log2(e) q.k_j,  m = max_j x_j
//
// Quantised cache: the key's scale multiplies the score and the value's scale
// the probability (a power of two: nothing is rounded for it).
//
// Split: the batch's tiles of 128 tokens, laid end to end over (sequence, key
// head, tile), are cut into equal contiguous ranges, one per CTA and one CTA
// per SM, whatever the lengths are.  A (sequence, head) that a cut divides
// leaves partial sums (unnormalised out, m, l) in the workspace, which
// combine_kernel joins in tile order.
//
// CTA: one producer warp, eight consumer warps.  The producer's lanes 0..7
// load one group of 16 tokens each (a group never crosses a page) as swizzled
// TMA boxes into a ring of stages; consumer warp w takes group w of every
// tile: S = Q K^T as m16n8k16 (16 rows, the invalid ones zero), its own
// running m, l and O, O += P V.  Warps meet only at the end of a (sequence,
// head).  mma.sync is enough here: a row block of 16 is an eighth of a
// tcgen05 tile, and the path is bound by HBM, not by the tensor pipe.
//
// Quantised cache: codes are expanded in registers (exact), keys to fp16, the
// cheaper conversion, values to bf16, whose range P needs: a probability keeps
// its 8 bits however small it is.  The
// contraction order over head_dim is free as long as Q uses the same, and so
// are the order of tokens (P's columns and V's rows) and of output columns;
// they are chosen so that each lane reads 16 consecutive bytes of a row,
// without bank conflicts, and needs no transposition.  Q is scaled per row by
// a power of two to [1, 2) before it is rounded to fp16, so that no value
// leaves fp16's range: q elements below 2^-14 of the row's largest lose bits
// that weigh less than 2^-25 of it.
#include <cuda.h>

#include "decode_common.h"
#include "kv_attend.h"

namespace ft {
namespace kv {
namespace {

constexpr int kConsumers = 8;
constexpr int kThreads = (kConsumers + 1) * 32;
constexpr int kGroup = 16;
static_assert(kTokenTile == kConsumers * kGroup, "a group per consumer warp");
constexpr int kRedRows = 4;  // rows joined across the warps at a time

template <int D, bool kFp8>
struct Layout {
  static constexpr int kEsz = kFp8 ? 1 : 2;
  static constexpr int kGroupBytes = kGroup * D * kEsz;  // K of a group; V follows
  static constexpr int kStageBytes = 2 * kConsumers * kGroupBytes;
  static constexpr int kStages = kStageBytes >= 65536 ? 3 : kStageBytes >= 32768 ? 6 : 8;
  static constexpr int kRowFloats = D + 4;
  static constexpr int kScaleOff = kStages * kStageBytes;
  static constexpr int kScaleBytes = kFp8 ? kStages * 2 * kTokenTile : 0;
  static constexpr int kRedOff = kScaleOff + kScaleBytes;
  static constexpr int kMlOff = kRedOff + kConsumers * kRedRows * kRowFloats * 4;
  static constexpr int kBarOff = kMlOff + kConsumers * 16 * 2 * 4;
  static constexpr int kSmem = kBarOff + 2 * kStages * 8 + 16 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kStages * kStageBytes >= (kMaxSeqs + 1) * 8 + 1024, "the prefix sums fit the ring before it fills");
};

__device__ __forceinline__ void mma_bf16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// scores: fp16 for the quantised cache
template <bool kFp8>
__device__ __forceinline__ void mma_score(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if (kFp8) mma_f16(c, a, b0, b1);
  else mma_bf16(c, a, b0, b1);
}
__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
          "r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(dec::smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t pair) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(pair & 0xffffu), __NV_E4M3);
  return (uint32_t)h.x | (uint32_t)h.y << 16;
}
__device__ __forceinline__ uint32_t e4m3x2_to_bf162(uint32_t pair) {
  const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(pair & 0xffffu), __NV_E4M3)));
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, bool half) {
  if (half) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ void bar_consumers() { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory"); }

// Order of a group's tokens in S's columns (and P's): column n of an 8-column
// block is token tok(n) of the block.  fp8 rows of 128 bytes: neighbouring
// rows of a quarter-warp differ in bit 2, which the swizzle turns into other
// banks.
template <int D, bool kFp8>
__device__ __forceinline__ int tok(int n) {
  return kFp8 && D == 128 ? (n >> 1) | ((n & 1) << 2) : n;
}
// Output column of accumulator block j, fragment column 2c + i.
template <int D, bool kFp8>
__device__ __forceinline__ int out_col(int j, int c, int i) {
  return !kFp8 ? 8 * j + 2 * c + i : D == 128 ? 16 * c + 64 * i + j : 16 * c + 8 * i + j;
}

template <int D, bool kFp8>
struct Warp {
  static constexpr int kKs = D / 16, kNb = D / 8;
  uint32_t qf[kKs][4];
  float o[kNb][4];
  float m[2], l[2], sc[2];  // rows lane / 4 and + 8: running maximum, this lane's sum, score factor
  int lo[2], hi[2];         // visible tokens [lo, hi) of those rows

  __device__ __forceinline__ void begin(const AttendArgs& a, const Seq& q, int h, int lane) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = g + 8 * half, i = r / a.G;
      const bool ok = i < q.m;
      const __nv_bfloat16* row = a.q + (long long)(q.q0 + i) * a.qts + (long long)(h * a.G + r % a.G) * a.qhs;
      const Span v = visible(a, q, ok ? i : 0);
      lo[half] = v.lo;
      hi[half] = ok ? v.hi : 0;
      m[half] = -INFINITY;
      l[half] = 0.0f;
      sc[half] = a.scale_log2;
#pragma unroll
      for (int ks = 0; ks < kKs; ++ks)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int d = !kFp8 ? 16 * ks + 8 * w + 2 * c : (ks < 4 ? 0 : 64) + 16 * c + 4 * (ks & 3) + 2 * w;
          qf[ks][2 * w + half] = ok ? __ldg(reinterpret_cast<const uint32_t*>(row + d)) : 0u;
        }
      if (kFp8) {  // to fp16, the row scaled to [1, 2)
        uint32_t top = 0;
#pragma unroll
        for (int ks = 0; ks < kKs; ++ks)
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const uint32_t u = qf[ks][2 * w + half];
            top = max(top, max((u << 16) & 0x7f800000u, u & 0x7f800000u));
          }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = min(max((int)(top >> 23), 1), 253);  // infinities and NaN stay what they are
        const float down = __uint_as_float((uint32_t)(254 - e) << 23);
        sc[half] *= __uint_as_float((uint32_t)e << 23);
#pragma unroll
        for (int ks = 0; ks < kKs; ++ks)
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const uint32_t u = qf[ks][2 * w + half];
            qf[ks][2 * w + half] = pack2(dec::bf16_lo(u) * down, dec::bf16_hi(u) * down, true);
          }
      }
    }
#pragma unroll
    for (int j = 0; j < kNb; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
  }

  // One group: tokens j0 .. j0 + 15 at shared addresses kb, vb; ksc, vsc their scale bytes.
  __device__ __forceinline__ void group(uint32_t kb, uint32_t vb, const uint8_t* ksc, const uint8_t* vsc, int j0,
                                        bool full, int m_new, int lane) {
    const int g = lane >> 2, c = lane & 3;
    float s[2][4] = {};
    if (!kFp8) {
      const int t = ((lane >> 4) << 3) + (lane & 7), ch = (lane >> 3) & 1;
#pragma unroll
      for (int ks = 0; ks < kKs; ++ks) {
        uint32_t b[4];
        ldsm4(b, kb + (ks >> 2) * (kGroup * 128) + t * 128 + (((2 * (ks & 3) + ch) ^ (t & 7)) << 4));
        mma_score<kFp8>(s[0], qf[ks], b[0], b[1]);
        mma_score<kFp8>(s[1], qf[ks], b[2], b[3]);
      }
    } else {
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) {
        const int t = nb * 8 + tok<D, kFp8>(g);
#pragma unroll
        for (int hf = 0; hf < D / 64; ++hf) {
          const int phys = D == 128 ? (c + 4 * hf) ^ (t & 7) : c ^ ((t >> 1) & 3);
          uint32_t w[4];
          asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                       : "r"(kb + t * D + (phys << 4)));
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mma_score<kFp8>(s[nb], qf[hf * 4 + i], e4m3x2_to_half2(w[i]), e4m3x2_to_half2(w[i] >> 16));
        }
      }
    }
    // scores to log2 domain, scales and masks
    float vs[4];  // value scales of this lane's four tokens
    float top[2] = {m[0], m[1]};
#pragma unroll
    for (int nb = 0; nb < 2; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = nb * 8 + tok<D, kFp8>(2 * c + i), u = 2 * nb + i;
        float kf = 1.0f;
        vs[u] = 1.0f;
        if (kFp8) {
          kf = scale_of(ksc[t]);
          vs[u] = scale_of(vsc[t]);
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float x = s[nb][2 * hf + i] * sc[hf];
          if (kFp8) x *= kf;
          if (!full && (j0 + t < lo[hf] || j0 + t >= hi[hf])) x = -INFINITY;
          s[nb][2 * hf + i] = x;
          top[hf] = fmaxf(top[hf], x);
        }
      }
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      top[hf] = fmaxf(top[hf], __shfl_xor_sync(0xffffffffu, top[hf], 1));
      top[hf] = fmaxf(top[hf], __shfl_xor_sync(0xffffffffu, top[hf], 2));
    }
    if (__any_sync(0xffffffffu, top[0] > m[0] || top[1] > m[1])) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const float f = top[hf] > m[hf] ? exp2_approx(m[hf] - top[hf]) : 1.0f;
        l[hf] *= f;
        m[hf] = top[hf];
#pragma unroll
        for (int j = 0; j < kNb; ++j) {
          o[j][2 * hf] *= f;
          o[j][2 * hf + 1] *= f;
        }
      }
    }
    uint32_t pf[4];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const float base = m[hf] == -INFINITY ? 0.0f : m[hf];
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) {
        float w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float x = s[nb][2 * hf + i];
          w[i] = exp2_approx(x - base);
          l[hf] += w[i];
          if (kFp8) w[i] = x == -INFINITY ? 0.0f : w[i] * vs[2 * nb + i];  // an unseen token's scale may be NaN
        }
        pf[2 * nb + hf] = pack2(w[0], w[1], false);
      }
    }
    // Tokens that no row sees hold anything (a page's unused end): their V is
    // taken as zero.  Where some rows see a token and others do not
    // (m_new > 1) and its V is not finite, 0 * V must not reach the others:
    // one product per new token, over the V that it sees, added to its rows.
    uint32_t keep[2] = {~0u, ~0u};
    bool split = false;
    if (!full) {
      const int any_lo = __shfl_sync(0xffffffffu, lo[0], 0);  // row 0 belongs to the first new token
      const int any_hi = max(hi[0], hi[1]);
      const int w_hi = max(any_hi, __shfl_xor_sync(0xffffffffu, any_hi, 4));
      const int x_hi = max(w_hi, __shfl_xor_sync(0xffffffffu, w_hi, 8));
      const int t_hi = max(x_hi, __shfl_xor_sync(0xffffffffu, x_hi, 16));
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) keep[nb] = keep_mask(nb, c, j0, any_lo, t_hi);
      split = m_new > 1;
    }
    accumulate(vb, pf, keep, full, split, j0, m_new, lane);
  }
  __device__ __forceinline__ uint32_t keep_mask(int nb, int c, int j0, int from, int to) const {
    uint32_t k = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = j0 + nb * 8 + tok<D, kFp8>(2 * c + i);
      if (j >= from && j < to) k |= 0xffffu << (16 * i);
    }
    return k;
  }
  // fragments (b0, b1) of kB consecutive blocks starting at block jb
  static constexpr int kB = kFp8 ? 4 : 2;
  __device__ __forceinline__ void v_frags(uint32_t vb, int jb, int lane, uint32_t (*b)[2]) const {
    const int g = lane >> 2, c = lane & 3;
    if (!kFp8) {
      const int t = (lane & 7) + (((lane >> 3) & 1) << 3), ch = jb + (lane >> 4);
      uint32_t r[4];
      ldsm4t(r, vb + (ch >> 3) * (kGroup * 128) + t * 128 + (((ch & 7) ^ (t & 7)) << 4));
      b[0][0] = r[0]; b[0][1] = r[1]; b[1][0] = r[2]; b[1][1] = r[3];
    } else {
      uint32_t w[2][2];
#pragma unroll
      for (int nb = 0; nb < 2; ++nb)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int t = nb * 8 + tok<D, kFp8>(2 * c + i);
          const int ch = D == 128 ? ((g >> 1) | ((g & 1) << 2)) ^ (t & 7) : (g >> 1) ^ ((t >> 1) & 3);
          const uint32_t at = vb + t * D + (ch << 4) + (D == 128 ? jb : (g & 1) * 8 + jb);
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[nb][i]) : "r"(at));
        }
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) {
        const uint32_t p = __byte_perm(w[nb][0], w[nb][1], 0x5140), q = __byte_perm(w[nb][0], w[nb][1], 0x7362);
        b[0][nb] = e4m3x2_to_bf162(p);
        b[1][nb] = e4m3x2_to_bf162(p >> 16);
        b[2][nb] = e4m3x2_to_bf162(q);
        b[3][nb] = e4m3x2_to_bf162(q >> 16);
      }
    }
  }
  __device__ __forceinline__ static bool not_finite(uint32_t b) {  // either 16-bit half an infinity or a NaN
    const uint32_t e = 0x7f80u;
    return (b & e) == e || ((b >> 16) & e) == e;
  }
  __device__ __forceinline__ void accumulate(uint32_t vb, const uint32_t* pf, const uint32_t* keep, bool full,
                                             bool split, int j0, int m_new, int lane) {
#pragma unroll
    for (int jb = 0; jb < kNb; jb += kB) {
      uint32_t b[kB][2];
      v_frags(vb, jb, lane, b);
      bool bad = false;
      if (!full) {
#pragma unroll
        for (int i = 0; i < kB; ++i)
#pragma unroll
          for (int nb = 0; nb < 2; ++nb) {
            b[i][nb] &= keep[nb];
            bad |= not_finite(b[i][nb]);
          }
      }
      if (!split || !__any_sync(0xffffffffu, bad)) {
#pragma unroll
        for (int i = 0; i < kB; ++i) mma_bf16(o[jb + i], pf, b[i][0], b[i][1]);
      } else {
        const int g = lane >> 2, c = lane & 3;
        for (int src = 0; src < 32; src += 4)  // the rows' distinct visible spans, row by row
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int from = __shfl_sync(0xffffffffu, lo[hf], src), to = __shfl_sync(0xffffffffu, hi[hf], src);
            const uint32_t k0 = keep_mask(0, c, j0, from, to), k1 = keep_mask(1, c, j0, from, to);
#pragma unroll
            for (int i = 0; i < kB; ++i) {
              float t[4] = {};
              mma_bf16(t, pf, b[i][0] & k0, b[i][1] & k1);
              if (g == src >> 2) {
                o[jb + i][2 * hf] += t[2 * hf];
                o[jb + i][2 * hf + 1] += t[2 * hf + 1];
              }
            }
          }
      }
    }
  }
};

template <int D, bool kFp8>
__global__ void __launch_bounds__(kThreads, 1)
    token_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                 const __grid_constant__ AttendArgs a) {
  using L = Layout<D, kFp8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (dec::smem_addr(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* empty = full + L::kStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + L::kStages);
  long long* s_pre = reinterpret_cast<long long*>(smem);  // in the ring, before it fills
  long long* s_scan = reinterpret_cast<long long*>(smem + L::kRedOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      dec::mbar_init(&full[i], 1);
      dec::mbar_init(&empty[i], kConsumers);
    }
    *abort_flag = 0;
    dec::mbar_init_fence();
  }
  dec::pdl_wait_primary();  // the batch, q and the pages may come from the kernel before
  const Range rg = token_range(a, s_pre, s_scan);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();  // the prefix sums are read; the ring may fill

  if (warp == kConsumers) {
    // ------------------------------------------------------------ producer
    int it = 0;
    bool go = true;
    TokenWalk w(a, rg);
    while (go && w.next(a)) {
      const int hi = w.hi, lo = w.lo;
      for (int t = w.t0; t < w.t1; ++t, ++it) {
        const int st = it % L::kStages, j0 = t * kTokenTile + lane * kGroup;
        const bool mine = lane < kConsumers && j0 < hi && j0 + kGroup > lo;
        int row = 0;
        if (mine) {
          const int page = max(0, load_page(a.p, a.b, w.s, j0 / a.p.page_tokens, a.status));
          row = (page * a.p.num_kv_heads + w.h) * a.p.page_tokens + j0 % a.p.page_tokens;
        }
        if (!wait_or_abort(&empty[st], ((it / L::kStages) & 1) ^ 1, a.status, abort_flag)) {
          go = false;
          break;
        }
        const int live = __popc(__ballot_sync(0xffffffffu, mine));
        if (lane == 0) dec::mbar_expect_tx(&full[st], live * (2 * L::kGroupBytes + (kFp8 ? 2 * kGroup : 0)));
        __syncwarp();
        if (mine) {
          const uint32_t kb = dec::smem_addr(smem + st * L::kStageBytes) + lane * (2 * L::kGroupBytes);
          const uint32_t vb = kb + L::kGroupBytes;
#pragma unroll
          for (int c = 0; c < (kFp8 ? 1 : D / 64); ++c) {
            tma_box(kb + c * kGroup * 128, &map_k, c * 64, row, &full[st]);
            tma_box(vb + c * kGroup * 128, &map_v, c * 64, row, &full[st]);
          }
          if (kFp8) {
            uint8_t* sc = smem + L::kScaleOff + st * 2 * kTokenTile + lane * kGroup;
            dec::bulk_g2s(sc, a.p.k_scale + row, kGroup, &full[st]);
            dec::bulk_g2s(sc + kTokenTile, a.p.v_scale + row, kGroup, &full[st]);
          }
        }
      }
    }
    // no copy may still be writing this CTA's shared memory when it exits
    for (int j = max(0, it - L::kStages); j < it; ++j)
      dec::mbar_wait(&full[j % L::kStages], (j / L::kStages) & 1, a.status);
  } else {
    // ------------------------------------------------------------ consumers
    float* red = reinterpret_cast<float*>(smem + L::kRedOff);
    float* ml = reinterpret_cast<float*>(smem + L::kMlOff);
    int it = 0;
    int4 begun = make_int4(-1, 0, 0, 0);
    TokenWalk w(a, rg);
    Warp<D, kFp8> ws;
    while (w.next(a)) {
      ws.begin(a, w.q, w.h, lane);
      const int hi = w.hi, lo = w.lo;
      // every row sees [all_lo, all_hi): the first new token's end, the last one's start
      const Span first = visible(a, w.q, 0), last = visible(a, w.q, max(0, w.q.m - 1));
      for (int t = w.t0; t < w.t1; ++t, ++it) {
        const int st = it % L::kStages, j0 = t * kTokenTile + warp * kGroup;
        const bool live = wait_or_abort(&full[st], (it / L::kStages) & 1, a.status, abort_flag);
        if (live && j0 < hi && j0 + kGroup > lo) {
          const uint32_t kb = dec::smem_addr(smem + st * L::kStageBytes) + warp * (2 * L::kGroupBytes);
          const uint8_t* sc = smem + L::kScaleOff + st * 2 * kTokenTile + warp * kGroup;
          ws.group(kb, kb + L::kGroupBytes, sc, sc + kTokenTile, j0, j0 >= last.lo && j0 + kGroup <= first.hi, w.q.m,
                   lane);
        }
        __syncwarp();
        if (lane == 0) dec::mbar_arrive(&empty[st]);
      }
      // join the eight warps, four rows at a time
      const int g = lane >> 2, c = lane & 3;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float l = ws.l[hf];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (c == 0) {
          ml[(warp * 16 + g + 8 * hf) * 2] = ws.m[hf];
          ml[(warp * 16 + g + 8 * hf) * 2 + 1] = l;
        }
      }
      bar_consumers();
      float top[2], f[2];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        top[hf] = -INFINITY;
        for (int x = 0; x < kConsumers; ++x) top[hf] = fmaxf(top[hf], ml[(x * 16 + g + 8 * hf) * 2]);
        f[hf] = ws.m[hf] == -INFINITY ? 0.0f : exp2_approx(ws.m[hf] - top[hf]);
      }
      const int rows = min(16, w.q.m * a.G);
      const bool whole = w.begins && w.ends;
      const long long slot = 2LL * blockIdx.x + w.begins;
      if (w.begins && !w.ends) begun = make_int4(w.s, w.h, 0, w.last_cta());
      for (int r0 = 0; r0 < rows; r0 += kRedRows) {
        const int hf = r0 >> 3;
        if ((g & ~(kRedRows - 1)) == (r0 & 7)) {
          float* dst = red + (warp * kRedRows + (g & (kRedRows - 1))) * L::kRowFloats;
          const float fx = hf ? f[1] : f[0];
#pragma unroll
          for (int j = 0; j < D / 8; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              dst[out_col<D, kFp8>(j, c, i)] = (hf ? ws.o[j][2 + i] : ws.o[j][i]) * fx;
        }
        bar_consumers();
        for (int e = threadIdx.x; e < kRedRows * D; e += kConsumers * 32) {
          const int rr = e / D, d = e % D, r = r0 + rr;
          if (r >= rows) continue;
          float sum = 0.0f, l = 0.0f, mm = -INFINITY;
#pragma unroll
          for (int x = 0; x < kConsumers; ++x) {
            sum += red[(x * kRedRows + rr) * L::kRowFloats + d];
            mm = fmaxf(mm, ml[(x * 16 + r) * 2]);
          }
#pragma unroll
          for (int x = 0; x < kConsumers; ++x) {
            const float mx = ml[(x * 16 + r) * 2];
            if (mx != -INFINITY) l += ml[(x * 16 + r) * 2 + 1] * exp2_approx(mx - mm);
          }
          if (whole) {
            a.out[out_at(a, w.q, w.h, r / a.G, r % a.G) + d] = __float2bfloat16(sum * inverse(l));
            if (d == 0) write_lse(a, w.q, w.h, r / a.G, r % a.G, mm, l);
          } else {
            a.part_o[(slot * kTokenRows + r) * D + d] = sum;
            if (d == 0) {
              a.part_ml[(slot * kTokenRows + r) * 2] = mm;
              a.part_ml[(slot * kTokenRows + r) * 2 + 1] = l;
            }
          }
        }
        bar_consumers();
      }
    }
    if (threadIdx.x == 0) a.desc[blockIdx.x] = begun;
  }
  dec::pdl_launch_dependents();
}

template <int D, bool kFp8>
cudaError_t launch(const AttendArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s) {
  const cudaError_t e = allow_smem<D * 2 + kFp8>(token_kernel<D, kFp8>, Layout<D, kFp8>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_dependent(token_kernel<D, kFp8>, a.grid, kThreads, Layout<D, kFp8>::kSmem, s, mk, mv, a);
}

}  // namespace

cudaError_t launch_attend_token(const AttendArgs& a, cudaStream_t s) {
  CUtensorMap mk, mv;
  if (!pages_map(&mk, a.p, a.p.k, kGroup) || !pages_map(&mv, a.p, a.p.v, kGroup)) return cudaErrorInvalidValue;
  const bool fp8 = a.p.kv_dtype == FT_KV_FP8E4M3;
  if (a.p.head_dim == 128) return fp8 ? launch<128, true>(a, mk, mv, s) : launch<128, false>(a, mk, mv, s);
  return fp8 ? launch<64, true>(a, mk, mv, s) : launch<64, false>(a, mk, mv, s);
}

}  // namespace kv
}  // namespace ft
