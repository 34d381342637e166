// Attention of a few rows over long sequences: every (sequence, key head) of
// the batch has at most 16 rows (new tokens x query heads of the group), as in
// decoding.  The work is reading K and V once: memory-bound.
//
//   out = sum_j w_j v_j / sum_j w_j,   w_j = 2^(x_j - m),  x_j = scale log2(e) q.k_j,  m >= max_j x_j - 8
//
// Quantised cache: the key's scale multiplies the score and the value's scale
// the probability (a power of two: nothing is rounded for it).
//
// Split: the batch's tiles of 64 tokens, laid end to end over (sequence, key
// head, tile), are cut into equal contiguous ranges, one per CTA and one CTA
// per SM, whatever the lengths are.  A (sequence, head) that a cut divides
// leaves partial sums (unnormalised out, m, l) in the workspace; the CTA that
// finishes the last part joins them, in tile order.  (A kernel of its own for
// that took 5 us and a launch; with every part from another CTA, 152 of them,
// one CTA reads 0.6 MB, some 5 us.)
//
// CTA: two producer warps (K, V) and kWarps consumer warps in sets.  The
// producers load a tile as swizzled TMA boxes of as many tokens as a page holds
// (64 at most: issuing a copy costs some 50 ns, and boxes of 16 tokens kept the
// consumers waiting) into a ring, several tiles at a time, each by a lane of its
// own (one after the other they kept the consumers waiting where tiles are small:
// eight e4m3 sequences of 2000-32500 tokens, head_dim 64, 24.9 -> 22.8 us); the sets take the tiles in turn, a warp a
// group of 16 tokens (with a quantised cache and at most 8 rows, two groups,
// whose chains of conversions and products interleave: 32.8 -> 31.2 us for
// eight sequences of 2000-32500 tokens).  S^T = K Q^T and O^T += V^T P^T as m16n8k16: tokens
// (then head_dim) are the 16 rows, so that 8 attention rows cost one block of
// columns and not a half-empty block of 16 rows.  Every warp has its own m, l
// and O; warps meet only at the end of a (sequence, head).  mma.sync is enough
// here: the path is bound by HBM and by what a code's expansion costs, not by
// the tensor pipe, and S^T's fragments become P^T's by one transposition of 8 x
// 8 registers.
//
// Quantised cache: codes are expanded in registers (exact), keys to fp16, the
// cheaper conversion, values to bf16, whose range P needs: a probability keeps
// its 8 bits however small it is.  The contraction order over head_dim is free
// as long as Q uses the same, and so are the order of tokens and of output
// columns; they are chosen so that each lane reads 16 consecutive bytes of a
// row, without bank conflicts.  Q is scaled per row by a power of two to [1, 2)
// before it is rounded to fp16, so that no value leaves fp16's range: q
// elements below 2^-14 of the row's largest lose bits that weigh less than
// 2^-25 of it.
//
// Bound: HBM.  64 bf16 sequences of 301-8000 tokens (head_dim 128, 8 key heads):
// 99.9 us, 6.2 TB/s.  Where a CTA's share is small its fixed cost shows (batch,
// cut, first page and tile 4 us, the end of a sequence and head 3 us), and with
// codes their expansion: eight e4m3 sequences of 2000-32500 tokens, 4 key heads, 27.5 us, 3.6 TB/s;
// one bf16 sequence of 1021 tokens 9 us, start and join.
#include <cuda.h>

#include "decode_common.h"
#include "kv_attend.h"

namespace ft {
namespace kv {
namespace {

constexpr int kGroup = 16;
constexpr float kGrow = 8.0f;  // log2 of the growth of a row's maximum that its sums' scale may lag behind

// NB: blocks of 8 rows.  Eight warps: with twelve or sixteen the quantised cache
// came no faster (eight e4m3 sequences of 2000-32500 tokens: 33.4, 34.5, 44 us).
template <int D, bool kFp8, int NB>
struct Layout {
  static constexpr int kWarps = 8;
  static constexpr int kGroups = kFp8 && NB == 1 ? 2 : 1;          // groups of a warp: independent chains to interleave
  static constexpr int kSet = kTokenTile / (kGroup * kGroups);     // warps of a set
  static constexpr int kSets = kWarps / kSet;
  static constexpr int kThreads = (kWarps + 2) * 32;
  static constexpr int kLine = kFp8 ? D : 128;                     // bytes of a token's row in a box
  static constexpr int kBoxes = kFp8 ? 1 : D / 64;                 // boxes side by side: 64 bf16 of a row each
  static constexpr int kHalfBytes = kTokenTile * kLine * kBoxes;   // a tile's K; its V follows
  static constexpr int kStageBytes = 2 * kHalfBytes;
  static constexpr int kStages = kStageBytes >= 32768 ? 6 : 12;    // a multiple of kSets: a stage is one set's
  static constexpr int kBurst = kStages / 3;                       // tiles that a producer issues at once
  static constexpr int kRedRows = 4;                               // rows joined across the warps at a time
  static constexpr int kRowFloats = D + 4;
  static constexpr int kScaleOff = kStages * kStageBytes;
  static constexpr int kScaleBytes = kFp8 ? kStages * 2 * kTokenTile : 0;
  static constexpr int kRedOff = kScaleOff + kScaleBytes;
  static constexpr int kRedBytes = kWarps * kRedRows * kRowFloats * 4, kFacBytes = kMostCtas * 8 * NB * 4;
  static constexpr int kMlOff = kRedOff + (kRedBytes > kFacBytes ? kRedBytes : kFacBytes);
  static constexpr int kTotOff = kMlOff + kWarps * 8 * NB * 2 * 4;  // a row's maximum and 1 / sum, of all warps
  static constexpr int kBarOff = kTotOff + 8 * NB * 2 * 4;
  static constexpr int kSmem = kBarOff + 2 * kStages * 8 + 16 + 1024;  // ..., abort and odd flags
  static_assert(kStages % kSets == 0, "a set that skipped a turn of a barrier would take it for the next");
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
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ uint32_t bits(__nv_bfloat162 b) { return *reinterpret_cast<const uint32_t*>(&b); }
__device__ __forceinline__ __half2 e4m3x2_to_half2(uint32_t pair) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)pair, __NV_E4M3));
}
__device__ __forceinline__ uint32_t e4m3x2_to_bf162(uint32_t pair) {
  const float2 f = __half22float2(e4m3x2_to_half2(pair));
  return bits(__floats2bfloat162_rn(f.x, f.y));
}

// Token of row n of an 8-row block of S^T.  fp8 rows of 128 bytes: neighbouring
// rows of a quarter-warp differ in bit 2, which the swizzle turns into other
// banks.
template <int D, bool kFp8>
__device__ __forceinline__ int tok(int n) {
  return kFp8 && D == 128 ? (n >> 1) | ((n & 1) << 2) : n;
}
// Output column of row g + 8 i of block mb of O^T.
template <int D, bool kFp8>
__device__ __forceinline__ int out_col(int mb, int g, int i) {
  return !kFp8 ? 16 * mb + 8 * i + g : (D == 128 ? 16 * ((g >> 1) | ((g & 1) << 2)) : 8 * g) + 2 * mb + i;
}

template <int D, bool kFp8, int NB, int NG>
struct Warp {
  static constexpr int kKs = D / 16, kMb = D / 16;
  uint32_t qf[NB][kKs][2];
  float o[NB][kMb][4];
  float m[NB][2], l[NB][2], sc[NB][2];  // rows 8 nb + 2c, + 1: running maximum, this lane's sum, score factor
  int lo[NB][2], hi[NB][2];             // visible tokens [lo, hi) of those rows
  bool started;

  __device__ __forceinline__ void begin(const AttendArgs& a, const Seq& q, int h, int lane) {
    const int g = lane >> 2, c = lane & 3;
    started = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int r = 8 * nb + g, i = r / a.G;
      const bool ok = i < q.m;
      const __nv_bfloat16* row = a.q + (long long)(q.q0 + i) * a.qts + (long long)(h * a.G + r % a.G) * a.qhs;
      uint32_t top = 0;
#pragma unroll
      for (int ks = 0; ks < kKs; ++ks)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int d = !kFp8 ? 16 * ks + 8 * w + 2 * c : (ks < 4 ? 0 : 64) + 16 * c + 4 * (ks & 3) + 2 * w;
          const uint32_t u = ok ? __ldg(reinterpret_cast<const uint32_t*>(row + d)) : 0u;
          qf[nb][ks][w] = u;
          top = max(top, max((u << 16) & 0x7f800000u, u & 0x7f800000u));
        }
      float up = 1.0f;
      if (kFp8) {  // to fp16, the row scaled to [1, 2)
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = min(max((int)(top >> 23), 1), 253);  // infinities and NaN stay what they are
        const float down = __uint_as_float((uint32_t)(254 - e) << 23);
        up = __uint_as_float((uint32_t)e << 23);
#pragma unroll
        for (int ks = 0; ks < kKs; ++ks)
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const uint32_t u = qf[nb][ks][w];
            qf[nb][ks][w] = bits(__floats2half2_rn(dec::bf16_lo(u) * down, dec::bf16_hi(u) * down));
          }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int rj = 8 * nb + 2 * c + j, ij = rj / a.G;
        const Span v = visible(a, q, ij < q.m ? ij : 0);
        lo[nb][j] = v.lo;
        hi[nb][j] = ij < q.m ? v.hi : 0;
        m[nb][j] = -INFINITY;
        l[nb][j] = 0.0f;
        sc[nb][j] = a.scale_log2 * __shfl_sync(0xffffffffu, up, (2 * c + j) * 4);
      }
#pragma unroll
      for (int mb = 0; mb < kMb; ++mb) o[nb][mb][0] = o[nb][mb][1] = o[nb][mb][2] = o[nb][mb][3] = 0.0f;
    }
  }

  // NG groups: tokens j0 .. j0 + 16 NG - 1 at shared addresses kb, vb (rows of
  // kLine bytes); ksc, vsc their scale bytes.  full: every row sees all of them.
  __device__ __forceinline__ void group(uint32_t kb, uint32_t vb, const uint8_t* ksc, const uint8_t* vsc, int j0,
                                        bool full, int lane) {
    const int g = lane >> 2, c = lane & 3;
    float s[NG][NB][4] = {};
    float vs[NG][2];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      if constexpr (!kFp8) {
        const int t = 16 * n + (lane & 15), ch = lane >> 4;
#pragma unroll
        for (int ks = 0; ks < kKs; ++ks) {
          uint32_t k[4];
          ldsm4(k, kb + (ks >> 2) * (kTokenTile * 128) + t * 128 + (((2 * (ks & 3) + ch) ^ (t & 7)) << 4));
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mma_bf16(s[n][nb], k, qf[nb][ks][0], qf[nb][ks][1]);
        }
      } else {
#pragma unroll
        for (int hf = 0; hf < D / 64; ++hf) {
          uint32_t w[2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int t = 16 * n + 8 * i + tok<D, kFp8>(g);
            const int phys = D == 128 ? (c + 4 * hf) ^ (t & 7) : c ^ ((t >> 1) & 3);
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3])
                         : "r"(kb + t * D + (phys << 4)));
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t f[4] = {bits(e4m3x2_to_half2(w[0][k] & 0xffffu)), bits(e4m3x2_to_half2(w[1][k] & 0xffffu)),
                                   bits(e4m3x2_to_half2(w[0][k] >> 16)), bits(e4m3x2_to_half2(w[1][k] >> 16))};
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma_f16(s[n][nb], f, qf[nb][hf * 4 + k][0], qf[nb][hf * 4 + k][1]);
          }
        }
      }
    }
    // scores in the log2 domain; s[n][nb][2 i + j]: token 16 n + 8 i + tok(g), row 8 nb + 2c + j
    bool grown = !started;
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = 16 * n + 8 * i + tok<D, kFp8>(g);
        float kf = 1.0f;
        vs[n][i] = 1.0f;
        if (kFp8) {
          kf = scale_of(ksc[t]);
          vs[n][i] = scale_of(vsc[t]);
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float x = s[n][nb][2 * i + j] * sc[nb][j];
            if (kFp8) x *= kf;
            if (!full && (j0 + t < lo[nb][j] || j0 + t >= hi[nb][j])) x = -INFINITY;
            s[n][nb][2 * i + j] = x;
            grown |= x > m[nb][j] + kGrow;
          }
      }
    if (__any_sync(0xffffffffu, grown)) {
      started = true;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float top = m[nb][j];
#pragma unroll
          for (int n = 0; n < NG; ++n) top = fmaxf(top, fmaxf(s[n][nb][j], s[n][nb][2 + j]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          const float f = top > m[nb][j] ? exp2_approx(m[nb][j] - top) : 1.0f;
          m[nb][j] = top;
          l[nb][j] *= f;
#pragma unroll
          for (int mb = 0; mb < kMb; ++mb) {
            o[nb][mb][j] *= f;
            o[nb][mb][2 + j] *= f;
          }
        }
    }
    uint32_t pf[NG][NB][2];
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float w[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float x = s[n][nb][2 * i + j], base = m[nb][j] == -INFINITY ? 0.0f : m[nb][j];
            w[j] = exp2_approx(x - base);
            l[nb][j] += w[j];
            if (kFp8) w[j] = x == -INFINITY ? 0.0f : w[j] * vs[n][i];  // an unseen token's scale may be NaN
          }
          pf[n][nb][i] = transpose8(bits(__floats2bfloat162_rn(w[0], w[1])));
        }
#pragma unroll
    for (int n = 0; n < NG; ++n) accumulate(vb, n, pf[n], lane);
  }
  __device__ __forceinline__ void product(int mb, const uint32_t* v, const uint32_t (*pf)[2]) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) mma_bf16(o[nb][mb], v, pf[nb][0], pf[nb][1]);
  }
  // O^T += V^T P^T
  __device__ __forceinline__ void accumulate(uint32_t vb, int n, const uint32_t (*pf)[2], int lane) {
    const int g = lane >> 2, c = lane & 3;
    if (!kFp8) {
      const int t = 16 * n + (lane & 7) + ((lane >> 4) << 3), ch = (lane >> 3) & 1;
#pragma unroll
      for (int mb = 0; mb < kMb; ++mb) {
        uint32_t v[4];
        ldsm4t(v, vb + (mb >> 2) * (kTokenTile * 128) + t * 128 + (((2 * (mb & 3) + ch) ^ (t & 7)) << 4));
        product(mb, v, pf);
      }
      return;
    }
    // this lane's 16 (8) codes of the four tokens of its fragments
    constexpr int kW = D / 32;
    uint32_t w[4][kW];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 16 * n + 8 * (i >> 1) + tok<D, kFp8>(2 * c + (i & 1));
      if (D == 128) {
        const uint32_t at = vb + t * D + ((((g >> 1) | ((g & 1) << 2)) ^ (t & 7)) << 4);
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][kW - 2]), "=r"(w[i][kW - 1])
                     : "r"(at));
      } else {
        const uint32_t at = vb + t * D + (((g >> 1) ^ ((t >> 1) & 3)) << 4) + (g & 1) * 8;
        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[i][0]), "=r"(w[i][1]) : "r"(at));
      }
    }
#pragma unroll
    for (int k = 0; k < kW; ++k) {
      // bytes 0..3 of the word, each of a pair of tokens
      const uint32_t a0 = __byte_perm(w[0][k], w[1][k], 0x5140), a1 = __byte_perm(w[0][k], w[1][k], 0x7362);
      const uint32_t b0 = __byte_perm(w[2][k], w[3][k], 0x5140), b1 = __byte_perm(w[2][k], w[3][k], 0x7362);
      uint32_t v[4] = {e4m3x2_to_bf162(a0 & 0xffffu), e4m3x2_to_bf162(a0 >> 16), e4m3x2_to_bf162(b0 & 0xffffu),
                       e4m3x2_to_bf162(b0 >> 16)};
      product(2 * k, v, pf);
      uint32_t u[4] = {e4m3x2_to_bf162(a1 & 0xffffu), e4m3x2_to_bf162(a1 >> 16), e4m3x2_to_bf162(b1 & 0xffffu),
                       e4m3x2_to_bf162(b1 >> 16)};
      product(2 * k + 1, u, pf);
    }
  }
};

// A group at the edge of what the rows see, by its warp.  vg: its V in the ring.
// Tokens [r0, r1) of it are seen by some row; the others hold anything (a page's
// unused end): their V becomes zero.  Of tokens that some rows see and others do
// not (outside [a0, a1)), bf16 values that are not finite become zero too, lest 0
// * V reach the others; the rows that see them add them in the end.  (A scale of
// NaN meets no unseen row's probability; codes of NaN: mend_codes.)  Returns
// whether there were any.
template <int D, bool kFp8, int kRowsHeld>
__device__ __noinline__ bool mend(uint8_t* vg, int r0, int r1, int a0, int a1, int lane) {
  constexpr int kLine = kFp8 ? D : 128, kBoxes = kFp8 ? 1 : D / 64, kPer = kLine / 16;
  bool odd = false;
  for (int i = lane; i < kRowsHeld * kPer * kBoxes; i += 32) {
    const int r = i / kPer % kRowsHeld, box = i / (kPer * kRowsHeld);
    uint4* at = reinterpret_cast<uint4*>(vg + box * kTokenTile * kLine + r * kLine + i % kPer * 16);
    if (r < r0 || r >= r1) {
      *at = make_uint4(0u, 0u, 0u, 0u);
    } else if (!kFp8 && (r < a0 || r >= a1)) {
      uint4 v = *at;
      uint32_t* x = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
      for (int k = 0; k < 4; ++k) {  // an exponent of all ones carries into the sign's place
        const uint32_t bad = ((x[k] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
        odd |= bad != 0u;
        x[k] &= ~((bad & 0x8000u ? 0xffffu : 0u) | (bad & 0x80000000u ? 0xffff0000u : 0u));
      }
      *at = v;
    }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the ring's next copies come after these writes
  return __any_sync(0xffffffffu, odd);
}
// The quantised cache's part of that, for several new tokens: codes of NaN become
// zero.  (Apart from mend, where it made one new token's call slower: 27.4 -> 27.7 us
// for eight sequences.  Four new tokens of 16 sequences of 500-9000 tokens: 44.4 -> 45.4.)
template <int D, int kRowsHeld>
__device__ __noinline__ bool mend_codes(uint8_t* vg, int r0, int r1, int a0, int a1, int lane) {
  bool odd = false;
  auto take = [&](int from, int to) {
    uint32_t* x = reinterpret_cast<uint32_t*>(vg);
#pragma unroll 1
    for (int i = from * (D / 4) + lane; i < to * (D / 4); i += 32) {
      const uint32_t nan = (x[i] & 0x7f7f7f7fu) + 0x01010101u & 0x80808080u;
      if (nan == 0u) continue;
      x[i] &= ~(nan / 128 * 255);
      odd = true;
    }
  };
  r0 = max(r0, 0);
  r1 = min(r1, kRowsHeld);
  take(r0, min(r1, a0));
  take(max(r0, a1), r1);
  return __any_sync(0xffffffffu, odd);  // (mend, which follows, has the fence)
}
// Sum of the values (codes) of tokens [from, to) outside [a0, a1) that are not finite, columns d and d + 1.
template <int D, bool kFp8>
__device__ __noinline__ float2 not_finite(const AttendArgs& a, int s, int h, int from, int to, int a0, int a1, int d) {
  float2 sum = make_float2(0.0f, 0.0f);
  for (int j = from; j < to; ++j) {
    if (j >= a0 && j < a1) continue;
    const int page = max(0, load_page(a.p, a.b, s, j / a.p.page_tokens, a.status));
    const long long at = (((long long)page * a.p.num_kv_heads + h) * a.p.page_tokens + j % a.p.page_tokens) * D + d;
    const float2 v = kFp8 ? __half22float2(e4m3x2_to_half2(*reinterpret_cast<const uint16_t*>(
                                static_cast<const uint8_t*>(a.p.v) + at)))
                          : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(
                                static_cast<const __nv_bfloat16*>(a.p.v) + at));
    if (!isfinite(v.x)) sum.x += v.x;
    if (!isfinite(v.y)) sum.y += v.y;
  }
  return sum;
}

template <int D, bool kFp8, int NB>
__global__ void __launch_bounds__(Layout<D, kFp8, NB>::kThreads, 1)
    token_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                 const __grid_constant__ AttendArgs a) {
  using L = Layout<D, kFp8, NB>;
  constexpr int kRows = 8 * NB, kConsumers = L::kWarps * 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (dec::smem_addr(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* empty = full + L::kStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + L::kStages);
  volatile int* odd_flag = abort_flag + 1;  // a mended group of this (sequence, head) had values that are not finite
  long long* s_pre = reinterpret_cast<long long*>(smem);  // in the ring, before it fills
  long long* s_scan = reinterpret_cast<long long*>(smem + L::kRedOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      dec::mbar_init(&full[i], 2);
      dec::mbar_init(&empty[i], L::kSet);
    }
    *abort_flag = 0;
    *odd_flag = 0;
    dec::mbar_init_fence();
  }
  dec::pdl_wait_primary();  // the batch, q and the pages may come from the kernel before
  const Range rg = token_range(a, s_pre, s_scan);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();  // the prefix sums are read; the ring may fill

  if (warp >= L::kWarps) {
    // ------------------------------------------------------------ producers
    // Lane l has the page row of box l of the next 32 boxes, and issues its copies.
    const bool v = warp > L::kWarps;
    const CUtensorMap* map = v ? &map_v : &map_k;
    const uint8_t* scales = v ? a.p.v_scale : a.p.k_scale;
    const int br = min(a.p.page_tokens, kTokenTile), per = kTokenTile / br;  // tokens of a box, boxes of a tile
    int it = 0;
    bool go = true;
    TokenWalk w(a, rg);
    while (go && w.next(a)) {
      const int hi = w.hi, lo = w.lo, t1 = w.t1;
      auto row_of = [&](int t) {  // of this lane's box, from tile t on; -1: no row sees a token of it
        const int j0 = t * kTokenTile + lane * br;
        if (j0 >= t1 * kTokenTile || j0 >= hi || j0 + br <= lo) return -1;
        const int page = max(0, load_page(a.p, a.b, w.s, j0 / a.p.page_tokens, a.status));
        return (page * a.p.num_kv_heads + w.h) * a.p.page_tokens + j0 % a.p.page_tokens;
      };
      int ahead = row_of(w.t0);
      for (int tb = w.t0; tb < t1 && go; tb += 32 / per) {
        const int row = ahead, te = min(t1, tb + 32 / per);
        ahead = row_of(te);  // on its way while these are issued
        const unsigned live = __ballot_sync(0xffffffffu, row >= 0);
        for (int t = tb; t < te && go;) {
          const int burst = min(te - t, L::kBurst), mine = lane / per - (t - tb);  // this lane's tile of the burst
          const bool in = mine >= 0 && mine < burst;
          const int i = in ? it + mine : it, st = i % L::kStages;
          go = wait_or_abort(&empty[st], ((i / L::kStages) & 1) ^ 1, a.status, abort_flag);
          if (!go) break;
          if (in && lane % per == 0)
            dec::mbar_expect_tx(&full[st],
                                __popc(live >> lane & ((1u << per) - 1u)) * br * (L::kLine * L::kBoxes + (kFp8 ? 1 : 0)));
          __syncwarp();
          if (in && row >= 0) {
            const int at = lane % per * br;
            const uint32_t dst = dec::smem_addr(smem + st * L::kStageBytes) + v * L::kHalfBytes + at * L::kLine;
#pragma unroll
            for (int c = 0; c < L::kBoxes; ++c) tma_box(dst + c * kTokenTile * 128, map, c * 64, row, &full[st]);
            if (kFp8)
              dec::bulk_g2s(smem + L::kScaleOff + (2 * st + v) * kTokenTile + at, scales + row, br, &full[st]);
          }
          t += burst;
          it += burst;
        }
      }
    }
    // no copy may still be writing this CTA's shared memory when it exits
    for (int j = max(0, it - L::kStages); j < it; ++j)
      if (!dec::mbar_wait(&full[j % L::kStages], (j / L::kStages) & 1, a.status)) break;  // a second: long enough for all
  } else {
    // ------------------------------------------------------------ consumers
    float* red = reinterpret_cast<float*>(smem + L::kRedOff);
    float2* ml = reinterpret_cast<float2*>(smem + L::kMlOff);
    float2* tot = reinterpret_cast<float2*>(smem + L::kTotOff);
    auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory"); };
    const int set = warp / L::kSet, grp = warp % L::kSet * L::kGroups;
    int it = 0;
    TokenWalk w(a, rg);
    Warp<D, kFp8, NB, L::kGroups> ws;
    while (w.next(a)) {
      ws.begin(a, w.q, w.h, lane);
      const int hi = w.hi, lo = w.lo;
      // every row sees [last.lo, first.hi): from the last new token's start to the first one's end
      const Span first = visible(a, w.q, 0), last = visible(a, w.q, max(0, w.q.m - 1));
      // this set's tiles: those whose place in the CTA's sequence of tiles is set modulo kSets
      const int first_turn = (set + L::kSets - it % L::kSets) % L::kSets;
      int st = (it + first_turn) % L::kStages;
      uint32_t ph = (it + first_turn) / L::kStages & 1;
      for (int t = w.t0 + first_turn; t < w.t1; t += L::kSets) {
        const int j0 = t * kTokenTile + grp * kGroup;
        const bool live = wait_or_abort(&full[st], ph, a.status, abort_flag);
        if (live && j0 < hi && j0 + kGroup * L::kGroups > lo) {
          uint8_t* kg = smem + st * L::kStageBytes + grp * kGroup * L::kLine;
          const uint8_t* sc = smem + L::kScaleOff + st * 2 * kTokenTile + grp * kGroup;
          const bool whole_group = j0 >= last.lo && j0 + kGroup * L::kGroups <= first.hi;  // every row sees all of it
          if (!whole_group) {
            uint8_t* vg = kg + L::kHalfBytes;
            const int a0 = last.lo - j0, a1 = first.hi - j0;
            if (kFp8 && w.q.m > 1 && mend_codes<D, kGroup * L::kGroups>(vg, lo - j0, hi - j0, a0, a1, lane)) *odd_flag = 1;
            if (mend<D, kFp8, kGroup * L::kGroups>(vg, lo - j0, hi - j0, a0, a1, lane)) *odd_flag = 1;
            __syncwarp();
          }
          const uint32_t kb = dec::smem_addr(kg);
          ws.group(kb, kb + L::kHalfBytes, sc, sc + kTokenTile, j0, whole_group, lane);
        }
        __syncwarp();
        if (lane == 0) dec::mbar_arrive(&empty[st]);
        st += L::kSets;
        if (st >= L::kStages) {
          st -= L::kStages;
          ph ^= 1;
        }
      }
      it += w.t1 - w.t0;
      // join the warps, kRedRows rows at a time
      const int g = lane >> 2, c = lane & 3;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float l = ws.l[nb][j];
          l += __shfl_xor_sync(0xffffffffu, l, 4);
          l += __shfl_xor_sync(0xffffffffu, l, 8);
          l += __shfl_xor_sync(0xffffffffu, l, 16);
          if (g == 0) {
            const int r = 8 * nb + 2 * c + j;
            ml[warp * kRows + r] = make_float2(ws.m[nb][j], l);
          }
        }
      sync();
      const bool odd = *odd_flag != 0;
      const int rows = min(kRows, w.q.m * a.G);
      const bool whole = w.begins && w.ends;
      const long long slot = 2LL * blockIdx.x + w.begins;
      if (threadIdx.x < rows) {  // (read after the next barrier)
        const int r = threadIdx.x;
        float mm = -INFINITY, l = 0.0f;
#pragma unroll
        for (int x = 0; x < L::kWarps; ++x) mm = fmaxf(mm, ml[x * kRows + r].x);
#pragma unroll
        for (int x = 0; x < L::kWarps; ++x) {
          const float2 y = ml[x * kRows + r];
          l += y.y * (y.x == -INFINITY ? 0.0f : exp2_approx(y.x - mm));  // (only scores of NaN: y.y is NaN, and so is l)
        }
        tot[r] = make_float2(mm, inverse(l));
        if (whole) {
          write_lse(a, w.q, w.h, r / a.G, r % a.G, mm, l);
        } else {
          a.part_ml[(slot * kTokenRows + r) * 2] = mm;
          a.part_ml[(slot * kTokenRows + r) * 2 + 1] = l;
        }
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float f[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float top = -INFINITY;
#pragma unroll
          for (int x = 0; x < L::kWarps; ++x) top = fmaxf(top, ml[x * kRows + 8 * nb + 2 * c + j].x);
          f[j] = ws.m[nb][j] == -INFINITY ? 0.0f : exp2_approx(ws.m[nb][j] - top);
        }
        for (int r0 = 8 * nb; r0 < min(rows, 8 * nb + 8); r0 += L::kRedRows) {
          if ((2 * c & ~(L::kRedRows - 1)) == (r0 & 7)) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float* dst = red + (warp * L::kRedRows + ((2 * c + j) & (L::kRedRows - 1))) * L::kRowFloats;
#pragma unroll
              for (int mb = 0; mb < D / 16; ++mb)
#pragma unroll
                for (int i = 0; i < 2; ++i) dst[out_col<D, kFp8>(mb, g, i)] = ws.o[nb][mb][2 * i + j] * f[j];
            }
          }
          sync();
          if (odd && threadIdx.x == 0) *odd_flag = 0;  // (everyone has read it)
          for (int e = threadIdx.x * 2; e < L::kRedRows * D; e += kConsumers * 2) {
            const int rr = e / D, d = e % D, r = r0 + rr;
            if (r >= rows) continue;
            float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int x = 0; x < L::kWarps; ++x) {
              const float2 y = *reinterpret_cast<const float2*>(&red[(x * L::kRedRows + rr) * L::kRowFloats + d]);
              sum.x += y.x;
              sum.y += y.y;
            }
            if (odd) {
              const Span v = visible(a, w.q, r / a.G);
              const float2 add = not_finite<D, kFp8>(a, w.s, w.h, max(v.lo, w.t0 * kTokenTile), min(v.hi, w.t1 * kTokenTile),
                                               last.lo, first.hi, d);
              sum.x += add.x;
              sum.y += add.y;
            }
            if (whole) {
              const float inv = tot[r].y;
              *reinterpret_cast<__nv_bfloat162*>(a.out + out_at(a, w.q, w.h, r / a.G, r % a.G) + d) =
                  __floats2bfloat162_rn(sum.x * inv, sum.y * inv);
            } else {
              *reinterpret_cast<float2*>(a.part_o + (slot * kTokenRows + r) * D + d) = sum;
            }
          }
          sync();
        }
      }
      if (whole) continue;
      // the last of the parts joins them
      const int c0 = w.first_cta(a), parts = w.last_cta(a) - c0 + 1;
      __threadfence();
      sync();
      if (threadIdx.x == 0) {
        const bool all = atomicAdd(&a.counter[c0], 1u) + 1u == (unsigned)parts;
        if (all) a.counter[c0] = 0u;
        tot[0].x = all ? 1.0f : 0.0f;
      }
      sync();
      const bool join = tot[0].x != 0.0f;
      sync();
      if (!join) continue;
      __threadfence();
      // part i: CTA c0's last slot, then the first slot of each CTA after it
      auto part = [&](int i, int r) { return (long long)(2 * (c0 + i) + (i == 0)) * kTokenRows + r; };
      float* fac = red;  // [parts][kRows] 2^(m_i - m)
      for (int r = warp; r < rows; r += L::kWarps) {
        float mm = -INFINITY, l = 0.0f;
        for (int i = lane; i < parts; i += 32) mm = fmaxf(mm, __ldcg(&a.part_ml[part(i, r) * 2]));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
        for (int i = lane; i < parts; i += 32) {
          const float2 y = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + part(i, r));
          const float f = y.x == -INFINITY ? 0.0f : exp2_approx(y.x - mm);
          fac[i * kRows + r] = f;
          l += f * y.y;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (lane == 0) {
          tot[r] = make_float2(mm, inverse(l));
          write_lse(a, w.q, w.h, r / a.G, r % a.G, mm, l);
        }
      }
      sync();
      for (int e = threadIdx.x * 4; e < rows * D; e += kConsumers * 4) {
        const int r = e / D, d = e % D;
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const float4* at = reinterpret_cast<const float4*>(a.part_o + ((2LL * c0 + 1) * kTokenRows + r) * D + d);
#pragma unroll 8
        for (int i = 0; i < parts; ++i) {
          const float4 y = __ldcg(at + (i ? (2 * i - 1) * (kTokenRows * D / 4) : 0));
          const float f = fac[i * kRows + r];
          sum.x += f * y.x;
          sum.y += f * y.y;
          sum.z += f * y.z;
          sum.w += f * y.w;
        }
        const float inv = tot[r].y;
        __nv_bfloat162* out =
            reinterpret_cast<__nv_bfloat162*>(a.out + out_at(a, w.q, w.h, r / a.G, r % a.G) + d);
        out[0] = __floats2bfloat162_rn(sum.x * inv, sum.y * inv);
        out[1] = __floats2bfloat162_rn(sum.z * inv, sum.w * inv);
      }
      sync();
    }
  }
  dec::pdl_launch_dependents();
}

template <int D, bool kFp8, int NB>
cudaError_t launch(const AttendArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s) {
  using L = Layout<D, kFp8, NB>;
  const cudaError_t e = allow_smem<(D * 2 + kFp8) * 2 + NB - 1>(token_kernel<D, kFp8, NB>, L::kSmem);
  if (e != cudaSuccess) return e;
  return launch_dependent(token_kernel<D, kFp8, NB>, a.grid, L::kThreads, L::kSmem, s, mk, mv, a);
}
template <int D, bool kFp8>
cudaError_t launch_rows(const AttendArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s) {
  return a.small <= 8 ? launch<D, kFp8, 1>(a, mk, mv, s) : launch<D, kFp8, 2>(a, mk, mv, s);
}

}  // namespace

cudaError_t launch_attend_token(const AttendArgs& a, cudaStream_t s) {
  CUtensorMap mk, mv;
  const int box = a.p.page_tokens < kTokenTile ? a.p.page_tokens : kTokenTile;
  if (!pages_map(&mk, a.p, a.p.k, box) || !pages_map(&mv, a.p, a.p.v, box)) return cudaErrorInvalidValue;
  const bool fp8 = a.p.kv_dtype == FT_KV_FP8E4M3;
  if (a.p.head_dim == 128) return fp8 ? launch_rows<128, true>(a, mk, mv, s) : launch_rows<128, false>(a, mk, mv, s);
  return fp8 ? launch_rows<64, true>(a, mk, mv, s) : launch_rows<64, false>(a, mk, mv, s);
}

}  // namespace kv
}  // namespace ft
