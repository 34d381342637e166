// Attention of many rows (prompt chunks, several new tokens) over the paged
// cache on the 5th-generation tensor cores.
//
//   S = Q K^T,  P = 2^(x - m),  O += P V,  out = O / sum P
//
// with a running maximum m per row and x = scale log2(e) S.  Quantised cache: a
// code times its power-of-two scale is a bf16 value, so its tiles are expanded
// to exactly that and the rest is the same.
//
// Item: a tile of 128 tokens for a row block of one (sequence, key head).  A
// row block is two sub-tiles of up to 128 rows, each the query heads of the
// group of 128 / G consecutive new tokens: the heads share the loaded K and V,
// and so do the sub-tiles.  The batch's items, laid end to end, are cut into
// equal ranges, one per CTA; a row block that a cut divides leaves partial sums,
// which the CTA that began it joins, or combine_kernel.  Each sub-tile has its own score tile, output
// accumulator and softmax warpgroup:
//
//   warps 0-3, 4-7   softmax of sub-tile 0, 1: per tile read S from TMEM (a
//                    thread per row), mask, exponentiate, write P (bf16) over
//                    S in TMEM; at the end scale O and store it, transposed
//                    through shared memory so that a store fills its lines
//   warp 8           walks the CTA's row blocks, tells the other warps of each
//                    through a small ring, and loads K and V tiles into another,
//                    one TMA box per page (or half page row), 128-byte swizzled
//   warp 9           tcgen05.mma: S_w = Q_w K^T (M 128, N 128), O_w += P_w V
//                    with P read from TMEM and V as it lies (token-major)
//   warp 10          Q of both sub-tiles by TMA as soon as the block before has
//                    its last score tile
//   warps 12-19      quantised cache: expand the codes of a raw ring, times their
//                    scales, into bf16 tiles of the layout that the MMA reads
//
// The MMA order PV_0(j-1) S_0(j) PV_1(j-1) S_1(j) keeps the tensor pipe on one
// sub-tile while the other's softmax runs; P comes in two halves, so that PV
// starts on the first while the second is made.  S_w(j)'s completion implies
// PV_w(j-1)'s, so the softmax of tile j may rescale O_w; it does so only when
// a row's maximum has grown by more than 2^8 since O_w's scale was set (P is
// then at most 2^8, and the final division removes any scale).
//
// Bound: the tensor pipe, 4 D flops per (row, token), if the softmax keeps up: a
// tile's exponentials take as long as its products (head_dim 128; twice as long
// with 64).  Measured: a prompt chunk of 16,384 tokens, 16 query heads over 4, bf16,
// 751-815 us, 1350-1465 TFLOP/s (the clock varies with the power); 2048 e4m3 tokens
// after 14,336, 227 us, 1135 TFLOP/s (expansion shares the issue slots: 64% used);
// five chunks of 501-1501 tokens under a window of 1000, 12 heads, head_dim 64, 46
// us, 230 TFLOP/s: 11 tiles a CTA, half of them at an edge, which take twice as
// long, after a start of 4 us (batch, cut, first block) and 1.5 us for the first tile.
#include "kv_attend.h"

namespace ft {
namespace kv {
namespace {

constexpr int kSub = kSubRows;
constexpr int kTile = 128;                    // tokens per tile
constexpr int kTmemCols = 512;                // S0 | S1 | O0 | O1, 128 columns each
constexpr int kUnits = 4;                     // ring of row blocks
// A block's fixed cost, in tiles, for the cut.  (2 / 3 / 4: a prompt of 16,384 tokens
// 752 / 733 / 740-750 us, of 4096 72.6 / 72.6 / 70.4, of 1024 27.1 / 28.7 / 28.6; windows
// 46.6 / 47 / 49; 8 is slower throughout.)
constexpr int kBlockItems = 3;
constexpr float kGrow = 8.0f;                 // log2 of the growth that O's scale may lag behind
constexpr int kBfThreads = 384, kFpThreads = 640;
// Registers of the quantised cache's warps (softmax, walker to Q, expanding),
// within what the block is launched with, 640 x 96.
constexpr int kFpSoft = 136, kFpRest = 80, kFpCvt = 64;
static_assert(256 * (kFpSoft + kFpCvt) + 128 * kFpRest <= kFpThreads * 96, "registers");
constexpr int kCvtWarps = 8;

template <int D, bool kFp8>
struct Layout {
  static constexpr int kQBytes = 2 * kSub * D * 2;
  static constexpr int kTileBytes = kTile * D * 2;                      // a K or V tile as the MMA reads it
  static constexpr int kRawBytes = kFp8 ? kTile * D : 0;
  static constexpr int kStages = (kFp8 ? 3 : 4) * (128 / D);
  static constexpr int kRaw = kFp8 ? 2 * (128 / D) : 0;
  static constexpr int kRingOff = kQBytes;
  static constexpr int kRawOff = kRingOff + kStages * kTileBytes;
  static constexpr int kLine = kFp8 ? 64 : 128;                         // bytes of a row in a softmax warp's staging
  static constexpr int kOutOff = kRawOff + kRaw * kRawBytes;
  static constexpr int kBarOff = kOutOff + 8 * 32 * kLine;
  static constexpr int kBars = 2 * kStages + 2 * kRaw + 2 * kUnits + 14 + 1;
  static constexpr int kUnitOff = kBarOff + (kBars * 8 + 15) / 16 * 16;
  static constexpr int kMiscOff = kUnitOff + kUnits * 96;
  static constexpr int kSmem = kMiscOff + 16 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kStages * kTileBytes >= (kMaxSeqs + 1) * 8 + 1024, "the prefix sums fit the ring before it fills");
};

// ---------------------------------------------------------------- PTX wrappers
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(dec::smem_addr(bar))
               : "memory");
}
// One thread of the warp, chosen so that the compiler knows the branch is uniform.
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// Shared-memory matrix descriptors, 128-byte swizzle, rows of 128 bytes, 8-row
// groups 1024 bytes apart: the low word holds the address (in 16 bytes) and the
// leading offset, the high word is a constant.  K-major (Q, K): the leading
// offset is not used.  N-major (V: a row is a token, 64 of head_dim wide): it
// leads to the next 64 columns, the next half of the tile.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lead = 16) { return (saddr >> 4) | (lead >> 4) << 16; }
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t ad, uint32_t bd, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "r"(ad), "r"(bd), "r"(idesc), "r"((uint32_t)acc), "r"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t at, uint32_t bd, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
      "r"(at), "r"(bd), "r"(idesc), "r"((uint32_t)acc), "r"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// 32 consecutive columns of this thread's TMEM lane; ld_wait() before use.
__device__ __forceinline__ void ld32(uint32_t t, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t));
}
__device__ __forceinline__ void st32(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
      "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(t)
      : "memory");
}
__device__ __forceinline__ void tma_box3(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(dec::smem_addr(bar))
      : "memory");
}
// kind::f16, fp32 accumulator, both operands bf16, B N-major or not.
__device__ constexpr uint32_t idesc(int N, bool b_n_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_n_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(kSub >> 4) << 24);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// ---------------------------------------------------------------- items

// A row block: what its rows see, in tokens and tiles, whole and per sub-tile.
struct Block {
  int lo, hi;            // tokens that some row sees
  int t0, t1;            // tiles of the block (at least one)
  int s0[2], s1[2];      // tiles of each sub-tile (none: s0 = s1)
  int all_lo, all_hi;    // tokens that every row sees
};
__device__ __forceinline__ Block block_of(const AttendArgs& a, const Seq& q, int rb) {
  Block b;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int i0 = (rb * 2 + w) * a.tps, i1 = min(q.m, i0 + a.tps) - 1;
    b.s0[w] = b.s1[w] = 0;
    if (i0 > i1) continue;
    const Span f = visible(a, q, i0), l = visible(a, q, i1);
    if (l.hi > f.lo) {
      b.s0[w] = f.lo / kTile;
      b.s1[w] = (l.hi + kTile - 1) / kTile;
    }
    if (w == 0) {
      b.lo = f.lo;
      b.all_hi = f.hi;
    }
    b.hi = l.hi;
    b.all_lo = l.lo;
  }
  b.t0 = b.lo / kTile;
  b.t1 = max(b.t0 + 1, (b.hi + kTile - 1) / kTile);
  return b;
}
__device__ __forceinline__ int blocks_of(const AttendArgs& a, const Seq& q) { return (q.m + 2 * a.tps - 1) / (2 * a.tps); }
__device__ __forceinline__ int tiles_of(const AttendArgs& a, const Seq& q, int rb) {
  const Block b = block_of(a, q, rb);
  return b.t1 - b.t0;
}
// Items of a block: its tiles, after kBlockItems that stand for its fixed cost.
__device__ __forceinline__ int items_of(const AttendArgs& a, const Seq& q, int rb) {
  return tiles_of(a, q, rb) + kBlockItems;
}
// Items of one head of a sequence, summed by the whole warp.
__device__ __forceinline__ long long head_items(const AttendArgs& a, const Seq& q, int lane) {
  long long n = 0;
  const int nb = blocks_of(a, q);
  for (int rb = lane; rb < nb; rb += 32) n += items_of(a, q, rb);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n;
}

// A CTA's part of a row block, as the other warps get it.
struct Unit {
  int s, h, rb;       // s < 0: no more
  int q0, m, n;
  int t0, t1;         // its tiles
  int f0[2], f1[2];   // those of them that each sub-tile has (none: f0 >= f1)
  int lo, hi, all_lo, all_hi;
  int begins, ends;
  int c0, parts;      // the block's first CTA and how many have a part
  int odd;            // some value of the part is not finite (see mend, expand)
  int pad[3];
  __device__ __forceinline__ Seq seq() const { return Seq{q0, m, n}; }
  __device__ __forceinline__ bool any(int sub) const { return f0[sub] < f1[sub]; }
  // V's tile t as the rows see it: tokens [r0, r1) of the tile are seen by some
  // row, [p0, p1) and [p2, p3) of them not by all
  struct Edge {
    int r0, r1, p0, p1, p2, p3;
  };
  __device__ __forceinline__ Edge edge(int t) const {
    Edge e;
    const int j0 = t * kTile;
    e.r0 = min(kTile, max(0, lo - j0));
    e.r1 = max(e.r0, min(kTile, hi - j0));
    e.p0 = e.r0;
    e.p1 = min(e.r1, all_lo - j0);
    e.p2 = max(e.r0, all_hi - j0);
    e.p3 = e.r1;
    return e;
  }
};
static_assert(sizeof(Unit) == 96, "Layout");

// The parts of row blocks in a CTA's range, one after the other (whole warp).
struct ChunkWalk {
  long long w, end, base, total, at;  // at: first item of the current block
  int n, s, h, rb, nb, items;
  Seq q;
  bool started;
  __device__ __forceinline__ ChunkWalk(const AttendArgs& a, const Range& r, int lane)
      : w(r.w0), end(r.w1), base(r.base), total(r.total), at(r.base), n(r.n), s(r.s), h(0), rb(0), nb(0), items(0),
        started(false) {
    if (w < end) find(a, lane);
  }
  __device__ __forceinline__ bool next(const AttendArgs& a, Unit& u) {
    for (;;) {
      if (w >= end) return false;
      if (!started) {
        started = true;
      } else {  // the range goes on: past a whole block
        at += items;
        if (++rb == nb) {
          rb = 0;
          if (++h == a.p.num_kv_heads) {
            h = 0;
            do {
              ++s;
              q = own_seq<false>(a, s);
            } while (q.m == 0);
            nb = blocks_of(a, q);
          }
        }
      }
      const Block b = block_of(a, q, rb);
      const int nt = b.t1 - b.t0;
      items = nt + kBlockItems;
      const int rel = (int)(w - at), cnt = (int)min((long long)(items - rel), end - w);
      const int r0 = max(0, rel - kBlockItems), r1 = max(0, rel + cnt - kBlockItems);
      w += cnt;
      if (r0 == r1) continue;  // only of the fixed cost
      u.s = s; u.h = h; u.rb = rb;
      u.q0 = q.q0; u.m = q.m; u.n = q.n;
      u.t0 = b.t0 + r0; u.t1 = b.t0 + r1;
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        u.f0[sub] = max(u.t0, b.s0[sub]);
        u.f1[sub] = min(u.t1, b.s1[sub]);
      }
      u.lo = b.lo; u.hi = b.hi; u.all_lo = b.all_lo; u.all_hi = b.all_hi;
      u.begins = r0 == 0;
      u.ends = r1 == nt;
      u.c0 = u.begins ? (int)blockIdx.x : cta_of(at + kBlockItems, total, n);
      u.parts = cta_of(at + items - 1, total, n) - u.c0 + 1;
      u.odd = 0;
      return true;
    }
  }
  // the head and row block of item w
  __device__ __forceinline__ void find(const AttendArgs& a, int lane) {
    long long per;
    for (;; ++s) {
      q = own_seq<false>(a, s);
      per = head_items(a, q, lane);
      if (w - base < per * a.p.num_kv_heads) break;
      base += per * a.p.num_kv_heads;
    }
    nb = blocks_of(a, q);
    h = (int)((w - base) / per);
    at = base + h * per;
    for (int r0 = 0;; r0 += 32) {
      const int mine = r0 + lane < nb ? items_of(a, q, r0 + lane) : 0;
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const unsigned past = __ballot_sync(0xffffffffu, at + incl > w);
      if (past) {
        const int l = __ffs(past) - 1;
        rb = r0 + l;
        at += __shfl_sync(0xffffffffu, incl - mine, l);
        return;
      }
      at += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
};

struct Shared {
  uint8_t* base;
  uint64_t *full, *empty, *rfull, *rempty, *ufull, *uempty;
  uint64_t *qfull, *qempty, *landed, *sfull, *pfull, *pfull2, *ofull;  // per sub-tile
  uint64_t* drain;
  Unit* unit;
  uint32_t* tmem;
  volatile int* abort_flag;
};

template <int D, bool kFp8>
__device__ __forceinline__ Shared carve(uint8_t* raw) {
  using L = Layout<D, kFp8>;
  Shared s;
  s.base = raw + ((1024u - (dec::smem_addr(raw) & 1023u)) & 1023u);
  uint64_t* b = reinterpret_cast<uint64_t*>(s.base + L::kBarOff);
  auto take = [&](int n) {
    uint64_t* r = b;
    b += n;
    return r;
  };
  s.full = take(L::kStages);
  s.empty = take(L::kStages);
  s.rfull = take(L::kRaw);
  s.rempty = take(L::kRaw);
  s.ufull = take(kUnits);
  s.uempty = take(kUnits);
  s.qfull = take(2);
  s.qempty = take(2);
  s.landed = take(2);
  s.sfull = take(2);
  s.pfull = take(2);
  s.pfull2 = take(2);
  s.ofull = take(2);
  s.drain = take(1);
  s.unit = reinterpret_cast<Unit*>(s.base + L::kUnitOff);
  s.tmem = reinterpret_cast<uint32_t*>(s.base + L::kMiscOff);
  s.abort_flag = reinterpret_cast<volatile int*>(s.tmem + 1);
  return s;
}

// A place in a ring of barriers and the parity of its turn.
template <int kN>
struct Turn {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++st == kN) {
      st = 0;
      ph ^= 1;
    }
  }
};

// A warp's view of the ring of row blocks.
struct Units {
  Turn<kUnits> at;
  // the next block, or null: no more (or the CTA has aborted)
  __device__ __forceinline__ Unit* next(const AttendArgs& a, const Shared& s) {
    if (!wait_or_abort(&s.ufull[at.st], at.ph, a.status, s.abort_flag)) return nullptr;
    Unit* u = &s.unit[at.st];
    return u->s < 0 ? nullptr : u;
  }
  __device__ __forceinline__ void done(const Shared& s, int lane) {
    __syncwarp();
    if (lane == 0) dec::mbar_arrive(&s.uempty[at.st]);
    at.next();
  }
};

// ---------------------------------------------------------------- producer

// The row blocks, and per tile K then V, the pages' boxes spread over the lanes.
template <int D, bool kFp8>
__device__ void produce(const AttendArgs& a, const Range& rg, const Shared& s, const CUtensorMap* map_k,
                        const CUtensorMap* map_v, int lane) {
  using L = Layout<D, kFp8>;
  constexpr int kSlots = kFp8 ? L::kRaw : L::kStages;
  constexpr int kHalves = kFp8 ? 1 : D / 64;
  uint64_t* full = kFp8 ? s.rfull : s.full;
  uint64_t* empty = kFp8 ? s.rempty : s.empty;
  const uint32_t ring = dec::smem_addr(s.base + (kFp8 ? L::kRawOff : L::kRingOff));
  constexpr uint32_t kBytes = kFp8 ? L::kRawBytes : L::kTileBytes;
  const int br = min(a.p.page_tokens, kTile);  // tokens of a box
  const int box = lane / kHalves, half = lane % kHalves;
  constexpr int kRowBytes = kFp8 ? D : 128;
  Turn<kSlots> at;
  Turn<kUnits> ut;
  int it = 0;
  bool go = true;
  ChunkWalk w(a, rg, lane);
  Unit u;
  while (go) {
    const bool more = w.next(a, u);
    if (!more) u.s = -1;
    if (!wait_or_abort(&s.uempty[ut.st], ut.ph ^ 1, a.status, s.abort_flag)) break;
    if (lane == 0) {
      s.unit[ut.st] = u;
      dec::mbar_arrive(&s.ufull[ut.st]);
    }
    ut.next();
    if (!more) break;
    for (int t = u.t0; t < u.t1 && go; ++t) {
      const int j0 = t * kTile + box * br;
      const bool mine = box * br < kTile && j0 < u.hi && j0 + br > u.lo;
      int row = 0;
      if (mine) {
        const int page = max(0, load_page(a.p, a.b, u.s, j0 / a.p.page_tokens, a.status));
        row = (page * a.p.num_kv_heads + u.h) * a.p.page_tokens + j0 % a.p.page_tokens;
      }
      const int live = __popc(__ballot_sync(0xffffffffu, mine));
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        if (!wait_or_abort(&empty[at.st], at.ph ^ 1, a.status, s.abort_flag)) {
          go = false;
          break;
        }
        if (lane == 0) dec::mbar_expect_tx(&full[at.st], live * br * kRowBytes);
        __syncwarp();
        if (mine)
          tma_box(ring + at.st * kBytes + half * (kTile * 128) + box * br * kRowBytes, kv ? map_v : map_k, half * 64,
                  row, &full[at.st]);
        at.next();
        ++it;
      }
    }
  }
  // no copy may still be writing this CTA's shared memory when it exits
  for (int j = max(0, it - kSlots); j < it; ++j)
    if (!dec::mbar_wait(&full[j % kSlots], (j / kSlots) & 1, a.status)) break;  // a second has passed: for all of them
}

// ---------------------------------------------------------------- V at the edge

// A bf16 tile at the edge of what the rows see, by the warpgroup whose P goes to
// it first.  Tokens that no row sees hold anything (a page's unused end, an
// evicted page): those within the MMA's 16-token steps are set to zero.  Of
// tokens that some rows see and others do not, values that are not finite are
// set to zero too, lest 0 * V reach the others; the rows that see them add them
// at the block's end.  Returns whether there were any (any thread's).
template <int D>
__device__ __forceinline__ bool mend(uint8_t* tile, const Unit::Edge& e, int tid) {
  constexpr int kPer = D / 8;
  // 16-byte chunk i of the tile (rows are mended whole, or chunk by chunk in place: the swizzle does not matter)
  auto chunk = [&](int i) {
    const int r = i / kPer, ch = i % kPer;
    return reinterpret_cast<uint4*>(tile + (ch >> 3) * (kTile * 128) + r * 128 + ((ch & 7) << 4));
  };
  auto zero = [&](int r0, int r1) {
    for (int i = r0 * kPer + tid; i < r1 * kPer; i += 128) *chunk(i) = make_uint4(0, 0, 0, 0);
  };
  bool odd = false;
  auto take = [&](int r0, int r1) {
#pragma unroll 4
    for (int i = r0 * kPer + tid; i < r1 * kPer; i += 128) {
      uint4 v = *chunk(i);
      uint32_t* x = reinterpret_cast<uint32_t*>(&v);
      // an exponent of all ones carries into the sign's place
      uint32_t hit = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) hit |= (x[k] & 0x7f807f80u) + 0x00800080u;
      if (!(hit & 0x80008000u)) continue;
      odd = true;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t bad = ((x[k] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
        x[k] &= ~((bad & 0x8000u ? 0xffffu : 0u) | (bad & 0x80000000u ? 0xffff0000u : 0u));
      }
      *chunk(i) = v;
    }
  };
  zero(e.r0 & ~15, e.r0);
  zero(e.r1, (e.r1 + 15) & ~15);
  if (e.p0 < e.p1) take(e.p0, e.p1);
  if (e.p2 < e.p3) take(e.p2, e.p3);
  return odd;
}

// ---------------------------------------------------------------- MMA

// The warp runs together and elects the issuing thread at each step: issued
// from a branch that one lane is in throughout, the MMAs came 10% slower.
template <int D, bool kFp8>
__device__ void multiply(const AttendArgs& a, const Shared& s, uint32_t tmem, int lane) {
  using L = Layout<D, kFp8>;
  const uint32_t ring = desc_lo(dec::smem_addr(s.base + L::kRingOff)), qd = desc_lo(dec::smem_addr(s.base));
  constexpr uint32_t id_s = idesc(kTile, false), id_o = idesc(D, true);
  constexpr uint32_t kVLead = ((kTile * 128 - 16) >> 4) << 16;  // a V descriptor's leading offset, from a K one's
  constexpr int kSteps = kTile / 16;
  Turn<L::kStages> kt, vt;  // places of the next K and V
  vt.next();
  uint32_t pq[2] = {0, 0}, pp[2] = {0, 0};
  auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_or_abort(bar, parity, a.status, s.abort_flag); };
  Units units;
  while (const Unit* u = units.next(a, s)) {
    bool live[2] = {false, false};  // O_w has been written in this part
    const int t0 = u->t0, t1 = u->t1;
    const int f0[2] = {u->f0[0], u->f0[1]}, f1[2] = {u->f1[0], u->f1[1]};
    // tiles [e0, e1) are seen whole by every row
    const int e0 = (max(u->lo, u->all_lo) + kTile - 1) / kTile, e1 = u->all_hi / kTile;
    for (int t = t0; t <= t1; ++t) {
      int k0 = 0, k1 = kSteps;  // 16-token steps of V(t - 1) with tokens that some row sees
      if (t > t0) {
        if (!wait(&s.full[vt.st], vt.ph)) goto out;
        if (t - 1 < e0 || t > e1) {
          const Unit::Edge e = u->edge(t - 1);
          k0 = e.r0 >> 4;
          k1 = (e.r1 + 15) >> 4;
        }
      }
      const uint32_t kd = ring + kt.st * (L::kTileBytes >> 4), vd = ring + vt.st * (L::kTileBytes >> 4) + kVLead;
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        const uint32_t S = tmem + sub * 128, O = tmem + 256 + sub * 128;
        if (t > f0[sub] && t <= f1[sub]) {  // O_sub += P_sub(t - 1) V(t - 1)
          if (!wait(&s.pfull[sub], pp[sub])) goto out;
          fence_after();
          if (k0 == 0 && k1 == kSteps) {
            if (elect()) {
#pragma unroll
              for (int k = 0; k < kSteps / 2; ++k) mma_ts(O, S + k * 8, vd + k * 128, id_o, k != 0 || live[sub]);
            }
            __syncwarp();
            if (!wait(&s.pfull2[sub], pp[sub])) goto out;
            fence_after();
            if (elect()) {
#pragma unroll
              for (int k = kSteps / 2; k < kSteps; ++k) mma_ts(O, S + k * 8, vd + k * 128, id_o, true);
            }
          } else {
            if (!wait(&s.pfull2[sub], pp[sub])) goto out;
            fence_after();
            if (elect())
              for (int k = k0; k < k1; ++k) mma_ts(O, S + k * 8, vd + k * 128, id_o, k != k0 || live[sub]);
          }
          if (t == f1[sub] && elect()) commit(&s.ofull[sub]);  // while the other sub-tile goes on
          __syncwarp();
          pp[sub] ^= 1;
          live[sub] = true;
        }
        if (t < t1) {  // S_sub = Q_sub K(t)^T
          if (sub == 0 && !wait(&s.full[kt.st], kt.ph)) goto out;
          if (t >= f0[sub] && t < f1[sub]) {
            if (t == f0[sub]) {
              if (!wait(&s.qfull[sub], pq[sub])) goto out;
              pq[sub] ^= 1;
            }
            fence_after();
            if (elect()) {
#pragma unroll
              for (int k = 0; k < D / 16; ++k)
                mma_ss(S, qd + sub * (kSub * D / 8) + (k >> 2) * (kSub * 8) + (k & 3) * 2,
                       kd + (k >> 2) * (kTile * 8) + (k & 3) * 2, id_s, k != 0);
              commit(&s.sfull[sub]);
              if (t + 1 == f1[sub]) commit(&s.qempty[sub]);
            }
            __syncwarp();
          }
        }
      }
      if (elect()) {
        if (t > t0) commit(&s.empty[vt.st]);
        if (t < t1) commit(&s.empty[kt.st]);
      }
      __syncwarp();
      if (t > t0) {
        vt.next();
        vt.next();
      }
      if (t < t1) {
        kt.next();
        kt.next();
      }
    }
    units.done(s, lane);
  }
out:
  // every MMA issued has completed before TMEM is freed
  if (elect()) {
    commit(s.drain);
    dec::mbar_wait(s.drain, 0, a.status);
  }
  __syncwarp();
}

// ---------------------------------------------------------------- Q

// Q of every block by TMA: a box of the group's heads x 128 / G tokens is the
// K-major tile.  (Rows past the sequence's end are the next one's, or zeros;
// rows past the box keep what they held.  Both are never stored.)  A negative
// softmax scale goes into Q's signs.
template <int D>
__device__ void load_q(const AttendArgs& a, const Shared& s, const CUtensorMap* map, int lane) {
  const bool flip = a.scale_log2 < 0.0f;  // then Q arrives on `landed` first
  uint32_t ph[2] = {0, 0};
  bool used[2] = {false, false};
  Units units;
  while (const Unit* u = units.next(a, s)) {
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      if (!u->any(sub)) continue;
      const uint32_t mine = ph[sub];
      if (!wait_or_abort(&s.qempty[sub], mine ^ 1, a.status, s.abort_flag)) goto out;
      ph[sub] ^= 1;
      used[sub] = true;
      uint8_t* Q = s.base + sub * kSub * D * 2;
      uint64_t* bar = flip ? &s.landed[sub] : &s.qfull[sub];
      if (lane == 0) {
        dec::mbar_expect_tx(bar, a.tps * a.G * D * 2);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          tma_box3(dec::smem_addr(Q + c * kSub * 128), map, c * 64, u->h * a.G, u->q0 + (u->rb * 2 + sub) * a.tps, bar);
      }
      if (flip) {
        if (!wait_or_abort(bar, mine, a.status, s.abort_flag)) goto out;
#pragma unroll 4
        for (int i = lane; i < kSub * D / 8; i += 32) {
          uint4* at = reinterpret_cast<uint4*>(Q) + i;
          uint4 v = *at;
          v.x ^= 0x80008000u; v.y ^= 0x80008000u; v.z ^= 0x80008000u; v.w ^= 0x80008000u;
          *at = v;
        }
        fence_async();
        __syncwarp();
        if (lane == 0) dec::mbar_arrive(&s.qfull[sub]);
      }
    }
    units.done(s, lane);
  }
out:
  // no copy may still be writing this CTA's shared memory when it exits (where the CTA aborts, nobody else has waited)
#pragma unroll 1
  for (int sub = 0; sub < 2; ++sub)
    if (used[sub]) dec::mbar_wait(flip ? &s.landed[sub] : &s.qfull[sub], ph[sub] ^ 1, a.status);
}

// ---------------------------------------------------------------- softmax

// A warp's 32 rows of kChunks 16-byte chunks in shared memory, swizzled so that
// neither a lane per row nor neighbouring lanes in a row collide.
template <int kChunks>
__device__ __forceinline__ uint4* stage_at(uint8_t* stage, int r, int c) {
  const int x = kChunks == 8 ? r & 7 : (r >> 1) & 3;
  return reinterpret_cast<uint4*>(stage + r * (kChunks * 16) + ((c ^ x) << 4));
}
template <int kChunks>
__device__ __forceinline__ void stage_put(uint8_t* stage, int r, int c, uint4 v) {
  *stage_at<kChunks>(stage, r, c) = v;
}
// Out to column `col` of the rows; at: element offset of this lane's row (-1: none).
template <int kChunks>
__device__ __forceinline__ void stage_out(uint8_t* stage, int lane, long long at, uint8_t* base, int esz, int col) {
  __syncwarp();
  constexpr int kRows = 32 / kChunks;
#pragma unroll
  for (int r0 = 0; r0 < 32; r0 += kRows) {
    const int r = r0 + lane / kChunks, c = lane % kChunks;
    const long long to = __shfl_sync(0xffffffffu, at, r);
    if (to >= 0) *reinterpret_cast<uint4*>(base + (to + col) * esz + c * 16) = *stage_at<kChunks>(stage, r, c);
  }
  __syncwarp();
}
// Adds to a row's columns k .. k + 31 the values of tokens [from, to) that are not finite.
template <int D>
__device__ __noinline__ void add_not_finite(const AttendArgs& a, int s, int h, int from, int to, int k, float* o) {
  for (int j = from; j < to; ++j) {
    const int page = max(0, load_page(a.p, a.b, s, j / a.p.page_tokens, a.status));
    const __nv_bfloat16* at =
        static_cast<const __nv_bfloat16*>(a.p.v) +
        (((long long)page * a.p.num_kv_heads + h) * a.p.page_tokens + j % a.p.page_tokens) * D + k;
    for (int i = 0; i < 32; ++i) {
      const float x = __bfloat162float(at[i]);
      if (!isfinite(x)) o[i] += x;
    }
  }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Two fp32 operations at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 d, a, b;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// Probabilities of kN of a row's scores, as bf16 pairs, and their sum.
template <int kN>
__device__ __forceinline__ float2 probabilities(const float* x, float c, float base, uint32_t* p) {
  const float2 c2 = make_float2(c, c), b2 = make_float2(-base, -base);
  float2 sum0 = make_float2(0.0f, 0.0f), sum1 = sum0;
#pragma unroll
  for (int k = 0; k < kN; k += 2) {
    const float2 y = fma2(make_float2(x[k], x[k + 1]), c2, b2);
    const float2 e = make_float2(exp2_approx(y.x), exp2_approx(y.y));
    if (k & 2) sum1 = add2(sum1, e);
    else sum0 = add2(sum0, e);
    p[k / 2] = pack2(e.x, e.y);
  }
  return add2(sum0, sum1);
}

// Quantised cache: the columns, a bit each, in which some of tokens [from, to) has
// no finite value.  Of tokens [all_lo, all_hi), which went through the product as
// they are, only scales of NaN count.
struct Columns {
  uint32_t bits[4];
};
template <int D>
__device__ __noinline__ Columns not_finite(const AttendArgs& a, int s, int h, int from, int to, int all_lo, int all_hi) {
  Columns c{};
  for (int j = from; j < to; ++j) {
    const int page = max(0, load_page(a.p, a.b, s, j / a.p.page_tokens, a.status));
    const long long row = ((long long)page * a.p.num_kv_heads + h) * a.p.page_tokens + j % a.p.page_tokens;
    const int e = a.p.v_scale[row];
    if (e == kNanScale) return Columns{{~0u, ~0u, ~0u, ~0u}};
    if (j >= all_lo && j < all_hi) continue;
    for (int d = 0; d < D; ++d) {
      const float x = __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(a.p.v)[row * D + d], __NV_E4M3)));
      if (!isfinite(x * scale_of(e)))
#pragma unroll
        for (int k = 0; k < 4; ++k) c.bits[k] |= d >> 5 == k ? 1u << (d & 31) : 0u;
    }
  }
  return c;
}

template <int D, bool kFp8>
__device__ void soften(const AttendArgs& a, const Shared& s, uint32_t tmem, int sub, int tid) {
  using L = Layout<D, kFp8>;
  const int lane = tid & 31, quarter = (tid >> 5) & 3;
  const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
  const uint32_t ts = tmem + lanes + sub * 128, to = tmem + lanes + 256 + sub * 128;
  const float c = fmaxf(fabsf(a.scale_log2), 1.17549435e-38f);  // never 0: 0 * -inf is not -inf
  const int my_token = tid / a.G;
  uint8_t* stage = s.base + L::kOutOff + (sub * 4 + quarter) * 32 * L::kLine;
  uint32_t ns = 0, no = 0;
  int tiles = 0;  // of the blocks before
  const int group = sub * 4 + quarter;  // of 32 rows
  if (lane == 0) a.desc[blockIdx.x * 8 + group] = make_int4(-1, 0, 0, 0);
  Units units;
  while (Unit* u = units.next(a, s)) {
    const int i_new = (u->rb * 2 + sub) * a.tps + my_token;  // this row's new token
    const bool mine = my_token < a.tps && i_new < u->m;
    const bool any = u->any(sub);
    const Span v = visible(a, u->seq(), mine ? i_new : 0);
    const int lo = mine ? v.lo : 0, hi = mine ? v.hi : 0;
    float m = -INFINITY, l = 0.0f;
    const int t_end = any ? u->f1[sub] : 0, all_lo = u->all_lo, all_hi = u->all_hi;
    bool first = true;
    for (int t = u->f0[sub]; t < t_end; ++t) {
      const int j0 = t * kTile;
      if (!wait_or_abort(&s.sfull[sub], ns, a.status, s.abort_flag)) return;
      ns ^= 1;
      fence_after();
      // A row's scores come by kHeld, once for the maximum and once more for P:
      // short loops, which with the other warps' fit the instruction cache
      // (unrolled over the row, the quantised cache's kernel took 1.35 times as
      // long, its warps waiting for instructions).
      constexpr int kHeld = 64;
      float x[kHeld];
      const bool edge = j0 < all_lo || j0 + kTile > all_hi;  // some row does not see all of the tile
      if (edge) {  // unseen scores become -inf in place, so that the loops below are short
        const int from = lo - j0, end = hi - j0;
#pragma unroll 1
        for (int col = 0; col < 128; col += 32) {
          if (__all_sync(0xffffffffu, from <= col && end >= col + 32)) continue;
          float y[32];
          ld32(ts + col, y);
          ld_wait();
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (k < from - col || k >= end - col) y[k] = -INFINITY;
          st32(ts + col, reinterpret_cast<const uint32_t*>(y));
        }
        st_wait();
      }
      auto load = [&](int col) {  // kHeld scores from column col
#pragma unroll
        for (int k = 0; k < kHeld; k += 32) ld32(ts + col + k, x + k);
        ld_wait();
      };
      float top = -INFINITY;
#pragma unroll 1
      for (int col = 0; col < 128; col += kHeld) {
        load(col);
        float top4[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) top4[k] = fmaxf(x[k], x[k + 4]);
#pragma unroll
        for (int k = 8; k < kHeld; k += 8)
#pragma unroll
          for (int i = 0; i < 4; ++i) top4[i] = max3(top4[i], x[k + i], x[k + 4 + i]);
        top = max3(top, max3(top4[0], top4[1], top4[2]), top4[3]);
      }
      top *= c;
      if (first) {
        m = top;
        first = false;
      } else if (__any_sync(0xffffffffu, mine && top > m + kGrow)) {  // (a row that is nobody's changes no other's rounding)
        const float mn = fmaxf(m, top), f = top > m ? exp2_approx(m - mn) : 1.0f;
        m = mn;
        l *= f;
        for (int k = 0; k < D; k += 32) {
          float o[32];
          ld32(to + k, o);
          ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= f;
          st32(to + k, reinterpret_cast<const uint32_t*>(o));
        }
      }
      const float base = m == -INFINITY ? 0.0f : m;
      float2 sum = make_float2(0.0f, 0.0f);
      // (sub-tile 0's P goes to V first, unless only the other has the tile)
      if (!kFp8 && edge && (sub == 0 || t < u->f0[0] || t >= u->f1[0])) {
        const int i = 2 * (tiles + t - u->t0) + 1;  // V's place among the ring's tiles
        if (!wait_or_abort(&s.full[i % L::kStages], i / L::kStages & 1, a.status, s.abort_flag)) return;
        if (mend<D>(s.base + L::kRingOff + i % L::kStages * L::kTileBytes, u->edge(t), tid))
          *reinterpret_cast<volatile int*>(&u->odd) = 1;
        fence_async();
      }
#pragma unroll 1
      for (int col = 0; col < 128; col += kHeld) {
        uint32_t p[kHeld / 2];
        load(col);
        sum = add2(sum, probabilities<kHeld>(x, c, base, p));
        st32(ts + col / 2, p);
        if ((col + kHeld) % 64 == 0) {  // half of P
          st_wait();
          fence_before();
          __syncwarp();
          if (lane == 0) dec::mbar_arrive(col >= 64 ? &s.pfull2[sub] : &s.pfull[sub]);
        }
      }
      l += sum.x + sum.y;
    }
    // ------------------------------------------------------------ the block's end
    if (any) {
      if (!wait_or_abort(&s.ofull[sub], no, a.status, s.abort_flag)) return;
      no ^= 1;
      fence_after();
    }
    // The CTA that begins a block of two parts comes to its own last, as a rule,
    // and the other first; then the other's is there, and they are joined here.
    // combine_kernel does what is left, with the same roundings.  (A prompt chunk
    // of 4096 tokens: 78.7 -> 73 us; blocks of three and four too came no faster.)
    const long long slot = 2LL * blockIdx.x + u->begins;
    const int parts = u->parts, row = group * 32 + lane;
    bool whole = parts == 1;
    float f0 = 1.0f, f1 = 0.0f;
    if (u->begins && parts == 2) {
      unsigned seen = 0;
      if (lane == 0) {
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(&a.arrived[u->c0 * 8 + group]) : "memory");
        __threadfence();
      }
      whole = __shfl_sync(0xffffffffu, seen, 0) == 1u;
      __syncwarp();
      if (whole) {
        const float2 x = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + 2 * (u->c0 + 1) * kChunkRows + row);
        const float top = fmaxf(m, x.x), base = top == -INFINITY ? 0.0f : top;
        f0 = exp2_approx(m - base);
        f1 = exp2_approx(x.x - base);
        l = join(join(0.0f, f0, l), f1, x.y);
        m = top;
      }
    }
    const bool joined = whole && parts > 1;
    const int my_head = tid - my_token * a.G;
    const long long at = !mine ? -1 : out_at(a, u->seq(), u->h, i_new, my_head);  // in elements; -1: no row
    if (mine) {
      if (whole)
        write_lse(a, u->seq(), u->h, i_new, my_head, m, l);
      else
        reinterpret_cast<float2*>(a.part_ml)[slot * kChunkRows + row] = make_float2(m, l);
    }
    const float inv = inverse(l);
    const bool odd = any && *const_cast<const volatile int*>(&u->odd) && mine;
    const int first_tok = max(lo, u->t0 * kTile), last_tok = min(hi, u->t1 * kTile);
    Columns nan{};
    if (kFp8 && odd) nan = not_finite<D>(a, u->s, u->h, first_tok, last_tok, all_lo, all_hi);
    float4 y[8];  // 32 columns of the other part
    auto other = [&](int k) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = __ldcg(part_at<D>(a, 2 * (u->c0 + 1), row, k + 4 * i));
    };
    if (joined) other(0);
    for (int k = 0; k < D; k += 32) {
      float o[32];
      if (any) {
        ld32(to + k, o);
        ld_wait();
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = 0.0f;
      }
      if (!kFp8 && odd) {  // (tokens that every row sees went through the product)
        float add[32] = {};
        add_not_finite<D>(a, u->s, u->h, first_tok, min(last_tok, all_lo), k, add);
        add_not_finite<D>(a, u->s, u->h, max(first_tok, max(all_lo, all_hi)), last_tok, k, add);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] += add[i];
      }
      if (kFp8 && odd) {
        const uint32_t here = k == 0 ? nan.bits[0] : k == 32 ? nan.bits[1] : k == 64 ? nan.bits[2] : nan.bits[3];
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = here >> i & 1u ? __uint_as_float(0x7fc00000u) : o[i];
      }
      if (joined) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          o[4 * i] = join(join(0.0f, f0, o[4 * i]), f1, y[i].x);
          o[4 * i + 1] = join(join(0.0f, f0, o[4 * i + 1]), f1, y[i].y);
          o[4 * i + 2] = join(join(0.0f, f0, o[4 * i + 2]), f1, y[i].z);
          o[4 * i + 3] = join(join(0.0f, f0, o[4 * i + 3]), f1, y[i].w);
        }
        if (k + 32 < D) other(k + 32);
      }
      if (whole) {  // rows through shared memory, so that neighbouring lanes store neighbouring bytes
        constexpr int kChunks = L::kLine / 16;
        constexpr int kHalf = L::kLine / 64;  // runs of 32 columns in a line
        const int run = kHalf == 2 ? k >> 5 & 1 : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          stage_put<kChunks>(stage, lane, run * 4 + i,
                             make_uint4(pack2(o[8 * i] * inv, o[8 * i + 1] * inv),
                                        pack2(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                        pack2(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                                        pack2(o[8 * i + 6] * inv, o[8 * i + 7] * inv)));
        if (run == kHalf - 1)
          stage_out<kChunks>(stage, lane, at, reinterpret_cast<uint8_t*>(a.out), 2, k & ~(kHalf * 32 - 1));
      } else if (mine) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *part_at<D>(a, slot, row, k + 4 * i) = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
      }
    }
    if (!whole) {
      if (u->begins) {
        if (lane == 0) a.desc[blockIdx.x * 8 + group] = make_int4(u->s, u->h, u->rb, u->c0 + parts - 1);
      } else {
        __threadfence();
        __syncwarp();
        if (lane == 0) atomicAdd(&a.arrived[u->c0 * 8 + group], 1u);
      }
    }
    tiles += u->t1 - u->t0;
    fence_before();  // the next block's MMAs write O after these reads
    units.done(s, lane);
  }
}

// ---------------------------------------------------------------- e4m3 codes to bf16 tiles

// Tokens that no row sees become zeros: they may hold anything.  So do the
// values of a token whose scale is NaN, lest 0 * NaN reach a row that does not
// see it, and codes of NaN, of tokens that some rows see and others do not; the
// block's end makes the rows that do NaN there.  (A key of NaN may stay: its
// scores are hidden, not multiplied.  Looking at the codes of edge tiles costs six
// chunks of 300 tokens 34.0 -> 34.7 us, a chunk beside 32 decoding sequences 72.8
// -> 73.6.)
template <int D>
__device__ void expand(const AttendArgs& a, const Shared& s, int tid) {
  using L = Layout<D, true>;
  const int lane = tid & 31;
  Turn<L::kRaw> rt;
  Turn<L::kStages> st;
  // A warp takes eight rows at a time, 64 codes of each (half a row of 128): a
  // lane 16 codes, four lanes a row.  The lanes of a quarter-warp are at rows r
  // and r ^ 5, whose chunks the swizzles put into different banks, where they
  // are read and where the two bf16 chunks are written.
  constexpr int kHalves = D / 64, kGroups = kCvtWarps / kHalves;
  const int half = (tid >> 5) % kHalves, ch = half * 4 + (lane & 3);
  const int r0 = (tid >> 5) / kHalves * 8 + ((lane >> 3) ^ (lane & 4 ? 5 : 0));  // then every kGroups * 8 rows
  constexpr int kRows = kGroups * 8;
  Units units;
  while (Unit* u = units.next(a, s)) {
    const int lo = u->lo, hi = u->hi, t1 = u->t1, all_lo = u->all_lo, all_hi = u->all_hi;
    // the scale bytes of tokens 4 lane .. + 3 of tile t (a page's tokens come in sixteens)
    auto scales = [&](int t, uint32_t* e) {
      const int j = t * kTile + 4 * lane;
      e[0] = e[1] = 0;
      if (t >= t1 || j + 3 < lo || j >= hi) return;
      const int page = max(0, load_page(a.p, a.b, u->s, j / a.p.page_tokens, a.status));
      const long long at = ((long long)page * a.p.num_kv_heads + u->h) * a.p.page_tokens + j % a.p.page_tokens;
      e[0] = __ldg(reinterpret_cast<const uint32_t*>(a.p.k_scale + at));
      e[1] = __ldg(reinterpret_cast<const uint32_t*>(a.p.v_scale + at));
    };
    uint32_t e[2];
    scales(u->t0, e);
    for (int t = u->t0; t < t1; ++t) {
      const int seen0 = lo - t * kTile, seen1 = hi - t * kTile, all0 = all_lo - t * kTile, all1 = all_hi - t * kTile;
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        if (!wait_or_abort(&s.rfull[rt.st], rt.ph, a.status, s.abort_flag)) return;
        const uint8_t* src = s.base + L::kRawOff + rt.st * L::kRawBytes;
        const uint32_t mine = kv ? e[1] : e[0];
        if (kv == 1) scales(t + 1, e);  // on their way while V is expanded
        // tokens that not every row sees, or scales of NaN, in this tile
        const bool odd = __any_sync(0xffffffffu, __vcmpeq4(mine, 0xffffffffu) != 0u) || all0 > 0 || all1 < kTile;
        if (!wait_or_abort(&s.empty[st.st], st.ph ^ 1, a.status, s.abort_flag)) return;
        uint8_t* dst = s.base + L::kRingOff + st.st * L::kTileBytes + (ch >> 2) * (kTile * 128);
#pragma unroll 1
        for (int r = r0; r < kTile; r += kRows) {
          const int phys = D == 128 ? ch ^ (r & 7) : ch ^ ((r >> 1) & 3);
          uint4 c = *reinterpret_cast<const uint4*>(src + r * D + (phys << 4));
          const uint32_t b = __shfl_sync(0xffffffffu, mine, r >> 2) >> ((r & 3) * 8) & 0xffu;
          uint32_t sc = b * 0x00800080u;  // 2^(b - 127) as a pair of bf16
          if (__builtin_expect(odd, 0)) {
            const bool nan = b == kNanScale, drop = r < seen0 || r >= seen1 || (kv == 1 && nan);
            if (drop) c = make_uint4(0, 0, 0, 0);
            if (nan || drop) sc = kv == 0 && nan ? 0x7fc07fc0u : 0u;
            bool hit = kv == 1 && nan && r >= seen0 && r < seen1;
            if (kv == 1 && (r < all0 || r >= all1)) {  // codes of NaN
              const uint32_t n0 = __vcmpeq4(c.x & 0x7f7f7f7fu, 0x7f7f7f7fu), n1 = __vcmpeq4(c.y & 0x7f7f7f7fu, 0x7f7f7f7fu),
                             n2 = __vcmpeq4(c.z & 0x7f7f7f7fu, 0x7f7f7f7fu), n3 = __vcmpeq4(c.w & 0x7f7f7f7fu, 0x7f7f7f7fu);
              c = make_uint4(c.x & ~n0, c.y & ~n1, c.z & ~n2, c.w & ~n3);
              hit |= (n0 | n1 | n2 | n3) != 0u;
            }
            if (hit) *reinterpret_cast<volatile int*>(&u->odd) = 1;
          }
          const __nv_bfloat162 sc2 = *reinterpret_cast<const __nv_bfloat162*>(&sc);
          const uint32_t q[4] = {c.x, c.y, c.z, c.w};
          uint32_t o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t pair = i & 1 ? q[i >> 1] >> 16 : q[i >> 1] & 0xffffu;
            const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)pair, __NV_E4M3)));
            const __nv_bfloat162 v = __hmul2(__floats2bfloat162_rn(f.x, f.y), sc2);  // exact
            o[i] = *reinterpret_cast<const uint32_t*>(&v);
          }
          uint8_t* row = dst + r * 128;
          const int d0 = (ch & 3) * 2;
          *reinterpret_cast<uint4*>(row + ((d0 ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(row + (((d0 + 1) ^ (r & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
        }
        fence_async();
        __syncwarp();
        if (lane == 0) {
          dec::mbar_arrive(&s.rempty[rt.st]);
          dec::mbar_arrive(&s.full[st.st]);
        }
        rt.next();
        st.next();
      }
    }
    units.done(s, lane);
  }
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(kFp8 ? kFpThreads : kBfThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                 const __grid_constant__ CUtensorMap map_q, const __grid_constant__ AttendArgs a) {
  using L = Layout<D, kFp8>;
  extern __shared__ uint8_t smem_raw[];
  const Shared s = carve<D, kFp8>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      dec::mbar_init(&s.full[i], kFp8 ? kCvtWarps : 1);
      dec::mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < L::kRaw; ++i) {
      dec::mbar_init(&s.rfull[i], 1);
      dec::mbar_init(&s.rempty[i], kCvtWarps);
    }
    for (int i = 0; i < kUnits; ++i) {
      dec::mbar_init(&s.ufull[i], 1);
      dec::mbar_init(&s.uempty[i], 8 + 2 + (kFp8 ? kCvtWarps : 0));  // softmax, MMA, Q, expanding
    }
    for (int i = 0; i < 2; ++i) {
      dec::mbar_init(&s.qfull[i], 1);
      dec::mbar_init(&s.qempty[i], 1);
      dec::mbar_init(&s.landed[i], 1);
      dec::mbar_init(&s.sfull[i], 1);
      dec::mbar_init(&s.pfull[i], 4);
      dec::mbar_init(&s.pfull2[i], 4);
      dec::mbar_init(&s.ofull[i], 1);
    }
    dec::mbar_init(s.drain, 1);
    *s.abort_flag = 0;
    dec::mbar_init_fence();
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dec::smem_addr(s.tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    fence_before();
  }
  // The batch, q and the pages may come from the kernel before.  Beside
  // token_kernel that is the one before it, which token_kernel has waited for
  // before any of its CTAs let this kernel start; with token_kernel itself this
  // one shares no data, so the wait for it is at the end (a chunk of 1000 tokens
  // beside 32 decoding sequences: 81 -> 78 us).
  if (!a.beside) dec::pdl_wait_primary();
  long long* pre = reinterpret_cast<long long*>(s.base + L::kRingOff);
  long long* scan = reinterpret_cast<long long*>(s.base);
  const Range rg = cut(a, pre, scan, [&](int seq) {
    // (a warp's lanes are at different sequences; a long one is summed by all)
    const Seq q = seq < a.b.num_seqs ? own_seq<false>(a, seq) : Seq{0, 0, 0};
    const int nb = blocks_of(a, q);
    long long n = 0;
    if (nb <= 8)
      for (int rb = 0; rb < nb; ++rb) n += items_of(a, q, rb);
    for (unsigned big = __ballot_sync(0xffffffffu, nb > 8); big; big &= big - 1) {
      const int src = __ffs(big) - 1;
      const Seq o{__shfl_sync(0xffffffffu, q.q0, src), __shfl_sync(0xffffffffu, q.m, src),
                  __shfl_sync(0xffffffffu, q.n, src)};
      const long long sum = head_items(a, o, lane);
      if (lane == src) n = sum;
    }
    return n * a.p.num_kv_heads;
  });
  fence_async();
  fence_before();
  __syncthreads();  // the prefix sums are read; the ring may fill; TMEM's address is there
  fence_after();
  const uint32_t tmem = *s.tmem;
  if (warp < 8) {
    if (kFp8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kFpSoft));
    soften<D, kFp8>(a, s, tmem, warp >> 2, threadIdx.x & 127);
    __syncwarp();
    st_wait();  // (a CTA that aborts may have stores to TMEM on their way)
  } else if (warp < 12) {
    if (kFp8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFpRest));
    if (warp == 8) produce<D, kFp8>(a, rg, s, &map_k, &map_v, lane);
    if (warp == 9) multiply<D, kFp8>(a, s, tmem, lane);
    if (warp == 10) load_q<D>(a, s, &map_q, lane);
  } else if (kFp8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFpCvt));
    expand<D>(a, s, threadIdx.x - 384);
  }
  fence_before();
  __syncthreads();
  if (warp == 9) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
  dec::pdl_launch_dependents();
  if (a.beside) dec::pdl_wait_primary();  // what follows in the stream follows token_kernel too
}

template <int D, bool kFp8>
cudaError_t launch(const AttendArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mq,
                   cudaStream_t s) {
  const cudaError_t e = allow_smem<4096 + D * 2 + kFp8>(chunk_kernel<D, kFp8>, Layout<D, kFp8>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_dependent(chunk_kernel<D, kFp8>, a.grid, kFp8 ? kFpThreads : kBfThreads, Layout<D, kFp8>::kSmem, s, mk,
                          mv, mq, a);
}

}  // namespace

cudaError_t launch_attend_chunk(const AttendArgs& a, cudaStream_t s) {
  CUtensorMap mk, mv, mq;
  const int box = a.p.page_tokens < kTile ? a.p.page_tokens : kTile;
  if (!pages_map(&mk, a.p, a.p.k, box) || !pages_map(&mv, a.p, a.p.v, box) || !queries_map(&mq, a, a.tps))
    return cudaErrorInvalidValue;
  const bool fp8 = a.p.kv_dtype == FT_KV_FP8E4M3;
  if (a.p.head_dim == 128) return fp8 ? launch<128, true>(a, mk, mv, mq, s) : launch<128, false>(a, mk, mv, mq, s);
  return fp8 ? launch<64, true>(a, mk, mv, mq, s) : launch<64, false>(a, mk, mv, mq, s);
}

}  // namespace kv
}  // namespace ft
