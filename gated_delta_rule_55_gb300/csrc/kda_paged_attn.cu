// Attention of new tokens over a paged cache (kda_paged_attention_fwd) on the tensor cores:
// bf16.
//
// Work.  An item is one sequence, one kv head and up to 256 of its query rows (tokens x query
// heads of that kv head).  Its visible keys come in tiles of 128; the tiles of all items, in
// order, form one line that is cut into equal stretches, one for each CTA (one CTA per SM).
// Ragged batches, causal triangles, windows and single tokens over long caches are thus
// balanced alike, and an item that a cut passes through leaves at most two partial results per
// CTA, joined by a second kernel.
//
// One CTA: two units, each with a score tile S [128 rows x 128 keys] and an output accumulator
// O [128 x D] in Tensor Memory and a warpgroup for the softmax.  They work in steps.  A wide item
// (more than 128 rows) gives each unit 128 rows and every key tile to both.  Two narrow ones
// (single tokens) of about the same length are taken side by side, one by each unit, so that one
// item's start and end pass beside the other's tiles (256 sequences of 100 to 1000 keys: 113 us
// for 156); any other narrow item gives both units the same rows and every other key tile, and
// their two results are joined at its end.
// A load warp brings key and value tiles by TMA (one box per page and 64 columns) through a
// ring of shared-memory stages; a warp of each unit issues the products
//   S = Q K^T  (both operands in shared memory),  O += P V  (P in Tensor Memory, V read as it
//   lies, keys along the contraction),
// so that the softmax of one unit runs while the tensor cores work for the other; another warp
// walks the items, puts the steps down for all roles a few ahead, and brings the query rows (a box
// where 128 rows are whole tokens).
//
// The code is kept small where it does not cost: each role's instructions push the others' out of
// the instruction cache.  Loops in place of unrolled copies in the cut, the load warp and the
// masked tiles' softmax took 30% of its length and 10 to 20% of the time of short items.
//
// The softmax subtracts a standing maximum: weights are made against the maximum so far while
// the tile's own is found beside them, and only where a row's has grown by more than 2^8 do the
// softmax warps rescale O and l (the sums stay far inside fp32).
//   D = 128: P lies over S's columns.  The product that makes S for the next tile is issued
//   behind the one that reads P, so S complete means O complete.  The lower half of a tile's
//   weights is handed over while the upper half is computed (1283 -> 1244 us for the long chunks
//   below), and a wide item's units take turns at the tensor cores.
//   D <= 64: P has columns of its own, and the next scores are made while the last tile's softmax
//   still runs (43.5 us for 45.6 on the mixed batch below); without a window, where few tiles are
//   masked, whole tiles are made in one pass as above.
//
// What bounds it, and measured (alone on the GPU):
//   64 single tokens over 512..8192 keys, 32 + 8 heads of 128: HBM; 167 us, 6.4 TB/s of the 6.8
//   of a copy.
//   2 chunks of 4096 tokens behind 12288 keys, the same heads: the tensor cores; 1.13 to
//   1.19 ms, 1.61 to 1.70 PFLOP/s of the 1.92 of a library product.
//   9 sequences of 1..700 tokens, window 1024, 16 + 2 heads of 64: 35 us, of which the start (the
//   cut, barriers, first loads) takes 4; then items' starts and ends.
//   One token over 1000 keys: 12 us of latencies in a row.
//
// Softmax weights are rounded to bf16 for the product (their sum is taken before, in fp32).
// Keys that no row of the item sees (behind the last one, outside the window, pages that are
// not loaded) have weight zero and their values are overwritten with zeros in shared memory,
// so what the cache holds there never counts.
#include "chunk_common.cuh"
#include "kda_paged.cuh"
#include "kda_paged_line.h"

namespace kda {
namespace {

using namespace chunk;

__device__ unsigned int g_paged_error;  // bit 6: a bounded wait gave up

constexpr int kKeys = 128;       // keys of a tile
constexpr int kRowsUnit = 128;   // query rows of a unit
constexpr int kRowsItem = 256;
constexpr int kThreads = 384;    // two softmax warpgroups, and one of the warps below
constexpr int kLoadWarp = 8, kMmaWarp = 9 /* and 10: one per unit */, kQueryWarp = 11;
// Registers: 168 a thread at launch (3 x 128 threads), moved to the softmax warpgroups:
// 2 x 216 + 72 = 3 x 168.
constexpr int kRegsSoftmax = 216, kRegsOther = 72;
// log2 growth of the maximum that O and l absorb.  (Rescaling only from some growth on, and two
// softmax warpgroups beside two score tiles, are published ways for attention on this hardware.)
constexpr float kRescale = 8.0f;

// What lies before the tiles: m and l of both units' rows (2 KB), barriers, the plan.
constexpr int kFront = 3 * 1024;

template <int D> struct Cfg {
  static constexpr int kStageBytes = kKeys * D * 2;
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr int kQBytes = kRowsUnit * D * 2;
  // Rows in shared memory: blocks of up to 64 columns, swizzled over their bytes.
  static constexpr int kRowBytes = D == 32 ? 64 : 128;
  static constexpr uint32_t kSwizzle = D == 32 ? 4 : kSwizzle128;  // 64-byte, 128-byte
  // D <= 64 leaves Tensor Memory for weights of their own (D = 128 keeps them over the scores):
  // the next scores are then made while the softmax of the last is still running.
  static constexpr bool kOwnP = D <= 64;
  static constexpr int kSmem = kFront + 2 * kQBytes + kStages * kStageBytes;
};

constexpr uint32_t kColS = 0, kColO = 256, kTmemCols = 512;  // + 128 * unit
constexpr uint32_t kColP64 = kColO + 64;                     // weights, D <= 64

// An item counts some units beside its tiles: what its start and end cost a CTA (the units lie
// before its tiles, and a cut among them falls to the item's first tile).  A wide one of D = 128
// counts 3: 12 sequences of 1 to 600 tokens, 32 + 8 heads, take 125 us for 132 with 2 and 145
// with 1; 256 single tokens 111 us with 2, 114 with 3; the mixed batch above 35.0 with 2, 35.7
// with 3.
constexpr int kOverhead = 2, kOverheadMost = 3;

struct Header {  // a CTA's part of the line, for the joining kernel
  int rows;       // rows of the item that starts in its stretch and is cut (0: none)
  int row0, h;    // its first row and kv head
  int nt;         // its tiles
  int start, total;  // place of its first tile in the line, the line's length
  int bos;        // its sequence's first token
};

// ------------------------------------------------------------------- items of the line

// x / G, G = Hq / Hkv, for 0 <= x < 2^31, by the host's multiplier (launch_t).
__device__ __forceinline__ int div_g(const PagedArgs& a, int x) {
  return (int)((__umulhi((uint32_t)x, a.g_mul) + (uint32_t)x) >> a.g_shift);
}

struct Geometry {
  int row0, rows;  // query rows of the item
  KeyRange kr;
  int t_lo, ns, nt;  // first window tile, sink tiles before it, tiles in all
  int extra;         // units of the line before its tiles
  __device__ __forceinline__ int units() const { return nt + extra; }
};

__device__ __forceinline__ Geometry geometry(const PagedArgs& a, const Seq& s, int G, int rt) {
  Geometry g;
  const int rows = s.len * G;
  g.row0 = rt * kRowsItem;
  g.rows = min(kRowsItem, rows - g.row0);
  g.extra = a.D == 128 && g.rows > kRowsUnit ? kOverheadMost : kOverhead;
  g.kr = key_range(a, s, div_g(a, g.row0), div_g(a, g.row0 + g.rows - 1));
  g.t_lo = g.kr.lo / kKeys;
  g.ns = min((g.kr.sinks + kKeys - 1) / kKeys, g.t_lo);
  // an item without keys still has one (empty) tile: its rows get their zeros
  g.nt = max(g.ns + (g.kr.hi + kKeys - 1) / kKeys - g.t_lo, 1);
  return g;
}

__device__ __forceinline__ Seq shfl_seq(const Seq& s, int src) {
  Seq t;
  t.bos = __shfl_sync(0xffffffffu, s.bos, src);
  t.len = __shfl_sync(0xffffffffu, s.len, src);
  t.kv = __shfl_sync(0xffffffffu, s.kv, src);
  t.pos0 = __shfl_sync(0xffffffffu, s.pos0, src);
  return t;
}

__device__ __forceinline__ int tile_start(const Geometry& g, int v) {
  return (v < g.ns ? v : g.t_lo + v - g.ns) * kKeys;
}

__device__ __forceinline__ int row_tiles(const Seq& s, int G) {
  return (int)(((long long)s.len * G + kRowsItem - 1) / kRowsItem);
}

struct Plan {  // in shared memory
  int total, first, end;  // units of the line, this CTA's stretch [first, end)
  int n, h, rt, x;        // where the stretch starts: an item and a unit of it (n < 0: nowhere)
  Seq s;                  // sequence n
};

// Walks the items of a CTA's stretch.  The next sequence's numbers are loaded while the current
// one is worked on.
struct Walker {
  int n, h, rt, v0, v1;
  int left;   // units of the stretch from the item's first one on
  int units;  // units of the item in the stretch
  Seq s;
  Geometry g;
  int c1, c2, kv1;  // the next sequence's offsets and keys

  __device__ __forceinline__ void ahead(const PagedArgs& a) {
    c1 = c2 = kv1 = 0;
    if (n + 1 < a.N) {
      c1 = a.cu_seqlens[n + 1];
      c2 = a.cu_seqlens[n + 2];
      kv1 = a.kv_lens[n + 1];
    }
  }
  // The item's tiles among its units [x, ...); false when the stretch ends before the first (it
  // is the stretch's last item then, and the next CTA takes it whole).
  __device__ __forceinline__ bool enter(const PagedArgs& a, int x) {
    g = geometry(a, s, a.G, rt);
    const int last = min(g.nt + g.extra, x + left);
    units = last - x;
    v0 = max(x - g.extra, 0);
    v1 = max(last - g.extra, 0);
    return v1 > v0;
  }
  __device__ __forceinline__ bool start(const PagedArgs& a, const Plan& p) {
    left = p.end - p.first;
    if (left <= 0 || p.n < 0) return false;
    n = p.n; h = p.h; rt = p.rt;
    s = p.s;
    ahead(a);
    return enter(a, p.x);
  }
  __device__ __forceinline__ bool next(const PagedArgs& a) {
    left -= units;
    if (left <= 0) return false;
    if (++rt >= row_tiles(s, a.G)) {
      rt = 0;
      if (++h >= a.Hkv) {
        h = 0;
        do {  // (the line has more units, so a later sequence has tokens)
          if (++n >= a.N) return false;
          s = make_seq(a, c1, c2, kv1);
          ahead(a);
        } while (s.len == 0);
      }
    }
    return enter(a, 0);
  }
  __device__ __forceinline__ int tiles() const { return v1 - v0; }
  __device__ __forceinline__ bool narrow() const { return g.rows <= kRowsUnit; }
};

constexpr int kPlanSeqs = 384;  // sequences whose units are looked at together

// Units of one head's items of a sequence, its row tiles spread over the warp's lanes.
__device__ __forceinline__ int head_units(const PagedArgs& a, const Seq& s, int G) {
  int x = 0;
  const int nrt = row_tiles(s, G);
#pragma unroll 1
  for (int rt = threadIdx.x & 31; rt < nrt; rt += 32) x += geometry(a, s, G, rt).units();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Notes the unit `off` of sequence n's units (`per` of them in each head) as the stretch's
// start; a whole warp calls.
__device__ __forceinline__ void note_start(const PagedArgs& a, Plan& plan, const Seq& s, int n,
                                           int per, int off) {
  const int lane = threadIdx.x & 31, G = a.G;
  const int h = (int)((unsigned)off / (unsigned)per);
  if (h >= a.Hkv) return;
  off -= h * per;
  const int nrt = row_tiles(s, G);
#pragma unroll 1
  for (int base = 0; base < nrt; base += 32) {
    const int rt = base + lane;
    const int nt = rt < nrt ? geometry(a, s, G, rt).units() : 0;
    int run = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += y;
    }
    if (off >= run - nt && off < run) {
      plan.n = n;
      plan.h = h;
      plan.rt = rt;
      plan.x = off - (run - nt);
      plan.s = s;
    }
    const int here = __shfl_sync(0xffffffffu, run, 31);
    if (off < here) break;
    off -= here;
  }
}

// The CTA's stretch of the line: all threads call.  s_units: kPlanSeqs entries, each of which
// fits 31 bits (paged_tc_index_ok).  So does the line when the offsets are in order; when they
// overlap, against the call's rules, it may not, and then every CTA's stretch is empty.
__device__ void make_plan(const PagedArgs& a, Plan& plan, int* s_units) {
  static_assert(kPlanSeqs == kThreads, "one sequence per thread");
  constexpr int W = kThreads / 32, kFew = 2 * W;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = a.G;
  const int rounds = (a.N + kPlanSeqs - 1) / kPlanSeqs;
  // Sequences r kPlanSeqs + ...: with few of them a warp takes two and its lanes the row tiles,
  // with many a thread takes one, and its warp helps where there are many row tiles.
  Seq s[2]{};
  int per[2], count = 0, sum = 0;
  if (threadIdx.x == 0) plan.n = -1;
  auto load = [&](int r) {
    count = min(a.N - r * kPlanSeqs, kPlanSeqs);
    __syncthreads();
    if (count <= kFew) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (warp + k * W < count) s[k] = load_seq(a, r * kPlanSeqs + warp + k * W);
#pragma unroll 1
      for (int k = 0; k < 2; ++k)
        if (warp + k * W < count) {
          const int y = head_units(a, k == 0 ? s[0] : s[1], G);
          if (lane == 0) s_units[warp + k * W] = y * a.Hkv;
          (k == 0 ? per[0] : per[1]) = y;
        }
    } else {
      const int i = threadIdx.x;
      if (i < count) s[0] = load_seq(a, r * kPlanSeqs + i);
      const int nrt = i < count ? row_tiles(s[0], G) : 0;
      per[0] = 0;
      if (nrt <= 4)
#pragma unroll 1
        for (int rt = 0; rt < nrt; ++rt) per[0] += geometry(a, s[0], G, rt).units();
#pragma unroll 1
      for (unsigned todo = __ballot_sync(0xffffffffu, nrt > 4); todo; todo &= todo - 1) {
        const int src = __ffs(todo) - 1;
        const int y = head_units(a, shfl_seq(s[0], src), G);
        if (lane == src) per[0] = y;
      }
      if (i < count) s_units[i] = per[0] * a.Hkv;
    }
    __syncthreads();
    sum = 0;
#pragma unroll 1
    for (int i = lane; i < count; i += 32) sum = line_add(sum, s_units[i]);
    // (in a loop: unrolled, long chunks take 1.7% longer, by where the later code then lies)
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) sum = line_add(sum, __shfl_xor_sync(0xffffffffu, sum, o));
  };
  // (one loop for the sum and the search: little code, which a call has to fetch first)
  int total = 0, before = 0, first = 0;
#pragma unroll 1
  for (int x = 0; x < 2 * rounds; ++x) {
    const int r = x < rounds ? x : x - rounds;
    if (x < rounds || rounds > 1) load(r);
    if (x < rounds) {
      total = line_add(total, sum);
      if (x + 1 < rounds) continue;
      if (total == kLineTooLong) total = 0;
      first = stretch(total, blockIdx.x);
      const int end = stretch(total, blockIdx.x + 1);
      if (threadIdx.x == 0) {
        plan.total = total;
        plan.first = first;
        plan.end = end;
      }
      if (first == end) return;  // (uniform)
      continue;
    }
    if (first >= before + sum) {  // (uniform)
      before += sum;
      continue;
    }
    // the sequence that holds the first unit, and the units before it
    int n = -1, pre = before;
#pragma unroll 1
    for (int base = 0; base < count; base += 32) {
      const int mine = base + lane < count ? s_units[base + lane] : 0;
      int run = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += y;
      }
      const unsigned b = __ballot_sync(0xffffffffu, first < pre + run);
      if (b) {
        const int src = __ffs(b) - 1;
        n = base + src;
        pre += __shfl_sync(0xffffffffu, run - mine, src);
        break;
      }
      pre += __shfl_sync(0xffffffffu, run, 31);
    }
    // its warp has it at hand
    const bool few = count <= kFew;
    if (n < 0 || (few ? n % W : n / 32) != warp) return;
    const int src = n & 31;
    note_start(a, plan, few ? (n < W ? s[0] : s[1]) : shfl_seq(s[0], src), r * kPlanSeqs + n,
               few ? (n < W ? per[0] : per[1]) : __shfl_sync(0xffffffffu, per[0], src),
               first - pre);
    return;
  }
}

// What a CTA's units work on together; made by the query warp, kSteps of them ahead at most.
enum Kind : int {
  kEnd,    // nothing more
  kWide,   // one item, 128 rows for each unit, every tile for both
  kSplit,  // one narrow item, the same rows for both units, every other tile for each
  kPair,   // two narrow items, one for each unit
};
struct Item {
  int n, h, bos, pos0;  // sequence, kv head, first token and its position
  int v0, v1;           // its tiles in the stretch
  Geometry g;
};
struct Step {
  int kind;
  Item it[2];
  __device__ __forceinline__ int tiles(int i) const { return it[i].v1 - it[i].v0; }
};
constexpr int kSteps = 4;
// Two narrow items next to each other are worked on side by side when neither has more than
// kSkew tiles more than the other: their starts and ends then pass beside the other's tiles.  What
// is left of a longer one would go through one unit alone.
constexpr int kSkew = 3;

// A step's order of key and value tiles in the ring, that in which the products use them:
// wide K0 V0 K1 V1 ...; otherwise K0 K1 V0 K2 V1 ... (the second unit's scores start before the
// first unit's values are needed), where tiles go to the units in turn, a pair's last ones to the
// unit of the longer item.
struct Order {
  int kind, n;  // tiles in all
  int turns;    // tiles that the units take in turn
  int longer;   // the unit that takes the others
  __device__ __forceinline__ explicit Order(const Step& s) {
    kind = s.kind;
    const int n0 = s.tiles(0), n1 = kind == kPair ? s.tiles(1) : 0;
    n = n0 + n1;
    turns = kind == kPair ? 2 * min(n0, n1) : n;
    longer = n1 > n0;
  }
  // Number of unit u's i-th tile (split: the item's i-th).
  __device__ __forceinline__ int tile(int u, int i) const {
    return kind == kPair ? (2 * i < turns ? 2 * i + u : turns / 2 + i) : i;
  }
  // Unit and place in its item of tile t of a pair.
  __device__ __forceinline__ int unit(int t) const { return t < turns ? t & 1 : longer; }
  __device__ __forceinline__ int place(int t) const { return t < turns ? t / 2 : t - turns / 2; }
  // Entry of tile t's keys, values.
  __device__ __forceinline__ uint32_t key(int t) const {
    return kind == kWide ? uint32_t(2 * t) : t == 0 ? 0u : uint32_t(2 * t - 1);
  }
  __device__ __forceinline__ uint32_t value(int t) const {
    return kind == kWide ? uint32_t(2 * t + 1) : uint32_t(min(2 * t + 2, 2 * n - 1));
  }
  // The tile of entry e.
  __device__ __forceinline__ int tile_of(int e) const {
    if (kind == kWide) return e / 2;
    return e == 0 ? 0 : e == 2 * n - 1 ? n - 1 : e & 1 ? (e + 1) / 2 : e / 2 - 1;
  }
  // The unit that uses entry e (not wide: both do).
  __device__ __forceinline__ int owner(int e) const { return unit(tile_of(e)); }
};

// ------------------------------------------------------------------------ small pieces

// 32 consecutive columns of the thread's lane: the load, and the wait after which (and only
// then) its registers may be read.
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32_finish(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]),
                 "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// Packed pairs of fp32: a b + c, a + b.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 32 bytes to a 32-byte boundary: a whole sector, where two 16-byte stores are two partial ones.
__device__ __forceinline__ void store32(void* p, const uint32_t* x) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(x[0]), "r"(x[1]),
               "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void tmem_st16_nowait(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32_nowait(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
      "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
      "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
      "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Byte offset of the 16-byte piece `ch` of row r in a 128-row tile, swizzled as TMA lays it.
template <int D>
__device__ __forceinline__ uint32_t piece_offset(int r, int ch) {
  if (D == 32) return uint32_t(r * 64 + ((ch ^ (r >> 1 & 3)) << 4));
  return sw128_offset<2>(128, r, ch * 8);
}

// Softmax weights of 32 scores: p = 2^(s sc + nb), packed to bf16; their sum (in fp32, before the
// rounding) and the largest score, started or carried on.
__device__ __forceinline__ void weights32(const uint32_t (&s)[32], float sc, float nb, uint32_t* p,
                                          float& sum, float& top, bool start) {
  const uint64_t sc2 = pack2(sc, sc), nb2 = pack2(nb, nb);
  uint64_t acc[4] = {0, 0, 0, 0};
  float c4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float s0 = __uint_as_float(s[2 * e]), s1 = __uint_as_float(s[2 * e + 1]);
    c4[e & 3] = max3(c4[e & 3], s0, s1);
    float x, y;
    unpack2(fma2(pack2(s0, s1), sc2, nb2), x, y);
    x = fast_exp2(x);
    y = fast_exp2(y);
    acc[e & 3] = add2(acc[e & 3], pack2(x, y));
    p[e] = pack_bf16(x, y);
  }
  float x, y;
  unpack2(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])), x, y);
  sum = start ? x + y : sum + (x + y);
  const float t = fmaxf(max3(c4[0], c4[1], c4[2]), c4[3]);
  top = start ? t : fmaxf(top, t);
}

struct Bars {
  uint64_t kv_full[8], kv_empty[8], q_full[2], q_empty[2], s_full[2], s_empty[2], p_full[2],
      o_full[2], turn[2], ph_full[2], oh_full[2], join, step_full[kSteps], step_empty[kSteps];
};

// A wait that gives up (after 2 to 8 seconds) marks the thread dead: it then runs through the
// rest of its step without waiting (its results are void) and leaves, so that every loop ends.
// Tries are counted, not timed: there are many of these loops, and their instructions push those
// of the softmax out of the cache.
__device__ __forceinline__ void wait_or_die(uint64_t* bar, uint32_t parity, bool& dead) {
  if (dead) return;
#pragma unroll 1
  for (int i = 0; !mbar_try_wait_short(bar, parity); ++i)
    if (i == 2000000) {
      dead = true;
      atomicOr(&g_paged_error, 64u);
      break;
    }
}

// ONE: whole tiles with weights of their own in one pass (D <= 64 without a window).
template <int D, bool ONE>
__global__ void __launch_bounds__(kThreads, 1)
paged_tc_kernel(PagedArgs a, const __grid_constant__ CUtensorMap qmap,
                const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap, int q_boxes, Header* headers,
                float* part_o, float2* part_ml) {
  using C = Cfg<D>;
  constexpr int NS = C::kStages, RB = C::kRowBytes, HALVES = D * 2 / RB;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  float2* s_ml = reinterpret_cast<float2*>(smem_raw);  // [2][128]: m, l of the units' rows
  struct Small {
    Bars bars;
    Plan plan;
    Step steps[kSteps];
    uint32_t tmem;
  };
  static_assert(2048 + sizeof(Small) <= kFront, "front");
  Small& small = *reinterpret_cast<Small*>(smem_raw + 2048);
  Bars& bars = small.bars;
  Plan& plan = small.plan;
  uint32_t& s_tmem = small.tmem;
  uint8_t* sQ = smem_raw + kFront;           // two 128-row tiles
  uint8_t* sKV = sQ + 2 * C::kQBytes;        // the ring

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == kMmaWarp) tmem_alloc(&s_tmem, kTmemCols);
  if (tid == 32 * kLoadWarp) {
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&bars.kv_full[i], 1);
      mbar_init(&bars.kv_empty[i], 2);  // both units let an entry go
    }
    for (int u = 0; u < 2; ++u) {
      mbar_init(&bars.q_full[u], 1);
      mbar_init(&bars.q_empty[u], 2);
      mbar_init(&bars.s_full[u], 1);
      mbar_init(&bars.s_empty[u], 4);
      mbar_init(&bars.p_full[u], 4);
      mbar_init(&bars.o_full[u], 1);
      mbar_init(&bars.turn[u], 1);
      mbar_init(&bars.ph_full[u], 4);
      mbar_init(&bars.oh_full[u], 1);
    }
    mbar_init(&bars.join, 8);
    for (int i = 0; i < kSteps; ++i) {
      mbar_init(&bars.step_full[i], 1);
      mbar_init(&bars.step_empty[i], 11);  // load, products, softmaxes: one for each warp
    }
    fence_mbar_init();
  }
  make_plan(a, plan, reinterpret_cast<int*>(sKV));  // (the ring is not in use yet)
  fence_async_smem();  // the plan's numbers lay where copies will land
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may be set up
  const uint32_t tm = s_tmem;
  bool dead = false;
  // The CTA's j-th step (null: none, or the warp has given up), and that the warp is done with it.
  auto step = [&](uint32_t j) -> const Step* {
    wait_or_die(&bars.step_full[j % kSteps], (j / kSteps) & 1, dead);
    dead = __any_sync(0xffffffffu, dead);
    const Step* s = &small.steps[j % kSteps];
    return dead || s->kind == kEnd ? nullptr : s;
  };
  auto step_done = [&](uint32_t j) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars.step_empty[j % kSteps]);
  };

  if (warp >= kLoadWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == kLoadWarp) {
      const int ps = a.page_size, ppt = kKeys / ps;  // pages of a tile: 8, 4, 2 or 1
      // Lane 8 x + p looks up and copies page p of the tiles x, x + 4, ..., four tiles ahead.
      const int quarter = lane >> 3, pi = lane & 7;
      uint32_t pos = 0, sg = 0, ph = 0;  // entries pushed, the next one's stage and phase
      for (uint32_t j = 0;; ++j) {
        const Step* st = step(j);
        if (!st) break;
        const Order o(*st);
        const bool pair = o.kind == kPair;
        int x = pair ? quarter & 1 : 0;  // the item of the lane's tiles
        Item w = st->it[x];
        int row = -1;       // of the page in the caches, for the lane's tile; -1: not needed
        bool fresh = true;  // a look-up that has not been made a row yet
        int page = 0, head = -1;
        auto look_up = [&](int t) {
          head = -1;
          fresh = true;
          if (pi >= ppt || t >= o.n) return;
          if (pair && o.unit(t) != x) {
            x = o.unit(t);
            w = st->it[x];
          }
          const int k0 = tile_start(w.g, w.v0 + (pair ? o.place(t) : t)) + pi * ps;
          if (k0 >= w.g.kr.hi || (k0 + ps <= w.g.kr.lo && k0 >= w.g.kr.sinks)) return;
          head = w.h;
          page = __ldg(a.block_table + (long long)w.n * a.max_pages + k0 / kKeys * ppt + pi);
        };
        auto settle = [&]() {  // (touches the loaded number: a tile later)
          if (fresh) row = head < 0 ? -1 : (min(max(page, 0), a.num_pages - 1) * a.Hkv + head) * ps;
          fresh = false;
        };
        look_up(quarter);
        settle();
        const bool wide = o.kind == kWide;
#pragma unroll 1
        for (int t = -1; t < o.n; ++t) {
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const bool keys = (z == 0) != wide;  // the next tile's; or this tile's values
            const int y = keys ? t + 1 : t;
            if (y < 0 || y >= o.n) continue;
            wait_or_die(&bars.kv_empty[sg], ph ^ 1, dead);
            const bool mine = (y & 3) == quarter && row >= 0;
            const unsigned need = __ballot_sync(0xffffffffu, mine);
            uint64_t* bar = &bars.kv_full[sg];
            if (lane == 0)
              mbar_arrive_expect_tx(bar, uint32_t(__popc(need)) * uint32_t(HALVES * ps * RB));
            __syncwarp();
            if (mine && !dead) {
              uint8_t* dst = sKV + sg * C::kStageBytes + pi * ps * RB;
#pragma unroll
              for (int hf = 0; hf < HALVES; ++hf)
                tma_load_2d(dst + hf * (kKeys * RB), keys ? &kmap : &vmap, bar, hf * 64, row);
            }
            __syncwarp();
            if (++sg == NS) {
              sg = 0;
              ph ^= 1;
            }
            ++pos;
          }
          if (t >= 0) {
            settle();
            if ((t & 3) == quarter) look_up(t + 4);
            __syncwarp();
          }
        }
        step_done(j);
      }
      // leave no copy in flight behind a give-up
      if (dead)
        for (uint32_t i = pos > NS ? pos - NS : 0; i < pos; ++i)
          mbar_wait(&bars.kv_full[i % NS], (i / NS) & 1, 100000000ull);
    } else if (warp < kQueryWarp) {
      // Products of unit u.  Each unit has a warp, so that one's waits pass while the tensor
      // cores work for the other.  The whole warp walks and waits, one lane issues.  Addresses
      // are made warp-uniform before the issuing branch: from values of one lane, eight
      // products took 800 to 1200 cycles to issue, twice their run time.
      const int u = warp - kMmaWarp;
      const uint32_t idesc_s = make_idesc(1, 128, kKeys);
      const uint32_t idesc_o = make_idesc(1, 128, D, false, true);
      const uint32_t tmu = __shfl_sync(0xffffffffu, tm + 128 * u, 0);
      const uint32_t q0 = smem_u32(sQ), kv0 = smem_u32(sKV);
      const bool leader = elect_one();
      uint32_t pos = 0, seen = 0, np = 0, items = 0, wides = 0, turns = 0, nscores = 0;
      // Ring entries up to `at` have landed.  Every entry is waited for in turn, and the other
      // unit's are let go at once: a stage is refilled only when both units have passed it, so
      // no barrier is ever more than the one phase away that a parity can tell.
      auto ready = [&](uint32_t at, const Order& o) {
        for (; (int)(at - seen) >= 0; ++seen) {
          wait_or_die(&bars.kv_full[seen % NS], (seen / NS) & 1, dead);
          if (o.kind != kWide && o.owner((int)(seen - pos)) != u && leader)
            mbar_arrive(&bars.kv_empty[seen % NS]);
        }
      };
      auto stage = [&](uint32_t at) {
        return __shfl_sync(0xffffffffu, kv0 + at % NS * C::kStageBytes, 0);
      };
      auto scores = [&](uint32_t q, uint32_t k) {  // S = Q K^T
        const uint64_t kd = make_sdesc(k, 16, 8 * RB, C::kSwizzle);
        const uint64_t qd = make_sdesc(q, 16, 8 * RB, C::kSwizzle);
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          // the K step's 32 bytes, in 16-byte units; 64-column blocks are 16 KB apart
          const uint64_t off = (s / 4) * (kKeys * RB / 16) + (s % 4) * 2;
          mma_ss(tmu + kColS, qd + off, kd + off, idesc_s, s > 0);
        }
      };
      // O (+)= P V over a part of the keys: halves of the tile, or all of it.
      constexpr int kHalf = kKeys / 32;
      auto values = [&](uint32_t v, bool first, bool lower, bool upper) {
        const uint64_t vd = make_sdesc(v, kKeys * RB, 8 * RB, C::kSwizzle);
#pragma unroll
        for (int s = 0; s < 2 * kHalf; ++s)
          if (s < kHalf ? lower : upper)
          mma_ts(tmu + kColO, tmu + (C::kOwnP ? kColP64 : kColS) + 8 * s, vd + s * (16 * RB / 16),
                 idesc_o, !(first && s == 0));
      };
      // Weights of their own: scores wait only for the last ones to have been read.
      auto scores_free = [&]() {
        if (C::kOwnP) wait_or_die(&bars.s_empty[u], (nscores & 1) ^ 1, dead);
        ++nscores;
      };
      for (uint32_t j = 0;; ++j) {
        const Step* st = step(j);
        if (!st) break;
        const Order o(*st);
        const int kind = o.kind, n = kind == kPair ? st->tiles(u) : o.n;
        const bool split = kind == kSplit;
        const int tile = split ? 0 : u;  // of the query rows
        const uint32_t q = __shfl_sync(0xffffffffu, q0 + tile * C::kQBytes, 0);
        const int first = split ? u : 0, by = split ? 2 : 1;
        // Every step fills the first tile; both units wait for it and let it go in each, so that
        // it never gets a phase ahead of either.  The second tile is unit 1's, which counts for
        // two.
        wait_or_die(&bars.q_full[0], items & 1, dead);
        if (tile) {
          if (leader) mbar_arrive(&bars.q_empty[0]);
          wait_or_die(&bars.q_full[1], wides & 1, dead);
        }
        ++items;
        wides += !split;
        if (first < n) {
          // the first scores
          const uint32_t k_at = pos + o.key(o.tile(u, first));
          ready(k_at, o);
          scores_free();
          tc_fence_after();
          const uint32_t k = stage(k_at);
          if (leader) {
            if (!dead) scores(q, k);
            mma_commit(&bars.s_full[u]);
            mma_commit(&bars.kv_empty[k_at % NS]);
            if (first + by >= n) {
              mma_commit(&bars.q_empty[tile]);
              if (tile) mma_commit(&bars.q_empty[tile]);
            }
          }
          __syncwarp();
        } else if (leader) {
          mbar_arrive(&bars.q_empty[tile]);
        }
        // a tile's values, then the unit's next scores
        for (int i = first; i < n; i += by) {
          const bool more = i + by < n;
          const uint32_t v_at = pos + o.value(o.tile(u, i));
          const uint32_t k_at = pos + o.key(o.tile(u, i + by));
          auto next_scores = [&](uint32_t k) {  // by the leader
            if (!dead) scores(q, k);
            mma_commit(&bars.s_full[u]);
            mma_commit(&bars.kv_empty[k_at % NS]);
            if (i + 2 * by >= n) {
              mma_commit(&bars.q_empty[tile]);
              if (tile) mma_commit(&bars.q_empty[tile]);
            }
          };
          if constexpr (C::kOwnP) {
            if (more) {
              ready(k_at, o);
              scores_free();
              tc_fence_after();
              const uint32_t k = stage(k_at);
              if (leader) next_scores(k);
              __syncwarp();
            }
            ready(v_at, o);
            const uint32_t v = stage(v_at);
            wait_or_die(&bars.p_full[u], np & 1, dead);
            ++np;
            tc_fence_after();
            if (leader) {
              if (!dead) values(v, i == first, true, true);
              mma_commit(&bars.o_full[u]);
              mma_commit(&bars.kv_empty[v_at % NS]);
            }
            __syncwarp();
          } else {
            ready(v_at, o);
            if (more) ready(k_at, o);
            const uint32_t v = stage(v_at), k = stage(k_at);
            // the lower half of the keys' weights comes first
            wait_or_die(&bars.ph_full[u], np & 1, dead);
            // A wide item's units take turns: interleaved, both would get their scores late and
            // their softmaxes would fall together; one after the other, one unit's softmax runs
            // beside the other's products.
            if (kind == kWide) {
              wait_or_die(&bars.turn[u], (turns & 1) ^ (u == 0), dead);
              ++turns;
            }
            tc_fence_after();
            if (leader) {
              if (!dead) values(v, i == first, true, false);
              mma_commit(&bars.oh_full[u]);
            }
            __syncwarp();
            wait_or_die(&bars.p_full[u], np & 1, dead);
            ++np;
            tc_fence_after();
            if (leader) {
              if (!dead) {
                values(v, false, false, true);
                if (more) scores(q, k);
              }
              if (kind == kWide) mbar_arrive(&bars.turn[u ^ 1]);
              mma_commit(more ? &bars.s_full[u] : &bars.o_full[u]);
              mma_commit(&bars.kv_empty[v_at % NS]);
              if (more) mma_commit(&bars.kv_empty[k_at % NS]);
              if (more && i + 2 * by >= n) {
                mma_commit(&bars.q_empty[tile]);
                if (tile) mma_commit(&bars.q_empty[tile]);
              }
            }
            __syncwarp();
          }
        }
        ready(pos + 2 * o.n - 1, o);
        pos += 2 * o.n;
        step_done(j);
      }
    } else {
      // The steps, one ahead of the query rows of each; a tile of rows as soon as the products on
      // its last rows are done.
      Walker w;
      bool live = w.start(a, plan);
      Header hd;
      hd.rows = 0;
      uint32_t nq0 = 0, nq1 = 0;
      for (uint32_t j = 0;; ++j) {
        wait_or_die(&bars.step_empty[j % kSteps], ((j / kSteps) & 1) ^ 1, dead);
        dead = __any_sync(0xffffffffu, dead);
        if (dead) break;
        Step& next = small.steps[j % kSteps];
        int kind = kEnd;
#pragma unroll 1
        for (int x = 0, n = 0; x < 2 && live; ++x) {
          if (x == 0) {
            kind = w.narrow() ? kSplit : kWide;
            n = w.tiles();
          } else {
            if (kind != kSplit || !w.narrow() || abs(w.tiles() - n) > kSkew) break;
            kind = kPair;
          }
          if (lane == 0) {
            Item& it = next.it[x];
            it.n = w.n; it.h = w.h; it.bos = w.s.bos; it.pos0 = w.s.pos0;
            it.v0 = w.v0; it.v1 = w.v1;
            it.g = w.g;
          }
          if (w.v0 == 0 && w.v1 < w.g.nt) {  // starts here and goes on: only the last item does
            hd.rows = w.g.rows;
            hd.row0 = w.g.row0;
            hd.h = w.h;
            hd.nt = w.g.nt;
            hd.bos = w.s.bos;
            hd.start = plan.end - w.v1;
            hd.total = plan.total;
          }
          live = w.next(a);
        }
        if (lane == 0) {
          next.kind = kind;
          mbar_arrive(&bars.step_full[j % kSteps]);
        }
        __syncwarp();
        // the rows of the step before
        const Step& st = small.steps[(j + kSteps - 1) % kSteps];
        const int before = j == 0 ? kEnd : st.kind;
#pragma unroll 1
        for (int t = 0; t < (before == kEnd ? 0 : before == kSplit ? 1 : 2); ++t) {
          const Item& it = st.it[before == kPair ? t : 0];
          const int skip = before == kWide ? t * kRowsUnit : 0;
          const int rows = min(it.g.rows - skip, kRowsUnit), row0 = it.g.row0 + skip;
          const int bos = it.bos, h = it.h;
          wait_or_die(&bars.q_empty[t], ((t ? nq1 : nq0) & 1) ^ 1, dead);
          if (t)
            ++nq1;
          else
            ++nq0;
          if (q_boxes && rows > 32) {
            // 128 rows are whole tokens: a box of 64 columns, the kv head's query heads and
            // those tokens (what lies behind the sequence is read and not used)
            if (lane == 0 && !dead) {
              mbar_arrive_expect_tx(&bars.q_full[t], C::kQBytes);
#pragma unroll
              for (int hf = 0; hf < HALVES; ++hf)
                tma_load_3d(sQ + t * C::kQBytes + hf * (kRowsUnit * RB), &qmap, &bars.q_full[t],
                            hf * 64, h * a.G, bos + div_g(a, row0));
            }
            __syncwarp();
            continue;
          }
          constexpr int CH = D / 8, RPI = 32 / CH;  // 16-byte pieces of a row, rows at a time
          const uint32_t dst = smem_u32(sQ + t * C::kQBytes);
          const int ch = lane % CH;
          for (int r = lane / CH; r < rows; r += RPI) {
            const int tk = div_g(a, row0 + r), hg = row0 + r - tk * a.G;
            const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) +
                                       (long long)(bos + tk) * a.q_stride +
                                       (long long)(h * a.G + hg) * D + ch * 8;
            cp_async16(dst + piece_offset<D>(r, ch), src);
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.q_full[t]);
        }
        if (kind == kEnd) break;
      }
      if (lane == 0) headers[blockIdx.x] = hd;
      // leave no copy in flight behind a give-up (each tile's last one at most)
      if (dead)
        for (int t = 0; t < 2; ++t)
          if ((t ? nq1 : nq0) > 0)
            mbar_wait(&bars.q_full[t], ((t ? nq1 : nq0) - 1) & 1, 100000000ull);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int u = warp >> 2, r = tid & 127;  // unit, row within it
    const uint32_t lanebits = uint32_t(warp & 3) << 21;  // (32 * warp of the group) << 16
    const uint32_t tS = tm + kColS + 128 * u + lanebits, tO = tm + kColO + 128 * u + lanebits;
    const uint32_t tO0 = tm + kColO + lanebits, tO1 = tO0 + 128;
    const uint32_t tP = C::kOwnP ? tm + kColP64 + 128 * u + lanebits : tS;
    const float sc = a.scale * kLog2E;
    uint32_t pos = 0, ns = 0, no = 0, joins = 0;
    auto join = [&]() {  // all softmax warps
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.join);
      wait_or_die(&bars.join, joins & 1, dead);
      ++joins;
    };
    for (uint32_t j = 0;; ++j) {
      const Step* st = step(j);
      if (!st) break;
      const Order order(*st);
      const bool split = order.kind == kSplit;
      const Item w = st->it[order.kind == kPair ? u : 0];
      const int n = w.v1 - w.v0;
      const int base = order.kind == kWide ? u * kRowsUnit : 0;  // first row of the unit's tile
      const int nr = min(w.g.rows - base, kRowsUnit);  // its rows (1 at least)
      const bool active = (warp & 3) * 32 < nr;      // (warp-uniform)
      const int row = w.g.row0 + base + min(r, nr - 1);
      const int tk = div_g(a, row);

      // 1. The unit's tiles.
      float m = -INFINITY, l = 0.f;
      int mine = 0;
      const int mypos = w.pos0 + tk;
      const int pos_first = w.pos0 + div_g(a, w.g.row0 + base);
      const int pos_last = w.pos0 + div_g(a, w.g.row0 + base + nr - 1);
      for (int i = split ? u : 0; i < n; i += split ? 2 : 1) {
        const int ks = tile_start(w.g, w.v0 + i);
        wait_or_die(&bars.s_full[u], ns & 1, dead);
        ++ns;
        tc_fence_after();
        bool halves = false;  // the lower half of the weights has been handed over
        // The scores are in the warp's registers (or it has no rows): the next may come.
        auto scores_read = [&]() {
          if (C::kOwnP) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.s_empty[u]);
          }
        };
        // The product that reads the last weights and adds to O is done.  Every warp waits for
        // it, rows or not: none may run ahead and arrive for a tile whose last is still open.
        auto weights_free = [&]() {
          if (C::kOwnP) {
            wait_or_die(&bars.o_full[u], (no & 1) ^ 1, dead);
            tc_fence_after();
          }
        };
        if (C::kOwnP && !active) {
          scores_read();
          weights_free();
        }
        if (active) {
          // a tile needs masks where some row of the unit does not see all of it
          const bool whole =
              ks + kKeys <= pos_first + 1 &&
              (a.window == 0 || ks > max(pos_last, 0) - a.window || ks + kKeys <= a.sinks);
          bool done = false;
          // O and l to another maximum (mine > 0, or O is not there yet).
          bool lower = false;  // the product of the tile's lower half is in O
          auto rescale = [&](float mn) {
            const float f = mn == -INFINITY ? 1.f : fast_exp2((m - mn) * sc);
            m = mn;
            l *= f;
            if (mine > 0 || lower) {
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                float o[16];
                tmem_ld16(tO + c, o);
                uint32_t x[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(o[e] * f);
                tmem_st16(tO + c, x);
              }
            }
          };
          constexpr bool kOnePass = !C::kOwnP || ONE;
          if (kOnePass && whole && mine == 0) {
            // no maximum yet: that of the first 32 keys
            uint32_t s[32];
            tmem_ld32_start(tS, s);
            tmem_ld32_finish(s);
            float c4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 32; c += 2)
              c4[c / 2 & 3] =
                  max3(c4[c / 2 & 3], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
            m = fmaxf(max3(c4[0], c4[1], c4[2]), c4[3]);
          }
          if (!C::kOwnP && whole) {
            // Weights against the maximum so far, which almost always stands, while the
            // tile's own maximum is found beside them; the scores stay until that is known.
            // The lower half of the keys is handed over while the upper is computed.
            const float nb = m == -INFINITY ? 0.f : -m * sc;
            uint32_t p[32], s[2][32];
            float sum, top;
            // (rows behind the item's last hold anything, and must not choose the way: the two
            // ways sum in different orders)
            auto outgrown = [&]() { return r < nr && top > m && (top - m) * sc > kRescale; };
            tmem_ld32_start(tS, s[0]);
            tmem_ld32_finish(s[0]);
            tmem_ld32_start(tS + 32, s[1]);
            weights32(s[0], sc, nb, p, sum, top, true);
            tmem_ld32_finish(s[1]);
            tmem_ld32_start(tS + 64, s[0]);
            weights32(s[1], sc, nb, p + 16, sum, top, false);
            done = !__any_sync(0xffffffffu, outgrown());
            if (done) {
              tmem_st32_nowait(tP, p);
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bars.ph_full[u]);
              l += sum;
            }
            tmem_ld32_finish(s[0]);
            if (done) {
              tmem_ld32_start(tS + 96, s[1]);
              weights32(s[0], sc, nb, p, sum, top, true);
              tmem_ld32_finish(s[1]);
              weights32(s[1], sc, nb, p + 16, sum, top, false);
              if (__any_sync(0xffffffffu, outgrown())) {
                // The upper half has outgrown the range: once the lower half's product is in O,
                // O and l are scaled down and the upper half's weights made again.
                wait_or_die(&bars.oh_full[u], (ns - 1) & 1, dead);
                tc_fence_after();
                lower = true;
                rescale(outgrown() ? top : m);
                const float nb2 = m == -INFINITY ? 0.f : -m * sc;
                tmem_ld32_start(tS + 64, s[0]);
                tmem_ld32_finish(s[0]);
                weights32(s[0], sc, nb2, p, sum, top, true);
                weights32(s[1], sc, nb2, p + 16, sum, top, false);
              }
              tmem_st32_nowait(tP + 32, p);
              l += sum;
              halves = true;
            }
          }
          if (C::kOwnP && kOnePass && whole) {
            // The same in one piece; the scores stay until the tile's own maximum is known.
            const float nb = m == -INFINITY ? 0.f : -m * sc;
            uint32_t p[2][32], s[2][32];
            float sum, top;
            tmem_ld32_start(tS, s[0]);
            tmem_ld32_finish(s[0]);
            tmem_ld32_start(tS + 32, s[1]);
            weights32(s[0], sc, nb, p[0], sum, top, true);
            tmem_ld32_finish(s[1]);
            tmem_ld32_start(tS + 64, s[0]);
            weights32(s[1], sc, nb, p[0] + 16, sum, top, false);
            tmem_ld32_finish(s[0]);
            tmem_ld32_start(tS + 96, s[1]);
            weights32(s[0], sc, nb, p[1], sum, top, false);
            tmem_ld32_finish(s[1]);
            weights32(s[1], sc, nb, p[1] + 16, sum, top, false);
            done = !__any_sync(0xffffffffu, r < nr && top > m && (top - m) * sc > kRescale);
            if (done) {
              scores_read();
              weights_free();
              tmem_st32_nowait(tP, p[0]);
              tmem_st32_nowait(tP + 32, p[1]);
              l += sum;
            }
          }
          if (!done) {
            // The first tile, masked ones, and a maximum that has outgrown the range: the
            // maximum first, then the weights.
            // Bits of the keys that the thread's row sees: not in the future, and in the
            // window or among the sinks.
            const int hi = whole ? kKeys : mypos - ks + 1;  // keys [0, hi) of the tile
            const int lo = a.window && !whole ? max(mypos, 0) - a.window - ks + 1 : 0;
            const int sk = a.window ? a.sinks - ks : 0;
            auto bits = [&](int q) -> uint32_t {
              auto below = [&](int x) -> uint32_t {  // bits [0, x - 32 q)
                const int b = x - 32 * q;
                return b <= 0 ? 0u : b >= 32 ? 0xffffffffu : (1u << b) - 1u;
              };
              return below(hi) & (~below(lo) | below(sk));
            };
            auto mask = [&](uint32_t(&s)[32], int q) {
              const uint32_t b = bits(q);
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(b >> c & 1)) s[c] = 0xff800000u;  // -inf: weight zero
            };
            float c4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            auto largest = [&](const uint32_t(&s)[32]) {
#pragma unroll
              for (int c = 0; c < 32; c += 2)
                c4[c / 2 & 3] =
                    max3(c4[c / 2 & 3], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
            };
            float nb = 0.f;
            auto standing = [&]() {
              const float mx = fmaxf(max3(c4[0], c4[1], c4[2]), c4[3]);
              weights_free();
              const bool grow = r < nr && mx > m && (mx - m) * sc > kRescale;  // (m = -inf: any)
              if (__any_sync(0xffffffffu, grow)) rescale(grow ? mx : m);
              nb = m == -INFINITY ? 0.f : -m * sc;
            };
            auto weigh = [&](const uint32_t(&s)[32], int q) {
              uint32_t p[16];
              float sum, top;
              weights32(s, sc, nb, p, sum, top, true);
              l += sum;
              tmem_st16_nowait(tP + 16 * q, p);
            };
            if constexpr (!kOnePass) {
              // the scores are read at once, so that the next can be made
              uint32_t s[4][32];
#pragma unroll
              for (int q = 0; q < 4; ++q) tmem_ld32_start(tS + 32 * q, s[q]);
#pragma unroll
              for (int q = 0; q < 4; ++q) tmem_ld32_finish(s[q]);
              scores_read();
              if (!whole) {
#pragma unroll
                for (int q = 0; q < 4; ++q) mask(s[q], q);
              }
#pragma unroll
              for (int q = 0; q < 4; ++q) largest(s[q]);
              standing();
#pragma unroll
              for (int q = 0; q < 4; ++q) weigh(s[q], q);
            } else {
              // twice, in loops: their instructions do not push the other roles' out of the cache
              // (weights go over scores that have been read)
              uint32_t s[32];
#pragma unroll 1
              for (int q = 0; q < 4; ++q) {
                tmem_ld32_start(tS + 32 * q, s);
                tmem_ld32_finish(s);
                if (!whole) mask(s, q);
                largest(s);
              }
              standing();
#pragma unroll 1
              for (int q = 0; q < 4; ++q) {
                tmem_ld32_start(tS + 32 * q, s);
                tmem_ld32_finish(s);
                if (q == 3) scores_read();
                if (!whole) mask(s, q);
                weigh(s, q);
              }
            }
          }
        }
        // Keys of this tile that no row of the item sees: their values become zeros (weight
        // zero times what the cache holds there need not be zero).  Behind the wait for the
        // scores: the products before them have used every earlier entry of the ring, so the
        // value stage's barrier is in the phase that is waited for.
        if (ks + kKeys > w.g.kr.hi || (ks < w.g.kr.lo && ks + kKeys > w.g.kr.sinks)) {
          const uint32_t at = pos + order.value(order.tile(u, i));
          wait_or_die(&bars.kv_full[at % NS], (at / NS) & 1, dead);
          const int key = ks + r;
          if (key >= w.g.kr.hi || (key < w.g.kr.lo && key >= w.g.kr.sinks)) {
            uint8_t* vrow = sKV + (at % NS) * C::kStageBytes + r * RB;
#pragma unroll
            for (int hf = 0; hf < HALVES; ++hf)
#pragma unroll
              for (int ch = 0; ch < RB / 16; ++ch)  // (from another piece in each lane: all banks)
                *reinterpret_cast<uint4*>(vrow + hf * (kKeys * RB) +
                                          ((ch + lane) & (RB / 16 - 1)) * 16) =
                    make_uint4(0, 0, 0, 0);
          }
          fence_async_smem();
        }
        if (active) tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (!C::kOwnP && !halves) mbar_arrive(&bars.ph_full[u]);
          mbar_arrive(&bars.p_full[u]);
        }
        ++mine;
        if (C::kOwnP) ++no;
      }

      // 2. The unit's result.  A narrow item's two are joined, half of the columns by each unit:
      // a warp reaches both accumulators' lanes.
      if (mine > 0) {  // (kOwnP: a phase for each tile, the last one of which is waited for)
        if (!C::kOwnP) ++no;
        wait_or_die(&bars.o_full[u], (no & 1) ^ 1, dead);
      }
      float f0 = 1.f, f1 = 0.f;  // of units 0 and 1 (wide: f0 is the unit's own)
      const bool both = split && n > 1;
      constexpr int kShare = D == 32 ? 32 : D / 2;  // columns of unit 0
      if (split) {
        s_ml[128 * u + r] = make_float2(m, l);
        tc_fence_before();
        join();
        const float2 x = s_ml[r], y = s_ml[128 + r];
        m = x.x;
        l = x.y;
        if (both) {
          m = fmaxf(x.x, y.x);
          const float b = m == -INFINITY ? 0.f : m;
          f0 = fast_exp2((x.x - b) * sc);
          f1 = fast_exp2((y.x - b) * sc);
          l = x.y * f0 + y.y * f1;
        }
      }
      tc_fence_after();
      const bool cut0 = w.v0 > 0, cut1 = w.v1 < w.g.nt;
      if (active) {
        const bool valid = r < nr;
        const long long orow =
            (long long)(w.bos + tk) * a.Hq + w.h * a.G + (row - tk * a.G);
        const float inv = l == 0.f ? 0.f : 1.0f / l;
        const long long prow =
            (long long)(2 * blockIdx.x + (cut0 ? 0 : 1)) * kRowsItem + base + r;
        __nv_bfloat16* orowp = static_cast<__nv_bfloat16*>(a.out) + orow * D;
        const bool wide_stores = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
#pragma unroll 1
        for (int c = split ? u * kShare : 0; c < (split && u == 0 ? kShare : D); c += 32) {
          uint32_t o[32], o1[32];
          tmem_ld32_start((split ? tO0 : tO) + c, o);
          tmem_ld32_start((both ? tO1 : split ? tO0 : tO) + c, o1);
          tmem_ld32_finish(o);
          tmem_ld32_finish(o1);
          if (both) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = __float_as_uint(__uint_as_float(o[e]) * f0 + __uint_as_float(o1[e]) * f1);
          }
          if (!valid) continue;
          if (cut0 || cut1) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) store32(part_o + prow * D + c + e, o + e);
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 16) {
              uint32_t x[8];
#pragma unroll
              for (int q = 0; q < 8; ++q)
                x[q] = l == 0.f ? 0u
                                : pack_bf16(__uint_as_float(o[e + 2 * q]) * inv,
                                            __uint_as_float(o[e + 2 * q + 1]) * inv);
              if (wide_stores) {
                store32(orowp + c + e, x);
              } else {
                uint4* dst = reinterpret_cast<uint4*>(orowp + c + e);
                dst[0] = make_uint4(x[0], x[1], x[2], x[3]);
                dst[1] = make_uint4(x[4], x[5], x[6], x[7]);
              }
            }
          }
        }
        if (valid && (!split || u == 0)) {
          if (cut0 || cut1)
            part_ml[prow] = make_float2(m * sc, l);
          else if (a.lse)
            a.lse[orow] =
                l == 0.f ? -INFINITY : (m * sc + log2f(l)) * 0.6931471805599453f;
        }
      }
      tc_fence_before();
      if (split) join();  // (neither overwrites what the other reads)
      pos += 2 * order.n;
      step_done(j);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) {
    tmem_relinquish();
    tmem_dealloc(tm, kTmemCols);
  }
}

// Joins the partial results of an item that was cut: the CTA it starts in has it in its second
// slot, the following ones in their first.  Blocks (c, .): the item that starts in CTA c's
// stretch; a thread has four columns of a row and takes four parts at a time, all their loads in
// flight together (eight: 39.8 against 37.5 us for a call with 150 items cut in two).
template <int D>
__global__ void __launch_bounds__(256) paged_join_kernel(PagedArgs a, const Header* headers,
                                                         const float* part_o,
                                                         const float2* part_ml) {
  constexpr int PIECES = D / 4, U = 4;
  const int c = blockIdx.x;
  // launched while the first kernel runs: wait for its results
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Header hd = headers[c];
  if (hd.rows == 0) return;
  // CTAs from this one to the one it ends in
  const int parts = stretch_of(hd.total, hd.start + hd.nt - 1) - c + 1;
  for (int at = blockIdx.y * 256 + threadIdx.x; at < hd.rows * PIECES; at += gridDim.y * 256) {
    const int r = at / PIECES, e = at % PIECES;
    // Row of the i-th part in the partial results, -1 if that CTA has no tile of the item.
    auto place = [&](int i) -> int {
      const int k = c + i;
      const int first = stretch(hd.total, k) - hd.start;
      const int last = min(stretch(hd.total, k + 1) - hd.start, hd.nt);
      return i < parts && last > max(first, 0) ? (2 * k + (i == 0)) * kRowsItem + r : -1;
    };
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < parts; i0 += U) {
      float2 ml[U];
      float4 x[U];
      float mn = m;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int p = place(i0 + i);
        ml[i] = p >= 0 ? part_ml[p] : make_float2(-INFINITY, 0.f);
        x[i] = p >= 0 ? *reinterpret_cast<const float4*>(part_o + (long long)p * D + 4 * e)
                      : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (ml[i].y != 0.f) mn = fmaxf(mn, ml[i].x);  // (a part that saw nothing has no say)
      const float b = mn == -INFINITY ? 0.f : mn, f = fast_exp2(m - b);
      m = mn;
      l *= f;
      o.x *= f; o.y *= f; o.z *= f; o.w *= f;
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (ml[i].y != 0.f) {
          const float g = fast_exp2(ml[i].x - b);
          l += ml[i].y * g;
          o.x += x[i].x * g;
          o.y += x[i].y * g;
          o.z += x[i].z * g;
          o.w += x[i].w * g;
        }
    }
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    const int tk = div_g(a, hd.row0 + r);
    const long long row =
        (long long)(hd.bos + tk) * a.Hq + hd.h * a.G + (hd.row0 + r - tk * a.G);
    uint2 w;
    w.x = pack_bf16(o.x * inv, o.y * inv);
    w.y = pack_bf16(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row * D + 4 * e) = w;
    if (e == 0 && a.lse)
      a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
  }
}

bool cache_map(CUtensorMap* map, const void* base, const PagedArgs& a) {
  const auto enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)a.D,
                              (cuuint64_t)a.num_pages * a.Hkv * (cuuint64_t)a.page_size};
  const cuuint64_t strides[1] = {(cuuint64_t)a.D * 2};
  const cuuint32_t box[2] = {a.D == 32 ? 32u : 64u, (cuuint32_t)a.page_size};
  const cuuint32_t es[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             a.D == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Query rows: 128 rows of a kv head as a box of whole tokens, where its query heads divide 128.
bool query_map(CUtensorMap* map, const PagedArgs& a) {
  const auto enc = encode_fn();
  if (!enc) return false;
  const cuuint32_t G = (cuuint32_t)(a.Hq / a.Hkv);
  const cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)a.Hq, (cuuint64_t)a.total_T};
  const cuuint64_t strides[2] = {(cuuint64_t)a.D * 2, (cuuint64_t)a.q_stride * 2};
  const cuuint32_t box[3] = {a.D == 32 ? 32u : 64u, G, kRowsUnit / G};
  const cuuint32_t es[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             a.D == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_t(PagedArgs a, void* workspace, cudaStream_t st) {
  // x / G = (mulhi(x, g_mul) + x) >> g_shift for x < 2^31
  const uint32_t G = (uint32_t)(a.Hq / a.Hkv);
  a.G = (int)G;
  a.g_shift = 0;
  while ((1u << a.g_shift) < G) ++a.g_shift;
  a.g_mul = (uint32_t)((((1ull << a.g_shift) - G) << 32) / G + 1);
  CUtensorMap qmap{}, kmap{}, vmap{};
  // Rows by TMA where the items are large: a call with one token for each of its sequences has
  // a few rows in each, which are copied one by one.
  const int q_boxes = kRowsUnit % G == 0 && (long long)a.total_T * G > 32 && query_map(&qmap, a);
  if (a.num_pages > 0 && a.max_pages > 0)
    if (!cache_map(&kmap, a.k_cache, a) || !cache_map(&vmap, a.v_cache, a))
      return cudaErrorInvalidValue;
  Header* headers = static_cast<Header*>(workspace);
  float2* ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + 8192);
  float* po = reinterpret_cast<float*>(ml + (size_t)2 * kCtas * kRowsItem);
  // D <= 64: chunks of 2048 behind 8192 keys, 32 + 4 heads of 64: 320 us for 352 with one pass over
  // whole tiles, 148 for 162 with D = 32.  Masked tiles are faster unrolled, which the one pass
  // does not go with; under a window they can be many (a third in the windowed batch above: 36.2 us for
  // 35.1).  How many there are lies in device memory, so any window counts as narrow: a chunk under
  // a wide one forgoes the gain.
  auto kernel = paged_tc_kernel<D, false>;
  if constexpr (Cfg<D>::kOwnP)
    if (a.window == 0) kernel = paged_tc_kernel<D, true>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  kernel<<<kCtas, kThreads, Cfg<D>::kSmem, st>>>(a, qmap, kmap, vmap, q_boxes, headers, po, ml);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // a thread per four columns of the largest item there can be
  const long long rows = (long long)a.total_T * G;
  const unsigned by = (unsigned)((rows < kRowsItem ? rows : kRowsItem) * (D / 4) + 255) / 256;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kCtas, by);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<D>, a, (const Header*)headers,
                            (const float*)po, (const float2*)ml);
}

}  // namespace

static_assert(sizeof(Header) * kCtas <= 8192, "headers");

// Whether the line of key tiles, at the block table's capacity, fits the kernel's indices.
bool paged_tc_index_ok(const PagedArgs& a) {
  const double rows = (double)a.total_T * (a.Hq / a.Hkv) / kRowsItem + a.N;
  const double tiles = (double)a.max_pages * a.page_size / kKeys + kOverheadMost + 2;
  return rows * tiles * a.Hkv < 2147483647.0;
}

size_t paged_tc_workspace(int D) {
  return 8192 + (size_t)2 * kCtas * kRowsItem * (sizeof(float2) + D * sizeof(float));
}

cudaError_t launch_paged_tc(const PagedArgs& a, void* workspace, cudaStream_t st) {
  return a.D == 32   ? launch_t<32>(a, workspace, st)
         : a.D == 64 ? launch_t<64>(a, workspace, st)
                     : launch_t<128>(a, workspace, st);
}

unsigned int paged_read_error(bool reset) {
  unsigned int v = 0;
  cudaMemcpyFromSymbol(&v, g_paged_error, sizeof(v));
  if (reset) {
    const unsigned int z = 0;
    cudaMemcpyToSymbol(g_paged_error, &z, sizeof(z));
  }
  return v;
}

}  // namespace kda
