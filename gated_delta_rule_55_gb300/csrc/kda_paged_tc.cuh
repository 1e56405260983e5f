// Attention of new tokens over a paged cache (kda_paged_attention_fwd, _q8_fwd,
// kda_paged_prefix_attention_fwd) on the tensor cores: bf16 queries.  Included once for each kind
// of call, by the file that launches it.
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
// Caches in 8 bits (Q8).  D = 128: a key tile is an operand as it lands, e4m3 with e4m3, the
// queries as two terms hi + lo of that type (made before, kda_cache_q8.cu), whose two products take
// the tensor cores as long as one of bf16; the scores are multiplied by their keys' scales, and a
// fourth warpgroup expands value tiles to bf16 where they landed, a thread for each key's row.  The
// columns of four change places on the way (kda_q8.cuh), and O's change back as it is read.  2
// chunks of 2048 tokens behind 8192 keys, 32 + 8 heads: 538 us, 61% of a library product's rate
// (over bf16 pages 394 to 406: the expanding takes 105 us of the softmax warps' issue slots, the
// keys' scales 37); with keys expanded too 932.  The expanding is a loop (unrolled: 618).  D <= 64:
// keys and values land in a ring of their own and are expanded, with their scales, into that of the
// products.
//
// Shared prefixes (PRE).  A row has two lists of keys, its group's prefix and its own, both of them
// items of the line; each item leaves its rows' (m, l, O), whole or in parts, and paged_rows_kernel
// joins a row's two sides.  64 single tokens behind 16384 shared and 16..1024 own keys, 32 + 8
// heads of 128: 54 us for 30 of bytes.  8 chunks of 100..512 tokens behind 8191 keys: 233 to 241 us
// (161 of flops); their groups go alone (kda_paged_plan.cuh).
//
// Softmax weights are rounded to bf16 for the product (their sum is taken before, in fp32).
// Keys that no row of the item sees (behind the last one, outside the window, pages that are
// not loaded) have weight zero and their values are overwritten with zeros in shared memory,
// so what the cache holds there never counts.
#pragma once

#include "kda_paged_line.h"

namespace kda {
namespace {
constexpr int kStretches = kCtas;  // one CTA per SM
constexpr int kRowsItem = 256;
constexpr int kRowsFew = 128;
// An item counts some units beside its tiles: what its start and end cost a CTA (the units lie
// before its tiles, and a cut among them falls to the item's first tile).  A wide one of D = 128
// counts 3: 12 sequences of 1 to 600 tokens, 32 + 8 heads, take 125 us for 132 with 2 and 145
// with 1; 256 single tokens 111 us with 2, 114 with 3; the mixed batch above 35.0 with 2, 35.7
// with 3.
//
// Behind prefixes, where the rows of a group fill wide items beside the narrow ones of the
// sequences' own keys, a wide tile counts 3 and a narrow one 2: as equals, the CTAs with the prefix
// of 64 single tokens behind 16384 keys took 56 us, the others 37.
constexpr int kTile = kPrefixes ? 2 : 1, kTileMost = kPrefixes ? 3 : 1;
constexpr int kOverhead = kPrefixes ? 4 : 2, kOverheadMost = kPrefixes ? 15 : 3;
}  // namespace
}  // namespace kda

#include "kda_paged_plan.cuh"

namespace kda {
namespace {

constexpr int kRowsUnit = 128;   // query rows of a unit
constexpr int kLoadWarp = 8, kMmaWarp = 9 /* and 10: one per unit */, kQueryWarp = 11;
constexpr int kExpandWarp = 12;  // and 13 to 15: caches in 8 bits

// Two softmax warpgroups, one of the warps above, and one that expands 8-bit tiles.  Registers: 168
// a thread at launch (3 x 128 threads), moved to the softmax warpgroups: 2 x 216 + 72 = 3 x 168;
// with the fourth warpgroup 128: 2 x 184 + 72 + 72 = 4 x 128.
template <bool Q8> struct Group {
  static constexpr int kThreads = Q8 ? 512 : 384;
  static constexpr int kRegsSoftmax = Q8 ? 184 : 216, kRegsOther = 72, kRegsExpand = 72;
};
// log2 growth of the maximum that O and l absorb.  (Rescaling only from some growth on, and two
// softmax warpgroups beside two score tiles, are published ways for attention on this hardware.)
// Weights, sums and O keep their relative precision whatever their size, so what bounds it is
// overflow: 2^32 leaves values times keys seen of 2^95 (values of 2^80 and 2^15 keys).  Keys of
// different magnitudes outgrow 2^8 in some row of a warp every few tiles, and such a tile goes the
// long way: 2 chunks of 2048 tokens behind 8192 keys in 8 bits whose magnitudes vary by e^0.7 took
// 1003 us.  bf16 pages, whose values may be larger, keep to 2^8, with prefixes as without.
template <bool Q8> constexpr float kRescaleOf = Q8 ? 32.0f : 8.0f;
// Direct keys (8 bits, D = 128): scores of e4m3 rows, up to 448^2 128 < 2^25, are multiplied by
// their keys' scales, up to 2^119, before the query row's own scale, so the keys' are kept 2^16
// lower and the rows' 2^16 higher: keys of all magnitudes stay inside fp32, the smallest scale
// (2^-110) a normal number.
constexpr float kKeyDown = 0x1p-16f, kRowUp = 0x1p16f;
// How far (log2) above the first 32 keys' maximum the standing one starts.
template <bool Q8> constexpr float kAheadOf = Q8 ? 24.0f : 0.0f;

template <int D, bool Q8> struct Cfg {
  // 8 bits and D = 128: keys are products' operands as they land (kDirect), in a ring of their own;
  // values land in the upper half of their stage and are expanded where they are.  Otherwise all
  // tiles are in one ring, and those in 8 bits land in another one.
  static constexpr bool kDirect = Q8 && D == 128;
  // What lies before the tiles: m and l of both units' rows (2 KB), barriers, the plan; 8 bits:
  // the scales of the tiles that have landed.
  static constexpr int kFront = (Q8 ? 4 : 3) * 1024;
  static constexpr int kStageBytes = kKeys * D * 2;
  // (direct: of each, and no fewer: a unit's values wait for its next keys, two tiles on)
  static constexpr int kStages = kDirect ? 3 : Q8 ? 6 : D == 128 ? 5 : 8;
  static constexpr int kBars = kDirect ? 2 * kStages : kStages;
  // A direct stage of keys: the tile, and the scales as fp32.
  static constexpr int kKeyBytes = kDirect ? kKeys * D + kKeys * 4 : 0;
  // Tiles in 8 bits, as they land.
  static constexpr int kRawStages = kDirect ? 6 : Q8 ? 6 : 0;
  static constexpr int kRawBytes = kKeys * D;
  static constexpr int kQBytes = kRowsUnit * D * 2;
  // Rows in shared memory: blocks of up to 64 columns, swizzled over their bytes.
  static constexpr int kRowBytes = D == 32 ? 64 : 128;
  static constexpr uint32_t kSwizzle = D == 32 ? 4 : kSwizzle128;  // 64-byte, 128-byte
  // D <= 64 leaves Tensor Memory for weights of their own (D = 128 keeps them over the scores):
  // the next scores are then made while the softmax of the last is still running.
  static constexpr bool kOwnP = D <= 64;
  static constexpr int kSmem = kFront + 2 * kQBytes + kStages * kStageBytes +
                               (kDirect ? kStages * kKeyBytes : kRawStages * kRawBytes);
};

constexpr uint32_t kColS = 0, kColO = 256, kTmemCols = 512;  // + 128 * unit
constexpr uint32_t kColP64 = kColO + 64;                     // weights, D <= 64

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
  int start_at;         // its first tile in the line
  Geometry g;
};
struct Step {
  int kind;
  Item it[2];
  __device__ __forceinline__ int tiles(int i) const { return it[i].v1 - it[i].v0; }
};
constexpr int kSteps = 4;

// A call with prefixes: what is known of each row, its prefix's first, [2][total_T][Hq].
struct Rows {
  int4* at;    // row_at()
  float2* ml;  // of items that are not cut: m and l
  float* o;    // [.][D]
};
// Where a row's parts are: the item's first tile in the line, its tiles (0: not cut; -1: it has no
// other side, and is joined as an item where it is cut); row in the item, units of a tile, this CTA
// (that it starts in), the number of CTAs to its last tile's; the line's length.
__device__ __forceinline__ int4 row_at(const Item& w, bool cut, int row, int total) {
  const int c = blockIdx.x, unit = w.g.cost();
  const int parts =
      cut ? stretch_of<kStretches>(total, w.start_at + unit * (w.g.nt - 1)) - c + 1 : 1;
  return make_int4(w.start_at, w.g.list >= 0 ? -1 : cut ? w.g.nt : 0,
                   row | unit << 8 | c << 12 | parts << 20, total);
}
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
  __device__ __forceinline__ bool is_key(int e) const {
    return kind == kWide ? !(e & 1) : e == 0 || ((e & 1) && e != 2 * n - 1);
  }
  // The unit that uses entry e (not wide: both do).
  __device__ __forceinline__ int owner(int e) const { return unit(tile_of(e)); }
};

// ------------------------------------------------------------------------ small pieces

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

template <bool B> struct Bool { static constexpr bool value = B; };

// 32 scores times their keys' scales.
__device__ __forceinline__ void scale32(uint32_t (&s)[32], const float* c) {
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(c + e);
    float x[4];
    unpack2(mul2(pack2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), f.x), x[0], x[1]);
    unpack2(mul2(pack2(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), f.y), x[2], x[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) s[e + i] = __float_as_uint(x[i]);
  }
}

// Softmax weights of 32 scores: p = 2^(s sc + nb), packed to bf16; their sum (in fp32, before the
// rounding) and the largest score, started or carried on.  SC: scores times their keys' scales c.
template <bool SC>
__device__ __forceinline__ void weights32(const uint32_t (&s)[32], const float* c, float sc,
                                          float nb, uint32_t* p, float& sum, float& top,
                                          bool start) {
  const uint64_t sc2 = pack2(sc, sc), nb2 = pack2(nb, nb);
  uint64_t acc[4] = {0, 0, 0, 0};
  float c4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  ulonglong2 f{};
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float s0 = __uint_as_float(s[2 * e]), s1 = __uint_as_float(s[2 * e + 1]);
    if constexpr (SC) {
      if (e % 2 == 0) f = *reinterpret_cast<const ulonglong2*>(c + 2 * e);
      unpack2(mul2(pack2(s0, s1), e % 2 ? f.y : f.x), s0, s1);
    }
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

template <int NR>  // stages that 8-bit tiles land in
struct Bars {
  uint64_t raw_full[NR ? NR : 1], raw_empty[NR ? NR : 1];
  uint64_t kv_full[8], kv_empty[8], q_full[2], q_empty[2], s_full[2], s_empty[2], p_full[2],
      o_full[2], turn[2], ph_full[2], oh_full[2], join, step_full[kSteps], step_empty[kSteps];
};

// ONE: whole tiles with weights of their own in one pass (D <= 64 without a window).  Q8: caches in
// 8 bits, whose tiles land in a ring of their own and are expanded into that of the products.
// PRE: every row has two lists of keys, a prefix and its own; results go to `rows` instead of out.
template <int D, bool ONE, bool Q8, bool PRE>
__global__ void __launch_bounds__(Group<Q8>::kThreads, 1)
paged_tc_kernel(PagedArgs a, const __grid_constant__ CUtensorMap qmap,
                const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap, int q_boxes, Header* headers,
                float* part_o, float2* part_ml, Rows rows) {
  using C = Cfg<D, Q8>;
  constexpr int NS = C::kStages, RB = C::kRowBytes, HALVES = D * 2 / RB;
  constexpr int NL = Q8 ? C::kRawStages : NS;  // stages of the ring that tiles land in
  constexpr bool KD = C::kDirect;
  constexpr float kRescale = kRescaleOf<Q8>, kAhead = kAheadOf<Q8>;
  constexpr int kThreads = Group<Q8>::kThreads, kFront = C::kFront;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  float2* s_ml = reinterpret_cast<float2*>(smem_raw);  // [2][128]: m, l of the units' rows
  struct Small {
    Bars<C::kRawStages> bars;
    Plan plan;
    Step steps[kSteps];
    uint32_t tmem;
    alignas(16) uint8_t scales[Q8 ? NL * kKeys : 16];  // of the tiles in 8 bits
  };
  static_assert(2048 + sizeof(Small) <= kFront, "front");
  Small& small = *reinterpret_cast<Small*>(smem_raw + 2048);
  Bars<C::kRawStages>& bars = small.bars;
  Plan& plan = small.plan;
  uint32_t& s_tmem = small.tmem;
  uint8_t* sQ = smem_raw + kFront;           // two 128-row tiles
  uint8_t* sKV = sQ + 2 * C::kQBytes;        // the ring
  uint8_t* sRaw = sKV + NS * C::kStageBytes;  // and that of tiles in 8 bits; or that of keys,
  float* sKeyScale = reinterpret_cast<float*>(sRaw + NS * C::kRawBytes);  // [NS][128] (direct)

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == kMmaWarp) tmem_alloc(&s_tmem, kTmemCols);
  if (tid == 32 * kLoadWarp) {
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  if (tid == 0) {
    for (int i = 0; i < C::kBars; ++i) {
      mbar_init(&bars.kv_full[i], Q8 ? 4 : 1);
      mbar_init(&bars.kv_empty[i], 2);  // both units let an entry go
    }
    for (int i = 0; i < C::kRawStages; ++i) {
      mbar_init(&bars.raw_full[i], 1);
      mbar_init(&bars.raw_empty[i], 4);
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
      // load, products, softmaxes, expanders: one for each warp
      mbar_init(&bars.step_empty[i], Q8 ? 15 : 11);
    }
    fence_mbar_init();
  }
  make_plan<kThreads>(a, plan, reinterpret_cast<int*>(sKV));  // (the ring is not in use yet)
  fence_async_smem();  // the plan's numbers lay where copies will land
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may be set up
  if (KD) asm volatile("griddepcontrol.wait;" ::: "memory");  // for the queries' terms
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

  // Barrier (and stage) and phase of a tile's keys and values, `pos` entries before its step.
  // (Direct: stages of keys, then of values.)
  struct Place {
    uint32_t at, phase;
  };
  auto ring = [](uint32_t i, uint32_t first) {
    return Place{first + i % NS, (i / NS) & 1};
  };
  auto key_place = [&](const Order& o, uint32_t pos, int t) {
    return KD ? ring(pos / 2 + t, 0) : ring(pos + o.key(t), 0);
  };
  auto value_place = [&](const Order& o, uint32_t pos, int t) {
    return KD ? ring(pos / 2 + t, NS) : ring(pos + o.value(t), 0);
  };
  auto entry_place = [&](const Order& o, uint32_t pos, int e) {
    return KD ? ring(pos / 2 + o.tile_of(e), o.is_key(e) ? 0 : NS) : ring(pos + e, 0);
  };

  if (Q8 && warp >= kExpandWarp) {
    if constexpr (Q8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Group<Q8>::kRegsExpand));
    // A thread has a key's row of each tile: its bytes into registers, the landing stage let go,
    // and the row written as bf16 in the products' layout.
    const int r = tid - 32 * kExpandWarp;
    uint32_t pos = 0;
    for (uint32_t j = 0;; ++j) {
      const Step* st = step(j);
      if (!st) break;
      const Order o(*st);
      const int n = 2 * o.n;
#pragma unroll 1
      for (int e = 0; e < n; ++e) {
        const Place to = entry_place(o, pos, e);
        const Place from = KD ? to : Place{(pos + e) % NL, ((pos + e) / NL) & 1};
        wait_or_die(&bars.raw_full[from.at], from.phase, dead);
        const uint32_t byte = small.scales[from.at * kKeys + r];
        if (KD && o.is_key(e)) {
          sKeyScale[to.at * kKeys + r] = q8::scale(byte) * kKeyDown;
        } else {
          const q8::Scale16 sc(byte);
          uint8_t* dst = sKV + (KD ? to.at - NS : to.at) * C::kStageBytes;
          const uint8_t* src = KD ? dst + C::kRawBytes : sRaw + from.at * C::kRawBytes;
          const bool big = __any_sync(0xffffffffu, sc.big);
          if (!KD) wait_or_die(&bars.kv_empty[to.at], to.phase ^ 1, dead);
          // In a loop: little code.  (Direct: the pieces that are written over the row's bytes are
          // behind those that have been read.)
          uint4 w = *reinterpret_cast<const uint4*>(src + raw_offset<D>(r, 0));
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
            if (c + 1 < D / 16)
              w = *reinterpret_cast<const uint4*>(src + raw_offset<D>(r, c + 1));
            uint32_t y[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (KD)  // (values: their columns change places)
                q8::expand4(x[k], sc, y[2 * k], y[2 * k + 1]);
              else
                q8::expand4_in_order(x[k], sc, y[2 * k], y[2 * k + 1]);
            }
            if (big)
#pragma unroll
              for (int k = 0; k < 8; ++k) y[k] = q8::mul_bf16x2(y[k], sc.more);
            *reinterpret_cast<uint4*>(dst + piece_offset<D>(r, 2 * c)) =
                make_uint4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<uint4*>(dst + piece_offset<D>(r, 2 * c + 1)) =
                make_uint4(y[4], y[5], y[6], y[7]);
          }
          if (!KD) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.raw_empty[from.at]);
          }
          fence_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.kv_full[to.at]);
      }
      pos += n;
      step_done(j);
    }
    }
  } else if (warp >= kLoadWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Group<Q8>::kRegsOther));
    if (warp == kLoadWarp) {
      const int ps = a.page_size, ppt = kKeys / ps;  // pages of a tile: 8, 4, 2 or 1
      // Lane 8 x + p looks up and copies page p of the tiles x, x + 4, ..., four tiles ahead.
      const int quarter = lane >> 3, pi = lane & 7;
      uint64_t *const landed = Q8 ? bars.raw_full : bars.kv_full;
      uint64_t *const gone = Q8 && !KD ? bars.raw_empty : bars.kv_empty;
      uint32_t pos = 0, sg = 0, ph = 0;  // entries pushed, the next one's stage and phase
      uint32_t keys_pushed = 0;
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
          const int v = w.v0 + (pair ? o.place(t) : t);
          const int k0 = tile_start(w.g, v) + pi * ps;
          const bool along = PRE && v < w.g.ns;  // a prefix's tile before the own ones
          if (PRE ? k0 >= (along ? w.g.kr.sinks : w.g.kr.hi)
                  : k0 >= w.g.kr.hi || (k0 + ps <= w.g.kr.lo && k0 >= w.g.kr.sinks))
            return;
          head = w.h;
          const int32_t* table = PRE ? table_of(a, along ? w.g.list : w.n)
                                     : a.block_table + (long long)w.n * a.max_pages;
          page = __ldg(table + k0 / kKeys * ppt + pi);
        };
        auto settle = [&]() {  // (touches the loaded number: a tile later)
          if (fresh) row = head < 0 ? -1 : (min(max(page, 0), a.num_pages - 1) * a.Hkv + head) * ps;
          fresh = false;
        };
        look_up(quarter);
        settle();
        const bool wide = o.kind == kWide;
        const uint32_t base = pos;
#pragma unroll 1
        for (int t = -1; t < o.n; ++t) {
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const bool keys = (z == 0) != wide;  // the next tile's; or this tile's values
            const int y = keys ? t + 1 : t;
            if (y < 0 || y >= o.n) continue;
            const Place at = !KD    ? Place{sg, ph}
                             : keys ? key_place(o, base, y)
                                    : value_place(o, base, y);
            wait_or_die(&gone[at.at], at.phase ^ 1, dead);
            const bool mine = (y & 3) == quarter && row >= 0;
            const unsigned need = __ballot_sync(0xffffffffu, mine);
            uint64_t* bar = &landed[at.at];
            if (lane == 0)
              mbar_arrive_expect_tx(bar, uint32_t(__popc(need)) *
                                             uint32_t(Q8 ? ps * (D + 1) : HALVES * ps * RB));
            __syncwarp();
            if (Q8 && mine && !dead) {
              uint8_t* dst = KD && !keys
                                 ? sKV + (at.at - NS) * C::kStageBytes + C::kRawBytes
                                 : sRaw + at.at * C::kRawBytes;
              tma_load_2d(dst + pi * ps * D, keys ? &kmap : &vmap, bar, 0, row);
              bulk_load(small.scales + at.at * kKeys + pi * ps,
                        (keys ? a.k_scale : a.v_scale) + row, ps, bar);
            }
            if (!Q8 && mine && !dead) {
              uint8_t* dst = sKV + at.at * C::kStageBytes + pi * ps * RB;
#pragma unroll
              for (int hf = 0; hf < HALVES; ++hf)
                tma_load_2d(dst + hf * (kKeys * RB), keys ? &kmap : &vmap, bar, hf * 64, row);
            }
            __syncwarp();
            if (!KD && ++sg == NL) {
              sg = 0;
              ph ^= 1;
            }
            ++pos;
            if (keys) ++keys_pushed;
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
      if (dead && KD)
        for (uint32_t v = 0; v < 2; ++v)
          for (uint32_t end = v ? pos - keys_pushed : keys_pushed, i = end > NS ? end - NS : 0;
               i < end; ++i)
            mbar_wait(&landed[v * NS + i % NS], (i / NS) & 1, 100000000ull);
      if (dead && !KD)
        for (uint32_t i = pos > NL ? pos - NL : 0; i < pos; ++i)
          mbar_wait(&landed[i % NL], (i / NL) & 1, 100000000ull);
    } else if (warp < kQueryWarp) {
      // Products of unit u.  Each unit has a warp, so that one's waits pass while the tensor
      // cores work for the other.  The whole warp walks and waits, one lane issues.  Addresses
      // are made warp-uniform before the issuing branch: from values of one lane, eight
      // products took 800 to 1200 cycles to issue, twice their run time.
      const int u = warp - kMmaWarp;
      const uint32_t idesc_s = make_idesc(KD ? 0 : 1, 128, kKeys);
      const uint32_t idesc_o = make_idesc(1, 128, D, false, true);
      const uint32_t tmu = __shfl_sync(0xffffffffu, tm + 128 * u, 0);
      const uint32_t q0 = smem_u32(sQ), kv0 = smem_u32(sKV);
      const bool leader = elect_one();
      uint32_t pos = 0, seen = 0, np = 0, items = 0, wides = 0, turns = 0, nscores = 0;
      uint32_t k_last = 0;  // stage of the last scores' keys
      // Ring entries up to number e of the step have landed.  Every entry is waited for in turn,
      // and the other unit's are let go at once: a stage is refilled only when both units have
      // passed it, so no barrier is ever more than the one phase away that a parity can tell.
      auto ready = [&](int e, const Order& o) {
        for (; (int)(pos + e - seen) >= 0; ++seen) {
          const int x = (int)(seen - pos);
          const Place at = entry_place(o, pos, x);
          wait_or_die(&bars.kv_full[at.at], at.phase, dead);
          if (o.kind != kWide && o.owner(x) != u && leader) mbar_arrive(&bars.kv_empty[at.at]);
        }
      };
      auto key_stage = [&](const Place& p) {
        return __shfl_sync(0xffffffffu,
                           KD ? smem_u32(sRaw) + p.at * C::kRawBytes : kv0 + p.at * C::kStageBytes,
                           0);
      };
      auto value_stage = [&](const Place& p) {
        return __shfl_sync(0xffffffffu, kv0 + (KD ? p.at - NS : p.at) * C::kStageBytes, 0);
      };
      auto scores = [&](uint32_t q, uint32_t k) {  // S = Q K^T
        const uint64_t kd = make_sdesc(k, 16, 8 * RB, C::kSwizzle);
        const uint64_t qd = make_sdesc(q, 16, 8 * RB, C::kSwizzle);
        if constexpr (KD) {  // the queries' two terms, in the halves of their tile
#pragma unroll
          for (int s = 0; s < 2 * (D / 32); ++s)
            mma_ss_f8(tmu + kColS, qd + (s / 4) * (kRowsUnit * 128 / 16) + (s % 4) * 2,
                      kd + (s % 4) * 2, idesc_s, s > 0);
          return;
        }
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
          const int t = o.tile(u, first);
          const Place k_at = key_place(o, pos, t);
          ready((int)o.key(t), o);
          scores_free();
          tc_fence_after();
          const uint32_t k = key_stage(k_at);
          k_last = k_at.at;
          if (leader) {
            if (!dead) scores(q, k);
            mma_commit(&bars.s_full[u]);
            if (!KD) mma_commit(&bars.kv_empty[k_at.at]);
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
          const int t = o.tile(u, i), t1 = o.tile(u, i + by);
          const Place v_at = value_place(o, pos, t), k_at = key_place(o, pos, t1);
          const int v_e = (int)o.value(t), k_e = (int)o.key(t1);
          auto next_scores = [&](uint32_t k) {  // by the leader
            if (!dead) scores(q, k);
            mma_commit(&bars.s_full[u]);
            mma_commit(&bars.kv_empty[k_at.at]);
            if (i + 2 * by >= n) {
              mma_commit(&bars.q_empty[tile]);
              if (tile) mma_commit(&bars.q_empty[tile]);
            }
          };
          if constexpr (C::kOwnP) {
            if (more) {
              ready(k_e, o);
              scores_free();
              tc_fence_after();
              const uint32_t k = key_stage(k_at);
              if (leader) next_scores(k);
              __syncwarp();
            }
            ready(v_e, o);
            const uint32_t v = value_stage(v_at);
            wait_or_die(&bars.p_full[u], np & 1, dead);
            ++np;
            tc_fence_after();
            if (leader) {
              if (!dead) values(v, i == first, true, true);
              mma_commit(&bars.o_full[u]);
              mma_commit(&bars.kv_empty[v_at.at]);
            }
            __syncwarp();
          } else {
            ready(v_e, o);
            if (more) ready(k_e, o);
            const uint32_t v = value_stage(v_at), k = key_stage(k_at);
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
              mma_commit(&bars.kv_empty[v_at.at]);
              // (direct keys: their scales were in use until the weights were there)
              if (KD) mma_commit(&bars.kv_empty[k_last]);
              if (!KD && more) mma_commit(&bars.kv_empty[k_at.at]);
              if (more && i + 2 * by >= n) {
                mma_commit(&bars.q_empty[tile]);
                if (tile) mma_commit(&bars.q_empty[tile]);
              }
            }
            __syncwarp();
            k_last = k_at.at;
          }
        }
        ready(2 * o.n - 1, o);
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
            kind = (w.g.rows <= kRowsUnit) ? kSplit : kWide;
            n = w.tiles();
          } else {
            if (kind != kSplit || w.g.rows > kRowsUnit || abs(w.tiles() - n) > kSkew) break;
            kind = kPair;
          }
          if (lane == 0) {
            Item& it = next.it[x];
            it.n = w.n; it.h = w.h; it.bos = w.s.bos; it.pos0 = w.s.pos0;
            it.v0 = w.v0; it.v1 = w.v1; it.start_at = w.start_at;
            it.g = w.g;
          }
          // starts here and goes on: only the last item does (and its rows have no other side)
          if (w.v0 == 0 && w.v1 < w.g.nt && (!PRE || w.g.list >= 0)) {
            hd.unit = w.g.cost();
            hd.rows = w.g.rows;
            hd.row0 = w.g.row0;
            hd.h = w.h;
            hd.nt = w.g.nt;
            hd.bos = w.s.bos;
            hd.start = w.start_at;
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
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Group<Q8>::kRegsSoftmax));
    const int u = warp >> 2, r = tid & 127;  // unit, row within it
    const uint32_t lanebits = uint32_t(warp & 3) << 21;  // (32 * warp of the group) << 16
    const uint32_t tS = tm + kColS + 128 * u + lanebits, tO = tm + kColO + 128 * u + lanebits;
    const uint32_t tO0 = tm + kColO + lanebits, tO1 = tO0 + 128;
    const uint32_t tP = C::kOwnP ? tm + kColP64 + 128 * u + lanebits : tS;
    float sc = a.scale * kLog2E;
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
      if (KD) {  // with the power of two of the row's terms
        const float x = a.scale * kLog2E;
        const float y =
            __ldg(a.q_scale + (long long)(w.bos + tk) * a.Hq + w.h * a.G + (row - tk * a.G));
        sc = x > 1.f ? x * y * kRowUp : x * kRowUp * y;  // (neither order leaves fp32 on the way)
        if (sc < 1.2e-38f) sc = 1.2e-38f;  // (zero times a hidden key's -inf would be NaN)
        if (sc > 3.4e38f) sc = 3.4e38f;    // (and infinity times a score of zero)
      }
      float m = -INFINITY, l = 0.f;
      int mine = 0;
      // (a prefix is seen to its last key by all)
      auto limit = [&](int x) { return PRE ? min(x, w.g.kr.hi - 1) : x; };
      const int mypos = limit(w.pos0 + tk);
      const int pos_first = limit(w.pos0 + div_g(a, w.g.row0 + base));
      const int pos_last = limit(w.pos0 + div_g(a, w.g.row0 + base + nr - 1));
      for (int i = split ? u : 0; i < n; i += split ? 2 : 1) {
        const int ks = tile_start(w.g, w.v0 + i);
        const bool along = PRE && w.v0 + i < w.g.ns;  // a prefix's tile before the own ones
        const int tile = order.tile(u, i);
        const float* cols = nullptr;
        if (KD) {
          const Place at = key_place(order, pos, tile);
          wait_or_die(&bars.kv_full[at.at], at.phase, dead);  // (written by the expanders)
          cols = sKeyScale + at.at * kKeys;
        }
        wait_or_die(&bars.s_full[u], ns & 1, dead);
        ++ns;
        tc_fence_after();
        bool halves = false;  // the lower half of the weights has been handed over
        // Scores from column c on, waited for, times the keys' scales.
        auto finish = [&](uint32_t(&s)[32], int c) {
          tmem_ld32_finish(s);
          if (KD) scale32(s, cols + c);
        };
        auto weights = [&](const uint32_t(&s)[32], int c, float nb, uint32_t* p, float& sum,
                           float& top, bool start) {
          weights32<KD>(s, cols + c, sc, nb, p, sum, top, start);
        };
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
              along ? ks + kKeys <= w.g.kr.sinks
                    : ks + kKeys <= pos_first + 1 &&
                          (a.window == 0 || ks > max(pos_last, 0) - a.window ||
                           ks + kKeys <= a.sinks);
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
            finish(s, 0);
            float c4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 32; c += 2)
              c4[c / 2 & 3] =
                  max3(c4[c / 2 & 3], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
            m = fmaxf(max3(c4[0], c4[1], c4[2]), c4[3]);
            if (kAhead > 0.f) m += fminf(kAhead / sc, 1e30f);  // (sc may be next to nothing)
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
            weights(s[0], 0, nb, p, sum, top, true);
            tmem_ld32_finish(s[1]);
            tmem_ld32_start(tS + 64, s[0]);
            weights(s[1], 32, nb, p + 16, sum, top, false);
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
              weights(s[0], 64, nb, p, sum, top, true);
              tmem_ld32_finish(s[1]);
              weights(s[1], 96, nb, p + 16, sum, top, false);
              if (__any_sync(0xffffffffu, outgrown())) {
                // The upper half has outgrown the range: once the lower half's product is in O,
                // O and l are scaled down and the upper half's weights made again.
                wait_or_die(&bars.oh_full[u], (ns - 1) & 1, dead);
                tc_fence_after();
                lower = true;
                rescale(outgrown() ? top : m);
                const float nb2 = m == -INFINITY ? 0.f : -m * sc;
                if constexpr (KD) {  // (rare, and little code)
                  sum = 0.f;
#pragma unroll 1
                  for (int q = 0; q < 2; ++q) {
                    tmem_ld32_start(tS + 64 + 32 * q, s[0]);
                    finish(s[0], 64 + 32 * q);
                    float part, t2;
                    weights32<false>(s[0], nullptr, sc, nb2, p, part, t2, true);
                    sum += part;
                    if (q == 0)
#pragma unroll
                      for (int e = 0; e < 16; ++e) s[1][e] = p[e];
                  }
#pragma unroll
                  for (int e = 0; e < 16; ++e) {
                    p[16 + e] = p[e];
                    p[e] = s[1][e];
                  }
                } else {
                  tmem_ld32_start(tS + 64, s[0]);
                  tmem_ld32_finish(s[0]);
                  weights(s[0], 64, nb2, p, sum, top, true);
                  weights(s[1], 96, nb2, p + 16, sum, top, false);
                }
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
            weights(s[0], 0, nb, p[0], sum, top, true);
            tmem_ld32_finish(s[1]);
            tmem_ld32_start(tS + 64, s[0]);
            weights(s[1], 0, nb, p[0] + 16, sum, top, false);
            tmem_ld32_finish(s[0]);
            tmem_ld32_start(tS + 96, s[1]);
            weights(s[0], 0, nb, p[1], sum, top, false);
            tmem_ld32_finish(s[1]);
            weights(s[1], 0, nb, p[1] + 16, sum, top, false);
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
            // keys [0, hi) of the tile
            const int hi = whole ? kKeys : along ? w.g.kr.sinks - ks : mypos - ks + 1;
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
              weights32<false>(s, nullptr, sc, nb, p, sum, top, true);
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
                finish(s, 32 * q);
                if (!whole) mask(s, q);
                largest(s);
              }
              standing();
#pragma unroll 1
              for (int q = 0; q < 4; ++q) {
                tmem_ld32_start(tS + 32 * q, s);
                finish(s, 32 * q);
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
        const int behind = along ? w.g.kr.sinks : w.g.kr.hi;
        if (ks + kKeys > behind || (!PRE && ks < w.g.kr.lo && ks + kKeys > w.g.kr.sinks)) {
          const Place at = value_place(order, pos, tile);
          wait_or_die(&bars.kv_full[at.at], at.phase, dead);
          const int key = ks + r;
          if (key >= behind || (!PRE && key < w.g.kr.lo && key >= w.g.kr.sinks)) {
            uint8_t* vrow = sKV + (KD ? at.at - NS : at.at) * C::kStageBytes + r * RB;
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
      // the rows' other side is to be joined
      const bool sides = PRE && w.g.list < 0;
      if (active) {
        const bool valid = r < nr;
        const long long orow =
            (long long)(w.bos + tk) * a.Hq + w.h * a.G + (row - tk * a.G);
        const float inv = l == 0.f ? 0.f : 1.0f / l;
        const long long prow =
            (long long)(2 * blockIdx.x + (cut0 ? 0 : 1)) * kRowsItem + base + r;
        const long long side = PRE ? (w.n < a.groups ? 0 : (long long)a.total_T * a.Hq) + orow : 0;
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
          if (KD) {  // (the expanded values' order)
            uint32_t x[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = o[q8::place(e)];
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = x[e];
          }
          if (sides || cut0 || cut1) {
            float* dst = PRE && !cut0 && !cut1 ? rows.o + side * D : part_o + prow * D;
#pragma unroll
            for (int e = 0; e < 32; e += 8) store32(dst + c + e, o + e);
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
          if (PRE && !cut0)
            rows.at[side] = row_at(w, cut1, base + r, plan.total);
          if (cut0 || cut1)
            part_ml[prow] = make_float2(m * sc, l);
          else if (sides)
            rows.ml[side] = make_float2(m * sc, l);
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

// Joins what a row has of its prefix and of its own keys, each of which lies whole in `rows` or in
// parts with the CTAs that its item was cut among.  A warp a row: half of its lanes look at a
// side's CTAs each, so that all parts' (m, l) and their columns, D / 32 of them a lane, are one
// round trip to memory.  A warp has `per` rows, one after the other.  The first `joins` blocks, a
// multiple of the CTAs, join the items whose rows have no other side.  (Whatever the numbers of a
// row that no item had are, they are made places inside the workspace.)
template <int D>
__global__ void __launch_bounds__(256) paged_rows_kernel(PagedArgs a, Rows rows, int per,
                                                         int joins, const Header* headers,
                                                         const float* part_o,
                                                         const float2* part_ml) {
  constexpr int C = D / 32, U = 8;
  if ((int)blockIdx.x < joins) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    join_items<D>(a, headers, part_o, part_ml, blockIdx.x % kCtas, blockIdx.x / kCtas,
                  joins / kCtas);
    return;
  }
  const int all = a.total_T * a.Hq;
  const int lane = threadIdx.x & 31, side = lane >> 4;
  const long long first = first_row(blockIdx.x - joins, threadIdx.x >> 5, per);
  auto owned = [&](int row, bool& grouped) {
    const int tok = (int)((unsigned)row / (unsigned)a.Hq);
    grouped = token_grouped(a, tok);
    return token_owned(a, tok);
  };
  bool grouped = false;
  const bool live = first < all && (per > 1 || owned((int)first, grouped));
  // launched while the first kernel runs: wait for its results.  (Without rows too: were every
  // block gone before the first kernel's end, what follows in the stream could begin beside it.)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!live) return;
  unsigned open = 1;  // rows that are not done
  if (per > 1)
    open = __ballot_sync(0xffffffffu,
                         lane < per && first + lane < all &&
                             rows.at[all + min(first + lane, all - 1ll)].y >= 0);
#pragma unroll 1
  for (; open; open &= open - 1) {
    const int row = (int)first + __ffs(open) - 1;
    if (per > 1 && !owned(row, grouped)) continue;
    const int4 at = rows.at[(long long)side * all + row];
    if (__shfl_sync(0xffffffffu, at.y, 16) < 0) continue;  // (a warp alike)
    const bool any = side || grouped, whole = at.y <= 0;
    const int unit = at.z >> 8 & 15, c = min(at.z >> 12 & 255, kCtas - 1);
    const int parts = !any ? 0 : whole ? 1 : min(at.z >> 20 & 255, kCtas - c);
    // the first tile that begins in a CTA's stretch or behind it
    auto first_of = [&](int cta) {
      const int x = stretch(max(at.w, 0), cta) - at.x;
      return x <= 0 ? 0 : min(unit == kTile ? (x + kTile - 1) / kTile
                                            : (x + kTileMost - 1) / kTileMost, at.y);
    };
    float m = -INFINITY, l = 0.f, o[C];
#pragma unroll
    for (int e = 0; e < C; ++e) o[e] = 0.f;
#pragma unroll 1
    for (int i = lane & 15; __any_sync(0xffffffffu, i < parts); i += 16) {
      const int cta = min(c + i, kCtas - 1);
      const bool there = i < parts && (whole || first_of(cta + 1) > first_of(cta));
      const int p = (2 * cta + (i == 0)) * kRowsItem + (at.z & 255);
      const float2* pm = whole ? rows.ml + (long long)side * all + row : part_ml + p;
      // (rows.o lies behind part_o)
      const long long at_o =
          whole ? (rows.o - part_o) + ((long long)side * all + row) * D : (long long)p * D;
      const float2 ml = there ? __ldcs(pm) : make_float2(-INFINITY, 0.f);
      unsigned todo = __ballot_sync(0xffffffffu, there);
      // the columns of up to U parts; src: their lanes
      float x[U][C];
      int src[U];
      auto fetch = [&]() {
#pragma unroll
        for (int k = 0; k < U; ++k) {
          src[k] = todo ? __ffs(todo) - 1 : -1;
          const float* po = part_o + __shfl_sync(0xffffffffu, at_o, max(src[k], 0)) + C * lane;
#pragma unroll
          for (int e = 0; e < C; ++e) x[k][e] = 0.f;
          if (todo) {
            if constexpr (C == 4) {
              const float4 y = __ldcs(reinterpret_cast<const float4*>(po));
              x[k][0] = y.x; x[k][1] = y.y; x[k][2] = y.z; x[k][3] = y.w;
            } else if constexpr (C == 2) {
              const float2 y = __ldcs(reinterpret_cast<const float2*>(po));
              x[k][0] = y.x; x[k][1] = y.y;
            } else {
              x[k][0] = __ldcs(po);
            }
          }
          todo &= todo - 1;
        }
      };
      fetch();
      const bool some = ml.y != 0.f;  // (a part that saw nothing has no say)
      float mn = some ? ml.x : -INFINITY;
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, w));
      mn = fmaxf(mn, m);
      const float b = mn == -INFINITY ? 0.f : mn, f = fast_exp2(m - b);
      const float g = some ? fast_exp2(ml.x - b) : 0.f;
      m = mn;
      l = l * f + warp_sum(some ? ml.y * g : 0.f);
#pragma unroll
      for (int e = 0; e < C; ++e) o[e] *= f;
#pragma unroll 1
      while (src[0] >= 0) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const float w = __shfl_sync(0xffffffffu, g, max(src[k], 0));
#pragma unroll
          for (int e = 0; e < C; ++e) o[e] += x[k][e] * (src[k] < 0 ? 0.f : w);
        }
        fetch();
      }
    }
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + (long long)row * D + C * lane;
    if constexpr (C == 4)
      *reinterpret_cast<uint2*>(dst) =
          make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
    else if constexpr (C == 2)
      *reinterpret_cast<uint32_t*>(dst) = pack_bf16(o[0] * inv, o[1] * inv);
    else
      *dst = __float2bfloat16_rn(o[0] * inv);
    if (lane == 0 && a.lse)
      a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
  }
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

template <int D, bool Q8, bool PRE>
cudaError_t launch_t(PagedArgs a, void* workspace, void* query_terms, cudaStream_t st) {
  set_divisor(a);
  const uint32_t G = (uint32_t)a.G;
  a.alone = PRE && (long long)a.total_T * G >= kAlone;
  if constexpr (Cfg<D, Q8>::kDirect) {
    const cudaError_t e = launch_query_terms(a, query_terms, st);
    if (e != cudaSuccess) return e;
  }
  CUtensorMap qmap{}, kmap{}, vmap{};
  // Rows by TMA where the items are large: a call with one token for each of its sequences has
  // a few rows in each, which are copied one by one.
  const int q_boxes = kRowsUnit % G == 0 && (long long)a.total_T * G > 32 && query_map(&qmap, a);
  if (a.num_pages > 0 && (a.max_pages > 0 || a.max_prefix_pages > 0))
    if (!cache_map<Q8>(&kmap, a.k_cache, a) || !cache_map<Q8>(&vmap, a.v_cache, a))
      return cudaErrorInvalidValue;
  Header* headers = static_cast<Header*>(workspace);
  float2* ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + 8192);
  float* po = reinterpret_cast<float*>(ml + (size_t)2 * kCtas * kRowsItem);
  // D <= 64: chunks of 2048 behind 8192 keys, 32 + 4 heads of 64: 320 us for 352 with one pass over
  // whole tiles, 148 for 162 with D = 32.  Masked tiles are faster unrolled, which the one pass
  // does not go with; under a window they can be many (a third in the windowed batch above: 36.2 us
  // for 35.1).  How many there are lies in device memory, so any window counts as narrow: a chunk
  // under a wide one forgoes the gain.
  using C = Cfg<D, Q8>;
  auto kernel = paged_tc_kernel<D, PRE && C::kOwnP, Q8, PRE>;  // (prefixes: no window)
  if constexpr (C::kOwnP && !PRE)
    if (a.window == 0) kernel = paged_tc_kernel<D, true, Q8, PRE>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::kSmem);
  if (e != cudaSuccess) return e;
  const long long all = (long long)a.total_T * a.Hq;
  Rows rows{};
  if (PRE) {
    rows.o = po + (size_t)2 * kCtas * kRowsItem * D;
    rows.at = reinterpret_cast<int4*>(rows.o + 2 * all * D);
    rows.ml = reinterpret_cast<float2*>(rows.at + 2 * all);
  }
  if constexpr (C::kDirect) {
    // set up beside the kernel that makes the queries' terms
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kCtas);
    cfg.blockDim = dim3(Group<Q8>::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, a, qmap, kmap, vmap, q_boxes, headers, po, ml, rows);
  } else {
    kernel<<<kCtas, Group<Q8>::kThreads, C::kSmem, st>>>(a, qmap, kmap, vmap, q_boxes, headers, po,
                                                         ml, rows);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  if constexpr (!PRE) return launch_join<D>(a, headers, po, ml, st);
  cudaLaunchConfig_t cfg{};
  // A warp looks at several rows, most of which may be done, where there are more than the SMs have
  // room for warps (with few, one after the other takes longer: 130 tokens of 16 heads 34 us for
  // 27).
  const int per = a.alone && all > kCtas * 64 ? 4 : 1, joins = a.alone ? 8 * kCtas : 0;
  cfg.gridDim = dim3((unsigned)(joins + (all + 8 * per - 1) / (8 * per)));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_rows_kernel<D>, a, rows, per, joins,
                            (const Header*)headers, (const float*)po,
                            (const float2*)ml);
}

// query_terms: 8 bits and D = 128, room for paged_query_terms() bytes.
template <bool Q8, bool PRE>
cudaError_t launch_any(const PagedArgs& a, void* workspace, void* query_terms, cudaStream_t st) {
  return a.D == 32   ? launch_t<32, Q8, PRE>(a, workspace, query_terms, st)
         : a.D == 64 ? launch_t<64, Q8, PRE>(a, workspace, query_terms, st)
                     : launch_t<128, Q8, PRE>(a, workspace, query_terms, st);
}

static_assert(sizeof(Header) * kCtas <= 8192, "headers");

}  // namespace
}  // namespace kda
