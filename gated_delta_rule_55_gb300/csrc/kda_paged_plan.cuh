// The line of key tiles that attention over pages cuts among its CTAs, as its tensor-core kernels
// walk it, the joining of the items that a cut passes through, and small pieces that they share.
// Included behind the including kernel's numbers:
//   kRowsItem    query rows of an item, at most
//   kStretches   CTAs of the line
//   kTile        units of the line that a tile counts; kTileMost, one of an item with more than
//                kRowsFew rows
//   kPrefixes    whether calls have prefixes
//   kOverhead    units that an item counts beside its tiles; kOverheadMost, one of D = 128 with
//                more than kRowsFew rows
#pragma once

#include "chunk_common.cuh"
#include "kda_paged.cuh"
#include "kda_paged_line.h"
#include "kda_q8.cuh"

namespace kda {
namespace {

using namespace chunk;

__device__ unsigned int g_paged_error;  // bit 6: a bounded wait gave up

constexpr int kKeys = 128;       // keys of a tile

struct Header {  // a CTA's part of the line, for the joining kernel
  int rows;       // rows of the item that starts in its stretch and is cut (0: none)
  int row0, h;    // its first row and kv head
  int nt;         // its tiles
  int start, total;  // place of its first tile in the line, the line's length
  int bos;        // its sequence's first token
  int unit;       // units of a tile
};

// ------------------------------------------------------------------- items of the line

// x / G, G = Hq / Hkv, for 0 <= x < 2^31, by the host's multiplier (launch_t).
__device__ __forceinline__ int div_g(const PagedArgs& a, int x) {
  return (int)((__umulhi((uint32_t)x, a.g_mul) + (uint32_t)x) >> a.g_shift);
}

struct Geometry {
  int row0, rows;  // query rows of the item
  KeyRange kr;
  int t_lo, ns, nt;  // first window tile, sink (prefix) tiles before it, tiles in all
  int list;          // the prefix whose tiles come first, kr.sinks keys of it (< 0: none)
  int extra;         // units of the line before its tiles
  // A tile's units: it is worked on where the first of them lies.
  __device__ __forceinline__ int cost() const {
    return kTile == kTileMost || rows <= kRowsFew ? kTile : kTileMost;
  }
  __device__ __forceinline__ int units() const { return nt * cost() + extra; }
  // Tiles that begin among the item's first x units.
  __device__ __forceinline__ int begun(int x) const {
    const int c = cost();
    return x <= extra ? 0 : c == 1 ? x - extra : min((x - extra + c - 1) / c, nt);
  }
};

// A group whose sequences have kAlone rows and more on average fills the products' tiles without
// its neighbours: its sequences take the prefix along with their own keys, as one list of tiles,
// and there is nothing to join.  (2300 tokens of 8 sequences behind 8191 keys, 32 + 8 heads of 128:
// 250 us when their prefix was worked on for all of them.)
//
// Sequences of 256, 512, 768, 1024 rows, prefix taken along / shared, us: 8 sequences behind 8191
// keys, D = 128, 68 / 73, 114 / 132, 158 / 194, 200 / 254; behind 2000 keys 41 / 45, 53 / 71, 68 /
// 101, 83 / 130; 3 sequences behind 4000 keys 36 / 30, 40 / 44, 52 / 59, 63 / 74; 8 behind 4000, D =
// 64, 39 / 58, 60 / 100, 82 / 139, 102 / 181; over 8-bit pages 60 / 67, 97 / 116, 129 / 171, 164 /
// 224.  So between 512 rows and the border sharing costs 10 to 40%; a prefix taken along is read
// once for each sequence, which more sequences of fewer rows pay for.
constexpr int kAlone = 768;

__device__ __forceinline__ bool group_alone(const PagedArgs& a, int g) {
  const int g0 = min(max(a.cu_groups[g], 0), a.N), g1 = min(max(a.cu_groups[g + 1], 0), a.N);
  const long long lo = a.cu_seqlens[g0], hi = a.cu_seqlens[g1];
  return g1 > g0 && (hi - lo) * a.G >= (long long)kAlone * (g1 - g0);
}
// List i from its raw numbers.
__device__ __forceinline__ Seq list_seq(const PagedArgs& a, int i, int lo, int hi, int kv) {
  Seq s = make_seq(a, lo, hi, kv, i < a.groups);
  if (kPrefixes && a.alone) {
    if (i < a.groups) {
      if (group_alone(a, i)) s.len = 0;
    } else {
      const int n = i - a.groups;
      int g = 0;  // the last group that begins at n or before it
      for (int end = a.groups; end - g > 1;) {
        const int mid = (g + end) >> 1;
        (a.cu_groups[mid] <= n ? g : end) = mid;
      }
      if (a.cu_groups[g] <= n && n < a.cu_groups[g + 1] && group_alone(a, g)) {
        s.list = g;
        s.pre = make_seq(a, 0, 0, a.prefix_lens[g], true).kv;
      }
    }
  }
  return s;
}
__device__ __forceinline__ Seq load_list(const PagedArgs& a, int i) {
  int lo, hi, kv;
  raw_seq(a, i, lo, hi, kv);
  return list_seq(a, i, lo, hi, kv);
}

__device__ __forceinline__ Geometry geometry(const PagedArgs& a, const Seq& s, int G, int rt) {
  Geometry g;
  const int rows = s.len * G;
  g.row0 = rt * kRowsItem;
  g.rows = min(kRowsItem, rows - g.row0);
  g.extra = a.D == 128 && g.rows > kRowsFew ? kOverheadMost : kOverhead;
  g.kr = key_range(a, s, div_g(a, g.row0), div_g(a, g.row0 + g.rows - 1));
  g.t_lo = g.kr.lo / kKeys;
  g.ns = min((g.kr.sinks + kKeys - 1) / kKeys, g.t_lo);
  g.list = -1;
  if (kPrefixes) {  // (no window: neither sinks nor tiles that it hides)
    g.list = s.list;
    g.kr.sinks = s.pre;
    g.ns = (s.pre + kKeys - 1) / kKeys;
  }
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
  t.list = t.pre = 0;
  if (kPrefixes) {
    t.list = __shfl_sync(0xffffffffu, s.list, src);
    t.pre = __shfl_sync(0xffffffffu, s.pre, src);
  }
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
  int end;       // the stretch's
  int start_at;  // the item's first tile in the line
  Seq s;
  Geometry g;
  int c1, c2, kv1;  // the next sequence's offsets and keys

  __device__ __forceinline__ void ahead(const PagedArgs& a) {
    c1 = c2 = kv1 = 0;
    if (n + 1 < lists(a)) raw_seq(a, n + 1, c1, c2, kv1);
  }
  // The item's tiles among its units [x, ...); false when the stretch ends before the first (it
  // is the stretch's last item then, and the next CTA takes it whole).
  __device__ __forceinline__ bool enter(const PagedArgs& a, int x) {
    g = geometry(a, s, a.G, rt);
    const int last = min(g.units(), x + left);
    units = last - x;
    v0 = g.begun(x);
    v1 = g.begun(last);
    start_at = end - left - x + g.extra;
    return v1 > v0;
  }
  __device__ __forceinline__ bool start(const PagedArgs& a, const Plan& p) {
    end = p.end;
    left = p.end - p.first;
    if (left <= 0 || p.n < 0) return false;
    n = p.n; h = p.h; rt = p.rt;
    s = p.s;
    ahead(a);
    if (enter(a, p.x)) return true;
    // (only units of a tile that the CTA before has)
    return kTileMost > 1 && left > units && next(a);
  }
  __device__ __forceinline__ bool next(const PagedArgs& a) {
    left -= units;
    if (left <= 0) return false;
    if (++rt >= row_tiles(s, a.G)) {
      rt = 0;
      if (++h >= a.Hkv) {
        h = 0;
        do {  // (the line has more units, so a later sequence has tokens)
          if (++n >= lists(a)) return false;
          s = list_seq(a, n, c1, c2, kv1);
          ahead(a);
        } while (s.len == 0);
      }
    }
    return enter(a, 0);
  }
  __device__ __forceinline__ int tiles() const { return v1 - v0; }
};

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

// The CTA's stretch of the line: all NT threads call.  s_units: NT entries, each of which
// fits 31 bits (paged_tc_index_ok).  So does the line when the offsets are in order; when they
// overlap, against the call's rules, it may not, and then every CTA's stretch is empty.
template <int NT>
__device__ void make_plan(const PagedArgs& a, Plan& plan, int* s_units) {
  constexpr int kPlanSeqs = NT;  // sequences (lists) whose units are looked at together
  constexpr int W = NT / 32, kFew = 2 * W;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = a.G;
  const int rounds = (lists(a) + kPlanSeqs - 1) / kPlanSeqs;
  // Sequences r kPlanSeqs + ...: with few of them a warp takes two and its lanes the row tiles,
  // with many a thread takes one, and its warp helps where there are many row tiles.
  Seq s[2]{};
  int per[2], count = 0, sum = 0;
  if (threadIdx.x == 0) plan.n = -1;
  auto load = [&](int r) {
    count = min(lists(a) - r * kPlanSeqs, kPlanSeqs);
    __syncthreads();
    if (count <= kFew) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (warp + k * W < count) s[k] = load_list(a, r * kPlanSeqs + warp + k * W);
#pragma unroll 1
      for (int k = 0; k < 2; ++k)
        if (warp + k * W < count) {
          const int y = head_units(a, k == 0 ? s[0] : s[1], G);
          if (lane == 0) s_units[warp + k * W] = y * a.Hkv;
          (k == 0 ? per[0] : per[1]) = y;
        }
    } else {
      const int i = threadIdx.x;
      if (i < count) s[0] = load_list(a, r * kPlanSeqs + i);
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
      first = stretch<kStretches>(total, blockIdx.x);
      const int end = stretch<kStretches>(total, blockIdx.x + 1);
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
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

// D[tmem] (+)= A[smem] * B[smem]^T of e4m3, issued by one thread.
__device__ __forceinline__ void mma_ss_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// A copy of `bytes` (a multiple of 16, both addresses on 16 bytes) that counts on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, "
      "[%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Byte offset of the 16-byte piece `ch` of row r in a 128-row tile of 8-bit numbers: swizzled over
// the row's D bytes, as TMA lays it.
template <int D>
__device__ __forceinline__ uint32_t raw_offset(int r, int ch) {
  const int x = D == 128 ? r & 7 : D == 64 ? r >> 1 & 3 : r >> 2 & 1;
  return uint32_t(r * D + ((ch ^ x) << 4));
}

// Byte offset of the 16-byte piece `ch` of row r in a 128-row tile, swizzled as TMA lays it.
template <int D>
__device__ __forceinline__ uint32_t piece_offset(int r, int ch) {
  if (D == 32) return uint32_t(r * 64 + ((ch ^ (r >> 1 & 3)) << 4));
  return sw128_offset<2>(128, r, ch * 8);
}

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

// Joins the partial results of an item that was cut: the CTA it starts in has it in its second
// slot, the following ones in their first.  Blocks (c, .): the item that starts in CTA c's
// stretch; a thread has four columns of a row and takes four parts at a time, all their loads in
// flight together (eight: 39.8 against 37.5 us for a call with 150 items cut in two).
// (c, y of ny): the block's number.
template <int D>
__device__ __forceinline__ void join_items(const PagedArgs& a, const Header* headers,
                                           const float* part_o, const float2* part_ml, int c,
                                           int y, int ny) {
  constexpr int PIECES = D / 4, U = 4;
  const Header hd = headers[c];
  if (hd.rows == 0) return;
  const int unit = kTileMost == 1 ? 1 : hd.unit;
  // CTAs from this one to the one it ends in
  const int parts = stretch_of<kStretches>(hd.total, hd.start + unit * (hd.nt - 1)) - c + 1;
  // The first of its tiles that begins in CTA k's stretch or behind it.
  auto first_of = [&](int k) {
    const int x = stretch<kStretches>(hd.total, k) - hd.start;
    if (kTileMost == 1) return x;
    return x <= 0 ? 0 : unit == kTile ? (x + kTile - 1) / kTile : (x + kTileMost - 1) / kTileMost;
  };
  for (int at = y * 256 + threadIdx.x; at < hd.rows * PIECES; at += ny * 256) {
    const int r = at / PIECES, e = at % PIECES;
    // Row of the i-th part in the partial results, -1 if that CTA has no tile of the item.
    auto place = [&](int i) -> int {
      const int k = c + i;
      const int first = first_of(k), last = min(first_of(k + 1), hd.nt);
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

template <int D>
__global__ void __launch_bounds__(256) paged_join_kernel(PagedArgs a, const Header* headers,
                                                         const float* part_o,
                                                         const float2* part_ml) {
  // launched while the first kernel runs: wait for its results
  asm volatile("griddepcontrol.wait;" ::: "memory");
  join_items<D>(a, headers, part_o, part_ml, blockIdx.x, blockIdx.y, gridDim.y);
}

// Pages of a cache: boxes of a page's rows, of up to 64 columns of bf16 or of all D bytes.
template <bool Q8>
bool cache_map(CUtensorMap* map, const void* base, const PagedArgs& a) {
  const auto enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)a.D,
                              (cuuint64_t)a.num_pages * a.Hkv * (cuuint64_t)a.page_size};
  const cuuint64_t strides[1] = {(cuuint64_t)a.D * (Q8 ? 1 : 2)};
  const cuuint32_t box[2] = {Q8 ? (cuuint32_t)a.D : a.D == 32 ? 32u : 64u,
                             (cuuint32_t)a.page_size};
  const cuuint32_t es[2] = {1, 1};
  if (Q8)
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
               es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               a.D == 32   ? CU_TENSOR_MAP_SWIZZLE_32B
               : a.D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                           : CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             a.D == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The joining kernel behind the one that left the parts.
template <int D>
cudaError_t launch_join(const PagedArgs& a, const Header* headers, const float* po,
                        const float2* ml, cudaStream_t st) {
  // a thread per four columns of the largest item there can be
  const long long most = (long long)a.total_T * a.G;
  const unsigned by = (unsigned)((most < kRowsItem ? most : kRowsItem) * (D / 4) + 255) / 256;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kStretches, by);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<D>, a, headers, po, ml);
}

// The host's numbers for div_g: x / G = (mulhi(x, g_mul) + x) >> g_shift for x < 2^31.
void set_divisor(PagedArgs& a) {
  const uint32_t G = (uint32_t)(a.Hq / a.Hkv);
  a.G = (int)G;
  a.g_shift = 0;
  while ((1u << a.g_shift) < G) ++a.g_shift;
  a.g_mul = (uint32_t)((((1ull << a.g_shift) - G) << 32) / G + 1);
}

unsigned int read_error(bool reset) {
  unsigned int v = 0;
  cudaMemcpyFromSymbol(&v, g_paged_error, sizeof(v));
  if (reset) {
    const unsigned int z = 0;
    cudaMemcpyToSymbol(g_paged_error, &z, sizeof(z));
  }
  return v;
}

}  // namespace
}  // namespace kda
