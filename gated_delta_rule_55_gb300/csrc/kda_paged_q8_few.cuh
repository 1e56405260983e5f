// Attention of few new tokens (single ones, or a handful) over a paged cache in 8 bits, D = 64 or
// 128, on the tensor cores: kda_paged_attention_q8_fwd where kda_paged_tc.cuh's tiles of 128 query
// rows would be almost empty.
//
// The products are turned round: keys and values are the 128 rows of the tiles, the query rows
// (kRowsItem at most: 16, or 32) the columns,
//   S^T = K Q^T,   O^T += V^T P^T,
// so that they take an eighth of the time, and a softmax thread has a key instead of a query row:
// all 128 work however few rows there are, scales of keys and values are one number of a thread,
// and its weights' sums stay in its registers until the item's end.
//
// K stays in 8 bits.  A query row (8 bits of mantissa) becomes two rows of e4m3 under a power of
// two:
//   q 2^-e = hi + lo,   hi = e4m3(q 2^-e),  lo = e4m3(q 2^-e - hi)
// which is exact where q is more than 2^-9 of the row's largest, and off by at most 2^-17 of that
// elsewhere; the products of e4m3 are exact in fp32, and their sum is scaled in fp32:
// (hi k + lo k) 2^e 2^scale(k).  V is expanded to bf16 without its scales, which go into the
// weights: bf16(p 2^scale(v)).
//
// One CTA is one line's stretch (kda_paged_plan.cuh) with a ring of two tiles of keys and two of
// values (D = 64: three), half of an SM's shared memory; two CTAs share an SM, and one's chain of
// waits (scores, softmax, values) passes beside the other's.  Items of 32 rows leave no room for
// weights and a second place for query rows: weights lie over the keys whose scores they come from
// (which are then free only behind the values' product), query rows in one place.
//
// What bounds it, and measured (alone on the GPU, 32 + 8 heads): 64 single tokens over 512..8192
// keys HBM, 97 us, 5.6 TB/s of the 6.8 of a copy (233 through tiles of 128 query rows), 14 of them
// the start and the join; 16 tokens over 30000 keys 163 us, 6.1 TB/s; 256 tokens over 100..1000
// keys 77 us, where items' starts and ends count; one token over 1000 keys 11.3 us of latencies in
// a row.  More rows, over the 512..8192 keys: 4 tokens (16 rows) 113 us, 5 (20 rows) 172, 8 (32)
// 176, the softmax's chain (through tiles of 128 query rows 241).  D = 64: single tokens 82 us (161
// through tiles of 128, 104 over bf16 pages) for 41 of bytes, 5 tokens 136 (162), 8 tokens 147.
// The code is kept small: what runs once or twice in an item is fetched anew every time, so it is
// in loops or shared out among lanes (unrolled, 256 sequences of 4 tokens over 100..1000 keys took
// 170 us for 121).  With the expanding unrolled the long caches take 2% less, the short ones 15%
// more.
#pragma once

#include "kda_paged_line.h"

namespace kda {
namespace {
constexpr int kStretches = 2 * kCtas;  // two CTAs per SM
constexpr int kRowsFew = kRowsItem;
constexpr bool kPrefixes = false;
constexpr int kTile = 1, kTileMost = 1;
constexpr int kOverhead = 2, kOverheadMost = 2;  // units of the line that an item counts
}  // namespace
}  // namespace kda

#include "kda_paged_plan.cuh"

namespace kda {
namespace {

constexpr int kThreads = 384;  // softmax, expanders, and the warps below
constexpr int kExpandWarp = 4, kLoadWarp = 8, kMmaWarp = 9, kQueryWarp = 10 /* and 11 */;
// Registers: 80 a thread at launch, 3 x 80 = 112 + 64 + 64.
constexpr int kRegsSoftmax = 112, kRegsExpand = 64, kRegsOther = 64;
constexpr float kRescale = 32.0f;  // log2 growth of the maximum that O and l absorb
constexpr int kSteps = 4;         // items put down ahead

constexpr int kFront = 5 * 1024;                  // barriers, the plan, scales
constexpr bool kWide = kRowsItem == 32;
constexpr int kPBytes = kRowsItem * kKeys * 2;
constexpr int kLand = kKeys * 128;  // where a slot's values land: D = 128, in its upper half
template <int D> struct Cfg {
  static constexpr int kStages = D == 128 ? 2 : 3;   // tiles of keys, of values
  static constexpr int kQBytes = 2 * kRowsItem * D;  // hi rows, lo rows
  static constexpr int kKBytes = kKeys * D;
  static constexpr int kVBytes = D == 128 ? 2 * kLand : kLand + kKBytes;
  static constexpr int kSmem = kFront + (kWide ? kQBytes : 2 * kQBytes + kPBytes) +
                               kStages * (kKBytes + kVBytes);
  static constexpr uint32_t kSwizzleK = D == 128 ? kSwizzle128 : 4;  // its rows: 128 or 64 bytes
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs on an SM");
  static_assert(!kWide || kPBytes <= kKBytes, "weights over their keys");
};
// Two of the scores, two of O.
constexpr uint32_t kColS = 0, kColO = 2 * kRowsItem, kTmemCols = 4 * kRowsItem;

struct Step {
  int live;             // 0: nothing more
  int n, h, bos, pos0;  // sequence, kv head, first token and its position
  int v0, v1;           // its tiles in the stretch
  Geometry g;
};

template <int NS> struct Small {
  uint64_t k_full[NS], k_empty[NS], vr_full[NS], v_full[NS], v_empty[NS], q_full[2], q_empty[2],
      s_full[2], s_empty[2], o_empty[2], q_read, p_full, pv_done, vote, step_full[kSteps],
      step_empty[kSteps];
  Plan plan;
  Step steps[kSteps];
  uint32_t tmem;
  alignas(16) uint8_t k_scale[NS][kKeys], v_scale[NS][kKeys];
  alignas(16) float row_scale[2][kRowsItem];  // 2^e scale log2(e)
  alignas(16) int row_pos[2][kRowsItem];
  alignas(16) int votes[2][4];
  alignas(16) float parts[2][4][kRowsItem];   // a warp's maxima, sums
  // For each warp: standing maxima (of more rows than 16), what they rise by, the factors.
  alignas(16) float m[4][kRowsItem], by[4][kRowsItem], f[4][kRowsItem];
};
static_assert(sizeof(Small<3>) <= kFront, "front");

template <int N> __device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[N]) {
  uint32_t r[N];
  if constexpr (N == 4) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(taddr)
        : "memory");
  } else if constexpr (N == 8) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(taddr)
        : "memory");
  } else {
    tmem_ld16(taddr, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]);
}
template <int N> __device__ __forceinline__ void tmem_st(uint32_t taddr, const float (&v)[N]) {
  if constexpr (N == 4) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3])
        : "memory");
  } else if constexpr (N == 8) {
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(v[i]);
    tmem_st8(taddr, r);
  } else {
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
    tmem_st16(taddr, r);
  }
}

template <int N> struct Int { static constexpr int value = N; };

// N values of each lane, each joined over the warp's lanes: a lane gives half of its values away
// and takes the other half's from its partner until one is left, number e of them, which `out` then
// has (N - 1 exchanges and those for the lanes that are left; 5 N one by one).
template <int N, class F>
__device__ __forceinline__ void join_lanes(float (&v)[N], float* out, F op) {
  const int lane = threadIdx.x & 31;
  int e = 0, o = 16;
#pragma unroll
  for (int n = N / 2; n > 0; n >>= 1, o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float y = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + n], o);
      v[i] = op(up ? v[i + n] : v[i], y);
    }
    if (up) e += n;
  }
  for (; o > 0; o >>= 1) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
  if ((lane & (32 / N - 1)) == 0) out[e] = v[0];
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
paged_q8_few_kernel(PagedArgs a, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap, Header* headers, float* part_o,
                    float2* part_ml) {
  using C = Cfg<D>;
  constexpr int NS = C::kStages, kQBytes = C::kQBytes, kKBytes = C::kKBytes,
                kVBytes = C::kVBytes;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Small<NS>& s = *reinterpret_cast<Small<NS>*>(smem_raw);
  uint8_t* sQ = smem_raw + kFront;   // two stages (wide: one)
  uint8_t* sP = sQ + 2 * kQBytes;    // (wide: over the tile of keys)
  uint8_t* sK = kWide ? sQ + kQBytes : sP + kPBytes;  // tiles, as they land
  uint8_t* sV = sK + NS * kKBytes;   // tiles as the products read them, and as they land
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == kMmaWarp) {
    tmem_alloc(&s.tmem, kTmemCols);
    tmem_relinquish();  // (the SM's other CTA allocates too)
  }
  if (tid == 32 * kLoadWarp) {
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&s.k_full[i], 1);
      mbar_init(&s.k_empty[i], 5);  // the scores' product (wide: the values'), the softmax warps
      mbar_init(&s.vr_full[i], 1);
      mbar_init(&s.v_full[i], 4);
      mbar_init(&s.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.q_full[i], 2);  // half of the rows by each query warp
      mbar_init(&s.q_empty[i], kWide ? 4 : 5);
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.s_empty[i], 4);
      mbar_init(&s.o_empty[i], 4);
    }
    mbar_init(&s.q_read, 1);
    mbar_init(&s.p_full, 4);
    mbar_init(&s.pv_done, 1);
    mbar_init(&s.vote, 4);
    for (int i = 0; i < kSteps; ++i) {
      mbar_init(&s.step_full[i], 1);
      // load, products, second query warp, expanders, softmax: one for each warp
      mbar_init(&s.step_empty[i], 11);
    }
    fence_mbar_init();
  }
  make_plan<kThreads>(a, s.plan, reinterpret_cast<int*>(sK));  // (not in use yet)
  fence_async_smem();  // the plan's numbers lay where copies will land
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may be set up
  const uint32_t tm = s.tmem;
  bool dead = false;
  auto step = [&](uint32_t j) -> const Step* {
    wait_or_die(&s.step_full[j % kSteps], (j / kSteps) & 1, dead);
    dead = __any_sync(0xffffffffu, dead);
    const Step* st = &s.steps[j % kSteps];
    return dead || !st->live ? nullptr : st;
  };
  auto step_done = [&](uint32_t j) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.step_empty[j % kSteps]);
  };

  // A half of item i's query rows as their two terms: 8 numbers a lane.
  auto convert = [&](uint32_t i, int half) {
    const uint32_t b = i & 1;
    const Step& it = s.steps[i % kSteps];
    const int rows = it.g.rows, row0 = it.g.row0, bos = it.bos, h = it.h, pos0 = it.pos0;
    uint8_t* q = kWide ? sQ : sQ + b * kQBytes;
    constexpr int L = D / 8, W = 32 / L;  // lanes of a row, rows of the warp
    constexpr int kHalf = kRowsItem / 2, U = kHalf / W;
    const int c = lane & (L - 1), r0 = half * kHalf, end = min(rows, r0 + kHalf);
    // (the rows are on their way while the place is waited for)
    auto free_rows = [&]() {
      wait_or_die(&s.q_empty[b], ((i >> 1) & 1) ^ 1, dead);
      if (kWide) wait_or_die(&s.q_read, (i & 1) ^ 1, dead);
      // rows that the item does not have: whatever lies there, no scores that grow
      if (lane < kHalf && r0 + lane >= rows) s.row_scale[b][r0 + lane] = 0.f;
    };
    if (r0 < end) {
      uint4 x[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int r = min(r0 + W * k + lane / L, rows - 1);
        const int tk = div_g(a, row0 + r), hg = row0 + r - tk * a.G;
        x[k] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                               (long long)(bos + tk) * a.q_stride +
                                               (long long)(h * a.G + hg) * D + c * 8);
      }
      free_rows();
      // In a loop that passes the rows along: little code.
#pragma unroll 1
      for (int r = r0 + lane / L; r < r0 + kHalf; r += W) {
        const uint32_t u[4] = {x[0].x, x[0].y, x[0].z, x[0].w};
#pragma unroll
        for (int k = 0; k + 1 < U; ++k) x[k] = x[k + 1];
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          top = max(top, max(u[e] << 16 & 0x7fff0000u, u[e] & 0x7fff0000u));
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1)
          top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const bool odd = top >= 0x7f800000u;  // an infinity or a NaN: the row's scores are NaN
        const int e = q8::exponent(top);
        const float f = odd ? 0.f : q8::power(-e);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const float y0 = odd ? 0.f : bf16_lo(u[p]) * f, y1 = odd ? 0.f : bf16_hi(u[p]) * f;
          hi[p] = q8::pack2(y0, y1);
          const float2 z = q8::unpack2(hi[p]);
          lo[p] = q8::pack2(y0 - z.x, y1 - z.y);
        }
        if (r < end) {
          uint8_t* dst = q + raw_offset<D>(r, c >> 1) + (c & 1) * 8;
          *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
          *reinterpret_cast<uint2*>(dst + kRowsItem * D) =
              make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
          if (c == 0) {
            s.row_scale[b][r] =
                odd ? __uint_as_float(0x7fc00000u) : q8::power(e) * (a.scale * kLog2E);
            s.row_pos[b][r] = pos0 + div_g(a, row0 + r);
          }
        }
      }
    } else {
      free_rows();
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.q_full[b]);
  };

  if (warp >= kLoadWarp)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
  if (warp == kLoadWarp) {
    const int ps = a.page_size, ppt = kKeys / ps;  // pages of a tile: 8, 4, 2 or 1
    // Lane 8 x + p looks up and copies page p of the tiles x, x + 4, ..., four tiles ahead.
    const int quarter = lane >> 3, pi = lane & 7;
    uint32_t kp = 0, vp = 0;  // tiles of keys and of values pushed
    for (uint32_t j = 0;; ++j) {
      const Step* st = step(j);
      if (!st) break;
      const Step w = *st;
      const int n = w.v1 - w.v0;
      int row = -1;  // of the page in the caches, for the lane's tile; -1: not needed
      int page = 0;
      bool fresh = true, need_it = false;  // a look-up that has not been made a row yet
      auto look_up = [&](int t) {
        need_it = false;
        fresh = true;
        if (pi >= ppt || t >= n) return;
        const int k0 = tile_start(w.g, w.v0 + t) + pi * ps;
        if (k0 >= w.g.kr.hi || (k0 + ps <= w.g.kr.lo && k0 >= w.g.kr.sinks)) return;
        need_it = true;
        page = __ldg(a.block_table + (long long)w.n * a.max_pages + k0 / kKeys * ppt + pi);
      };
      auto settle = [&]() {  // (touches the loaded number: a tile later)
        if (fresh)
          row = need_it ? (min(max(page, 0), a.num_pages - 1) * a.Hkv + w.h) * ps : -1;
        fresh = false;
      };
      look_up(quarter);
      settle();
#pragma unroll 1
      for (int t = -1; t < n; ++t) {
#pragma unroll 1
        for (int z = 0; z < 2; ++z) {  // the next tile's keys, this one's values
          const bool keys = z == 0;
          const int y = keys ? t + 1 : t;
          if (y < 0 || y >= n) continue;
          const uint32_t at = keys ? kp++ : vp++, slot = at % NS;
          wait_or_die(keys ? &s.k_empty[slot] : &s.v_empty[slot], ((at / NS) & 1) ^ 1, dead);
          const bool mine = (y & 3) == quarter && row >= 0;
          const unsigned need = __ballot_sync(0xffffffffu, mine);
          uint64_t* bar = keys ? &s.k_full[slot] : &s.vr_full[slot];
          if (lane == 0)
            mbar_arrive_expect_tx(bar, uint32_t(__popc(need)) * uint32_t(ps * (D + 1)));
          __syncwarp();
          if (mine && !dead) {
            uint8_t* dst = keys ? sK + slot * kKBytes : sV + slot * kVBytes + kLand;
            tma_load_2d(dst + pi * ps * D, keys ? &kmap : &vmap, bar, 0, row);
            bulk_load((keys ? s.k_scale[slot] : s.v_scale[slot]) + pi * ps,
                      (keys ? a.k_scale : a.v_scale) + row, ps, bar);
          }
          __syncwarp();
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
    if (dead) {
      for (uint32_t i = kp > NS ? kp - NS : 0; i < kp; ++i)
        mbar_wait(&s.k_full[i % NS], (i / NS) & 1, 100000000ull);
      for (uint32_t i = vp > NS ? vp - NS : 0; i < vp; ++i)
        mbar_wait(&s.vr_full[i % NS], (i / NS) & 1, 100000000ull);
    }
  } else if (warp == kMmaWarp) {
    // Products: a tile's scores one tile ahead of the values.  The whole warp walks and waits, one
    // lane issues, from warp-uniform addresses.
    const uint32_t idesc_s = make_idesc(0, 128, kRowsItem);
    const uint32_t idesc_o = make_idesc(1, D, kRowsItem, true, false);
    const uint32_t tmu = __shfl_sync(0xffffffffu, tm, 0);
    const uint32_t q0 = smem_u32(sQ), p0 = smem_u32(sP), k0 = smem_u32(sK), v0 = smem_u32(sV);
    const bool leader = elect_one();
    uint32_t jq = 0, tq = 0, jp = 0, tp = 0;  // items and tiles of the scores, of the values
    int iq = 0, ip = 0;
    const Step* sq = step(0);
    int nq = sq ? sq->v1 - sq->v0 : 0, np = nq;
    auto scores = [&]() {
      if (!sq) return;
      if (iq == 0) wait_or_die(&s.q_full[jq & 1], (jq >> 1) & 1, dead);
      const uint32_t b = tq & 1, slot = tq % NS;
      wait_or_die(&s.k_full[slot], (tq / NS) & 1, dead);
      wait_or_die(&s.s_empty[b], ((tq >> 1) & 1) ^ 1, dead);
      tc_fence_after();
      const uint64_t kd = make_sdesc(__shfl_sync(0xffffffffu, k0 + slot * kKBytes, 0), 16, 8 * D,
                                     C::kSwizzleK);
      const uint64_t qd = make_sdesc(
          __shfl_sync(0xffffffffu, kWide ? q0 : q0 + (jq & 1) * kQBytes, 0), 16, 8 * D,
          C::kSwizzleK);
      const uint32_t to = __shfl_sync(0xffffffffu, tmu + kColS + kRowsItem * b, 0);
      ++iq;
      if (leader) {
        if (!dead)
#pragma unroll
          for (int x = 0; x < D / 16; ++x)  // with the first terms, with the second ones
            mma_ss_f8(to, kd + x % (D / 32) * 2,
                      qd + x % (D / 32) * 2 + x / (D / 32) * (kRowsItem * D / 16), idesc_s, x > 0);
        mma_commit(&s.s_full[b]);
        if (!kWide) mma_commit(&s.k_empty[slot]);
        if (iq == nq) mma_commit(kWide ? &s.q_read : &s.q_empty[jq & 1]);
      }
      __syncwarp();
      ++tq;
      if (iq == nq) {
        iq = 0;
        sq = step(++jq);
        nq = sq ? sq->v1 - sq->v0 : 0;
      }
    };
    scores();
    while (tp < tq) {
      scores();
      const uint32_t b = tp % NS;
      if (ip == 0) wait_or_die(&s.o_empty[jp & 1], ((jp >> 1) & 1) ^ 1, dead);
      wait_or_die(&s.v_full[b], (tp / NS) & 1, dead);
      wait_or_die(&s.p_full, tp & 1, dead);
      tc_fence_after();
      const uint64_t vd = make_sdesc(__shfl_sync(0xffffffffu, v0 + b * kVBytes, 0), kKeys * 128,
                                     1024, kSwizzle128);
      const uint64_t pd = make_sdesc(
          __shfl_sync(0xffffffffu, kWide ? k0 + b * kKBytes : p0, 0), 16, 1024, kSwizzle128);
      const uint32_t to = __shfl_sync(0xffffffffu, tmu + kColO + kRowsItem * (jp & 1), 0);
      if (leader) {
        if (!dead)
#pragma unroll
          for (int x = 0; x < kKeys / 16; ++x)
            mma_ss(to, vd + x * (16 * 128 / 16),
                   pd + (x / 4) * (kRowsItem * 128 / 16) + (x % 4) * 2, idesc_o, ip > 0 || x > 0);
        mma_commit(&s.pv_done);
        mma_commit(&s.v_empty[b]);
        if (kWide) mma_commit(&s.k_empty[b]);
      }
      __syncwarp();
      ++tp;
      if (++ip == np) {
        step_done(jp);
        ip = 0;
        ++jp;
        const Step& nx = s.steps[jp % kSteps];
        np = tp < tq ? nx.v1 - nx.v0 : 0;
      }
    }
  } else if (warp > kQueryWarp) {
    for (uint32_t j = 0; step(j); ++j) {
      convert(j, 1);
      step_done(j);
    }
  } else if (warp == kQueryWarp) {
    // The items, one ahead of the query rows of each.
    Walker w;
    bool live = w.start(a, s.plan);
    Header hd;
    hd.rows = 0;
    for (uint32_t j = 0;; ++j) {
      wait_or_die(&s.step_empty[j % kSteps], ((j / kSteps) & 1) ^ 1, dead);
      dead = __any_sync(0xffffffffu, dead);
      if (dead) break;
      Step& next = s.steps[j % kSteps];
      const bool here = live;
      if (here) {
        if (lane == 0) {
          next.n = w.n; next.h = w.h; next.bos = w.s.bos; next.pos0 = w.s.pos0;
          next.v0 = w.v0; next.v1 = w.v1;
          next.g = w.g;
        }
        if (w.v0 == 0 && w.v1 < w.g.nt) {  // starts here and goes on: only the last item does
          hd.rows = w.g.rows;
          hd.row0 = w.g.row0;
          hd.h = w.h;
          hd.nt = w.g.nt;
          hd.bos = w.s.bos;
          hd.start = w.start_at;
          hd.total = s.plan.total;
        }
        live = w.next(a);
      }
      if (lane == 0) {
        next.live = here;
        mbar_arrive(&s.step_full[j % kSteps]);
      }
      __syncwarp();
      if (j > 0) convert(j - 1, 0);  // the rows of the item before
      if (!here) break;
    }
    if (lane == 0) headers[blockIdx.x] = hd;
  } else if (warp >= kExpandWarp && warp < kLoadWarp) {
    // A thread has a key's row of each tile of values: its bytes, where they landed, into
    // registers, and the row as bf16 into the slot in the products' layout (whose pieces in the
    // upper half, D = 128, lie where the row's own bytes did).
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsExpand));
    const int r = tid - 32 * kExpandWarp;
    const q8::Scale16 one(q8::kBias);
    uint32_t t = 0;
    for (uint32_t j = 0;; ++j) {
      const Step* st = step(j);
      if (!st) break;
      const int n = st->v1 - st->v0;
#pragma unroll 1
      for (int i = 0; i < n; ++i, ++t) {
        const uint32_t b = t % NS;
        wait_or_die(&s.vr_full[b], (t / NS) & 1, dead);
        uint8_t* slot = sV + b * kVBytes;
        // In a loop: little code, which a small call has to fetch.  (The pieces that are written
        // over the row's bytes are behind those that have been read.)
        uint4 w = *reinterpret_cast<const uint4*>(slot + kLand + raw_offset<D>(r, 0));
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          const uint32_t x[4] = {w.x, w.y, w.z, w.w};
          if (c + 1 < D / 16)
            w = *reinterpret_cast<const uint4*>(slot + kLand + raw_offset<D>(r, c + 1));
          uint32_t y[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) q8::expand4(x[k], one, y[2 * k], y[2 * k + 1]);
          *reinterpret_cast<uint4*>(slot + piece_offset<D>(r, 2 * c)) =
              make_uint4(y[0], y[1], y[2], y[3]);
          *reinterpret_cast<uint4*>(slot + piece_offset<D>(r, 2 * c + 1)) =
              make_uint4(y[4], y[5], y[6], y[7]);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.v_full[b]);
      }
      step_done(j);
    }
  } else if (warp < kExpandWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int r = tid;  // the thread's key in the tile
    // The column whose lane of O is the thread's: with D = 64 a warp has sixteen.
    const int d = q8::place(D == 128 ? tid : warp * 16 + (lane & 15));
    const bool has = D == 128 || lane < 16;
    const uint32_t lanebits = uint32_t(warp) << 21;  // (32 * warp) << 16
    const uint32_t prow = (r >> 6) * (kRowsItem * 128) + (r & 7) * 2;
    const uint32_t pchunk = uint32_t(r >> 3 & 7) << 4;
    uint32_t t = 0, nv = 0;
    // All softmax warps: what one wrote before it, the others see behind it.
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.vote);
      wait_or_die(&s.vote, nv & 1, dead);
      ++nv;
    };
    for (uint32_t j = 0;; ++j) {
      const Step* st = step(j);
      if (!st) break;
      const Step w = *st;
      const int n = w.v1 - w.v0, nr = w.g.rows;
      const uint32_t qb = j & 1, tO = tm + kColO + kRowsItem * qb + lanebits;
      wait_or_die(&s.q_full[qb], (j >> 1) & 1, dead);
      const int pos_first = w.pos0 + div_g(a, w.g.row0);
      const int pos_last = w.pos0 + div_g(a, w.g.row0 + nr - 1);
      // NR: rows that the item's are padded to.
      auto item = [&](auto nrc) {
        constexpr int NR = decltype(nrc)::value;
        constexpr int NH = NR < 16 ? NR : 16;  // rows that are read and joined at a time
        // The standing maxima, of more rows than 16 in shared memory, a copy for each warp; rows
        // that have seen nothing yet (bits of none) stand at 0.
        constexpr bool kFar = NR > 16;
        float m[kFar ? 1 : NR], l[NR];
        uint32_t none = 0xffffffffu >> (32 - nr);
        float* const fm = s.m[warp];
        float* const fb = s.by[warp];
        float* const ff = s.f[warp];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          if (!kFar) m[kFar ? 0 : i] = 0.f;
          l[i] = 0.f;
        }
        if (kFar) {
          __syncwarp();
          if (lane < kRowsItem) fm[lane] = 0.f;
          __syncwarp();
        }
#pragma unroll 1
        for (int i = 0; i < n; ++i, ++t) {
          const int ks = tile_start(w.g, w.v0 + i), key = ks + r;
          const uint32_t b = t & 1, slot = t % NS, ph = (t / NS) & 1;
          wait_or_die(&s.k_full[slot], ph, dead);
          const float ck = q8::scale(s.k_scale[slot][r]);
          wait_or_die(&s.s_full[b], (t >> 1) & 1, dead);
          tc_fence_after();
          float x[NR];
#pragma unroll
          for (int e0 = 0; e0 < NR; e0 += NH) {
            float y[NH];
            tmem_ld<NH>(tm + kColS + kRowsItem * b + lanebits + e0, y);
#pragma unroll
            for (int e = 0; e < NH; ++e) x[e0 + e] = y[e];
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&s.s_empty[b]);
            mbar_arrive(&s.k_empty[slot]);
          }
          const bool whole =
              ks + kKeys <= pos_first + 1 &&
              (a.window == 0 || ks > max(pos_last, 0) - a.window || ks + kKeys <= a.sinks);
          // Scores, in log2 and less the standing maximum.
#pragma unroll
          for (int e = 0; e < NR; e += 4) {
            const float4 rs = *reinterpret_cast<const float4*>(&s.row_scale[qb][e]);
            const float4 mx = kFar ? *reinterpret_cast<const float4*>(fm + e)
                                   : make_float4(m[kFar ? 0 : e], m[kFar ? 0 : e + 1],
                                                 m[kFar ? 0 : e + 2], m[kFar ? 0 : e + 3]);
            x[e] = fmaf(x[e], ck * rs.x, -mx.x);
            x[e + 1] = fmaf(x[e + 1], ck * rs.y, -mx.y);
            x[e + 2] = fmaf(x[e + 2], ck * rs.z, -mx.z);
            x[e + 3] = fmaf(x[e + 3], ck * rs.w, -mx.w);
          }
          if (!whole) {
            // the position that sees the key no more
            const uint32_t until =
                a.window == 0 || key < a.sinks ? 0xffffffffu : (uint32_t)key + a.window;
#pragma unroll
            for (int e = 0; e < NR; ++e) {
              const int pos = s.row_pos[qb][e];
              if (key > pos || until <= (uint32_t)pos) x[e] = -INFINITY;
            }
          }
          bool grown = i == 0;
#pragma unroll
          for (int e = 0; e < NR; ++e) grown |= x[e] > kRescale;
          if (none && i > 0) {
#pragma unroll
            for (int e = 0; e < NR; ++e) grown |= (none >> e & 1) && x[e] > -INFINITY;
          }
          // One maximum for all warps: where one's has grown, all look for the new one.
          const bool any = __any_sync(0xffffffffu, grown);
          if (lane == 0) s.votes[nv & 1][warp] = any;
          const int4* vt = reinterpret_cast<const int4*>(s.votes[nv & 1]);
          meet();
          const int4 v = *vt;
          if (v.x | v.y | v.z | v.w) {
            float f[NH];
#pragma unroll
            for (int e0 = 0; e0 < NR; e0 += NH) {
#pragma unroll
              for (int e = 0; e < NH; ++e) f[e] = x[e0 + e];
              join_lanes(f, s.parts[nv & 1][warp] + e0,
                         [](float y, float z) { return fmaxf(y, z); });
            }
            const float(*all)[kRowsItem] = s.parts[nv & 1];
            meet();
            // What row e's maximum rises by, and the factor of what has been summed up: by lane e.
            bool up = false;
            if (lane < kRowsItem) {
              const float y = fmaxf(fmaxf(all[0][lane], all[1][lane]),
                                    fmaxf(all[2][lane], all[3][lane]));
              const bool first = none >> lane & 1;
              up = y > (first ? -INFINITY : kRescale);
              const float by = up ? y : 0.f;
              ff[lane] = !up ? 1.f : first ? 0.f : fast_exp2(-y);
              fb[lane] = by;
              if (kFar) fm[lane] += by;
            }
            none &= ~__ballot_sync(0xffffffffu, up);
            __syncwarp();
            if (i > 0) {  // O as far as it is
              wait_or_die(&s.pv_done, (t - 1) & 1, dead);
              tc_fence_after();
            }
#pragma unroll
            for (int e0 = 0; e0 < NR; e0 += NH) {
#pragma unroll
              for (int e = 0; e < NH; ++e) {
                const float by = fb[e0 + e];
                f[e] = ff[e0 + e];
                if (!kFar) m[kFar ? 0 : e] += by;
                l[e0 + e] *= f[e];
                x[e0 + e] -= by;
              }
              if (i > 0) {
                float o[NH];
                tmem_ld<NH>(tO + e0, o);
#pragma unroll
                for (int e = 0; e < NH; ++e) o[e] *= f[e];
                tmem_st<NH>(tO + e0, o);
              }
            }
          }
          wait_or_die(&s.vr_full[slot], ph, dead);
          const float cv = q8::scale(s.v_scale[slot][r]);
#pragma unroll
          for (int e = 0; e < NR; ++e) {
            const float p = fast_exp2(x[e]);
            l[e] += p;
            x[e] = p * cv;
          }
          if (!whole && cv != cv) {  // a NaN counts where it is seen
#pragma unroll
            for (int e = 0; e < NR; ++e)
              if (!visible(a, s.row_pos[qb][e], key)) x[e] = 0.f;
          }
          if (t > 0) wait_or_die(&s.pv_done, (t - 1) & 1, dead);  // the last weights were read
#pragma unroll
          for (int e = 0; e < NR; ++e)
            *reinterpret_cast<__nv_bfloat16*>((kWide ? sK + slot * kKBytes : sP) + prow +
                                              (e >> 3) * 1024 + (e & 7) * 128 +
                                              (pchunk ^ uint32_t((e & 7) << 4))) =
                __float2bfloat16_rn(x[e]);
          fence_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.p_full);
        }
        // The item's result: the keys' sums joined, columns of O by each thread.
#pragma unroll
        for (int e0 = 0; e0 < NR; e0 += NH) {
          float y[NH];
#pragma unroll
          for (int e = 0; e < NH; ++e) y[e] = l[e0 + e];
          join_lanes(y, s.parts[nv & 1][warp] + e0, [](float y, float z) { return y + z; });
        }
        const float(*all)[kRowsItem] = s.parts[nv & 1];
        meet();
        wait_or_die(&s.pv_done, (t - 1) & 1, dead);
        tc_fence_after();
        // What the rows need, row e's by lane e: where they go, and what they are divided by.
        const bool cut0 = w.v0 > 0, cut = cut0 || w.v1 < w.g.nt;
        float inv = 1.f;
        long long at;
        {
          const int e = min(lane, nr - 1), row = w.g.row0 + e, tk = div_g(a, row);
          const float sum = (all[0][e] + all[1][e]) + (all[2][e] + all[3][e]);
          float mx = kFar ? fm[e] : m[0];
#pragma unroll
          for (int k = 1; k < (kFar ? 1 : NR); ++k) mx = e == k ? m[k] : mx;
          const bool writes = warp == 0 && lane < nr;
          if (cut) {
            at = (long long)(2 * blockIdx.x + (cut0 ? 0 : 1)) * kRowsItem + e;
            if (writes) part_ml[at] = make_float2(mx, sum);
          } else {
            at = (long long)(w.bos + tk) * a.Hq + w.h * a.G + (row - tk * a.G);
            inv = sum == 0.f ? -1.f : 1.0f / sum;
            if (writes && a.lse)
              a.lse[at] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * 0.6931471805599453f;
          }
          at *= D;
        }
#pragma unroll 1
        for (int e0 = 0; e0 < (kFar ? nr : 1); e0 += NH) {
          float o[NH];
          tmem_ld<NH>(tO + e0, o);
          if (e0 + NH >= nr) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&s.o_empty[qb]);
              mbar_arrive(&s.q_empty[qb]);
            }
          }
          // In a loop that passes the values along: little code.
#pragma unroll 1
          for (int e = e0; e < min(nr, e0 + NH); e += 4) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float f = __shfl_sync(0xffffffffu, inv, e + k);
              const long long to = __shfl_sync(0xffffffffu, at, e + k) + d;
              if (has && e + k < nr) {
                if (cut)
                  part_o[to] = o[k];
                else
                  static_cast<__nv_bfloat16*>(a.out)[to] =
                      __float2bfloat16_rn(f < 0.f ? 0.f : o[k] * f);
              }
            }
#pragma unroll
            for (int k = 0; k + 4 < NH; ++k) o[k] = o[k + 4];
          }
        }
      };
      if constexpr (kWide) {
        if (nr <= 16)
          item(Int<16>{});
        else
          item(Int<32>{});
      } else if (nr <= 4) {
        item(Int<4>{});
      } else if (nr <= 8) {
        item(Int<8>{});
      } else {
        item(Int<16>{});
      }
      step_done(j);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tm, kTmemCols);
}

static_assert(sizeof(Header) * kStretches <= 16384, "headers");
static_assert(kStretches * kRowsItem <= 152 * 256, "inside the workspace of the other kernel");

template <int D>
cudaError_t launch_t(const PagedArgs& a, void* workspace, cudaStream_t st) {
  CUtensorMap kmap{}, vmap{};
  if (a.num_pages > 0 && a.max_pages > 0)
    if (!cache_map<true>(&kmap, a.k_cache, a) || !cache_map<true>(&vmap, a.v_cache, a))
      return cudaErrorInvalidValue;
  Header* headers = static_cast<Header*>(workspace);
  float2* ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + 16384);
  float* po = reinterpret_cast<float*>(ml + (size_t)2 * kStretches * kRowsItem);
  cudaError_t e = cudaFuncSetAttribute(
      paged_q8_few_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  paged_q8_few_kernel<D>
      <<<kStretches, kThreads, Cfg<D>::kSmem, st>>>(a, kmap, vmap, headers, po, ml);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_join<D>(a, headers, po, ml, st);
}

cudaError_t launch_few(PagedArgs a, void* workspace, cudaStream_t st) {
  set_divisor(a);
  return a.D == 64 ? launch_t<64>(a, workspace, st) : launch_t<128>(a, workspace, st);
}

}  // namespace
}  // namespace kda
