// Attention of new tokens over a paged cache (kda_paged_attention_fwd, _q8_fwd,
// kda_paged_prefix_attention_fwd) in fp32.  (bf16 runs on the tensor cores: kda_paged_tc.cuh.)
//
// A block takes 16 query rows (tokens x query heads of one kv head) of one sequence and one
// part of its visible keys, and keeps for every row the running maximum m, the sum l of
// e^{s - m} and the unnormalised output, so the keys are read once.  Keys are taken 32 at a
// time into shared memory: a lane scores one key against the warp's rows, and then owns D / 32
// output columns of those rows.  Bound by latency (a step of keys is a round trip to memory), so
// a long key range is cut into parts (for few rows) whose (m, l, o) are joined by a second
// kernel, and blocks share an SM.  5 sequences of 1..17 tokens over up to 700 keys, 4 + 4 heads
// of 64: 11.5 us.  Chunks take taller tiles (below), which the FMA pipes bound.
//
// Rows in 8 bits are expanded to fp32 on their way into shared memory.  With prefixes the parts of
// both of a row's lists are joined by the second kernel.
#include "kda_paged.cuh"
#include "kda_q8.cuh"

namespace kda {
namespace {

constexpr int kRows = 16;    // query rows of a block
constexpr int kWarps = 4;    // of a block
constexpr int kKeys = 32;    // keys of a step
constexpr int kThreads = 128;
constexpr int kMaxParts = 32;
constexpr int kMinPartKeys = kKeys;  // one step: a step is a round trip to memory

// 16 bytes, or zeros.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src), "r"(there ? 16 : 0)
               : "memory");
}

// 16 numbers of an 8-bit row, from column c on, as fp32 (or zeros).  Their rounding to 8 bits is
// undone exactly, so the arithmetic behind it is that of an fp32 cache.
__device__ __forceinline__ void expand16(float* dst, const void* cache, const uint8_t* scales,
                                         long long row, int D, int c, bool there) {
  uint4 w = make_uint4(0, 0, 0, 0);
  float s = 1.f;
  if (there) {
    w = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(cache) + row * D + c));
    s = q8::scale(__ldg(scales + row));
  }
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = q8::unpack2(x[i]), b = q8::unpack2(x[i] >> 16);
    *reinterpret_cast<float4*>(dst + 4 * i) = make_float4(a.x * s, a.y * s, b.x * s, b.y * s);
  }
}

// Place of a row's part in the partial results: those of prefixes come first.
__device__ __forceinline__ long long part_row(const PagedArgs& a, int n, int part, int parts,
                                              long long row) {
  const int side = a.groups > 0 && n >= a.groups;
  return ((long long)side * parts + part) * a.total_T * a.Hq + row;
}

template <int D> struct Short {
  static constexpr int PK = D + 4;  // K pitch: 16-byte rows, lanes on different banks
  float k[kKeys * PK], v[kKeys * D], q[kRows * D];
};

// One row tile of list n, RW rows for each warp; all threads of the block call.
template <int D, int RW, bool Q8>
__device__ void row_tile(const PagedArgs& a, const Seq& q, int n, int r0, int nr, int parts,
                         Short<D>& sm, float* part_o, float2* part_ml) {
  constexpr int PK = Short<D>::PK;
  constexpr int C = D / 32;  // output columns of a lane
  float *sK = sm.k, *sV = sm.v, *sQ = sm.q;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.Hq / a.Hkv;
  const int hkv = blockIdx.y, part = blockIdx.z;
  const KeyRange kr = key_range(a, q, r0 / G, (r0 + nr - 1) / G);
  const int total = kr.sinks + kr.hi - kr.lo;
  int np = min(parts, (total + kMinPartKeys - 1) / kMinPartKeys);
  np = max(np, 1);
  const int per = (total + np - 1) / np;
  const int v0 = min(part * per, total), v1 = part < np ? min(v0 + per, total) : v0;

  for (int i = tid; i < kRows * (D / 4); i += kThreads) {
    const int r = i / (D / 4), c = i % (D / 4) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < nr) {
      const long long tok = (long long)q.bos + (r0 + r) / G;
      const float* p = static_cast<const float*>(a.q) + tok * a.q_stride +
                   (long long)(hkv * G + (r0 + r) % G) * D + c;
      x = *reinterpret_cast<const float4*>(p);
    }
    const float sc = a.scale * 1.4426950408889634f;  // scores in log2 units
    *reinterpret_cast<float4*>(&sQ[r * D + c]) =
        make_float4(x.x * sc, x.y * sc, x.z * sc, x.w * sc);
  }

  float m[RW], l[RW], o[RW][C];
  int pos[RW];
#pragma unroll
  for (int r = 0; r < RW; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
    const int rr = warp * RW + r;
    pos[r] = rr < nr ? q.pos0 + (r0 + rr) / G : -1;
#pragma unroll
    for (int c = 0; c < C; ++c) o[r][c] = 0.f;
  }
  const bool busy = warp * RW < nr;
  // A step's K and V rows; places behind the part's end hold zeros.
  constexpr int PIECES = D / 4;
  auto fetch = [&](int vb) {
    if constexpr (Q8) {
      constexpr int P16 = D / 16;
#pragma unroll
      for (int i = tid; i < kKeys * P16; i += kThreads) {
        const int key_i = i / P16, c = i % P16 * 16;
        const bool there = vb + key_i < v1;
        const long long row = there ? cache_row(a, n, hkv, virtual_key(kr, vb + key_i)) : 0;
        expand16(&sK[key_i * PK + c], a.k_cache, a.k_scale, row, D, c, there);
        expand16(&sV[key_i * D + c], a.v_cache, a.v_scale, row, D, c, there);
      }
      return;
    }
#pragma unroll
    for (int k = 0; k < kKeys * PIECES / kThreads; ++k) {
      const int i = tid + k * kThreads;
      const int key_i = i / PIECES, c = i % PIECES * 4;
      const bool there = vb + key_i < v1;
      const long long off =
          there ? cache_row(a, n, hkv, virtual_key(kr, vb + key_i)) * D + c : 0;
      copy16(&sK[key_i * PK + c], static_cast<const float*>(a.k_cache) + off, there);
      copy16(&sV[key_i * D + c], static_cast<const float*>(a.v_cache) + off, there);
    }
  };
  if (v0 < v1) fetch(v0);
  for (int vb = v0; vb < v1; vb += kKeys) {
    if (vb > v0) {
      __syncthreads();  // the last step's are done with
      fetch(vb);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    if (!busy) continue;
    float s[RW];
#pragma unroll
    for (int r = 0; r < RW; ++r) s[r] = 0.f;
#pragma unroll 8
    for (int c = 0; c < D; c += 4) {
      const float4 kx = *reinterpret_cast<const float4*>(&sK[lane * PK + c]);
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        const float4 qx = *reinterpret_cast<const float4*>(&sQ[(warp * RW + r) * D + c]);
        s[r] += qx.x * kx.x + qx.y * kx.y + qx.z * kx.z + qx.w * kx.w;
      }
    }
    const bool in = vb + lane < v1;
    const int key = in ? virtual_key(kr, vb + lane) : 0;
    float p[RW];
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      const bool see = in && visible(a, pos[r], key);
      const float x = see ? s[r] : -INFINITY;
      float mx = x;
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, mx, w);
        mx = (y > mx || y != y) ? y : mx;  // a NaN score stays
      }
      const float mn = (mx > m[r] || mx != mx) ? mx : m[r];
      const float base = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(m[r] - base);
      p[r] = see ? exp2f(x - base) : 0.f;
      m[r] = mn;
      l[r] = l[r] * f + p[r];  // the lane's own share; joined at the end
#pragma unroll
      for (int c = 0; c < C; ++c) o[r][c] *= f;
    }
    const int steps = min(kKeys, v1 - vb);
    for (int j = 0; j < steps; ++j) {
      float vx[C];
#pragma unroll
      for (int c = 0; c < C; ++c) vx[c] = sV[j * D + c * 32 + lane];
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        const float pj = __shfl_sync(0xffffffffu, p[r], j);
        if (pj != 0.f) {  // a hidden key's value never counts, whatever it holds
#pragma unroll
          for (int c = 0; c < C; ++c) o[r][c] += pj * vx[c];
        }
      }
    }
  }
  if (!busy) return;
#pragma unroll
  for (int r = 0; r < RW; ++r) {
    const float lt = warp_sum(l[r]);
    const int rr = warp * RW + r;
    if (rr >= nr) continue;
    const long long tok = (long long)q.bos + (r0 + rr) / G;
    const long long row = tok * a.Hq + hkv * G + (r0 + rr) % G;
    if (parts > 1 || a.groups > 0) {
      const long long at = part_row(a, n, part, parts, row);
#pragma unroll
      for (int c = 0; c < C; ++c) part_o[at * D + c * 32 + lane] = o[r][c];
      if (lane == 0) part_ml[at] = make_float2(m[r], lt);
    } else {
      const float inv = lt == 0.f ? 0.f : 1.0f / lt;  // (NaN stays NaN)
#pragma unroll
      for (int c = 0; c < C; ++c)
        static_cast<float*>(a.out)[row * D + c * 32 + lane] = o[r][c] * inv;
      if (lane == 0 && a.lse)
        a.lse[row] = lt == 0.f ? -INFINITY : (m[r] + log2f(lt)) * 0.6931471805599453f;
    }
  }
}

// ------------------------------------------------------------------------- tall row tiles
//
// The same for chunks: 64 rows against 64 keys at a time.  A thread of a block of 16 x 8 scores
// the rows ty + 16 i against the keys tx + 8 j (NI x 8 products, in pairs along D), and then owns
// D / 8 output columns of those rows; the weights pass through shared memory, over the keys.
// Bound by the FMA pipes, closely followed by shared memory: a warp's 16-byte load takes a cycle
// for each half of it, however many lanes share an address, so 12 loads for 128 multiply-adds of
// a thread are three quarters of what the FMA pipes take (16 x 16 threads: 24 cycles of loads for
// 16).  Two blocks share an SM, and one computes while the other waits for its keys.
// NI: the rows of a thread that the tile needs.

constexpr int kTallRows = 64, kTallKeys = 64;

template <int D> struct Tall {
  static constexpr int PQ = D + 4;             // pitches: 16-byte rows, neighbours on other banks
  static constexpr int PP = kTallKeys + 8;
  static constexpr int KP = PQ > PP ? PQ : PP;  // keys, then weights
  static constexpr int CG = D / 32;            // groups of 4 neighbouring columns of a thread
  static constexpr int kSmem = (kTallRows * PQ + kTallKeys * KP + kTallKeys * D) * 4;
};

__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 split(uint64_t p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
template <int D, int NI, bool Q8>
__device__ void tall_tile(const PagedArgs& a, const Seq& q, int n, int r0, int nr, int parts,
                          float* smem, float* part_o, float2* part_ml) {
  using T = Tall<D>;
  constexpr int PQ = T::PQ, PP = T::PP, CG = T::CG, NC = 2 * CG, NJ = kTallKeys / 8;
  float* sQ = smem;
  float* sK = sQ + kTallRows * PQ;
  float* sP = sK;
  float* sV = sK + kTallKeys * T::KP;
  const int tid = threadIdx.x, tx = tid & 7, ty = tid >> 3;
  const int G = a.Hq / a.Hkv, hkv = blockIdx.y, part = blockIdx.z;
  const KeyRange kr = key_range(a, q, r0 / G, (r0 + nr - 1) / G);
  const int total = kr.sinks + kr.hi - kr.lo;
  const int np = max(min(parts, (total + kTallKeys - 1) / kTallKeys), 1);
  const int per = (total + np - 1) / np;
  const int v0 = min(part * per, total), v1 = part < np ? min(v0 + per, total) : v0;
  const int shift = __ffs(a.page_size) - 1;

  const int32_t* table = table_of(a, n);
  auto fetch = [&](int vb) {
    constexpr int PIECES = Q8 ? D / 16 : D / 4;
#pragma unroll 4
    for (int i = tid; i < kTallKeys * PIECES; i += kThreads) {
      const int key_i = i / PIECES, c = i % PIECES * (D / PIECES);
      const bool there = vb + key_i < v1;
      const int key = there ? virtual_key(kr, vb + key_i) : 0;
      const int p = there ? __ldg(table + (key >> shift)) : 0;
      const long long row =
          (((long long)min(max(p, 0), a.num_pages - 1) * a.Hkv + hkv) << shift) +
          (key & (a.page_size - 1));
      if constexpr (Q8) {
        expand16(&sK[key_i * PQ + c], a.k_cache, a.k_scale, row, D, c, there);
        expand16(&sV[key_i * D + c], a.v_cache, a.v_scale, row, D, c, there);
        continue;
      }
      copy16(&sK[key_i * PQ + c], static_cast<const float*>(a.k_cache) + row * D + c, there);
      copy16(&sV[key_i * D + c], static_cast<const float*>(a.v_cache) + row * D + c, there);
    }
  };
  if (v0 < v1) fetch(v0);
  for (int i = tid; i < NI * 16 * (D / 4); i += kThreads) {
    const int row = i / (D / 4), c = i % (D / 4) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < nr) {
      const long long tok = (long long)q.bos + (r0 + row) / G;
      x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + tok * a.q_stride +
                                           (long long)(hkv * G + (r0 + row) % G) * D + c);
    }
    const float sc = a.scale * 1.4426950408889634f;  // scores in log2 units
    *reinterpret_cast<float4*>(&sQ[row * PQ + c]) =
        make_float4(x.x * sc, x.y * sc, x.z * sc, x.w * sc);
  }
  float m[NI], l[NI];
  int pos[NI];
  uint64_t o[NI][NC];  // pairs of columns
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
    pos[i] = ty + 16 * i < nr ? q.pos0 + (r0 + ty + 16 * i) / G : -1;
#pragma unroll
    for (int c = 0; c < NC; ++c) o[i][c] = 0;
  }
  const int pos_first = q.pos0 + r0 / G, pos_last = q.pos0 + (r0 + nr - 1) / G;
  for (int vb = v0; vb < v1; vb += kTallKeys) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    // Values that are not finite: then hidden keys are left out one by one (zero times them
    // would not be zero).
    if (Q8) __syncthreads();  // (the pieces below are others' here)
    float odd = 0.f;
#pragma unroll 4
    for (int i = tid; i < kTallKeys * (D / 4); i += kThreads) {
      const float4 x = *reinterpret_cast<const float4*>(&sV[i * 4]);
      odd += x.x * 0.f + x.y * 0.f + x.z * 0.f + x.w * 0.f;
    }
    const bool careful = __syncthreads_or(odd != 0.f);  // (each thread has read its own pieces)
    uint64_t s2[NI][NJ];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) s2[i][j] = 0;
#pragma unroll 2
    for (int c = 0; c < D; c += 4) {
      ulonglong2 k[NJ];
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        k[j] = *reinterpret_cast<const ulonglong2*>(&sK[(tx + 8 * j) * PQ + c]);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(&sQ[(ty + 16 * i) * PQ + c]);
#pragma unroll
        for (int j = 0; j < NJ; ++j) s2[i][j] = fma2(x.y, k[j].y, fma2(x.x, k[j].x, s2[i][j]));
      }
    }
    const int first = virtual_key(kr, vb);
    const bool whole = vb + kTallKeys <= v1 && virtual_key(kr, vb + kTallKeys - 1) <= pos_first &&
                       (a.window == 0 || first > pos_last - a.window);
    __syncthreads();  // the keys are done with
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      float s[NJ], mx = -INFINITY;
      bool see[NJ];
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const float2 h = split(s2[i][j]);
        const int v = vb + tx + 8 * j;
        see[j] = whole || (v < v1 && visible(a, pos[i], virtual_key(kr, v)));
        s[j] = see[j] ? h.x + h.y : -INFINITY;
        mx = (s[j] > mx || s[j] != s[j]) ? s[j] : mx;  // a NaN score stays
      }
#pragma unroll
      for (int w = 4; w > 0; w >>= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, mx, w);
        mx = (y > mx || y != y) ? y : mx;
      }
      const float mn = (mx > m[i] || mx != mx) ? mx : m[i];
      const float base = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(m[i] - base);
      m[i] = mn;
      l[i] *= f;  // the thread's own share; joined at the end
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const float p = see[j] ? exp2f(s[j] - base) : 0.f;
        l[i] += p;
        sP[(ty + 16 * i) * PP + tx + 8 * j] = p;
      }
      const uint64_t f2 = pair(f, f);
#pragma unroll
      for (int c = 0; c < NC; ++c) o[i][c] = mul2(o[i][c], f2);
    }
    __syncthreads();
    auto values = [&](int k, uint64_t(&v)[NC]) {  // columns 4 tx + 32 g + ...
#pragma unroll
      for (int g = 0; g < CG; ++g) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(&sV[k * D + 4 * tx + 32 * g]);
        v[2 * g] = x.x;
        v[2 * g + 1] = x.y;
      }
    };
    if (!careful) {
#pragma unroll 2
      for (int k = 0; k < kTallKeys; k += 4) {
        uint64_t v[4][NC];
#pragma unroll
        for (int e = 0; e < 4; ++e) values(k + e, v[e]);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const float4 p = *reinterpret_cast<const float4*>(&sP[(ty + 16 * i) * PP + k]);
          const uint64_t p2[4] = {pair(p.x, p.x), pair(p.y, p.y), pair(p.z, p.z), pair(p.w, p.w)};
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int c = 0; c < NC; ++c) o[i][c] = fma2(p2[e], v[e][c], o[i][c]);
        }
      }
    } else {
#pragma unroll 1
      for (int k = 0; k < kTallKeys; ++k) {
        uint64_t v[NC];
        values(k, v);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const float p = sP[(ty + 16 * i) * PP + k];
          if (p != 0.f)
#pragma unroll
            for (int c = 0; c < NC; ++c) o[i][c] = fma2(pair(p, p), v[c], o[i][c]);
        }
      }
    }
    __syncthreads();
    if (vb + kTallKeys < v1) fetch(vb + kTallKeys);
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    float lt = l[i];
#pragma unroll
    for (int w = 4; w > 0; w >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, w);
    const int rr = ty + 16 * i;
    if (rr >= nr) continue;
    const long long tok = (long long)q.bos + (r0 + rr) / G;
    const long long row = tok * a.Hq + hkv * G + (r0 + rr) % G;
    const bool partial = parts > 1 || a.groups > 0;
    const long long at = part_row(a, n, part, parts, row);
    const float inv = partial ? 1.f : lt == 0.f ? 0.f : 1.0f / lt;  // (NaN stays NaN)
    float* dst = partial ? part_o + at * D : static_cast<float*>(a.out) + row * D;
#pragma unroll
    for (int g = 0; g < CG; ++g) {
      const float2 x = split(o[i][2 * g]), y = split(o[i][2 * g + 1]);
      *reinterpret_cast<float4*>(dst + 4 * tx + 32 * g) =
          make_float4(x.x * inv, x.y * inv, y.x * inv, y.y * inv);
    }
    if (tx == 0) {
      if (partial)
        part_ml[at] = make_float2(m[i], lt);
      else if (a.lse)
        a.lse[row] = lt == 0.f ? -INFINITY : (m[i] + log2f(lt)) * 0.6931471805599453f;
    }
  }
}

// Blocks are numbered over the sequences' row tiles; with many sequences, where the search for a
// block's tile would cost more than the tile, over the sequences.
constexpr int kSearch = 1024;

template <int D, bool Q8>
__global__ void __launch_bounds__(kThreads, 4) paged_simt_kernel(PagedArgs a, int parts,
                                                              float* part_o, float2* part_ml) {
  __shared__ int s_find[2];
  __shared__ __align__(16) Short<D> sm;
  // Few rows are spread over the warps (16 single tokens over 4096 keys, 32 + 8 heads of 128:
  // 159 us; 350 when one warp had all of them).
  auto tile_of = [&](int n, int tile) {
    const Seq q = load_seq(a, n);
    const int rows = q.len * (a.Hq / a.Hkv), r0 = tile * kRows;
    const int nr = min(kRows, rows - r0);
    if (nr <= kWarps)
      row_tile<D, 1, Q8>(a, q, n, r0, nr, parts, sm, part_o, part_ml);
    else
      row_tile<D, 4, Q8>(a, q, n, r0, nr, parts, sm, part_o, part_ml);
  };
  if (lists(a) > kSearch) {
    const int n = blockIdx.x, G = a.Hq / a.Hkv;
    const int tiles = (int)(((long long)load_seq(a, n).len * G + kRows - 1) / kRows);
    for (int tile = 0; tile < tiles; ++tile) {
      __syncthreads();  // the last tile's shared memory is free
      tile_of(n, tile);
    }
  } else {
    int n, tile;
    if (find_row_tile<kThreads>(a, kRows, (int)blockIdx.x, s_find, n, tile)) tile_of(n, tile);
  }
}

template <int D, bool Q8>
__global__ void __launch_bounds__(kThreads, 2) paged_tall_kernel(PagedArgs a, int parts,
                                                                 float* part_o, float2* part_ml) {
  extern __shared__ __align__(16) float smem[];
  __shared__ int s_find[2];
  auto tile_of = [&](int n, int tile) {
    const Seq q = load_seq(a, n);
    const int rows = q.len * (a.Hq / a.Hkv), r0 = tile * kTallRows;
    const int nr = min(kTallRows, rows - r0);
    if (nr <= 16)
      tall_tile<D, 1, Q8>(a, q, n, r0, nr, parts, smem, part_o, part_ml);
    else if (nr <= 32)
      tall_tile<D, 2, Q8>(a, q, n, r0, nr, parts, smem, part_o, part_ml);
    else
      tall_tile<D, 4, Q8>(a, q, n, r0, nr, parts, smem, part_o, part_ml);
  };
  if (lists(a) > kSearch) {
    const int n = blockIdx.x, G = a.Hq / a.Hkv;
    const int tiles = (int)(((long long)load_seq(a, n).len * G + kTallRows - 1) / kTallRows);
    for (int tile = 0; tile < tiles; ++tile) {
      __syncthreads();  // the last tile's shared memory is free
      tile_of(n, tile);
    }
  } else {
    int n, tile;
    if (find_row_tile<kThreads>(a, kTallRows, (int)blockIdx.x, s_find, n, tile)) tile_of(n, tile);
  }
}

// One warp per query row: o = sum_i e^{m_i - m} o_i / sum_i e^{m_i - m} l_i over the parts.  A
// lane looks up one part's (m, l), so that the parts' outputs are then independent loads.
template <int D>
__global__ void __launch_bounds__(128) paged_simt_join_kernel(PagedArgs a, int parts,
                                                              const float* part_o,
                                                              const float2* part_ml) {
  constexpr int C = D / 32;
  static_assert(kMaxParts <= 32, "a part per lane");
  const long long rows = (long long)a.total_T * a.Hq;
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  // a programmatic launch behind the first kernel, which gives no early trigger: it may begin once
  // that one's blocks have left, so wait for what they wrote
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (row >= rows || !token_owned(a, row / a.Hq)) return;
  // with prefixes, twice as many parts, the first half for the tokens that have one
  const int all = a.groups > 0 ? 2 * parts : parts;
  const int none = a.groups > 0 && !token_grouped(a, row / a.Hq) ? parts : 0;
  const float2 ml = lane >= none && lane < all ? part_ml[lane * rows + row] : make_float2(0.f, 0.f);
  const bool some = ml.y != 0.f;  // (a NaN is something)
  float m = some ? ml.x : -INFINITY;
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, m, w);
    m = (y > m || y != y) ? y : m;
  }
  const float base = m == -INFINITY ? 0.f : m;
  const float g = some ? exp2f(ml.x - base) : 0.f;
  const float l = warp_sum(some ? ml.y * g : 0.f);
  float o[C];
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] = 0.f;
  unsigned todo = __ballot_sync(0xffffffffu, some);
  while (todo) {
    constexpr int U = 8;  // parts in flight
    float x[U][C], gw[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int j = todo ? __ffs(todo) - 1 : -1;
      todo &= todo - 1;
      gw[i] = __shfl_sync(0xffffffffu, g, max(j, 0));
      const float* src = part_o + (max(j, 0) * rows + row) * D + lane;
#pragma unroll
      for (int c = 0; c < C; ++c) x[i][c] = j >= 0 ? src[c * 32] : 0.f;
      if (j < 0) gw[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] += x[i][c] * gw[i];
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
#pragma unroll
  for (int c = 0; c < C; ++c)
    static_cast<float*>(a.out)[row * D + c * 32 + lane] = o[c] * inv;
  if (lane == 0 && a.lse)
    a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// Row tiles of a call, about (with prefixes, of the two lists that every row has).
long long row_tiles(bool big, const PagedArgs& a) {
  const long long height = big ? kTallRows : kRows;
  const long long tiles = ((long long)a.total_T * (a.Hq / a.Hkv) + height - 1) / height;
  auto side = [&](int n) {
    const long long seqs = n < a.total_T ? n : a.total_T;
    return tiles < seqs ? seqs : tiles;
  };
  return side(a.N) + (a.groups > 0 ? side(a.groups) : 0);
}

// Tall tiles where a sequence has 32 rows or more on average and the caches (at the block table's
// capacity) make a step of 64 keys for every place on the SMs.  16 sequences of 8 new tokens and
// 500 cached keys, 16 + 4 heads of 64: 24 us for 29; of 32 and 1000, 8 + 8 heads of 128: 118 for
// 223; but 200 tokens alone, 8 + 8 heads of 64: 19 for 14.  With prefixes the lists count as
// sequences, and the larger capacity.
bool tall(const PagedArgs& a) {
  const long long sides = a.groups > 0 ? 2 : 1;
  if (sides * a.total_T * (a.Hq / a.Hkv) < 32ll * (a.N + a.groups)) return false;
  const int pages = a.max_pages > a.max_prefix_pages ? a.max_pages : a.max_prefix_pages;
  const double steps = (double)pages * a.page_size / kTallKeys + 1;
  return row_tiles(true, a) * steps * a.Hkv >= 2 * 152;
}

// Parts of the key range: enough blocks for eight (tall: two) on each SM when there are few rows.
int simt_parts(bool big, const PagedArgs& a) {
  const long long tiles = row_tiles(big, a);
  if (tiles <= 0) return 1;
  const int most = a.groups > 0 ? kMaxParts / 2 : kMaxParts;  // (of each side)
  const long long p = 152 * (big ? 2 : 8) / (tiles * a.Hkv);
  return (int)(p < 1 ? 1 : p > most ? most : p);
}

// Partial results of `rows` query rows (tokens x heads), counted for each part.
size_t simt_bytes(long long rows, int D) { return (size_t)rows * (D + 2) * sizeof(float); }

// Rows of partial results of a call (0: it writes its output at once).
long long part_rows(const PagedArgs& a, int parts) {
  const long long rows = (long long)a.total_T * a.Hq;
  return a.groups > 0 ? 2 * parts * rows : parts > 1 ? parts * rows : 0;
}

template <int D, bool Q8>
cudaError_t launch_t(const PagedArgs& a, void* workspace, cudaStream_t st) {
  const bool big = tall(a);
  const int parts = simt_parts(big, a);
  const long long rows = (long long)a.total_T * a.Hq;
  float* po = static_cast<float*>(workspace);
  float2* pml = reinterpret_cast<float2*>(po + part_rows(a, parts) * D);
  const long long G = a.Hq / a.Hkv;
  const int height = big ? kTallRows : kRows;
  const int n = a.N + a.groups;
  const long long tiles =
      (a.groups > 0 ? 2 : 1) * ((a.total_T * G + height - 1) / height) + n;  // upper bound
  const dim3 grid((unsigned)(n > kSearch ? n : tiles), (unsigned)a.Hkv, (unsigned)parts);
  if (big) {
    const cudaError_t e = cudaFuncSetAttribute(
        paged_tall_kernel<D, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, Tall<D>::kSmem);
    if (e != cudaSuccess) return e;
    paged_tall_kernel<D, Q8><<<grid, kThreads, Tall<D>::kSmem, st>>>(a, parts, po, pml);
  } else {
    paged_simt_kernel<D, Q8><<<grid, kThreads, 0, st>>>(a, parts, po, pml);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || part_rows(a, parts) == 0) return e;
  // Programmatic: 14.3 us for 16.4 in the small case above, called from the host (in a graph the
  // same).
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((rows + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_simt_join_kernel<D>, a, parts, (const float*)po,
                            (const float2*)pml);
}

}  // namespace

size_t paged_simt_need(const PagedArgs& a) {
  return simt_bytes(part_rows(a, simt_parts(tall(a), a)), a.D);
}

// The most that a call of up to total_T tokens can need, so that a buffer for a program's largest
// batch serves every smaller one: simt_parts' parts times row tiles are at most its blocks.  With
// prefixes one part of each side at least.
size_t paged_simt_workspace(int total_T, int Hq, int D, bool prefix) {
  constexpr long long kMost = 152ll * 8 * kRows;
  static_assert(kMost == 152ll * 2 * kTallRows, "rows in flight, short and tall tiles");
  const long long tokens = (long long)total_T * Hq, all = kMaxParts * tokens;
  const long long rows = all < kMost ? all : kMost;
  return simt_bytes(prefix && rows < 2 * tokens ? 2 * tokens : rows, D);
}

cudaError_t launch_paged_simt(const PagedArgs& a, void* workspace, cudaStream_t st) {
  const bool q8 = a.k_scale != nullptr;
  switch (a.D) {
    case 32:
      return q8 ? launch_t<32, true>(a, workspace, st) : launch_t<32, false>(a, workspace, st);
    case 64:
      return q8 ? launch_t<64, true>(a, workspace, st) : launch_t<64, false>(a, workspace, st);
    default:
      return q8 ? launch_t<128, true>(a, workspace, st) : launch_t<128, false>(a, workspace, st);
  }
}

}  // namespace kda
