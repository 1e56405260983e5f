// RMS norm of every query and key head with the position rotation in the same pass
// (kda_qk_norm_rope_fwd / _append / _append_q8 / _bwd).
//
// Per head row x [D] of a token at position p, with weight w [D]:
//   r = 1 / sqrt(mean(x^2) + eps),   n = x r w,   y = Rot(p) n
// where Rot turns the pairs (i, i + R/2) (or (2i, 2i + 1), interleaved) of the first R elements
// by the angle whose cosine and sine are row p of the caller's tables.  Backward, with
// g = Rot(p)^T dy:
//   dw = sum over rows of g x r,   dx = r (g w - x r^2 mean(g w x)).
//
// Bound by HBM: every element is read once and written once (backward: two reads, one write)
// with ~8 flops between, so what costs is instructions, and the layout saves them: a row lies
// across D / VE lanes, each with two pieces of VE / 2 elements.  For half-split pairs the second
// piece holds the partners of the first (R / 2 elements on), so that a rotation needs no other
// lane and a lane needs one cosine and sine per pair; the mean is a few shuffles.  A warp takes
// a token's queries, keys or copied values: the lane's cosines, sines and weights are loaded
// once for all of them, and kUnroll row groups are in flight together.  16384 tokens of 32 + 8
// heads of 128, bf16: 53 us, 6.5 TB/s of the 6.8 of a copy (55.5 with 8 warps a block instead
// of 4); 80 when the rotation exchanged partners between lanes.  Of 4095 tokens of 16 + 2 + 2
// heads into the pages: 10.1 us for 6.3 of bytes, in almost three waves of blocks; the two thirds
// of them that have the keys or values find one row group, of two heads, and load it kUnroll
// times over.  Into pages in 8 bits 11.9 us.
#include "kda_internal.cuh"
#include "kda_q8.cuh"

namespace kda {
namespace {

constexpr int kUnroll = 4;    // row groups in flight
constexpr int kWarps = 4;     // warps of a block, forward
constexpr int kBwdWarps = 16;  // and backward
constexpr int kBwdUnroll = 2;  // row groups of a backward part
constexpr int kParts = 2;      // parts of a unit, at most
constexpr int kRing = 3;       // parts in a warp's ring

// Lane pieces of T as fp32: 8 bytes each.
template <typename T> struct Piece;
template <> struct Piece<float> {
  static constexpr int PE = 2;
  static __device__ __forceinline__ void unpack(uint2 w, float (&x)[2]) {
    x[0] = __uint_as_float(w.x);
    x[1] = __uint_as_float(w.y);
  }
  static __device__ __forceinline__ uint2 pack(const float (&x)[2]) {
    return make_uint2(__float_as_uint(x[0]), __float_as_uint(x[1]));
  }
};
template <> struct Piece<__nv_bfloat16> {
  static constexpr int PE = 4;
  static __device__ __forceinline__ void unpack(uint2 w, float (&x)[4]) {
    x[0] = __uint_as_float(w.x << 16);
    x[1] = __uint_as_float(w.x & 0xffff0000u);
    x[2] = __uint_as_float(w.y << 16);
    x[3] = __uint_as_float(w.y & 0xffff0000u);
  }
  static __device__ __forceinline__ uint2 pack(const float (&x)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]);
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2], x[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                      *reinterpret_cast<const uint32_t*>(&b));
  }
};

// Where a lane's two pieces start in a row, and its pairs' cosines and sines.
template <typename T, int D>
struct Lane {
  static constexpr int PE = Piece<T>::PE, VE = 2 * PE, L = D / VE, RPW = 32 / L;
  int a, b;             // first elements of the pieces
  float c[PE], s[PE];   // 1, 0 behind the rotated part

  __device__ __forceinline__ void place(const NormRopeArgs& g, int li, bool interleaved) {
    const bool split = !interleaved && li * VE < g.R;
    a = split ? li * PE : li * VE;
    b = split ? a + g.R / 2 : a + PE;
  }
  __device__ __forceinline__ void load_turn(const NormRopeArgs& g, long long tok, int li) {
#pragma unroll
    for (int i = 0; i < PE; ++i) {
      c[i] = 1.f;
      s[i] = 0.f;
    }
    if (li * VE < g.R) {
      const int p = min(max(g.positions[tok], 0), g.max_position - 1);
      const long long off = (long long)p * (g.R / 2) + li * PE;
#pragma unroll
      for (int i = 0; i < PE; i += 2) {
        const float2 x = __ldg(reinterpret_cast<const float2*>(g.cos_table + off + i));
        const float2 y = __ldg(reinterpret_cast<const float2*>(g.sin_table + off + i));
        c[i] = x.x; c[i + 1] = x.y;
        s[i] = y.x; s[i + 1] = y.y;
      }
    }
  }
  __device__ __forceinline__ void load_weight(const float* w, float (&wa)[PE],
                                              float (&wb)[PE]) const {
#pragma unroll
    for (int i = 0; i < PE; i += 2) {
      const float2 x = w ? __ldg(reinterpret_cast<const float2*>(w + a + i))
                         : make_float2(1.f, 1.f);
      const float2 y = w ? __ldg(reinterpret_cast<const float2*>(w + b + i))
                         : make_float2(1.f, 1.f);
      wa[i] = x.x; wa[i + 1] = x.y;
      wb[i] = y.x; wb[i + 1] = y.y;
    }
  }
  // The k-th of the lane's PE pairs within its VE elements (a's first, then b's).
  template <bool IL>
  static __device__ __forceinline__ constexpr int lo(int k) { return IL ? 2 * k : k; }
  template <bool IL>
  static __device__ __forceinline__ constexpr int hi(int k) { return IL ? 2 * k + 1 : k + PE; }
};

template <int L>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Both pieces of a row into x[VE].
template <typename T, int D>
__device__ __forceinline__ void unpack_row(uint2 pa, uint2 pb, float (&x)[Lane<T, D>::VE]) {
  constexpr int PE = Lane<T, D>::PE;
  float u[PE], v[PE];
  Piece<T>::unpack(pa, u);
  Piece<T>::unpack(pb, v);
#pragma unroll
  for (int i = 0; i < PE; ++i) {
    x[i] = u[i];
    x[PE + i] = v[i];
  }
}
template <typename T, int D>
__device__ __forceinline__ void store_row(T* row, const Lane<T, D>& l,
                                          const float (&x)[Lane<T, D>::VE]) {
  constexpr int PE = Lane<T, D>::PE;
  float u[PE], v[PE];
#pragma unroll
  for (int i = 0; i < PE; ++i) {
    u[i] = x[i];
    v[i] = x[PE + i];
  }
  *reinterpret_cast<uint2*>(row + l.a) = Piece<T>::pack(u);
  *reinterpret_cast<uint2*>(row + l.b) = Piece<T>::pack(v);
}
// A row in 8 bits: the lane's two pieces, and the scale's byte by the row's first lane.  The whole
// warp calls; `keep`: the row is one.
template <typename T, int D>
__device__ __forceinline__ void store_row_q8(uint8_t* row, uint8_t* scale, const Lane<T, D>& l,
                                             const float (&x)[Lane<T, D>::VE], int li, bool keep) {
  constexpr int PE = Lane<T, D>::PE, L = Lane<T, D>::L;
  uint32_t top = 0;  // magnitudes as integers: infinities above numbers, NaNs above those
#pragma unroll
  for (int e = 0; e < 2 * PE; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const bool odd = top >= 0x7f800000u;
  const int e = q8::exponent(top);
  const float f = odd ? 0.f : q8::power(-e);
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    uint32_t b[PE / 2];
#pragma unroll
    for (int i = 0; i < PE; i += 2) {
      const float u = odd ? 0.f : x[part * PE + i], v = odd ? 0.f : x[part * PE + i + 1];
      b[i / 2] = q8::pack2(u * f, v * f);
    }
    uint8_t* dst = row + (part ? l.b : l.a);
    if (!keep) continue;
    if constexpr (PE == 4)
      *reinterpret_cast<uint32_t*>(dst) = b[0] | b[PE / 2 - 1] << 16;
    else
      *reinterpret_cast<uint16_t*>(dst) = (uint16_t)b[0];
  }
  if (keep && li == 0) *scale = (uint8_t)(odd ? q8::kNaN : e + q8::kBias);
}
template <typename T>
__device__ __forceinline__ uint2 load_piece(const T* p) {
  return __ldcs(reinterpret_cast<const uint2*>(p));
}

// Forward: queries to query_out; keys to key_out, or (append) keys and values to their place
// in the pages, as they are or (Q8) in 8 bits.  blockIdx.y numbers a token's units of `per` heads
// of one kind.
template <typename T, int D, bool IL, bool Q8>
__global__ void __launch_bounds__(32 * kWarps) norm_rope_kernel(NormRopeArgs a, int per, int qu,
                                                                int ku) {
  using Ln = Lane<T, D>;
  constexpr int PE = Ln::PE, VE = Ln::VE, L = Ln::L, RPW = Ln::RPW;
  const int lane = threadIdx.x & 31, li = lane % L, rw = lane / L;
  const long long tok = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (tok >= a.T) return;
  int u = blockIdx.y;
  const int kind = u < qu ? 0 : u < qu + ku ? 1 : 2;  // queries, keys, values
  u -= kind == 0 ? 0 : kind == 1 ? qu : qu + ku;
  const int h0 = u * per, h1 = min(h0 + per, kind == 0 ? a.Hq : a.Hkv);
  Ln l;
  l.place(a, li, IL);
  const T* src = static_cast<const T*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) +
                 tok * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride);
  uint2 ra[kUnroll], rb[kUnroll];
  auto fetch = [&](int h) {
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int r = h + i * RPW + rw;
      const T* p = src + (long long)min(r, h1 - 1) * D;
      ra[i] = load_piece(p + l.a);
      rb[i] = load_piece(p + l.b);
    }
  };
  fetch(h0);
  // Where head h of this token goes: dst + h * dst_head.
  T* dst;
  uint8_t *dst8 = nullptr, *scale8 = nullptr;  // (Q8)
  long long dst_head = D;
  if (kind == 0) {
    dst = static_cast<T*>(a.q_out) + tok * a.Hq * D;
  } else if (!a.slots) {
    dst = static_cast<T*>(a.k_out) + tok * a.Hkv * D;
  } else {
    const long long slot = a.slots[tok];
    if (slot < 0 || slot >= (long long)a.num_pages * a.page_size) return;  // not kept
    const long long page = slot >> a.page_shift;
    dst_head = (long long)a.page_size * D;
    const long long in_page = slot - (page << a.page_shift);
    if constexpr (Q8) {
      dst = nullptr;
      dst8 = static_cast<uint8_t*>(kind == 1 ? a.k_cache : a.v_cache) + page * a.Hkv * dst_head +
             in_page * D;
      scale8 = (kind == 1 ? a.k_scale : a.v_scale) + page * a.Hkv * a.page_size + in_page;
    } else {
      dst = static_cast<T*>(kind == 1 ? a.k_cache : a.v_cache) + page * a.Hkv * dst_head +
            in_page * D;
    }
  }
  if (kind == 2) {
    for (int h = h0;;) {
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int r = h + i * RPW + rw;
        if constexpr (Q8) {
          if (h + i * RPW >= h1) break;  // (a warp alike; a row in 8 bits is more than a copy)
          float x[VE];
          unpack_row<T, D>(ra[i], rb[i], x);
          store_row_q8<T, D>(dst8 + r * dst_head, scale8 + (long long)r * a.page_size, l, x, li,
                             r < h1);
        } else if (r < h1) {
          T* row = dst + r * dst_head;
          *reinterpret_cast<uint2*>(row + l.a) = ra[i];
          *reinterpret_cast<uint2*>(row + l.b) = rb[i];
        }
      }
      if ((h += kUnroll * RPW) >= h1) return;
      fetch(h);
    }
  }
  float wa[PE], wb[PE];
  l.load_weight(kind == 0 ? a.q_weight : a.k_weight, wa, wb);
  l.load_turn(a, tok, li);
  // weight and turn in one: (y_lo, y_hi) = r (x_lo p0 - x_hi p1, x_lo p2 + x_hi p3)
  float p0[PE], p1[PE], p2[PE], p3[PE];
#pragma unroll
  for (int k = 0; k < PE; ++k) {
    const int e0 = Ln::template lo<IL>(k), e1 = Ln::template hi<IL>(k);
    const float w0 = e0 < PE ? wa[e0 % PE] : wb[e0 % PE];
    const float w1 = e1 < PE ? wa[e1 % PE] : wb[e1 % PE];
    p0[k] = w0 * l.c[k];
    p1[k] = w1 * l.s[k];
    p2[k] = w0 * l.s[k];
    p3[k] = w1 * l.c[k];
  }
  for (int h = h0;;) {
    float x[kUnroll][VE];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) unpack_row<T, D>(ra[i], rb[i], x[i]);
    const int now = h;
    h += kUnroll * RPW;
    if (h < h1) fetch(h);  // the next groups, while these are computed
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int row = now + i * RPW + rw;
      if (Q8 && now + i * RPW >= h1) break;
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < VE; ++e) ss += x[i][e] * x[i][e];
      const float v = row_sum<L>(ss) * (1.0f / D) + a.eps;
      float r = rsqrtf(v), y[VE];
      if (Q8 && kind == 1 && v < INFINITY) {
        // Of these only 8 bits stay, but which of two neighbours is nearest can hang on the last
        // bit: r by a Newton step with its residual exact, and multiplied last.  (Squares whose sum
        // leaves fp32 go the other way, whose r = 0 makes zeros; here zero times infinity would
        // make NaNs.)
        const float h = v * r, rest = fmaf(v, r, -h);
        r = fmaf(0.5f * r, fmaf(-h, r, 1.0f) - rest * r, r);
#pragma unroll
        for (int k = 0; k < PE; ++k) {
          const int e0 = Ln::template lo<IL>(k), e1 = Ln::template hi<IL>(k);
          y[e0] = (x[i][e0] * p0[k] - x[i][e1] * p1[k]) * r;
          y[e1] = (x[i][e0] * p2[k] + x[i][e1] * p3[k]) * r;
        }
      } else {
#pragma unroll
        for (int k = 0; k < PE; ++k) {
          const int e0 = Ln::template lo<IL>(k), e1 = Ln::template hi<IL>(k);
          const float x0 = x[i][e0] * r, x1 = x[i][e1] * r;
          y[e0] = x0 * p0[k] - x1 * p1[k];
          y[e1] = x0 * p2[k] + x1 * p3[k];
        }
      }
      if (Q8 && kind == 1)  // (warp-uniform)
        store_row_q8<T, D>(dst8 + row * dst_head, scale8 + (long long)row * a.page_size, l, y, li,
                           row < h1);
      else if (row < h1)
        store_row<T, D>(dst + row * dst_head, l, y);
    }
    if (h >= h1) break;
  }
}

// Two fp32 numbers in one register pair, and arithmetic on both at once.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void split(uint64_t p, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p));
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

__device__ __forceinline__ void copy8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// Backward: a fixed grid of warps walks the tokens, the first q_blocks blocks their queries and
// the others their keys, so that a warp sums its share of dw in registers; the block's sums go to
// partial[blockIdx.x][D].  A unit is up to kParts parts of kBwdUnroll row groups of a token; the
// grid sweeps the units in order, so that all warps read one neighbourhood of memory.  What a
// warp reads comes through a ring of its own in shared memory, kRing - 1 parts ahead, each lane
// copying what it will use itself: no register waits for memory, so that 16 warps of 118
// registers fit.
// 16384 tokens of 32 + 8 heads of 128: 84 to 86 us, 6.0 TB/s of the 6.8 of a copy; the instructions
// take 60% of the issue slots beside it.  91.5 with the loads in registers, 87 with single
// instead of packed fp32 arithmetic or 20 warps, 94 with 18, 108 with a ring of 6 (which leaves
// the tables no L1), 96 with one row group a part.
template <typename T, int D, bool IL>
__global__ void __launch_bounds__(32 * kBwdWarps) norm_rope_bwd_kernel(NormRopeArgs a,
                                                                       int q_blocks,
                                                                       float* partial) {
  using Ln = Lane<T, D>;
  constexpr int PE = Ln::PE, VE = Ln::VE, L = Ln::L, RPW = Ln::RPW, U = kBwdUnroll;
  __shared__ float s_dw[kBwdWarps][D];
  extern __shared__ __align__(16) uint2 s_ring[];  // [warp][kRing][U][4][lane]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, li = lane % L, rw = lane / L;
  const bool isk = (int)blockIdx.x >= q_blocks;
  const int first = isk ? blockIdx.x - q_blocks : blockIdx.x;
  const int blocks = isk ? gridDim.x - q_blocks : q_blocks;
  const int H = isk ? a.Hkv : a.Hq;
  Ln l;
  l.place(a, li, IL);
  // A lane's values of a row as pairs of pairs: v[j] the lower elements of its pairs 2j and
  // 2j + 1, v[NP + j] the upper ones.
  constexpr int NP = PE / 2;
  auto arrange = [](const float (&x)[VE], uint64_t (&v)[2 * NP]) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      v[j] = pair(x[Ln::template lo<IL>(2 * j)], x[Ln::template lo<IL>(2 * j + 1)]);
      v[NP + j] = pair(x[Ln::template hi<IL>(2 * j)], x[Ln::template hi<IL>(2 * j + 1)]);
    }
  };
  auto restore = [](const uint64_t (&v)[2 * NP], float (&x)[VE]) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      split(v[j], x[Ln::template lo<IL>(2 * j)], x[Ln::template lo<IL>(2 * j + 1)]);
      split(v[NP + j], x[Ln::template hi<IL>(2 * j)], x[Ln::template hi<IL>(2 * j + 1)]);
    }
  };
  uint64_t w[2 * NP], dw[2 * NP];
  {
    float wa[PE], wb[PE], both[VE];
    l.load_weight(isk ? a.k_weight : a.q_weight, wa, wb);
#pragma unroll
    for (int e = 0; e < PE; ++e) {
      both[e] = wa[e];
      both[PE + e] = wb[e];
    }
    arrange(both, w);
  }
#pragma unroll
  for (int j = 0; j < 2 * NP; ++j) dw[j] = pair(0.f, 0.f);
  const int parts = min(kParts, (H + U * RPW - 1) / (U * RPW));
  const int per = (H + parts * U * RPW - 1) / (parts * U * RPW);  // units of a token
  const int W = blocks * kBwdWarps, step_tok = W / per, step_unit = W % per;
  const T* src = static_cast<const T*>(isk ? a.k : a.q);
  const T* gsrc = static_cast<const T*>(isk ? a.dk_out : a.dq_out);
  T* dst = static_cast<T*>(isk ? a.dk : a.dq);
  const long long stride = isk ? a.k_stride : a.q_stride;
  const uint2* ring = s_ring + warp * (kRing * U * 4 * 32) + lane;
  const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  // token and unit in it, of the loads and of the sums
  int ltok = (warp * blocks + first) / per, lunit = (warp * blocks + first) % per, lpart = 0;
  int tok = ltok, unit = lunit, lslot = 0, slot = 0;
  auto next = [&](int& tk, int& un) {
    tk += step_tok;
    un += step_unit;
    if (un >= per) {
      un -= per;
      ++tk;
    }
  };
  auto load = [&] {
    if (ltok < a.T) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int h = min(((lunit * parts + lpart) * U + i) * RPW + rw, H - 1);
        const T* x = src + ltok * stride + h * D;
        const T* g = gsrc + ((long long)ltok * H + h) * D;
        const uint32_t at = ring_at + (lslot * U + i) * (4 * 32 * 8);
        copy8(at, x + l.a);
        copy8(at + 256, x + l.b);
        copy8(at + 512, g + l.a);
        copy8(at + 768, g + l.b);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    lslot = lslot + 1 == kRing ? 0 : lslot + 1;
    if (++lpart == parts || (lunit * parts + lpart) * (U * RPW) >= H) {
      lpart = 0;
      next(ltok, lunit);
    }
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) load();
  if (tok < a.T) l.load_turn(a, tok, li);
  while (tok < a.T) {
    int tok2 = tok, unit2 = unit;
    next(tok2, unit2);
    Ln nx = l;
    if (tok2 < a.T) nx.load_turn(a, tok2, li);
    for (int part = 0; part < parts && (unit * parts + part) * (U * RPW) < H; ++part) {
      uint64_t x[U][2 * NP], g[U][2 * NP];
      asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const uint2* at = ring + (slot * U + i) * (4 * 32);
        float raw[VE];
        unpack_row<T, D>(at[0], at[32], raw);
        arrange(raw, x[i]);
        unpack_row<T, D>(at[64], at[96], raw);
        arrange(raw, g[i]);
      }
      slot = slot + 1 == kRing ? 0 : slot + 1;
      load();  // into the part used before this one
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int row = ((unit * parts + part) * U + i) * RPW + rw;
        uint64_t gw[2 * NP], ss2 = pair(0.f, 0.f), sd2 = ss2;
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          const uint64_t c = pair(l.c[2 * j], l.c[2 * j + 1]);
          const uint64_t s = pair(l.s[2 * j], l.s[2 * j + 1]);
          const uint64_t ns = pair(-l.s[2 * j], -l.s[2 * j + 1]);
          const uint64_t d0 = g[i][j], d1 = g[i][NP + j];
          g[i][j] = fma2(d0, c, mul2(d1, s));
          g[i][NP + j] = fma2(d1, c, mul2(d0, ns));
        }
#pragma unroll
        for (int j = 0; j < 2 * NP; ++j) {
          gw[j] = mul2(g[i][j], w[j]);
          ss2 = fma2(x[i][j], x[i][j], ss2);
          sd2 = fma2(gw[j], x[i][j], sd2);
        }
        float ss, sd, hs, hd;
        split(ss2, ss, hs);
        split(sd2, sd, hd);
        const float r = rsqrtf(row_sum<L>(ss + hs) * (1.0f / D) + a.eps);
        const float c = row_sum<L>(sd + hd) * (-1.0f / D) * r * r;
        const bool in = row < H;
        // a lane behind the last head has read that head and adds it times zero
        const float rd = in ? r : 0.f;
        const uint64_t r2 = pair(r, r), c2 = pair(c, c), rd2 = pair(rd, rd);
#pragma unroll
        for (int j = 0; j < 2 * NP; ++j) {
          dw[j] = fma2(g[i][j], mul2(x[i][j], rd2), dw[j]);
          gw[j] = mul2(r2, fma2(x[i][j], c2, gw[j]));
        }
        float y[VE];
        restore(gw, y);
        if (in) store_row<T, D>(dst + ((long long)tok * H + row) * D, l, y);
      }
    }
    l = nx;
    tok = tok2;
    unit = unit2;
  }
  float sums[VE];
  restore(dw, sums);
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    float v = sums[e];
#pragma unroll
    for (int o = L; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (rw == 0) s_dw[warp][e < PE ? l.a + e : l.b + e - PE] = v;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += 32 * kBwdWarps) {
    float v = 0.f;
#pragma unroll
    for (int wp = 0; wp < kBwdWarps; ++wp) v += s_dw[wp][i];
    partial[(long long)blockIdx.x * D + i] = v;
  }
}

// dw[e] = sum over the blocks' partial sums (queries: the first q_blocks), in block order within
// a lane and a fixed tree across lanes; in 64 bits, which cost nothing here.  One warp per
// element.
__global__ void __launch_bounds__(256) norm_rope_dw_kernel(const float* partial, int q_blocks,
                                                           int blocks, int D, float* dqw,
                                                           float* dkw) {
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  // a programmatic launch behind the sums, which give no early trigger: it may begin once their
  // blocks have left, so wait for what they wrote
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (i >= 2 * D) return;
  const bool isk = i >= D;
  const int e = isk ? i - D : i, last = isk ? blocks : q_blocks;
  double v = 0.0;
#pragma unroll 8
  for (int b = (isk ? q_blocks : 0) + lane; b < last; b += 32)
    v += (double)partial[(long long)b * D + e];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  float* out = isk ? dkw : dqw;
  if (lane == 0 && out) out[e] = (float)v;
}

// The walking grid: one block an SM.
constexpr int kBwdBlocks = 152;
constexpr int kRingBytes = kBwdWarps * kRing * kBwdUnroll * 4 * 32 * (int)sizeof(uint2);

template <typename T, int D, bool Q8>
cudaError_t launch_fwd_t(const NormRopeArgs& a, cudaStream_t st) {
  constexpr int step = Lane<T, D>::RPW * kUnroll;
  // A warp takes all heads of a kind, or, with few tokens, as many as it has in flight (32 + 8
  // heads of 128: 9.1 us for 10.8 with 2048 tokens, 7.1 for 6.9 with 1024).
  const bool whole = a.T >= 152 * 8;
  const int per = whole ? (a.Hq > a.Hkv ? a.Hq : a.Hkv) : step;
  const int qu = (a.Hq + per - 1) / per, ku = (a.Hkv + per - 1) / per;
  const dim3 grid((a.T + kWarps - 1) / kWarps, qu + ku + (a.slots ? ku : 0));
  if (a.interleaved)
    norm_rope_kernel<T, D, true, Q8><<<grid, 32 * kWarps, 0, st>>>(a, per, qu, ku);
  else
    norm_rope_kernel<T, D, false, Q8><<<grid, 32 * kWarps, 0, st>>>(a, per, qu, ku);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_bwd_t(const NormRopeArgs& a, float* dqw, float* dkw, float* partial,
                         cudaStream_t st) {
  // Blocks in proportion to the parts, and no more than there are units for.  (In proportion to
  // the heads, 16 + 2 heads of 64, whose two keys fill a quarter of a part, took 85 us for 30.)
  constexpr int rows = kBwdUnroll * Lane<T, D>::RPW;
  const int qp = (a.Hq + rows - 1) / rows, kp = (a.Hkv + rows - 1) / rows;
  const long long units = (long long)a.T * (((qp < kp ? kp : qp) + kParts - 1) / kParts);
  const int need = (int)min((units + kBwdWarps - 1) / kBwdWarps, (long long)kBwdBlocks);
  int qb = (int)((long long)kBwdBlocks * qp / (qp + kp));
  qb = qb < 1 ? 1 : qb > kBwdBlocks - 1 ? kBwdBlocks - 1 : qb;
  int kb = kBwdBlocks - qb;
  if (qb > need) qb = need;
  if (kb > need) kb = need;
  const int blocks = qb + kb;
  if (blocks > 0) {
    auto kernel =
        a.interleaved ? norm_rope_bwd_kernel<T, D, true> : norm_rope_bwd_kernel<T, D, false>;
    cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (e != cudaSuccess) return e;
    kernel<<<blocks, 32 * kBwdWarps, kRingBytes, st>>>(a, qb, partial);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !(dqw || dkw)) return e;
  // Programmatic: 86.9 us for 89.4 with 16384 tokens, called from the host (in a graph the same).
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((2 * D + 7) / 8);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_rope_dw_kernel, (const float*)partial, qb, blocks, D, dqw,
                            dkw);
}

}  // namespace

size_t norm_rope_bwd_workspace(int D) { return (size_t)kBwdBlocks * D * sizeof(float); }

namespace {
template <int D>
cudaError_t launch_fwd_d(const NormRopeArgs& a, bool bf16, cudaStream_t st) {
  if (a.k_scale)
    return bf16 ? launch_fwd_t<__nv_bfloat16, D, true>(a, st) : launch_fwd_t<float, D, true>(a, st);
  return bf16 ? launch_fwd_t<__nv_bfloat16, D, false>(a, st) : launch_fwd_t<float, D, false>(a, st);
}
}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, bool bf16, cudaStream_t st) {
  return a.D == 32   ? launch_fwd_d<32>(a, bf16, st)
         : a.D == 64 ? launch_fwd_d<64>(a, bf16, st)
                     : launch_fwd_d<128>(a, bf16, st);
}

cudaError_t launch_norm_rope_bwd(const NormRopeArgs& a, float* dqw, float* dkw, void* workspace,
                                 bool bf16, cudaStream_t st) {
  float* p = static_cast<float*>(workspace);
  switch (a.D) {
    case 32:
      return bf16 ? launch_bwd_t<__nv_bfloat16, 32>(a, dqw, dkw, p, st)
                  : launch_bwd_t<float, 32>(a, dqw, dkw, p, st);
    case 64:
      return bf16 ? launch_bwd_t<__nv_bfloat16, 64>(a, dqw, dkw, p, st)
                  : launch_bwd_t<float, 64>(a, dqw, dkw, p, st);
    default:
      return bf16 ? launch_bwd_t<__nv_bfloat16, 128>(a, dqw, dkw, p, st)
                  : launch_bwd_t<float, 128>(a, dqw, dkw, p, st);
  }
}

}  // namespace kda
