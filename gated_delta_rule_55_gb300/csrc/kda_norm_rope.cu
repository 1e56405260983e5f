// RMS norm of every query and key head with the position rotation in the same pass
// (kda_qk_norm_rope_fwd / _append / _bwd).
//
// Per head row x [D] of a token at position p, with weight w [D]:
//   r = 1 / sqrt(mean(x^2) + eps),   n = x r w,   y = Rot(p) n
// where Rot turns the pairs (i, i + R/2) (or (2i, 2i + 1), interleaved) of the first R elements
// by the angle whose cosine and sine are row p of the caller's tables.  Backward, with
// g = Rot(p)^T dy:
//   dw = sum over rows of g x r,   dx = r (g w - x r^2 mean(g w x)).
//
// Bound by HBM: every element is read once and written once (backward: two reads, one write)
// with ~8 flops between.  A row lies across D / VE lanes as 16-byte vectors, so the mean is a
// few shuffles, and the rotation's partner is in the same lane (interleaved) or R / (2 VE)
// lanes away.  A warp takes kUnroll row groups of one token and one kind (queries, keys or
// copied values): the lane's cosines, sines and weights are then the same for all of them and
// are loaded once, and all its row loads are in flight together.
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kUnroll = 4;   // row groups of a warp's unit
constexpr int kWarps = 8;    // warps of a block

template <typename T> struct Row;  // 16-byte vectors of T as fp32
template <> struct Row<float> {
  static constexpr int VE = 4;
  static __device__ __forceinline__ void unpack(uint4 w, float (&x)[4]) {
    x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};
template <> struct Row<__nv_bfloat16> {
  static constexpr int VE = 8;
  static __device__ __forceinline__ void unpack(uint4 w, float (&x)[8]) {
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(r[i] << 16);
      x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      r[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
  }
};

// A lane's share of the rotation at one position: for each of its elements e, y_e = c_e n_e +
// s_e n_partner(e), with the sine's sign folded in.  Elements behind R have c = 1, s = 0.
template <int VE>
struct Turn {
  float c[VE], s[VE];
  int partner;  // lane holding the partners (half-split pairs)
};

template <int VE>
__device__ __forceinline__ Turn<VE> load_turn(const NormRopeArgs& a, long long tok, int li,
                                              int lane) {
  Turn<VE> t;
  t.partner = lane;
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    t.c[e] = 1.f;
    t.s[e] = 0.f;
  }
  const int e0 = li * VE;
  if (e0 < a.R) {
    const int p = min(max(a.positions[tok], 0), a.max_position - 1);
    const int half = a.R / 2;
    const float* cp = a.cos_table + (long long)p * half;
    const float* sp = a.sin_table + (long long)p * half;
    if (a.interleaved) {
#pragma unroll
      for (int i = 0; i < VE / 2; i += 2) {
        const float2 c = __ldg(reinterpret_cast<const float2*>(cp + e0 / 2 + i));
        const float2 s = __ldg(reinterpret_cast<const float2*>(sp + e0 / 2 + i));
        t.c[2 * i] = t.c[2 * i + 1] = c.x;
        t.c[2 * i + 2] = t.c[2 * i + 3] = c.y;
        t.s[2 * i] = -s.x; t.s[2 * i + 1] = s.x;
        t.s[2 * i + 2] = -s.y; t.s[2 * i + 3] = s.y;
      }
    } else {
      const bool low = e0 < half;
      const int i0 = low ? e0 : e0 - half;
      t.partner = low ? lane + half / VE : lane - half / VE;
#pragma unroll
      for (int i = 0; i < VE; i += 4) {
        const float4 c = __ldg(reinterpret_cast<const float4*>(cp + i0 + i));
        const float4 s = __ldg(reinterpret_cast<const float4*>(sp + i0 + i));
        t.c[i] = c.x; t.c[i + 1] = c.y; t.c[i + 2] = c.z; t.c[i + 3] = c.w;
        t.s[i] = low ? -s.x : s.x; t.s[i + 1] = low ? -s.y : s.y;
        t.s[i + 2] = low ? -s.z : s.z; t.s[i + 3] = low ? -s.w : s.w;
      }
    }
  }
  return t;
}

// Applies the rotation (TRANSPOSE: its transpose, the angle negated) to one row's lane share.
template <int VE, bool TRANSPOSE>
__device__ __forceinline__ void turn(float (&x)[VE], const Turn<VE>& t, bool interleaved) {
  float y[VE];
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < VE; ++e) y[e] = x[e ^ 1];
  } else {
#pragma unroll
    for (int e = 0; e < VE; ++e) y[e] = __shfl_sync(0xffffffffu, x[e], t.partner);
  }
#pragma unroll
  for (int e = 0; e < VE; ++e) x[e] = x[e] * t.c[e] + (TRANSPOSE ? -t.s[e] : t.s[e]) * y[e];
}

template <int VE>
__device__ __forceinline__ void load_weight(const float* w, int li, float (&out)[VE]) {
#pragma unroll
  for (int e = 0; e < VE; e += 4) {
    const float4 v = w ? __ldg(reinterpret_cast<const float4*>(w + li * VE + e))
                       : make_float4(1.f, 1.f, 1.f, 1.f);
    out[e] = v.x; out[e + 1] = v.y; out[e + 2] = v.z; out[e + 3] = v.w;
  }
}

template <int L>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Forward: queries to query_out; keys to key_out, or (append) keys and values to their place
// in the pages.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarps) norm_rope_kernel(NormRopeArgs a) {
  constexpr int VE = Row<T>::VE, L = D / VE, RPW = 32 / L;
  const int lane = threadIdx.x & 31, li = lane % L, rw = lane / L;
  const int per = RPW * kUnroll;  // heads of a unit
  const int qu = (a.Hq + per - 1) / per, ku = (a.Hkv + per - 1) / per;
  const int tu = qu + ku + (a.slots ? ku : 0);  // units of a token
  const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (unit >= (long long)a.T * tu) return;
  const long long tok = unit / tu;
  int u = (int)(unit - tok * tu);
  const int kind = u < qu ? 0 : u < qu + ku ? 1 : 2;  // queries, keys, values
  if (kind == 1) u -= qu;
  if (kind == 2) u -= qu + ku;
  const int H = kind == 0 ? a.Hq : a.Hkv;
  const T* src = static_cast<const T*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) +
                 tok * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride);
  // Where head h of this token goes: dst + h * dst_head.
  T* dst;
  long long dst_head = D;
  if (kind == 0) {
    dst = static_cast<T*>(a.q_out) + tok * a.Hq * D;
  } else if (!a.slots) {
    dst = static_cast<T*>(a.k_out) + tok * a.Hkv * D;
  } else {
    const long long slot = a.slots[tok];
    if (slot < 0 || slot >= (long long)a.num_pages * a.page_size) return;  // not kept
    const long long page = slot / a.page_size;
    dst_head = (long long)a.page_size * D;
    dst = static_cast<T*>(kind == 1 ? a.k_cache : a.v_cache) + page * a.Hkv * dst_head +
          (slot - page * a.page_size) * D;
  }
  uint4 raw[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int h = u * per + i * RPW + rw;
    raw[i] = h < H ? __ldcs(reinterpret_cast<const uint4*>(src + (long long)h * D + li * VE))
                   : make_uint4(0, 0, 0, 0);
  }
  if (kind == 2) {
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int h = u * per + i * RPW + rw;
      if (h < H) *reinterpret_cast<uint4*>(dst + h * dst_head + li * VE) = raw[i];
    }
    return;
  }
  float w[VE];
  load_weight<VE>(kind == 0 ? a.q_weight : a.k_weight, li, w);
  const Turn<VE> t = load_turn<VE>(a, tok, li, lane);
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int h = u * per + i * RPW + rw;
    float x[VE];
    Row<T>::unpack(raw[i], x);
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < VE; ++e) ss += x[e] * x[e];
    const float r = 1.0f / sqrtf(row_sum<L>(ss) * (1.0f / D) + a.eps);
#pragma unroll
    for (int e = 0; e < VE; ++e) x[e] *= r * w[e];
    turn<VE, false>(x, t, a.interleaved);
    if (h < H) *reinterpret_cast<uint4*>(dst + h * dst_head + li * VE) = Row<T>::pack(x);
  }
}

// Backward: units of (token, row groups) as above, walked by a fixed grid so that a warp sums
// its share of dw in registers; the block's sums go to partial[block][2][D].
template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarps) norm_rope_bwd_kernel(NormRopeArgs a,
                                                                    float* partial) {
  constexpr int VE = Row<T>::VE, L = D / VE, RPW = 32 / L, U = 2;
  __shared__ float s_dw[kWarps][2][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, li = lane % L, rw = lane / L;
  const int per = RPW * U;
  const int qu = (a.Hq + per - 1) / per, ku = (a.Hkv + per - 1) / per, tu = qu + ku;
  const long long units = (long long)a.T * tu;
  float dw[2][VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) dw[0][e] = dw[1][e] = 0.f;
  for (long long unit = (long long)blockIdx.x * kWarps + warp; unit < units;
       unit += (long long)gridDim.x * kWarps) {
    const long long tok = unit / tu;
    int u = (int)(unit - tok * tu);
    const bool isk = u >= qu;
    if (isk) u -= qu;
    const int H = isk ? a.Hkv : a.Hq;
    const T* src = static_cast<const T*>(isk ? a.k : a.q) + tok * (isk ? a.k_stride : a.q_stride);
    const T* gsrc = static_cast<const T*>(isk ? a.dk_out : a.dq_out) + tok * H * D;
    T* dst = static_cast<T*>(isk ? a.dk : a.dq) + tok * H * D;
    uint4 raw[U], graw[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = u * per + i * RPW + rw;
      const bool in = h < H;
      raw[i] = in ? __ldcs(reinterpret_cast<const uint4*>(src + (long long)h * D + li * VE))
                  : make_uint4(0, 0, 0, 0);
      graw[i] = in ? __ldcs(reinterpret_cast<const uint4*>(gsrc + (long long)h * D + li * VE))
                   : make_uint4(0, 0, 0, 0);
    }
    float w[VE];
    load_weight<VE>(isk ? a.k_weight : a.q_weight, li, w);
    const Turn<VE> t = load_turn<VE>(a, tok, li, lane);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = u * per + i * RPW + rw;
      float x[VE], g[VE];
      Row<T>::unpack(raw[i], x);
      Row<T>::unpack(graw[i], g);
      turn<VE, true>(g, t, a.interleaved);
      float ss = 0.f, sd = 0.f;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        ss += x[e] * x[e];
        sd += g[e] * w[e] * x[e];
      }
      const float r = 1.0f / sqrtf(row_sum<L>(ss) * (1.0f / D) + a.eps);
      const float c = row_sum<L>(sd) * (1.0f / D) * r * r;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float add = g[e] * x[e] * r;  // 0 for rows behind the last head
        if (isk) dw[1][e] += add; else dw[0][e] += add;
        x[e] = r * (g[e] * w[e] - x[e] * c);
      }
      if (h < H) __stcs(reinterpret_cast<uint4*>(dst + (long long)h * D + li * VE),
                        Row<T>::pack(x));
    }
  }
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      float v = dw[m][e];
#pragma unroll
      for (int o = L; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (rw == 0) s_dw[warp][m][li * VE + e] = v;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += 32 * kWarps) {
    float v = 0.f;
#pragma unroll
    for (int wp = 0; wp < kWarps; ++wp) v += s_dw[wp][i / D][i % D];
    partial[(long long)blockIdx.x * 2 * D + i] = v;
  }
}

// dw[m][e] = sum over the blocks' partial sums in block order within a lane and a fixed tree
// across lanes; in 64 bits, which cost nothing here.  One warp per element.
__global__ void __launch_bounds__(256) norm_rope_dw_kernel(const float* partial, int blocks,
                                                           int D, float* dqw, float* dkw) {
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (i >= 2 * D) return;
  double v = 0.0;
  for (int b = lane; b < blocks; b += 32) v += (double)partial[(long long)b * 2 * D + i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  float* out = i < D ? dqw : dkw;
  if (lane == 0 && out) out[i < D ? i : i - D] = (float)v;
}

constexpr int kBwdBlocks = 152 * 4;  // the walking grid: four blocks on each SM

template <typename T, int D>
cudaError_t launch_fwd_t(const NormRopeArgs& a, cudaStream_t st) {
  constexpr int per = 32 / (D / Row<T>::VE) * kUnroll;
  const int qu = (a.Hq + per - 1) / per, ku = (a.Hkv + per - 1) / per;
  const long long units = (long long)a.T * (qu + ku + (a.slots ? ku : 0));
  norm_rope_kernel<T, D><<<(unsigned)((units + kWarps - 1) / kWarps), 32 * kWarps, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_bwd_t(const NormRopeArgs& a, float* dqw, float* dkw, float* partial,
                         cudaStream_t st) {
  constexpr int per = 32 / (D / Row<T>::VE) * 2;
  const int qu = (a.Hq + per - 1) / per, ku = (a.Hkv + per - 1) / per;
  const long long need = ((long long)a.T * (qu + ku) + kWarps - 1) / kWarps;
  const int blocks = (int)(need < kBwdBlocks ? need : kBwdBlocks);
  if (blocks > 0) norm_rope_bwd_kernel<T, D><<<blocks, 32 * kWarps, 0, st>>>(a, partial);
  if (dqw || dkw)
    norm_rope_dw_kernel<<<(2 * D + 7) / 8, 256, 0, st>>>(partial, blocks, D, dqw, dkw);
  return cudaGetLastError();
}

}  // namespace

size_t norm_rope_bwd_workspace(int D) { return (size_t)kBwdBlocks * 2 * D * sizeof(float); }

cudaError_t launch_norm_rope(const NormRopeArgs& a, bool bf16, cudaStream_t st) {
  switch (a.D) {
    case 32: return bf16 ? launch_fwd_t<__nv_bfloat16, 32>(a, st) : launch_fwd_t<float, 32>(a, st);
    case 64: return bf16 ? launch_fwd_t<__nv_bfloat16, 64>(a, st) : launch_fwd_t<float, 64>(a, st);
    default:
      return bf16 ? launch_fwd_t<__nv_bfloat16, 128>(a, st) : launch_fwd_t<float, 128>(a, st);
  }
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
