// Serving form of the kernel_delta_attention call (kda_attention_step): a few new tokens for
// each of N requests against a pool of fp32 states, with grouped value heads.
//
// Per (request, value head), with d = e^{decay} (one factor for all channels) and the state
// S [dk, dv], one token does
//   p_k = S^T k^,  p_q = S^T q^                       (reductions over dk)
//   u   = beta (v - d p_k)        (literal order: beta (v - p_k))
//   S   = d S + k^ u^T,   o = d p_q + u (k^ . q^)
// The decay is one number per head, so it multiplies the two reductions' results instead of
// every element before them, and the output needs no second pass over the new state.
//
// Bound by HBM: 8 dk dv bytes of state per (request, value head) against ~7 flops per state
// element and token.  Value columns never interact, so a warp owns 32 of them for all dk rows
// and works alone: lane (rg, cg) holds columns 4cg..4cg+3 of the rows rg, rg + 4, ... (a row's
// 32 columns are one 128-byte line), the reductions over dk are the lane's own sum and two
// shuffles, and tokens follow each other with no block barrier.  The whole slice (16 KB at
// dk = 128) is put in flight before anything else, and eight tokens' q, k, v right behind it
// into shared memory; while the state arrives the tokens are made ready there (norms, q^, k^),
// so that the loop over tokens waits for no memory.
//   64 requests x 1 token, 32 heads of 128 x 128: 43.6 us, 6.2 TB/s of the 6.8 of a copy (53 with
//   the state behind the tokens, 45.4 with each token loaded when the loop came to it).
//   37 requests x up to 6 tokens, 16 heads of 64 x 128, fp32: 13.2 us, a third of it the chain of
//   the tokens.  One request, 32 heads: 2.9 us.
// Packed fp32 arithmetic does not pay: over pairs of rows 26 us for 29 at eight tokens of 64
// requests, but 44.7 for 43.6 at one; over pairs of columns it spills.
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kCols = 32;               // value columns of a warp
constexpr int kColGroups = kCols / 4;   // lanes across a row slice
constexpr int kRowGroups = 32 / kColGroups;
constexpr int kTokens = 8;              // tokens made ready together
constexpr int kWarps = 2;               // warps of a block, at most

template <typename T> struct Vec4;
template <> struct Vec4<float> {
  static __device__ __forceinline__ float4 load(const float* p) {
    return *reinterpret_cast<const float4*>(p);
  }
  static __device__ __forceinline__ void store(float* p, float4 x) {
    *reinterpret_cast<float4*>(p) = x;
  }
};
template <> struct Vec4<__nv_bfloat16> {
  static __device__ __forceinline__ float4 load(const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, float4 x) {
    __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    uint2 w;
    w.x = *reinterpret_cast<const uint32_t*>(&a);
    w.y = *reinterpret_cast<const uint32_t*>(&b);
    *reinterpret_cast<uint2*>(p) = w;
  }
};

__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}

__device__ __forceinline__ float dot4(float4 x, float4 y) {
  return x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
}

// Blocks that share an SM: as many as the state in registers allows.
template <int DK> constexpr int kBlocks = DK == 128 ? 4 : DK == 64 ? 8 : 12;

template <typename T, int DK, int DV>
__global__ void __launch_bounds__(32 * kWarps, kBlocks<DK>) step_kernel(StepArgs a) {
  constexpr int RPT = DK / kRowGroups;  // rows of a lane
  __shared__ __align__(16) float2 s_kq[kWarps][kTokens][DK];  // (k^, q^) of a warp's tokens
  __shared__ __align__(16) T s_v[kWarps][kTokens][kCols];
  __shared__ __align__(16) float4 s_sc[kWarps][kTokens];  // beta, d, k^ . q^
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cg = lane % kColGroups, rg = lane / kColGroups;
  constexpr int slices = DV / kCols;
  const long long unit = (long long)blockIdx.x * (blockDim.x >> 5) + warp;
  if (unit >= (long long)a.N * a.Hv * slices) return;
  const int sl = (int)(unit % slices);
  const int hv = (int)(unit / slices % a.Hv);
  const int n = (int)(unit / slices / a.Hv);
  const int hk = hv / (a.Hv / a.Hk);
  const int col = sl * kCols + 4 * cg;

  const int slot = a.slots[n];
  if (slot < 0 || slot >= a.num_slots) return;  // a request that is not there
  const int out_slot = a.out_slots ? a.out_slots[n] : slot;
  const bool store = out_slot >= 0 && out_slot < a.num_slots;

  const long long slice_off = ((long long)hv * DK + rg) * DV + col;
  const float* Sp = a.state + (long long)slot * a.Hv * (DK * DV) + slice_off;
  float4 s[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i)
    s[i] = __ldcs(reinterpret_cast<const float4*>(Sp + (i * kRowGroups) * DV));

  long long bos;
  int len;
  if (a.cu_seqlens) {
    int lo = a.cu_seqlens[n], hi = a.cu_seqlens[n + 1];
    lo = min(max(lo, 0), a.T);
    hi = min(max(hi, lo), a.T);
    bos = lo;
    len = hi - lo;
  } else {
    bos = (long long)n * a.T;
    len = a.T;
  }

  for (int t0 = 0; t0 < len; t0 += kTokens) {
    const int nt = min(len - t0, kTokens);
    // raw rows: q, then k, where the token's (k^, q^) will be
    constexpr int VE = 16 / sizeof(T), PQ = DK / VE, PV = kCols / VE;  // 16-byte pieces
    for (int i = lane; i < nt * PQ; i += 32) {
      const int j = i / PQ, c = i % PQ;
      const long long row = bos + t0 + j;
      uint8_t* dst = reinterpret_cast<uint8_t*>(s_kq[warp][j]) + c * 16;
      copy16(dst, static_cast<const T*>(a.q) + row * a.q_stride + hk * DK + c * VE);
      copy16(dst + DK * sizeof(T), static_cast<const T*>(a.k) + row * a.k_stride + hk * DK + c * VE);
    }
    for (int i = lane; i < nt * PV; i += 32) {
      const int j = i / PV, c = i % PV;
      copy16(&s_v[warp][j][c * VE], static_cast<const T*>(a.v) + (bos + t0 + j) * a.v_stride +
                                        hv * DV + sl * kCols + c * VE);
    }
    float beta1 = 0.f, decay1 = 0.f;  // lane j: token j's
    if (lane < nt) {
      beta1 = a.beta[(bos + t0 + lane) * a.Hv + hv];
      if (a.decay) decay1 = a.decay[(bos + t0 + lane) * a.Hv + hv];
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    const float d1 = expf(decay1);
#pragma unroll 2
    for (int j = 0; j < nt; ++j) {
      float4 q = make_float4(0.f, 0.f, 0.f, 0.f), k = q;
      if (lane < DK / 4) {
        const T* raw = reinterpret_cast<const T*>(s_kq[warp][j]);
        q = Vec4<T>::load(raw + 4 * lane);
        k = Vec4<T>::load(raw + DK + 4 * lane);
      }
      const float kk = warp_sum(dot4(k, k)), qq = warp_sum(dot4(q, q)), kq = warp_sum(dot4(k, q));
      const float rk = a.no_l2norm ? 1.0f : rsqrtf(kk + kL2Eps);
      const float rq = a.no_l2norm ? a.scale : a.scale * rsqrtf(qq + kL2Eps);
      __syncwarp();  // every lane has its raw values
      if (lane < DK / 4) {
        float4* dst = reinterpret_cast<float4*>(&s_kq[warp][j][4 * lane]);
        dst[0] = make_float4(k.x * rk, q.x * rq, k.y * rk, q.y * rq);
        dst[1] = make_float4(k.z * rk, q.z * rq, k.w * rk, q.w * rq);
      }
      if (lane == j) s_sc[warp][j] = make_float4(beta1, d1, kq * rk * rq, 0.f);
    }
    __syncwarp();
    for (int j = 0; j < nt; ++j) {
      const float2* kqs = s_kq[warp][j];
      float4 pk = make_float4(0.f, 0.f, 0.f, 0.f), pq = pk;
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const float2 c = kqs[i * kRowGroups + rg];
        pk.x += s[i].x * c.x; pk.y += s[i].y * c.x; pk.z += s[i].z * c.x; pk.w += s[i].w * c.x;
        pq.x += s[i].x * c.y; pq.y += s[i].y * c.y; pq.z += s[i].z * c.y; pq.w += s[i].w * c.y;
      }
#pragma unroll
      for (int o = kColGroups; o < 32; o <<= 1) {
        pk.x += __shfl_xor_sync(0xffffffffu, pk.x, o);
        pk.y += __shfl_xor_sync(0xffffffffu, pk.y, o);
        pk.z += __shfl_xor_sync(0xffffffffu, pk.z, o);
        pk.w += __shfl_xor_sync(0xffffffffu, pk.w, o);
        pq.x += __shfl_xor_sync(0xffffffffu, pq.x, o);
        pq.y += __shfl_xor_sync(0xffffffffu, pq.y, o);
        pq.z += __shfl_xor_sync(0xffffffffu, pq.z, o);
        pq.w += __shfl_xor_sync(0xffffffffu, pq.w, o);
      }
      const float4 sc = s_sc[warp][j];
      const float4 v = Vec4<T>::load(&s_v[warp][j][4 * cg]);
      const float beta = sc.x, d = sc.y, kq = sc.z;
      const float dp = a.literal ? 1.0f : d;
      float4 u;
      u.x = beta * (v.x - dp * pk.x);
      u.y = beta * (v.y - dp * pk.y);
      u.z = beta * (v.z - dp * pk.z);
      u.w = beta * (v.w - dp * pk.w);
      if (rg == 0)
        Vec4<T>::store(static_cast<T*>(a.out) + ((bos + t0 + j) * a.Hv + hv) * DV + col,
                       make_float4(d * pq.x + u.x * kq, d * pq.y + u.y * kq, d * pq.z + u.z * kq,
                                   d * pq.w + u.w * kq));
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const float kr = kqs[i * kRowGroups + rg].x;
        s[i].x = s[i].x * d + kr * u.x;
        s[i].y = s[i].y * d + kr * u.y;
        s[i].z = s[i].z * d + kr * u.z;
        s[i].w = s[i].w * d + kr * u.w;
      }
    }
    __syncwarp();  // the tokens' places are free again
  }
  if (!store || (len == 0 && out_slot == slot)) return;
  float* So = a.state + (long long)out_slot * a.Hv * (DK * DV) + slice_off;
#pragma unroll
  for (int i = 0; i < RPT; ++i)
    __stcs(reinterpret_cast<float4*>(So + (i * kRowGroups) * DV), s[i]);
}

template <typename T, int DK, int DV>
cudaError_t launch_t(const StepArgs& a, cudaStream_t st) {
  const long long units = (long long)a.N * a.Hv * (DV / kCols);
  // Warps are independent: one per block spreads a small batch over more SMs.  (Two against
  // four per block for a large one: 13.5 against 14.1 us for 2368 warps with up to 6 tokens.)
  const int warps = units <= 152 * 4 ? 1 : kWarps;
  step_kernel<T, DK, DV><<<(unsigned)((units + warps - 1) / warps), 32 * warps, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T, int DK>
cudaError_t launch_dv(const StepArgs& a, cudaStream_t st) {
  switch (a.dv) {
    case 32: return launch_t<T, DK, 32>(a, st);
    case 64: return launch_t<T, DK, 64>(a, st);
    default: return launch_t<T, DK, 128>(a, st);
  }
}

template <typename T>
cudaError_t launch_dk(const StepArgs& a, cudaStream_t st) {
  switch (a.dk) {
    case 32: return launch_dv<T, 32>(a, st);
    case 64: return launch_dv<T, 64>(a, st);
    default: return launch_dv<T, 128>(a, st);
  }
}

}  // namespace

cudaError_t launch_step(const StepArgs& a, bool bf16, cudaStream_t st) {
  return bf16 ? launch_dk<__nv_bfloat16>(a, st) : launch_dk<float>(a, st);
}

}  // namespace kda
