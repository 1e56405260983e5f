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
// dk = 128) is put in flight before anything else; a token's q, k, v are loaded while the
// token before it is computed.
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kCols = 32;               // value columns of a warp
constexpr int kColGroups = kCols / 4;   // lanes across a row slice
constexpr int kRowGroups = 32 / kColGroups;

template <typename T> struct Vec4;
template <> struct Vec4<float> {
  static __device__ __forceinline__ float4 load(const float* p) {
    return __ldg(reinterpret_cast<const float4*>(p));
  }
  static __device__ __forceinline__ void store(float* p, float4 x) {
    *reinterpret_cast<float4*>(p) = x;
  }
};
template <> struct Vec4<__nv_bfloat16> {
  static __device__ __forceinline__ float4 load(const __nv_bfloat16* p) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
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

// One token's inputs as a lane holds them: q, k in DK / 4 lanes, v by column group.
struct Token {
  float4 q, k, v;
  float beta, decay;
};

template <typename T, int DK>
__device__ __forceinline__ Token load_token(const StepArgs& a, long long row, int hk, int hv,
                                            int col, int lane) {
  Token t;
  t.q = t.k = make_float4(0.f, 0.f, 0.f, 0.f);
  if (lane < DK / 4) {
    t.q = Vec4<T>::load(static_cast<const T*>(a.q) + row * a.q_stride + hk * DK + 4 * lane);
    t.k = Vec4<T>::load(static_cast<const T*>(a.k) + row * a.k_stride + hk * DK + 4 * lane);
  }
  t.v = Vec4<T>::load(static_cast<const T*>(a.v) + row * a.v_stride + hv * a.dv + col);
  t.beta = a.beta[row * a.Hv + hv];
  t.decay = a.decay ? a.decay[row * a.Hv + hv] : 0.f;
  return t;
}

__device__ __forceinline__ float dot4(float4 x, float4 y) {
  return x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
}

template <typename T, int DK>
__global__ void __launch_bounds__(128) step_kernel(StepArgs a) {
  constexpr int RPT = DK / kRowGroups;  // rows of a lane
  __shared__ __align__(16) float2 s_kq[4][DK];  // (k^, q^) of the warp's current token
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cg = lane % kColGroups, rg = lane / kColGroups;
  const int slices = a.dv / kCols;
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

  const long long slice_off = (long long)hv * DK * a.dv + col;
  const float* Sp = a.state + (long long)slot * a.Hv * DK * a.dv + slice_off;
  float4 s[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i)
    s[i] = __ldcs(reinterpret_cast<const float4*>(Sp + (long long)(i * kRowGroups + rg) * a.dv));

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

  Token nxt;
  if (len > 0) nxt = load_token<T, DK>(a, bos, hk, hv, col, lane);
  for (int t = 0; t < len; ++t) {
    const Token cur = nxt;
    if (t + 1 < len) nxt = load_token<T, DK>(a, bos + t + 1, hk, hv, col, lane);
    float kk = warp_sum(dot4(cur.k, cur.k)), qq = warp_sum(dot4(cur.q, cur.q));
    float kq = warp_sum(dot4(cur.k, cur.q));
    const float rk = a.no_l2norm ? 1.0f : 1.0f / sqrtf(kk + kL2Eps);
    const float rq = a.no_l2norm ? a.scale : a.scale / sqrtf(qq + kL2Eps);
    kq *= rk * rq;
    __syncwarp();  // the previous token's k^, q^ have been read
    if (lane < DK / 4) {
      s_kq[warp][4 * lane + 0] = make_float2(cur.k.x * rk, cur.q.x * rq);
      s_kq[warp][4 * lane + 1] = make_float2(cur.k.y * rk, cur.q.y * rq);
      s_kq[warp][4 * lane + 2] = make_float2(cur.k.z * rk, cur.q.z * rq);
      s_kq[warp][4 * lane + 3] = make_float2(cur.k.w * rk, cur.q.w * rq);
    }
    __syncwarp();
    float4 pk = make_float4(0.f, 0.f, 0.f, 0.f), pq = pk;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const float2 c = s_kq[warp][i * kRowGroups + rg];
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
    const float d = expf(cur.decay);
    const float dp = a.literal ? 1.0f : d;
    float4 u, o4;
    u.x = cur.beta * (cur.v.x - dp * pk.x);
    u.y = cur.beta * (cur.v.y - dp * pk.y);
    u.z = cur.beta * (cur.v.z - dp * pk.z);
    u.w = cur.beta * (cur.v.w - dp * pk.w);
    o4.x = d * pq.x + u.x * kq;
    o4.y = d * pq.y + u.y * kq;
    o4.z = d * pq.z + u.z * kq;
    o4.w = d * pq.w + u.w * kq;
    if (rg == 0)
      Vec4<T>::store(static_cast<T*>(a.out) + ((bos + t) * a.Hv + hv) * a.dv + col, o4);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const float kr = s_kq[warp][i * kRowGroups + rg].x;
      s[i].x = s[i].x * d + kr * u.x;
      s[i].y = s[i].y * d + kr * u.y;
      s[i].z = s[i].z * d + kr * u.z;
      s[i].w = s[i].w * d + kr * u.w;
    }
  }
  if (!store || (len == 0 && out_slot == slot)) return;
  float* So = a.state + (long long)out_slot * a.Hv * DK * a.dv + slice_off;
#pragma unroll
  for (int i = 0; i < RPT; ++i)
    __stcs(reinterpret_cast<float4*>(So + (long long)(i * kRowGroups + rg) * a.dv), s[i]);
}

template <typename T, int DK>
cudaError_t launch_t(const StepArgs& a, cudaStream_t st) {
  const long long units = (long long)a.N * a.Hv * (a.dv / kCols);
  // Warps are independent: one per block spreads a small batch over more SMs, four per block
  // cost fewer block launches for a large one.
  const int warps = units <= 152 * 4 ? 1 : 4;
  step_kernel<T, DK><<<(unsigned)((units + warps - 1) / warps), 32 * warps, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_dk(const StepArgs& a, cudaStream_t st) {
  switch (a.dk) {
    case 32: return launch_t<T, 32>(a, st);
    case 64: return launch_t<T, 64>(a, st);
    default: return launch_t<T, 128>(a, st);
  }
}

}  // namespace

cudaError_t launch_step(const StepArgs& a, bool bf16, cudaStream_t st) {
  return bf16 ? launch_dk<__nv_bfloat16>(a, st) : launch_dk<float>(a, st);
}

}  // namespace kda
