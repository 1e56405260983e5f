// Reading tokens back from a cache in 8 bits (kda_paged_cache_read_q8): keys and values of given
// slots as dense rows of fp32 or bf16, which both hold them exactly.
//
// And queries as two e4m3 terms, for attention whose keys stay in 8 bits (kda_paged_tc.cuh).
//
// Reading is bound by HBM: D + 1 bytes in and 2 D or 4 D out per row.  A thread has 16 numbers of a
// token's key and value of one head, so that its loads are 16 bytes and its four loads of the two
// rows (numbers and scales) are in flight together behind the slot's.  Stores are whole sectors of
// 32 bytes: 16384 tokens of 8 heads of 128 take 14.2 us, 7.1 TB/s (part of it from L2); 19.3 with
// two stores of 16 bytes.
#include "kda_q8.cuh"

namespace kda {
namespace {

constexpr int kThreads = 64;  // of a block

// 32 bytes: a whole sector, where the address allows it.
__device__ __forceinline__ void store32(void* p, const uint32_t (&x)[8], bool whole) {
  if (whole) {
    asm volatile("st.global.cs.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(x[0]),
                 "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
  } else {
    __stcs(static_cast<uint4*>(p), make_uint4(x[0], x[1], x[2], x[3]));
    __stcs(static_cast<uint4*>(p) + 1, make_uint4(x[4], x[5], x[6], x[7]));
  }
}
__device__ __forceinline__ void put(float* dst, const uint4& w, float s, bool whole) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t y[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = q8::unpack2(x[2 * i + j / 2] >> (j % 2 * 16));
      y[2 * j] = __float_as_uint(a.x * s);
      y[2 * j + 1] = __float_as_uint(a.y * s);
    }
    store32(dst + 8 * i, y, whole);
  }
}
__device__ __forceinline__ void put(__nv_bfloat16* dst, const uint4& w, float s, bool whole) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
  uint32_t y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 a = q8::unpack2(x[j / 2] >> (j % 2 * 16));
    const __nv_bfloat162 b = __floats2bfloat162_rn(a.x * s, a.y * s);
    y[j] = *reinterpret_cast<const uint32_t*>(&b);
  }
  store32(dst, y, whole);
}

// A block has pieces of one token: a thread 16 numbers of its key and value of one head.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(CacheReadArgs a) {
  constexpr int PIECES = D / 16;
  const int i = blockIdx.y * kThreads + threadIdx.x;
  if (i >= a.Hkv * PIECES) return;
  const int h = i / PIECES, c = i % PIECES * 16;
  const long long tok = blockIdx.x;
  const long long slot = __ldg(a.slots + tok);
  uint4 k = make_uint4(0, 0, 0, 0), v = k;
  uint32_t ks = q8::kBias, vs = q8::kBias;
  if (slot >= 0 && slot < (long long)a.num_pages * a.page_size) {
    const long long page = slot >> a.page_shift;
    const long long at = (page * a.Hkv + h) * a.page_size + (slot - (page << a.page_shift));
    k = __ldg(reinterpret_cast<const uint4*>(a.k_cache + at * D + c));
    v = __ldg(reinterpret_cast<const uint4*>(a.v_cache + at * D + c));
    ks = __ldg(a.k_scale + at);
    vs = __ldg(a.v_scale + at);
  }
  const long long row = tok * a.Hkv + h;
  T *kd = static_cast<T*>(a.k_out) + row * D + c, *vd = static_cast<T*>(a.v_out) + row * D + c;
  put(kd, k, q8::scale(ks), (reinterpret_cast<uintptr_t>(kd) & 31) == 0);
  put(vd, v, q8::scale(vs), (reinterpret_cast<uintptr_t>(vd) & 31) == 0);
}

template <int D>
cudaError_t launch_t(const CacheReadArgs& a, bool bf16, cudaStream_t st) {
  const dim3 grid((unsigned)a.T, (unsigned)((a.Hkv * (D / 16) + kThreads - 1) / kThreads));
  if (bf16)
    cache_read_kernel<__nv_bfloat16, D><<<grid, kThreads, 0, st>>>(a);
  else
    cache_read_kernel<float, D><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

// A query row of bf16 (8 bits of mantissa) under a power of two as the sum of two rows of e4m3 (4
// each):  q 2^-e = hi + lo,  hi = e4m3(q 2^-e), lo = e4m3(q 2^-e - hi).  Exact where q is more than
// 2^-9 of the row's largest, and off by at most 2^-17 of that elsewhere (e4m3 ends at 2^-9).
// Sixteen lanes a row; hi and lo lie where the row's 256 bytes would.
constexpr int kTermThreads = 256;
__global__ void __launch_bounds__(kTermThreads) query_terms_kernel(PagedArgs a, uint8_t* terms,
                                                               float* scales) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the products may be set up
  const long long row = (long long)blockIdx.x * (kTermThreads / 16) + threadIdx.x / 16;
  const int c = threadIdx.x & 15;
  const long long rows = (long long)a.total_T * a.Hq;
  const long long src = row < rows ? row : rows - 1;
  const long long tok = src / a.Hq;
  const uint4 x = __ldcs(reinterpret_cast<const uint4*>(
      static_cast<const __nv_bfloat16*>(a.q) + tok * a.q_stride + (src - tok * a.Hq) * 128 +
      c * 8));
  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, max(u[i] << 16 & 0x7fff0000u, u[i] & 0x7fff0000u));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const bool odd = top >= 0x7f800000u;  // an infinity or a NaN: the row's scores are NaN
  const int e = q8::exponent(top);
  const float f = odd ? 0.f : q8::power(-e);
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float y0 = odd ? 0.f : __uint_as_float(u[i] << 16) * f;
    const float y1 = odd ? 0.f : __uint_as_float(u[i] & 0xffff0000u) * f;
    hi[i] = q8::pack2(y0, y1);
    const float2 z = q8::unpack2(hi[i]);
    lo[i] = q8::pack2(y0 - z.x, y1 - z.y);
  }
  if (row >= rows) return;
  uint8_t* dst = terms + row * 256 + c * 8;
  *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
  *reinterpret_cast<uint2*>(dst + 128) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
  if (c == 0) scales[row] = odd ? __uint_as_float(0x7fc00000u) : q8::power(e);
}

}  // namespace

size_t paged_query_terms(int total_T, int Hq) {
  return (size_t)total_T * Hq * (256 + sizeof(float));
}

cudaError_t launch_query_terms(PagedArgs& a, void* terms, cudaStream_t st) {
  const long long rows = (long long)a.total_T * a.Hq;
  uint8_t* t = static_cast<uint8_t*>(terms);
  float* scales = reinterpret_cast<float*>(t + rows * 256);
  constexpr int per = kTermThreads / 16;
  query_terms_kernel<<<(unsigned)((rows + per - 1) / per), kTermThreads, 0, st>>>(a, t, scales);
  a.q = t;
  a.q_stride = (long long)a.Hq * 128;
  a.q_scale = scales;
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const CacheReadArgs& a, bool bf16, cudaStream_t st) {
  return a.D == 32   ? launch_t<32>(a, bf16, st)
         : a.D == 64 ? launch_t<64>(a, bf16, st)
                     : launch_t<128>(a, bf16, st);
}

}  // namespace kda
