// The C ABI of the serving operators (declared in include/kda.h): the delta-rule step over a
// state pool, head norms with rotation, attention over a paged cache.  Host-side argument
// validation and launches on the caller's stream; nothing here allocates memory.
#include <math.h>

#include "kda_internal.cuh"

namespace {

constexpr double kMaxElems = 1099511627776.0;  // 2^40: far inside the kernels' 64-bit offsets

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
bool head_dim_ok(int d) { return d == 32 || d == 64 || d == 128; }
bool page_size_ok(int s) { return s == 16 || s == 32 || s == 64 || s == 128; }
bool dtype_ok(int t) { return t == KDA_F32 || t == KDA_BF16; }

template <size_t K>
bool all_aligned16(const void* const (&ptrs)[K]) {
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return false;
  return true;
}

// A token stride in elements: a token's size at least, rows on 16-byte boundaries, and the
// whole axis inside the index limits.
int check_stride(long long stride, long long token, long long rows, int dtype) {
  if (stride < token || stride % (dtype == KDA_F32 ? 4 : 8) != 0) return KDA_ERR_STRIDE;
  return (double)stride * (double)rows >= kMaxElems ? KDA_ERR_TOO_LARGE : KDA_OK;
}

int launch_status(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH; }

// Checks of the three norm-and-rotate calls that they share; fills the common arguments.
int fill_norm_rope(kda::NormRopeArgs& a, const void* query, const void* key,
                   const float* query_weight, const float* key_weight, const float* cos_table,
                   const float* sin_table, const int32_t* positions, float eps, int T, int Hq,
                   int Hkv, int D, int R, int max_position, long long query_stride,
                   long long key_stride, int flags, int dtype) {
  if (T < 0 || Hq <= 0 || Hkv <= 0) return KDA_ERR_BAD_SHAPE;
  if (!head_dim_ok(D)) return KDA_ERR_HEAD_DIM;
  if (R < 0 || R > D || R % 16 != 0) return KDA_ERR_ROTARY;
  if (R > 0 && max_position <= 0) return KDA_ERR_BAD_SHAPE;
  if (!(eps > 0.f) || !isfinite(eps)) return KDA_ERR_SCALE;
  if (flags & ~KDA_ROPE_INTERLEAVED) return KDA_ERR_FLAGS;
  if (!dtype_ok(dtype)) return KDA_ERR_DTYPE;
  if (T > 0 && (!query || !key || (R > 0 && (!cos_table || !sin_table || !positions))))
    return KDA_ERR_NULL_POINTER;
  const void* const ptrs[] = {query,     key,       query_weight, key_weight,
                              cos_table, sin_table, positions};
  if (!all_aligned16(ptrs)) return KDA_ERR_MISALIGNED;
  int s = check_stride(query_stride, (long long)Hq * D, T, dtype);
  if (s == KDA_OK) s = check_stride(key_stride, (long long)Hkv * D, T, dtype);
  if (s != KDA_OK) return s;
  // tokens and a token's units of work (at most one per head) are grid dimensions
  if ((double)Hq + 2.0 * Hkv > 65535.0 || (double)T * ((double)Hq + 2.0 * Hkv) >= 2147483647.0)
    return KDA_ERR_TOO_LARGE;
  a = kda::NormRopeArgs{};
  a.q = query; a.k = key; a.q_weight = query_weight; a.k_weight = key_weight;
  a.cos_table = cos_table; a.sin_table = sin_table; a.positions = positions; a.eps = eps;
  a.q_stride = query_stride; a.k_stride = key_stride;
  a.T = T; a.Hq = Hq; a.Hkv = Hkv; a.D = D; a.R = R; a.max_position = max_position;
  a.interleaved = (flags & KDA_ROPE_INTERLEAVED) ? 1 : 0;
  return KDA_OK;
}

}  // namespace

extern "C" {

int kda_attention_step(const void* query, const void* key, const void* value, const float* beta,
                       const float* decay, float* state, const int32_t* slots,
                       const int32_t* out_slots, const int32_t* cu_seqlens, void* out,
                       float softmax_scale, int N, int T, int Hk, int Hv, int dk, int dv,
                       int num_slots, long long query_stride, long long key_stride,
                       long long value_stride, int flags, int dtype, kda_stream_t stream) {
  if (N < 0 || T < 0 || Hk <= 0 || Hv <= 0 || Hv % Hk != 0 || num_slots < 0)
    return KDA_ERR_BAD_SHAPE;
  if (flags & ~(KDA_ATTN_NO_QK_L2NORM | KDA_ATTN_ORDER_LITERAL)) return KDA_ERR_FLAGS;
  if (!head_dim_ok(dk) || !head_dim_ok(dv)) return KDA_ERR_HEAD_DIM;
  if (!isfinite(softmax_scale)) return KDA_ERR_SCALE;
  if (softmax_scale <= 0.f) softmax_scale = 1.0f / sqrtf((float)dk);
  if (!dtype_ok(dtype)) return KDA_ERR_DTYPE;
  if (N > 0 && (!state || !slots)) return KDA_ERR_NULL_POINTER;
  if (N > 0 && T > 0 && (!query || !key || !value || !beta || !out)) return KDA_ERR_NULL_POINTER;
  const void* const ptrs[] = {query, key,       value,      beta, decay,
                              state, slots,     out_slots,  cu_seqlens, out};
  if (!all_aligned16(ptrs)) return KDA_ERR_MISALIGNED;
  const double rows = cu_seqlens ? (double)T : (double)N * T;
  if (rows > 2147483647.0 || rows * Hv * dv >= kMaxElems ||
      (double)num_slots * Hv * dk * dv >= kMaxElems ||
      (double)N * Hv * (dv / 32) > 2147483647.0)
    return KDA_ERR_TOO_LARGE;
  int s = check_stride(query_stride, (long long)Hk * dk, (long long)rows, dtype);
  if (s == KDA_OK) s = check_stride(key_stride, (long long)Hk * dk, (long long)rows, dtype);
  if (s == KDA_OK) s = check_stride(value_stride, (long long)Hv * dv, (long long)rows, dtype);
  if (s != KDA_OK) return s;
  s = kda::check_current_device();
  if (s != KDA_OK) return s;
  if (N == 0) return KDA_OK;
  kda::StepArgs a{};
  a.q = query; a.k = key; a.v = value; a.q_stride = query_stride; a.k_stride = key_stride;
  a.v_stride = value_stride; a.beta = beta; a.decay = decay; a.state = state; a.slots = slots;
  a.out_slots = out_slots; a.cu_seqlens = cu_seqlens; a.out = out; a.scale = softmax_scale;
  a.N = N; a.T = T; a.Hk = Hk; a.Hv = Hv; a.dk = dk; a.dv = dv; a.num_slots = num_slots;
  a.no_l2norm = (flags & KDA_ATTN_NO_QK_L2NORM) ? 1 : 0;
  a.literal = (flags & KDA_ATTN_ORDER_LITERAL) ? 1 : 0;
  return launch_status(
      kda::launch_step(a, dtype == KDA_BF16, reinterpret_cast<cudaStream_t>(stream)));
}

int kda_qk_norm_rope_fwd(const void* query, const void* key, const float* query_weight,
                         const float* key_weight, const float* cos_table,
                         const float* sin_table, const int32_t* positions, void* query_out,
                         void* key_out, float eps, int T, int Hq, int Hkv, int D, int R,
                         int max_position, long long query_stride, long long key_stride,
                         int flags, int dtype, kda_stream_t stream) {
  kda::NormRopeArgs a;
  int s = fill_norm_rope(a, query, key, query_weight, key_weight, cos_table, sin_table, positions,
                         eps, T, Hq, Hkv, D, R, max_position, query_stride, key_stride, flags,
                         dtype);
  if (s != KDA_OK) return s;
  if (T > 0 && (!query_out || !key_out)) return KDA_ERR_NULL_POINTER;
  const void* const ptrs[] = {query_out, key_out};
  if (!all_aligned16(ptrs)) return KDA_ERR_MISALIGNED;
  s = kda::check_current_device();
  if (s != KDA_OK) return s;
  if (T == 0) return KDA_OK;
  a.q_out = query_out; a.k_out = key_out;
  return launch_status(
      kda::launch_norm_rope(a, dtype == KDA_BF16, reinterpret_cast<cudaStream_t>(stream)));
}

int kda_qk_norm_rope_append(const void* query, const void* key, const void* value,
                            const float* query_weight, const float* key_weight,
                            const float* cos_table, const float* sin_table,
                            const int32_t* positions, const int64_t* slots, void* query_out,
                            void* k_cache, void* v_cache, float eps, int T, int Hq, int Hkv,
                            int D, int R, int max_position, int num_pages, int page_size,
                            long long query_stride, long long key_stride,
                            long long value_stride, int flags, int dtype, kda_stream_t stream) {
  kda::NormRopeArgs a;
  int s = fill_norm_rope(a, query, key, query_weight, key_weight, cos_table, sin_table, positions,
                         eps, T, Hq, Hkv, D, R, max_position, query_stride, key_stride, flags,
                         dtype);
  if (s != KDA_OK) return s;
  if (num_pages < 0) return KDA_ERR_BAD_SHAPE;
  if (!page_size_ok(page_size)) return KDA_ERR_PAGE_SIZE;
  if (T > 0 && (!value || !slots || !query_out || (num_pages > 0 && (!k_cache || !v_cache))))
    return KDA_ERR_NULL_POINTER;
  const void* const ptrs[] = {value, slots, query_out, k_cache, v_cache};
  if (!all_aligned16(ptrs)) return KDA_ERR_MISALIGNED;
  s = check_stride(value_stride, (long long)Hkv * D, T, dtype);
  if (s != KDA_OK) return s;
  if ((double)num_pages * Hkv * page_size * D >= kMaxElems) return KDA_ERR_TOO_LARGE;
  s = kda::check_current_device();
  if (s != KDA_OK) return s;
  if (T == 0) return KDA_OK;
  a.v = value; a.v_stride = value_stride; a.slots = slots; a.q_out = query_out;
  a.k_cache = k_cache; a.v_cache = v_cache; a.num_pages = num_pages; a.page_size = page_size;
  a.page_shift = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
  return launch_status(
      kda::launch_norm_rope(a, dtype == KDA_BF16, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_qk_norm_rope_bwd_workspace_size(int T, int Hq, int Hkv, int D) {
  if (T < 0 || Hq <= 0 || Hkv <= 0 || !head_dim_ok(D)) return 0;
  return kda::norm_rope_bwd_workspace(D);
}

int kda_qk_norm_rope_bwd(const void* query, const void* key, const float* query_weight,
                         const float* key_weight, const float* cos_table,
                         const float* sin_table, const int32_t* positions,
                         const void* d_query_out, const void* d_key_out, void* d_query,
                         void* d_key, float* d_query_weight, float* d_key_weight, float eps,
                         int T, int Hq, int Hkv, int D, int R, int max_position,
                         long long query_stride, long long key_stride, int flags, int dtype,
                         void* workspace, size_t workspace_bytes, kda_stream_t stream) {
  kda::NormRopeArgs a;
  int s = fill_norm_rope(a, query, key, query_weight, key_weight, cos_table, sin_table, positions,
                         eps, T, Hq, Hkv, D, R, max_position, query_stride, key_stride, flags,
                         dtype);
  if (s != KDA_OK) return s;
  if (T > 0 && (!d_query_out || !d_key_out || !d_query || !d_key)) return KDA_ERR_NULL_POINTER;
  const void* const ptrs[] = {d_query_out, d_key_out,      d_query,
                              d_key,       d_query_weight, d_key_weight};
  if (!all_aligned16(ptrs)) return KDA_ERR_MISALIGNED;
  if (!workspace || !aligned256(workspace) ||
      workspace_bytes < kda::norm_rope_bwd_workspace(D))
    return KDA_ERR_WORKSPACE;
  s = kda::check_current_device();
  if (s != KDA_OK) return s;
  a.dq_out = d_query_out; a.dk_out = d_key_out; a.dq = d_query; a.dk = d_key;
  return launch_status(kda::launch_norm_rope_bwd(a, d_query_weight, d_key_weight, workspace,
                                                 dtype == KDA_BF16,
                                                 reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_paged_attention_fwd_workspace_size(int N, int total_T, int Hq, int Hkv, int D,
                                              int dtype) {
  if (N <= 0 || total_T <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || !head_dim_ok(D) ||
      !dtype_ok(dtype))
    return 0;
  return dtype == KDA_BF16 ? kda::paged_tc_workspace(D)
                           : kda::paged_simt_workspace(total_T, Hq, D);
}

int kda_paged_attention_fwd(const void* query, const void* k_cache, const void* v_cache,
                            const int32_t* block_table, const int32_t* cu_seqlens,
                            const int32_t* kv_lens, void* out, float* lse, float softmax_scale,
                            int N, int total_T, int Hq, int Hkv, int D, int num_pages,
                            int page_size, int max_pages, int window, int sinks,
                            long long query_stride, int dtype, void* workspace,
                            size_t workspace_bytes, kda_stream_t stream) {
  if (N < 0 || total_T < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || num_pages < 0 ||
      max_pages < 0 || window < 0 || sinks < 0)
    return KDA_ERR_BAD_SHAPE;
  if (!head_dim_ok(D)) return KDA_ERR_HEAD_DIM;
  if (!page_size_ok(page_size)) return KDA_ERR_PAGE_SIZE;
  if (!isfinite(softmax_scale)) return KDA_ERR_SCALE;
  if (softmax_scale <= 0.f) softmax_scale = 1.0f / sqrtf((float)D);
  if (!dtype_ok(dtype)) return KDA_ERR_DTYPE;
  const bool work = N > 0 && total_T > 0;
  if (work && (!query || !out || !cu_seqlens || !kv_lens ||
               (num_pages > 0 && max_pages > 0 && (!k_cache || !v_cache || !block_table))))
    return KDA_ERR_NULL_POINTER;
  const void* const ptrs[] = {query, k_cache, v_cache, block_table, cu_seqlens, kv_lens, out, lse};
  if (!all_aligned16(ptrs)) return KDA_ERR_MISALIGNED;
  const int s0 = check_stride(query_stride, (long long)Hq * D, total_T, dtype);
  if (s0 != KDA_OK) return s0;
  if ((double)num_pages * Hkv * page_size > 2147483647.0 ||
      (double)max_pages * page_size > 2147483647.0 || (double)total_T * Hq > 2147483647.0 ||
      (double)N * max_pages >= kMaxElems || N > 65535 || Hkv > 65535)
    return KDA_ERR_TOO_LARGE;
  kda::PagedArgs a{};
  a.q = query; a.q_stride = query_stride; a.k_cache = k_cache; a.v_cache = v_cache;
  a.block_table = block_table; a.cu_seqlens = cu_seqlens; a.kv_lens = kv_lens; a.out = out;
  a.lse = lse; a.scale = softmax_scale; a.N = N; a.total_T = total_T; a.Hq = Hq; a.Hkv = Hkv;
  a.D = D; a.num_pages = num_pages; a.page_size = page_size; a.max_pages = max_pages;
  // a window that no position can leave hides nothing
  a.window = (double)window >= (double)max_pages * page_size ? 0 : window;
  a.sinks = sinks;
  if (dtype == KDA_BF16 && !kda::paged_tc_index_ok(a)) return KDA_ERR_TOO_LARGE;
  const size_t need = !work                 ? 0
                      : dtype == KDA_BF16 ? kda::paged_tc_workspace(D)
                                          : kda::paged_simt_need(a);
  if (need > 0 && (!workspace || !aligned256(workspace) || workspace_bytes < need))
    return KDA_ERR_WORKSPACE;
  const int s = kda::check_current_device();
  if (s != KDA_OK) return s;
  if (!work) return KDA_OK;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return launch_status(dtype == KDA_BF16 ? kda::launch_paged_tc(a, workspace, st)
                                         : kda::launch_paged_simt(a, workspace, st));
}

}  // extern "C"
