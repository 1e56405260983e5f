// Attention over a paged cache of bf16 on the tensor cores (kda_paged_attention_fwd), and what the
// kinds of call share.
namespace kda {
namespace {
constexpr bool kPrefixes = false;
}  // namespace
}  // namespace kda

#include "kda_paged_tc.cuh"

namespace kda {

// Whether the line of key tiles, at the block tables' capacity, fits the kernel's indices.
bool paged_tc_index_ok(const PagedArgs& a) {
  const double rows = (double)a.total_T * (a.Hq / a.Hkv) / kRowsItem;
  auto units = [&](int n, int pages) {
    const double tiles = (double)pages * a.page_size / kKeys + kOverheadMost + 2;
    return (rows + n) * tiles * a.Hkv * (a.groups > 0 ? 3 : 1);  // (units of a tile, at most)
  };
  // (sequences may take their prefix along)
  const int along = a.groups > 0 ? a.max_prefix_pages : 0;
  if ((double)a.max_pages + along > 2147483647.0) return false;
  const double shared = a.groups > 0 ? units(a.groups, a.max_prefix_pages) : 0.0;
  return units(a.N, a.max_pages + along) + shared < 2147483647.0;
}

size_t paged_tc_workspace(int D) {
  return 8192 + (size_t)2 * kCtas * kRowsItem * (sizeof(float2) + D * sizeof(float));
}

// Behind it: a query's terms (caches in 8 bits, D = 128), and every row's two results, where they
// are not cut and where they are (prefixes).
size_t paged_q8_tc_workspace(int total_T, int Hq, int D) {
  return paged_tc_workspace(D) + (D == 128 ? paged_query_terms(total_T, Hq) : 0);
}

size_t paged_prefix_tc_workspace(int total_T, int Hq, int D, bool q8) {
  return (q8 ? paged_q8_tc_workspace(total_T, Hq, D) : paged_tc_workspace(D)) +
         (size_t)2 * total_T * Hq * (sizeof(float2) + sizeof(int4) + D * sizeof(float));
}

cudaError_t launch_paged_tc(const PagedArgs& a, void* workspace, cudaStream_t st) {
  const bool q8 = a.k_scale != nullptr;
  if (a.groups > 0)
    return q8 ? launch_paged_tc_prefix_q8(a, workspace, st)
              : launch_paged_tc_prefix(a, workspace, st);
  // By the rows of a sequence on average, items of 16, of 32 or of 256 rows.  64 sequences, 32 + 8
  // heads: D = 128, 16 rows 113 us for 241 (items of 32, 20 rows: 172 for 253 with items of 16), 32
  // rows 176 for 241, 36 rows 244; D = 64, 4 rows 82 for 161, 20 rows 136, 32 rows 147 for 162.
  // The lengths lie in device memory, so the host has only the average, and one kernel takes all
  // sequences of a call.  Where they are of two kinds that costs one of them, D = 128: 64 single
  // tokens over 512..8192 keys with a chunk of 512 behind 8192 (35 rows on average: tiles of 256
  // rows) 335 us, alone 110 and 80, over bf16 pages 281; 200 single tokens with that chunk (14
  // rows: items of 16, for each of which the chunk's keys are read again) 641, alone 291 and 80,
  // bf16 673; 255 over 100..1000 keys with a chunk of 1700 behind 4096 (31 rows: items of 32) 825,
  // alone 76 and 148, bf16 236.  Two calls, one for each kind, take the sum of what they take alone.
  // Smaller items are more of them, whose line has to fit the indices as well (paged_tc_index_ok).
  const long long rows = (long long)a.total_T * (a.Hq / a.Hkv);
  const double line =
      (rows / 16.0 + a.N) * a.Hkv * ((double)a.max_pages * a.page_size / kKeys + 4);
  if (q8 && a.D >= 64 && rows <= 32ll * a.N && line < 2147483647.0)
    return rows <= 16ll * a.N ? launch_paged_tc_q8_few(a, workspace, st)
                              : launch_paged_tc_q8_few32(a, workspace, st);
  return q8 ? launch_paged_tc_q8(a, workspace, st)
            : launch_any<false, false>(a, workspace, nullptr, st);
}

unsigned int paged_read_error(bool reset) {
  return read_error(reset) | paged_q8_read_error(reset) | paged_q8_few_read_error(reset) |
         paged_q8_few32_read_error(reset) | paged_prefix_read_error(reset) |
         paged_prefix_q8_read_error(reset);
}

}  // namespace kda
