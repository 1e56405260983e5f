// Attention behind shared prefixes, caches in 8 bits, on the tensor cores
// (kda_paged_prefix_attention_fwd).
namespace kda {
namespace {
constexpr bool kPrefixes = true;
}  // namespace
}  // namespace kda

#include "kda_paged_tc.cuh"

namespace kda {

cudaError_t launch_paged_tc_prefix_q8(const PagedArgs& a, void* workspace, cudaStream_t st) {
  void* terms = static_cast<uint8_t*>(workspace) +
                paged_prefix_tc_workspace(a.total_T, a.Hq, a.D, false);
  return launch_any<true, true>(a, workspace, terms, st);
}

unsigned int paged_prefix_q8_read_error(bool reset) { return read_error(reset); }

}  // namespace kda
