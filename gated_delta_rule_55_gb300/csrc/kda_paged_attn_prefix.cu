// Attention behind shared prefixes, caches of bf16, on the tensor cores
// (kda_paged_prefix_attention_fwd).
namespace kda {
namespace {
constexpr bool kPrefixes = true;
}  // namespace
}  // namespace kda

#include "kda_paged_tc.cuh"

namespace kda {

cudaError_t launch_paged_tc_prefix(const PagedArgs& a, void* workspace, cudaStream_t st) {
  return launch_any<false, true>(a, workspace, nullptr, st);
}

unsigned int paged_prefix_read_error(bool reset) { return read_error(reset); }

}  // namespace kda
