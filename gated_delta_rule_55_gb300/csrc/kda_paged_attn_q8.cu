// Attention over a paged cache in 8 bits on the tensor cores (kda_paged_attention_q8_fwd).
namespace kda {
namespace {
constexpr bool kPrefixes = false;
}  // namespace
}  // namespace kda

#include "kda_paged_tc.cuh"

namespace kda {

cudaError_t launch_paged_tc_q8(const PagedArgs& a, void* workspace, cudaStream_t st) {
  return launch_any<true, false>(a, workspace,
                                 static_cast<uint8_t*>(workspace) + paged_tc_workspace(a.D), st);
}

unsigned int paged_q8_read_error(bool reset) { return read_error(reset); }

}  // namespace kda
