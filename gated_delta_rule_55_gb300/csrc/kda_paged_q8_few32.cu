// Attention of few new tokens over a paged cache in 8 bits: items of 32 query rows at most
// (kda_paged_q8_few.cuh).
namespace kda {
namespace {
constexpr int kRowsItem = 32;
}  // namespace
}  // namespace kda

#include "kda_paged_q8_few.cuh"

namespace kda {

cudaError_t launch_paged_tc_q8_few32(const PagedArgs& a, void* workspace, cudaStream_t st) {
  return launch_few(a, workspace, st);
}

unsigned int paged_q8_few32_read_error(bool reset) { return read_error(reset); }

}  // namespace kda
