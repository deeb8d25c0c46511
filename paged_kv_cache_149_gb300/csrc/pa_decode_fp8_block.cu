// Paged decode attention over FP8 (E4M3) K/V blocks with a scale for each (block, kv head):
// the instantiations of the kernel in pa_decode_kernel.cuh.
#include "pa_decode_kernel.cuh"

namespace pa {
namespace decode {
int launch_fp8_block(const Params& p, int grid, int head_dim, bool bf16, cudaStream_t stream) {
  return launch_format<kKvFp8Block, false>(p, grid, head_dim, bf16, stream);
}
}  // namespace decode
}  // namespace pa
