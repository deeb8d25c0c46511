// Paged decode attention over FP8 (E4M3) K/V blocks with a scale for each (block, kv head):
// the instantiations of the kernel in pa_decode_kernel.cuh.  HBM-bound like the others there;
// applying the scales costs little against one scale per cache.  On GB300, device time: 64
// sequences of 128..2048 tokens, 32 query / 8 kv heads of 128: 36.2 us (per-tensor scales 33.7,
// bytes at the copy rate 22.1), with 128 / 8 heads 71.8 (22.6; 255 registers and spills);
// 128 sequences with 32 / 32 heads 109 (104.5, 96.2); 8 sequences of 8-32 K tokens 62.1 (59.5,
// 40.8).
#include "pa_decode_kernel.cuh"

namespace pa {
namespace decode {
int launch_fp8_block(const Params& p, int grid, int head_dim, bool bf16, cudaStream_t stream) {
  return launch_format<kKvFp8Block, false>(p, grid, head_dim, bf16, stream);
}
}  // namespace decode
}  // namespace pa
