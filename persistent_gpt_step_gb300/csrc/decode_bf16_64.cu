// Instances of the decode attention kernels for bf16 heads of up to 64 elements.
#include "decode_attention.cuh"

namespace pgs {
int decode_bf16_64(const DecodeParams& p, const Plan& pl, cudaStream_t st) {
  if (pl.chunk <= 4) return launch_form<Bf16Path, 4, 64>(p, pl, st);
  if (pl.chunk <= 8) return launch_form<Bf16Path, 8, 64>(p, pl, st);
  return launch_form<Bf16Path, 16, 64>(p, pl, st);
}
}  // namespace pgs
