// Instances of the decode attention kernels for bf16 heads of up to 128 elements.
#include "decode_attention.cuh"

namespace pgs {
int decode_bf16_128(const DecodeParams& p, const Plan& pl, cudaStream_t st) {
  if (pl.chunk <= 4) return launch_form<Bf16Path, 4, 128>(p, pl, st);
  if (pl.chunk <= 8) return launch_form<Bf16Path, 8, 128>(p, pl, st);
  return launch_form<Bf16Path, 16, 128>(p, pl, st);
}
}  // namespace pgs
