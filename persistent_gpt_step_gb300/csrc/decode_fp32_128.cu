// Instances of the decode attention kernels for fp32 heads of up to 128 elements.
#include "decode_attention.cuh"

namespace pgs {
int decode_fp32_128(const DecodeParams& p, const Plan& pl, cudaStream_t st) {
  if (pl.chunk <= 1) return launch_form<Fp32Path, 1, 128>(p, pl, st);
  if (pl.chunk <= 4) return launch_form<Fp32Path, 4, 128>(p, pl, st);
  return launch_form<Fp32Path, 8, 128>(p, pl, st);
}
}  // namespace pgs
