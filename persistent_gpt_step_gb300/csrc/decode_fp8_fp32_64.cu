// decode_fp8_fp32_64.cu — gpt_decode_attention_fp8's kernels for fp32 queries, heads of up to 64.
#include "decode_fp8.cuh"

int pgs::decode_fp8_fp32_64(const DecodeParams& p, const Plan& pl, cudaStream_t st) {
  return pl.chunk <= 4 ? launch_fp8<float, 4, 64>(p, pl, st) : launch_fp8<float, 8, 64>(p, pl, st);
}
