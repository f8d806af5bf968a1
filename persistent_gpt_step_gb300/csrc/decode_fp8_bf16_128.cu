// decode_fp8_bf16_128.cu — gpt_decode_attention_fp8's kernels for bf16 queries, heads of 65 to 128.
#include "decode_fp8.cuh"

int pgs::decode_fp8_bf16_128(const DecodeParams& p, const Plan& pl, cudaStream_t st) {
  if (pl.chunk <= 4) return launch_fp8<__nv_bfloat16, 4, 128>(p, pl, st);
  return pl.chunk <= 8 ? launch_fp8<__nv_bfloat16, 8, 128>(p, pl, st) : launch_fp8<__nv_bfloat16, 16, 128>(p, pl, st);
}
