// next_token.cu — gpt_next_token: repeated-token penalties, biases and grammar
// masks on the logits, the greedy choice and the log-sum-exp of what is left.
#include <cmath>

#include "decode_ops.h"

namespace pgs {
namespace {

constexpr int kThreads = 512;
constexpr int kChunk = 4096;              // ids of a row handled at once
constexpr uint32_t kSeen = 0x80000000u;   // flag beside the count of an id

__device__ __forceinline__ float rescale(float x, float m) { return x == m ? 1.0f : __expf(x - m); }

__device__ __forceinline__ float load(const float* x) { return *x; }
__device__ __forceinline__ float load(const __nv_bfloat16* x) { return __bfloat162float(*x); }

// One block per row, in chunks of ids: the chunk's occurrences in the history
// are counted in shared memory, the biases of the chunk added up there, then
// every logit of the chunk is read once.
template <typename T>
__global__ void __launch_bounds__(kThreads) next_token_kernel(const __grid_constant__ gpt_next_token_args a) {
  __shared__ uint32_t count[kChunk];
  __shared__ float bias[kChunk];
  __shared__ float red_m[kThreads / 32], red_s[kThreads / 32];
  __shared__ int red_i[kThreads / 32];
  const int64_t b = blockIdx.x;
  const T* z_in = (const T*)a.logits + b * a.logits_stride;
  const int32_t* hist = a.history ? a.history + b * a.history_stride : nullptr;
  int n_hist = 0, n_prompt = 0;
  if (hist) {
    n_hist = a.history_lens ? a.history_lens[b] : a.max_history;
    n_prompt = a.prompt_lens ? a.prompt_lens[b] : 0;
    if (n_hist < 0 || n_hist > a.max_history) {
      if (threadIdx.x == 0) set_status(a.status, GPT_STATUS_BAD_POS);
      n_hist = n_hist < 0 ? 0 : a.max_history;
    }
  }
  const float rep = a.repetition ? a.repetition[b] : 1.f, pres = a.presence ? a.presence[b] : 0.f;
  const float freq = a.frequency ? a.frequency[b] : 0.f;
  float m = -INFINITY, sum = 0.f;
  int best = 0x7fffffff;
  for (int c0 = 0; c0 < a.vocab; c0 += kChunk) {
    const int n = min(kChunk, a.vocab - c0);
    for (int i = threadIdx.x; i < n; i += kThreads) count[i] = 0, bias[i] = 0.f;
    __syncthreads();
    for (int j = threadIdx.x; j < n_hist; j += kThreads) {
      const int id = hist[j];
      if (id < 0 || id >= a.vocab) {
        set_status(a.status, GPT_STATUS_BAD_TOKEN);
        continue;
      }
      const int i = id - c0;
      if (i < 0 || i >= n) continue;
      atomicOr(&count[i], kSeen);
      if (j >= n_prompt) atomicAdd(&count[i], 1u);
    }
    if (threadIdx.x == 0 && a.bias_ids)
      for (int j = 0; j < a.n_bias; ++j) {
        const int id = a.bias_ids[b * a.bias_stride + j];
        if (id >= a.vocab) set_status(a.status, GPT_STATUS_BAD_TOKEN);
        if (id >= c0 && id < c0 + n) bias[id - c0] += a.bias_values[b * a.bias_stride + j];
      }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const int id = c0 + i;
      float z = load(z_in + id);
      const uint32_t k = count[i];
      if (k & kSeen) z = z > 0.f ? __fdiv_rn(z, rep) : __fmul_rn(z, rep);
      if (k & ~kSeen) z = __fsub_rn(__fsub_rn(z, __fmul_rn(freq, (float)(k & ~kSeen))), pres);
      z = __fadd_rn(z, bias[i]);
      if (a.allowed && !((a.allowed[b * a.allowed_stride + (id >> 5)] >> (id & 31)) & 1u)) z = -INFINITY;
      if (a.out) a.out[b * a.out_stride + id] = z;
      if (z > m) {
        sum = sum * rescale(m, z) + 1.f;
        m = z;
        best = id;
      } else {
        sum += z == -INFINITY ? 0.f : rescale(z, m);
      }
    }
    __syncthreads();
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, w), s2 = __shfl_xor_sync(0xffffffffu, sum, w);
    const int i2 = __shfl_xor_sync(0xffffffffu, best, w);
    const float top = fmaxf(m, m2);
    sum = sum * rescale(m, top) + s2 * rescale(m2, top);
    best = m == m2 ? min(best, i2) : (m > m2 ? best : i2);
    m = top;
  }
  if (lane == 0) red_m[warp] = m, red_s[warp] = sum, red_i[warp] = best;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kThreads / 32; ++w) {
      const float top = fmaxf(m, red_m[w]);
      sum = sum * rescale(m, top) + red_s[w] * rescale(red_m[w], top);
      best = m == red_m[w] ? min(best, red_i[w]) : (m > red_m[w] ? best : red_i[w]);
      m = top;
    }
    if (a.token) a.token[b] = best == 0x7fffffff ? -1 : best;
    if (a.lse) a.lse[b] = m + logf(sum);
  }
}

}  // namespace
}  // namespace pgs

using namespace pgs;

extern "C" int gpt_next_token(const gpt_next_token_args* a, void* cuda_stream) {
  clear_call_error();
  if (!a) return call_error(GPT_ERR_INVALID_ARG, "args must be non-NULL");
  if (a->dtype != GPT_DTYPE_FP32 && a->dtype != GPT_DTYPE_BF16)
    return call_error(GPT_ERR_INVALID_ARG, "dtype must be GPT_DTYPE_FP32 or GPT_DTYPE_BF16");
  if (a->rows < 0 || a->vocab < 1 || a->max_history < 0 || a->n_bias < 0)
    return call_error(GPT_ERR_INVALID_ARG, "sizes must not be negative, vocab must be positive");
  if (a->rows == 0) return GPT_OK;
  if (!a->out && !a->token && !a->lse) return call_error(GPT_ERR_INVALID_ARG, "out, token and lse are all NULL");
  if (!a->logits) return call_error(GPT_ERR_INVALID_ARG, "logits must be non-NULL");
  if (a->rows > 1 && (a->logits_stride < a->vocab || (a->out && a->out_stride < a->vocab) ||
                      (a->history && a->history_stride < a->max_history) ||
                      (a->bias_ids && a->bias_stride < a->n_bias) ||
                      (a->allowed && a->allowed_stride < (a->vocab + 31) / 32)))
    return call_error(GPT_ERR_INVALID_ARG, "a row stride is smaller than its row");
  if (!a->history && (a->history_lens || a->prompt_lens))
    return call_error(GPT_ERR_INVALID_ARG, "history_lens and prompt_lens go with history");
  if ((a->bias_ids != nullptr) != (a->bias_values != nullptr))
    return call_error(GPT_ERR_INVALID_ARG, "bias_ids and bias_values go together");
  if ((const void*)a->out == a->logits && (a->dtype != GPT_DTYPE_FP32 || (a->rows > 1 && a->out_stride != a->logits_stride)))
    return call_error(GPT_ERR_INVALID_ARG, "in place needs fp32 logits and equal strides");
  const cudaStream_t st = (cudaStream_t)cuda_stream;
  if (a->dtype == GPT_DTYPE_BF16) next_token_kernel<__nv_bfloat16><<<a->rows, kThreads, 0, st>>>(*a);
  else next_token_kernel<float><<<a->rows, kThreads, 0, st>>>(*a);
  return check_launch("gpt_next_token");
}
