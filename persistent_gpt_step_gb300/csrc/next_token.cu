// next_token.cu — gpt_next_token: repeated-token penalties, biases and grammar
// masks on the logits, the greedy choice and the log-sum-exp of what is left.
//
// Bound: HBM (each logit read once, written once as fp32).  A row is the work of a
// cluster of blocks, each with a range of its ids, so that one row is spread over
// SMs and the row's maximum and sum are joined through shared memory: one launch,
// no workspace.  Few ids have a penalty or a bias.  Each block marks those of its
// range in a bitmap, gives them places in a compact table by the bitmap's running
// popcounts, and counts occurrences and adds biases there; the pass over the logits
// then looks at one byte of the bitmap per eight ids.
#include <cooperative_groups.h>

#include <cmath>
#include <utility>

#include "decode_ops.h"

namespace pgs {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMarked = 4096;            // places of the compact table
constexpr int kRange = 32768;            // ids marked at once, where the history and the biases fit the table
constexpr int kNoToken = 0x7fffffff;
constexpr float kLog2e = 1.4426950408889634f;

// exp(x - m) between partial maxima: 1 where both are the same, infinities too.
__device__ __forceinline__ float rescale(float x, float m) { return x == m ? 1.0f : exp2f((x - m) * kLog2e); }

struct Best {  // maximum, sum of exp(z - m), smallest id of the maximum
  float m, sum;
  int id;
};
__device__ __forceinline__ Best join(const Best& a, const Best& b) {
  const float top = fmaxf(a.m, b.m);
  return Best{top, a.sum * rescale(a.m, top) + b.sum * rescale(b.m, top), a.m == b.m ? min(a.id, b.id) : a.m > b.m ? a.id : b.id};
}

// Eight logits on a 16-byte boundary as floats.
__device__ __forceinline__ void load8(const float* z, float* x) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(z)), b = __ldcs(reinterpret_cast<const float4*>(z) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* z, float* x) {
  Piece<__nv_bfloat16>::unpack(__ldcs(reinterpret_cast<const uint4*>(z)), x);
}
__device__ __forceinline__ void load1(const float* z, float* x) { *x = *z; }
__device__ __forceinline__ void load1(const __nv_bfloat16* z, float* x) { *x = __bfloat162float(*z); }

// Units of eight ids: unit u holds ids 8 u - shift .., the shift chosen so that
// units of the logits lie on 16-byte boundaries whatever the row's address is.
template <typename T>
__global__ void __launch_bounds__(kThreads) next_token_kernel(const __grid_constant__ gpt_next_token_args a) {
  __shared__ uint32_t bitmap[kRange / 32];
  __shared__ uint16_t place[kRange / 32];   // marked ids before a word's
  __shared__ uint32_t seen[kMarked];        // in the history: 2^31; occurrences after the prompt
  __shared__ float bias[kMarked];
  __shared__ Best warp_best[kWarps], block_best[8];
  __shared__ uint32_t scan[kWarps];
  cg::cluster_group cluster = cg::this_cluster();
  auto started = cluster.barrier_arrive();  // waited for before another block's memory is written
  const int blocks = cluster.num_blocks(), part = cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t b = blockIdx.x / blocks;
  const T* z_in = (const T*)a.logits + b * a.logits_stride;
  float* z_out = a.out ? a.out + b * a.out_stride : nullptr;
  const uint32_t* allowed = a.allowed ? a.allowed + b * a.allowed_stride : nullptr;
  const int32_t* bias_ids = a.bias_ids ? a.bias_ids + b * a.bias_stride : nullptr;
  const int32_t* hist = a.history ? a.history + b * a.history_stride : nullptr;
  int n_hist = 0, n_prompt = 0;
  if (hist) {
    n_hist = a.history_lens ? a.history_lens[b] : a.max_history;
    n_prompt = a.prompt_lens ? a.prompt_lens[b] : 0;
    if (n_hist < 0 || n_hist > a.max_history) {
      if (tid == 0) set_status(a.status, GPT_STATUS_BAD_POS);
      n_hist = n_hist < 0 ? 0 : a.max_history;
    }
  }
  const int n_bias = bias_ids ? a.n_bias : 0;
  const bool marks = n_hist > 0 || n_bias > 0;
  const float rep = a.repetition ? a.repetition[b] : 1.f, pres = a.presence ? a.presence[b] : 0.f;
  const float freq = a.frequency ? a.frequency[b] : 0.f;

  const int shift = (int)((reinterpret_cast<uintptr_t>(z_in) & 15) / sizeof(T));
  const bool wide_out = z_out && ((reinterpret_cast<uintptr_t>(z_out) / 4 - shift) & 3) == 0;
  const int units = (int)(((int64_t)a.vocab + shift + 7) / 8);
  const int u0 = (int)((int64_t)part * units / blocks), u1 = (int)((int64_t)(part + 1) * units / blocks);
  const int step = ((int64_t)n_hist + n_bias <= kMarked ? kRange : kMarked) / 8;  // units marked at once: a place for each id in any case

  Best best{-INFINITY, 0.f, kNoToken};
  for (int v0 = u0; v0 < u1; v0 += step) {
    const int v1 = min(u1, v0 + step), words = (v1 - v0 + 3) / 4;
    const int64_t first = (int64_t)v0 * 8 - shift;  // the id of bit 0
    const int ids = (v1 - v0) * 8;
    if (marks) {
      for (int i = tid; i < words; i += kThreads) bitmap[i] = 0;
      __syncthreads();
      for (int j = tid; j < n_hist; j += kThreads) {
        const int id = hist[j];
        if (id < 0 || id >= a.vocab) { set_status(a.status, GPT_STATUS_BAD_TOKEN); continue; }
        const int64_t i = id - first;
        if (i >= 0 && i < ids) atomicOr(&bitmap[i >> 5], 1u << (i & 31));
      }
      for (int j = tid; j < n_bias; j += kThreads) {
        const int id = bias_ids[j];
        if (id >= a.vocab) { set_status(a.status, GPT_STATUS_BAD_TOKEN); continue; }
        const int64_t i = id - first;
        if (id >= 0 && i >= 0 && i < ids) atomicOr(&bitmap[i >> 5], 1u << (i & 31));
      }
      __syncthreads();
      // places: running popcounts, kRange / 32 / kThreads words a thread
      constexpr int kPer = kRange / 32 / kThreads;
      uint32_t mine = 0, sum;
#pragma unroll
      for (int i = 0; i < kPer; ++i) mine += tid * kPer + i < words ? __popc(bitmap[tid * kPer + i]) : 0;
      sum = mine;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, sum, x);
        if (lane >= x) sum += y;
      }
      if (lane == 31) scan[warp] = sum;
      __syncthreads();
      sum -= mine;
      uint32_t marked = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w == warp) sum += marked;
        marked += scan[w];
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (tid * kPer + i < words) {
          place[tid * kPer + i] = (uint16_t)sum;
          sum += __popc(bitmap[tid * kPer + i]);
        }
      for (uint32_t i = tid; i < marked; i += kThreads) seen[i] = 0, bias[i] = 0.f;
      __syncthreads();
      auto place_of = [&](int64_t i) { return place[i >> 5] + __popc(bitmap[i >> 5] & ((1u << (i & 31)) - 1u)); };
      for (int j = tid; j < n_hist; j += kThreads) {
        const int64_t i = hist[j] - first;
        if (hist[j] < 0 || hist[j] >= a.vocab || i < 0 || i >= ids) continue;
        atomicOr(&seen[place_of(i)], 0x80000000u);
        if (j >= n_prompt) atomicAdd(&seen[place_of(i)], 1u);
      }
      if (warp == 0)  // biases of one id in the order of their entries: the entry's rank among the equal ones takes turns
        for (int j0 = 0; j0 < n_bias; j0 += 32) {
          const int id = j0 + lane < n_bias ? bias_ids[j0 + lane] : -1;
          const int64_t i = id - first;
          const bool mine_too = id >= 0 && id < a.vocab && i >= 0 && i < ids;
          const float v = mine_too ? a.bias_values[b * a.bias_stride + j0 + lane] : 0.f;
          const uint32_t same = __match_any_sync(0xffffffffu, id);
          const int rank = mine_too ? __popc(same & ((1u << lane) - 1u)) : -1;
          for (int r = 0; __any_sync(0xffffffffu, rank >= r); ++r) {
            if (rank == r) bias[place_of(i)] += v;
            __syncwarp();
          }
        }
      __syncthreads();
    }

    constexpr int kUnroll = 2;
    for (int w0 = v0 + tid; w0 < v1; w0 += kUnroll * kThreads) {
      float x[kUnroll][8];
      uint32_t open[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int w = w0 + k * kThreads;
        const int64_t id0 = (int64_t)w * 8 - shift;
        open[k] = 0xffu;
        if (w >= v1) continue;
        if (id0 >= 0 && id0 + 8 <= a.vocab) {
          load8(z_in + id0, x[k]);
          if (allowed) {
            open[k] = allowed[id0 >> 5] >> (id0 & 31);
            if ((id0 & 31) > 24) open[k] |= allowed[(id0 >> 5) + 1] << (32 - (id0 & 31));
          }
        } else {
          open[k] = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int64_t id = id0 + i;
            const bool there = id >= 0 && id < a.vocab;
            x[k][i] = -INFINITY;
            if (there) load1(z_in + id, &x[k][i]);
            if (there && (!allowed || (allowed[id >> 5] >> (id & 31)) & 1u)) open[k] |= 1u << i;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int w = w0 + k * kThreads;
        if (w >= v1) continue;
        const int64_t id0 = (int64_t)w * 8 - shift;
        if (marks) {
          const int i0 = (w - v0) * 8;
          const uint32_t word = bitmap[i0 >> 5];
          if ((word >> (i0 & 31)) & 0xffu) {
            uint32_t at = place[i0 >> 5] + __popc(word & ((1u << (i0 & 31)) - 1u));
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if ((word >> ((i0 & 31) + i)) & 1u) {
                const uint32_t c = seen[at];
                float z = x[k][i];
                if (c) z = z > 0.f ? __fdiv_rn(z, rep) : __fmul_rn(z, rep);
                if (c & 0x7fffffffu) z = __fsub_rn(__fsub_rn(z, __fmul_rn(freq, (float)(c & 0x7fffffffu))), pres);
                x[k][i] = __fadd_rn(z, bias[at]);
                ++at;
              }
          }
        }
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (!((open[k] >> i) & 1u)) x[k][i] = -INFINITY;
          top = fmaxf(top, x[k][i]);
        }
        if (z_out) {
          if (wide_out && id0 >= 0 && id0 + 8 <= a.vocab) {
            __stcs(reinterpret_cast<float4*>(z_out + id0), make_float4(x[k][0], x[k][1], x[k][2], x[k][3]));
            __stcs(reinterpret_cast<float4*>(z_out + id0) + 1, make_float4(x[k][4], x[k][5], x[k][6], x[k][7]));
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (id0 + i >= 0 && id0 + i < a.vocab) z_out[id0 + i] = x[k][i];
          }
        }
        if (top > best.m) {  // ids only rise here: the first of equal maxima stays
          best.sum *= rescale(best.m, top);
          best.m = top;
#pragma unroll
          for (int i = 7; i >= 0; --i)
            if (x[k][i] == top) best.id = (int)id0 + i;
        }
        const float off = isinf(best.m) ? 0.f : best.m;  // of an infinite maximum: sums of infinities, as log-sum-exp has them
#pragma unroll
        for (int i = 0; i < 8; ++i) best.sum += exp2f((x[k][i] - off) * kLog2e);
      }
    }
    if (v1 < u1) __syncthreads();
  }

#pragma unroll
  for (int w = 16; w > 0; w >>= 1)
    best = join(best, Best{__shfl_xor_sync(0xffffffffu, best.m, w), __shfl_xor_sync(0xffffffffu, best.sum, w), __shfl_xor_sync(0xffffffffu, best.id, w)});
  if (lane == 0) warp_best[warp] = best;
  __syncthreads();
  cluster.barrier_wait(std::move(started));
  if (tid == 0) {
    for (int w = 1; w < kWarps; ++w) best = join(best, warp_best[w]);
    cluster.map_shared_rank(block_best, 0)[part] = best;
  }
  cluster.sync();
  if (part == 0 && tid == 0) {
    for (int r = 1; r < blocks; ++r) best = join(best, block_best[r]);
    if (a.token) a.token[b] = best.id == kNoToken ? -1 : best.id;
    if (a.lse) a.lse[b] = best.m + logf(best.sum);
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
  if (reinterpret_cast<uintptr_t>(a->logits) % elem_size(a->dtype) || reinterpret_cast<uintptr_t>(a->out) % 4)
    return call_error(GPT_ERR_INVALID_ARG, "logits and out must lie on their elements' boundaries");
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
  // Blocks of a row: as many as fill the GPU a few times over, with 1,024 ids each at least.
  int blocks = 8;
  while (blocks > 1 && ((int64_t)a->rows * blocks > 1216 || a->vocab / blocks < 1024)) blocks /= 2;
  if ((int64_t)a->rows * blocks > INT32_MAX) return call_error(GPT_ERR_UNSUPPORTED, "too many rows");
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = blocks, attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a->rows * blocks), cfg.blockDim = dim3(kThreads), cfg.stream = (cudaStream_t)cuda_stream;
  cfg.attrs = &attr, cfg.numAttrs = 1;
  if (a->dtype == GPT_DTYPE_BF16) cudaLaunchKernelEx(&cfg, next_token_kernel<__nv_bfloat16>, *a);
  else cudaLaunchKernelEx(&cfg, next_token_kernel<float>, *a);
  return check_launch("gpt_next_token");
}
