// next_token.cu — gpt_next_token: repeated-token penalties, biases and grammar
// masks on the logits, the greedy choice and the log-sum-exp of what is left.
//
// Bound: HBM (each logit read once, written once as fp32).  A row is the work of a
// cluster of blocks, each with a range of its ids, so that one row is spread over
// SMs and the row's maximum and sum are joined through shared memory: one launch,
// no workspace.  Few ids have a penalty or a bias.  Each block marks those of its
// range in a bitmap, gives them places in a compact table by the bitmap's running
// popcounts, counts occurrences and adds biases there, works them off one a thread,
// and writes them over what the pass over the logits left: that pass looks at one
// byte of the bitmap per eight ids and has no branch for them.  (With the penalties,
// or only separate stores, inside the pass 512 rows of 131,072 logits and 2,048 tokens
// took 150 us: nearly every warp has a marked id among its 256; now 113, 4.9 TB/s.)
#include <cooperative_groups.h>

#include <cmath>

#include "decode_ops.h"

namespace pgs {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRange = 32768;            // ids of a range at most
constexpr int kMarked = 2048;            // places of the compact table; a range with more marked ids ends before them
constexpr int kBatch = 16;               // history ids of a thread at a time
constexpr int kHistory = kBatch * kThreads;
constexpr int kNoToken = 0x7fffffff;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * kLog2e));
  return y;
}
// exp(x - m) between partial maxima: 1 where both are the same, infinities too.
__device__ __forceinline__ float rescale(float x, float m) { return x == m ? 1.0f : exp_fast(x - m); }

struct Best {  // maximum, sum of exp(z - m), smallest id of the maximum
  float m, sum;
  int id;
};
__device__ __forceinline__ Best join(const Best& a, const Best& b) {
  const float top = fmaxf(a.m, b.m);
  return Best{top, a.sum * rescale(a.m, top) + b.sum * rescale(b.m, top), a.m == b.m ? min(a.id, b.id) : a.m > b.m ? a.id : b.id};
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// Eight logits as loaded (fp32: on a 32-byte, bf16: on a 16-byte boundary), unpacked
// where they are used: nothing waits for them before, nor for the mask's words after
// them (unpacked at once 512 rows of 131,072 in bf16 118 us, so 112).
template <typename T> struct Eight;
template <> struct Eight<float> {
  float x[8];
  __device__ __forceinline__ void load(const float* z) {
    asm volatile("ld.global.L1::no_allocate.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
                 : "l"(z) : "memory");
  }
  __device__ __forceinline__ void load1(const float* z, int i, bool there) { x[i] = there ? *z : 0.f; }
  __device__ __forceinline__ float* values(float*) { return x; }
};
template <> struct Eight<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* z) {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(z) : "memory");
  }
  __device__ __forceinline__ void load1(const __nv_bfloat16* z, int i, bool there) {
    const uint32_t bits = there ? *reinterpret_cast<const uint16_t*>(z) : 0u;
    uint32_t& w = (&u.x)[i / 2];
    w = i & 1 ? w | bits << 16 : bits;
  }
  __device__ __forceinline__ float* values(float* to) const {
    Piece<__nv_bfloat16>::unpack(u, to);
    return to;
  }
};
__device__ __forceinline__ void store8(float* z, const float* x) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(z), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]),
               "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
               : "memory");
}

// Units of eight ids: unit u holds ids 8 u - shift .., the shift chosen so that
// units of the logits lie on boundaries of their size whatever the row's address is.
// kAhead: a thread has its next two units under way instead of one.
template <typename T, bool kAhead>
__global__ void __launch_bounds__(kThreads, 4) next_token_kernel(const __grid_constant__ gpt_next_token_args a) {
  __shared__ __align__(16) uint32_t bitmap[kRange / 32];
  __shared__ uint16_t place[kRange / 32];   // marked ids before a word's
  __shared__ uint16_t where[kMarked];       // the marked id of a place, from the range's first on
  __shared__ __align__(16) uint32_t seen[kMarked];  // occurrences after the prompt; 2^31: in the prompt
  __shared__ __align__(16) float bias[kMarked];
  __shared__ Best warp_best[kWarps], block_best[8];
  __shared__ uint32_t scan[kWarps];
  __shared__ int fit;
  cg::cluster_group cluster = cg::this_cluster();
  after_stream();
  const int blocks = cluster.num_blocks(), part = cluster.block_rank();
  if (blocks > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");  // waited for before another block's memory is written
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t b = blockIdx.x / blocks;
  const T* z_in = (const T*)a.logits + b * a.logits_stride;
  float* z_out = a.out ? a.out + b * a.out_stride : nullptr;
  const uint32_t* allowed = a.allowed ? a.allowed + b * a.allowed_stride : nullptr;
  const int32_t* bias_ids = a.bias_ids ? a.bias_ids + b * a.bias_stride : nullptr;
  const int shift = (int)((reinterpret_cast<uintptr_t>(z_in) / sizeof(T)) & 7);
  const bool wide_out = z_out && ((reinterpret_cast<uintptr_t>(z_out) / 4 - shift) & 7) == 0;
  const int units = (int)(((int64_t)a.vocab + shift + 7) / 8);
  const int u0 = (int)((int64_t)part * units / blocks), u1 = (int)((int64_t)(part + 1) * units / blocks);
  const int32_t* hist = a.history ? a.history + b * a.history_stride : nullptr;
  const int most = hist ? a.max_history : 0;
  int n_hist = hist && a.history_lens ? a.history_lens[b] : most;
  const int n_prompt = hist && a.prompt_lens ? a.prompt_lens[b] : 0;

  // Unit w of the logits as loaded, and the mask's words of its ids; at the row's ends
  // the first is the mask of its ids itself.
  auto inner = [&](int w) { return (int64_t)w * 8 - shift >= 0 && (int64_t)w * 8 - shift + 8 <= a.vocab; };
  auto load = [&](int w, Eight<T>& x, uint32_t& m0, uint32_t& m1) {
    const int64_t id0 = (int64_t)w * 8 - shift;
    m0 = m1 = 0xffffffffu;
    if (w >= u1) return;
    if (inner(w)) {
      x.load(z_in + id0);
      if (allowed) {
        m0 = allowed[id0 >> 5];
        if ((id0 & 31) > 24) m1 = allowed[(id0 >> 5) + 1];
      }
    } else {
      m0 = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t id = id0 + i;
        const bool there = id >= 0 && id < a.vocab;
        x.load1(z_in + id, i, there);
        if (there && (!allowed || (allowed[id >> 5] >> (id & 31)) & 1u)) m0 |= 1u << i;
      }
    }
  };
  Eight<T> raw;
  uint32_t m0, m1;
  load(u0 + tid, raw, m0, m1);  // every thread's first, under way while the ids are marked
  auto clear = [&] {
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    for (int i = tid; i < kRange / 128; i += kThreads) reinterpret_cast<uint4*>(bitmap)[i] = zero;
    for (int i = tid; i < kMarked / 4; i += kThreads) reinterpret_cast<uint4*>(seen)[i] = reinterpret_cast<uint4*>(bias)[i] = zero;
    if (tid == 0) fit = kRange / 32;
    __syncthreads();
  };

  // The history, kBatch ids of a thread at a time.  One that fits is read once, before
  // its length is known.
  const bool at_once = most <= kHistory;
  int recent[kBatch];
  auto read_history = [&](int j0, int n) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int j = j0 + i * kThreads + tid;
      recent[i] = j < n ? hist[j] : -1;
    }
  };
  if (at_once) read_history(0, most);
  const int n_bias = bias_ids ? a.n_bias : 0;
  int bias_id = -1;  // the first 32 entries, a lane of the last warp each
  float bias_value = 0.f;
  const bool adds = warp == kWarps - 1;
  if (adds && lane < n_bias) bias_id = bias_ids[lane], bias_value = a.bias_values[b * a.bias_stride + lane];
  if (hist || n_bias > 0) clear();  // (before the loads above are waited for)
  const float rep = a.repetition ? a.repetition[b] : 1.f, pres = a.presence ? a.presence[b] : 0.f;
  const float freq = a.frequency ? a.frequency[b] : 0.f;
  if (n_hist < 0 || n_hist > most || n_prompt < 0) {  // (a prompt longer than the history: none of that counts)
    if (tid == 0) set_status(a.status, GPT_STATUS_BAD_POS);
    n_hist = min(max(n_hist, 0), most);
  }
  const bool marks = n_hist > 0 || n_bias > 0;
  uint32_t bad = 0;

  Best best{-INFINITY, 0.f, kNoToken};
  for (int v0 = u0, v1; v0 < u1; v0 = v1) {
    v1 = min(u1, v0 + kRange / 8);
    const int words = (v1 - v0 + 3) / 4;
    const int first = (int)((int64_t)v0 * 8 - shift);  // the id of bit 0
    uint32_t ids = (v1 - v0) * 8, marked = 0;
    auto inside = [&](int id) { return (uint32_t)id < (uint32_t)a.vocab && (uint32_t)(id - first) < ids; };
    if (v0 > u0) load(v0 + tid, raw, m0, m1);
    if (marks) {
      if (v0 > u0) clear();
      auto mark = [&](int id) {
        if (inside(id)) atomicOr(&bitmap[(id - first) >> 5], 1u << ((id - first) & 31));
      };
      for (int j0 = 0; j0 < n_hist; j0 += kHistory) {
        if (!at_once) read_history(j0, n_hist);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int j = j0 + i * kThreads;
          if (j >= n_hist) break;
          const bool there = j + tid < n_hist;
          bad |= there && (uint32_t)recent[i] >= (uint32_t)a.vocab;
          if (there) mark(recent[i]);
        }
      }
      if (adds)
        for (int j = lane; j < n_bias; j += 32) {
          const int id = j < 32 ? bias_id : bias_ids[j];
          bad |= id >= a.vocab;
          mark(id);
        }
      __syncthreads();
      // places: running popcounts, kRange / 32 / kThreads words a thread
      constexpr int kPer = kRange / 32 / kThreads;
      uint32_t mine = 0, sum;
#pragma unroll
      for (int i = 0; i < kPer; ++i) mine += tid * kPer + i < words ? __popc(bitmap[tid * kPer + i]) : 0;
      sum = mine;
#pragma unroll
      for (int y = 1; y < 32; y <<= 1) {
        const uint32_t z = __shfl_up_sync(0xffffffffu, sum, y);
        if (lane >= y) sum += z;
      }
      if (lane == 31) scan[warp] = sum;
      __syncthreads();
      sum -= mine;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w == warp) sum += marked;
        marked += scan[w];
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (tid * kPer + i < words) {
          place[tid * kPer + i] = (uint16_t)sum;
          if (sum <= kMarked && sum + __popc(bitmap[tid * kPer + i]) > kMarked) fit = tid * kPer + i;  // the first word without places
          sum += __popc(bitmap[tid * kPer + i]);
        }
      __syncthreads();
      if (marked > kMarked) {  // the range ends before that word
        marked = place[fit];
        v1 = v0 + fit * 4;
        ids = fit * 32;
      }
      auto place_of = [&](int id) {
        const int i = id - first;
        return place[i >> 5] + __popc(bitmap[i >> 5] & ((1u << (i & 31)) - 1u));
      };
      for (int j0 = 0; j0 < n_hist; j0 += kHistory) {  // integer sums: the same in any order
        if (!at_once) read_history(j0, n_hist);
#pragma unroll
        for (int i0 = 0; i0 < kBatch; i0 += 4) {  // lookups before updates, so that they do not wait for one another
          if (j0 + i0 * kThreads >= n_hist) break;
          int at[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            at[i] = j0 + (i0 + i) * kThreads + tid < n_hist && inside(recent[i0 + i]) ? place_of(recent[i0 + i]) : -1;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (at[i] >= 0) {
              where[at[i]] = (uint16_t)(recent[i0 + i] - first);
              if (j0 + (i0 + i) * kThreads + tid >= n_prompt) atomicAdd(&seen[at[i]], 1u);
              else atomicOr(&seen[at[i]], 0x80000000u);
            }
        }
      }
      if (adds)  // biases of one id in the order of their entries: the entry's rank among the equal ones takes turns
        for (int j0 = 0; j0 < n_bias; j0 += 32) {
          if (j0 > 0) {
            bias_id = j0 + lane < n_bias ? bias_ids[j0 + lane] : -1;
            bias_value = j0 + lane < n_bias ? a.bias_values[b * a.bias_stride + j0 + lane] : 0.f;
          }
          const uint32_t same = __match_any_sync(0xffffffffu, bias_id);
          const int rank = inside(bias_id) ? __popc(same & ((1u << lane) - 1u)) : -1;
          if (rank >= 0) where[place_of(bias_id)] = (uint16_t)(bias_id - first);
          for (int r = 0; __any_sync(0xffffffffu, rank >= r); ++r) {
            if (rank == r) bias[place_of(bias_id)] += bias_value;
            __syncwarp();
          }
        }
      if (adds && n_bias > 32 && v1 < u1) bias_id = bias_ids[lane], bias_value = a.bias_values[b * a.bias_stride + lane];
      __syncthreads();
      // The marked ids themselves, one a thread.  The pass over the logits leaves them
      // out of the maximum and the sum, and their values are written over its own.
      for (uint32_t k = tid; k < marked; k += kThreads) {
        const int id = first + where[k];
        const uint32_t c = seen[k];
        float z = to_float(z_in[id]);
        if (c) z = z > 0.f ? __fdiv_rn(z, rep) : __fmul_rn(z, rep);
        if (c & 0x7fffffffu) z = __fsub_rn(__fsub_rn(z, __fmul_rn(freq, (float)(c & 0x7fffffffu))), pres);
        z = __fadd_rn(z, bias[k]);
        if (allowed && !((allowed[id >> 5] >> (id & 31)) & 1u)) z = -INFINITY;
        bias[k] = z;
        const float top = fmaxf(z, -INFINITY);  // NaN is never the maximum
        best = join(best, Best{top, top > -INFINITY ? 1.f : isnan(z) ? z : 0.f, top > -INFINITY ? id : kNoToken});
      }
      if ((const void*)z_out == (const void*)z_in) __syncthreads();  // before anything is written over
    }

    auto process = [&](int w, Eight<T>& raw, uint32_t m0, uint32_t m1) {
      const int64_t id0 = (int64_t)w * 8 - shift;
      const int i0 = (w - v0) * 8;
      const bool inside_row = inner(w);
      uint32_t open = inside_row ? __funnelshift_r(m0, m1, id0 & 31) : m0;
      float to[8], *x = raw.values(to);
      if (marks) open &= ~(bitmap[i0 >> 5] >> (i0 & 31));
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (!((open >> i) & 1u)) x[i] = -INFINITY;
        top = fmaxf(top, x[i]);
      }
      if (z_out) {
        if (wide_out && inside_row) {
          store8(z_out + id0, x);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (id0 + i >= 0 && id0 + i < a.vocab) z_out[id0 + i] = x[i];
        }
      }
      if (top >= best.m && top > -INFINITY) {
        best.sum *= rescale(best.m, top);
        int id = kNoToken;  // the first of equal maxima
#pragma unroll
        for (int i = 7; i >= 0; --i)
          if (x[i] == top) id = (int)id0 + i;
        best.id = top == best.m ? min(best.id, id) : id;
        best.m = top;
      }
      const float off = isinf(best.m) ? 0.f : best.m;  // of an infinite maximum: sums of infinities, as log-sum-exp has them
#pragma unroll
      for (int i = 0; i < 8; ++i) best.sum += exp_fast(x[i] - off);
    };
    if constexpr (kAhead) {
      Eight<T> raw2;
      uint32_t n0, n1;
      if (v0 + tid + kThreads < v1) load(v0 + tid + kThreads, raw2, n0, n1);
      for (int w = v0 + tid; w < v1; w += 2 * kThreads) {
        process(w, raw, m0, m1);
        if (w + 2 * kThreads < v1) load(w + 2 * kThreads, raw, m0, m1);
        if (w + kThreads < v1) {
          process(w + kThreads, raw2, n0, n1);
          if (w + 3 * kThreads < v1) load(w + 3 * kThreads, raw2, n0, n1);
        }
      }
    } else {
      for (int w = v0 + tid; w < v1; w += kThreads) {
        if (w > v0 + tid) load(w, raw, m0, m1);
        process(w, raw, m0, m1);
      }
    }
    if (marks && z_out) {
      __syncthreads();
      for (uint32_t k = tid; k < marked; k += kThreads) z_out[first + where[k]] = bias[k];
    }
    if (v1 < u1) __syncthreads();
  }

#pragma unroll
  for (int w = 16; w > 0; w >>= 1)
    best = join(best, Best{__shfl_xor_sync(0xffffffffu, best.m, w), __shfl_xor_sync(0xffffffffu, best.sum, w), __shfl_xor_sync(0xffffffffu, best.id, w)});
  if (bad) set_status(a.status, GPT_STATUS_BAD_TOKEN);
  if (lane == 0) warp_best[warp] = best;
  __syncthreads();
  if (tid == 0)
    for (int w = 1; w < kWarps; ++w) best = join(best, warp_best[w]);
  if (blocks > 1) {
    asm volatile("barrier.cluster.wait;" ::: "memory");
    if (tid == 0) cluster.map_shared_rank(block_best, 0)[part] = best;
    cluster.sync();
    if (part > 0) return;
    if (tid == 0)
      for (int r = 1; r < blocks; ++r) best = join(best, block_best[r]);
  }
  if (tid == 0) {
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
  if (a->max_history > (1 << 30) || a->n_bias > (1 << 30) || a->vocab > (1 << 30))
    return call_error(GPT_ERR_UNSUPPORTED, "max_history, n_bias and vocab must not exceed 2^30");
  if (a->rows == 0) return GPT_OK;
  if (!a->out && !a->token && !a->lse) return call_error(GPT_ERR_INVALID_ARG, "out, token and lse are all NULL");
  if (!a->logits) return call_error(GPT_ERR_INVALID_ARG, "logits must be non-NULL");
  if (reinterpret_cast<uintptr_t>(a->logits) % elem_size(a->dtype) || reinterpret_cast<uintptr_t>(a->out) % 4)
    return call_error(GPT_ERR_INVALID_ARG, "logits and out must lie on their elements' boundaries");
  auto narrow = [&](int64_t stride, int64_t width) { return a->rows > 1 && stride != 0 && stride < width; };  // 0: all rows read the same
  if (narrow(a->logits_stride, a->vocab) || (a->out && a->rows > 1 && a->out_stride < a->vocab) ||
      (a->history && narrow(a->history_stride, a->max_history)) || (a->bias_ids && narrow(a->bias_stride, a->n_bias)) ||
      (a->allowed && narrow(a->allowed_stride, (a->vocab + 31) / 32)))
    return call_error(GPT_ERR_INVALID_ARG, "a row stride is smaller than its row");
  if (!a->history && (a->history_lens || a->prompt_lens))
    return call_error(GPT_ERR_INVALID_ARG, "history_lens and prompt_lens go with history");
  if ((a->bias_ids != nullptr) != (a->bias_values != nullptr))
    return call_error(GPT_ERR_INVALID_ARG, "bias_ids and bias_values go together");
  if ((const void*)a->out == a->logits && (a->dtype != GPT_DTYPE_FP32 || (a->rows > 1 && a->out_stride != a->logits_stride)))
    return call_error(GPT_ERR_INVALID_ARG, "in place needs fp32 logits and equal strides");
  // Blocks of a row, a power of two of 512 ids at least each.  Up to two blocks an SM (304
  // on 152 SMs) more blocks are better (one row of 50,304 13, 10 and 9 us in clusters of 2,
  // 4 and 8); up to four (608), where a block keeps 8,192 ids (140 rows of 50,304 16.6 us in
  // clusters of 4, 19.5 of 2, but 64 rows 12.0 of 8, 10.7 of 4; 70 rows of 131,072 18.3 of
  // 8, 22.9 of 4).  Never a second wave, which repeats the marking of ids (200 rows of 50,304 23 us
  // in clusters of 2, 29 of 4, 35 of 8; 75 rows 12.3 of 4, 16.7 of 8: larger clusters do
  // not fill every place).
  int blocks = 1;
  auto fits = [&](int n) {
    const int64_t all = (int64_t)a->rows * n;
    return n <= 8 && a->vocab / n >= 512 && (all <= 304 || (all <= (n == 2 ? 608 : 568) && a->vocab / n >= 8192));
  };
  while (fits(2 * blocks)) blocks *= 2;
  if ((int64_t)a->rows * blocks > INT32_MAX) return call_error(GPT_ERR_UNSUPPORTED, "too many rows");
  const dim3 grid(a->rows * blocks);
  const cudaStream_t st = (cudaStream_t)cuda_stream;
  // Two units under way where a thread has eight or more (512 rows of 131,072 112.8 us and
  // 118.8, in bf16 106 and 112; 198 of 102,855 in bf16 38.0 and 40.5); below, the registers
  // it costs weigh more (64 rows of 50,304 in clusters of 4 11.7 and 11.4).
  const bool ahead = a->vocab / blocks >= 8 * 8 * kThreads;
  auto launch = [&](auto kernel, auto ahead_kernel) {
    return launch_after("gpt_next_token", ahead ? ahead_kernel : kernel, grid, kThreads, 0, blocks, st, *a);
  };
  if (a->dtype == GPT_DTYPE_BF16) return launch(next_token_kernel<__nv_bfloat16, false>, next_token_kernel<__nv_bfloat16, true>);
  return launch(next_token_kernel<float, false>, next_token_kernel<float, true>);
}
