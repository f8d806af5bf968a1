// sample_token.cu — gpt_sample_token: a token drawn from a row of logits with
// temperature, top-k, top-p and min-p, from a given number.
//
// Weights are integers: w = round(2^U exp((z - m) / T)), U such that a row's sum fits 64
// bits.  Sums of integers are the same in any order, so every limit (a count or a sum over
// the tokens above a value) and the draw itself (a running sum by id) are exact, whatever
// threads add.  All three limits keep a prefix of the tokens in order of falling z, so the
// kept ones are those above a key, and the first few, by id, of those that have it.
#include <cmath>

#include "decode_ops.h"

namespace pgs {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
using u64 = unsigned long long;

struct SampleParams {
  gpt_sample_token_args a;
  int32_t unit;  // U
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// Ascends with z; 0: no token.  Both zeros are one value.
__device__ __forceinline__ uint32_t key_of(float z) {
  if (!(z > -INFINITY)) return 0u;
  const uint32_t b = __float_as_uint(z + 0.f);
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) { return __uint_as_float(key >> 31 ? key & 0x7fffffffu : ~key); }

struct Row {
  float m;        // the largest z
  double c;       // log2 e / T
  int unit;
  __device__ __forceinline__ u64 weight(uint32_t key) const {
    const float z = value_of(key);
    if (z == m) return 1ull << unit;
    if (m == INFINITY) return 0ull;
    return __double2ull_rn(exp2(((double)z - (double)m) * c + unit));
  }
};

// The least integer that is at least f x, the largest that is at most f x, for 0 <= f < 1.
__device__ __forceinline__ u64 part_of(float f, u64 x, bool up) {
  const uint32_t b = __float_as_uint(f), e = b >> 23;
  const uint32_t mant = e ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
  const int shift = 150 - (int)(e ? e : 1);  // f = mant 2^-shift
  const unsigned __int128 p = (unsigned __int128)mant * x;
  if (shift >= 100) return up && mant && x ? 1 : 0;
  const u64 q = (u64)(p >> shift);
  return q + (up && (p & (((unsigned __int128)1 << shift) - 1)) != 0);
}

template <typename V, typename Op>
__device__ __forceinline__ V block_reduce(V v, V* scratch, Op op) {
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, x));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  v = scratch[threadIdx.x & 31];
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, x));
  return v;
}
__device__ __forceinline__ u64 add(u64 a, u64 b) { return a + b; }

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_token_kernel(const __grid_constant__ SampleParams p) {
  __shared__ u64 scratch[kWarps], mass[256];
  __shared__ uint32_t count[256];
  __shared__ struct { uint32_t key; u64 rest; } found;
  const gpt_sample_token_args& a = p.a;
  after_stream();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x;
  const T* z = (const T*)a.logits + b * a.logits_stride;
  auto key_at = [&](int i) { return key_of(to_float(z[i])); };

  // the first token in order: the largest key, of these the smallest id
  u64 best = 0, there = 0;
  for (int i = tid; i < a.vocab; i += kThreads) {
    const uint32_t key = key_at(i);
    if (key) best = max(best, (u64)key << 32 | ~(uint32_t)i), ++there;
  }
  best = block_reduce(best, scratch, [](u64 x, u64 y) { return max(x, y); });
  there = block_reduce(there, scratch, add);
  auto answer = [&](int token, float logprob, int kept) {
    if (tid > 0) return;
    if (a.token) a.token[b] = token;
    if (a.logprob) a.logprob[b] = logprob;
    if (a.kept) a.kept[b] = kept;
  };
  if (there == 0) return answer(-1, -INFINITY, 0);
  const float temperature = a.temperature ? a.temperature[b] : 1.f;
  if (!(temperature > 0.f)) return answer((int)~(uint32_t)best, 0.f, 1);
  const uint32_t top_key = (uint32_t)(best >> 32);
  const Row row{value_of(top_key), 1.4426950408889634 / (double)temperature, p.unit};

  // The prefix of `target` tokens, or of the least weight of at least that: its last key,
  // and how many tokens have that key in it (as many as it takes).
  auto select = [&](bool by_mass, u64 target) {
    uint32_t prefix = 0;
    u64 rest = target;
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kThreads) mass[i] = 0, count[i] = 0;
      __syncthreads();
      for (int i = tid; i < a.vocab; i += kThreads) {
        const uint32_t key = key_at(i);
        if (key == 0 || (shift < 24 && key >> (shift + 8) != prefix)) continue;
        if (by_mass) atomicAdd(&mass[key >> shift & 255u], row.weight(key));
        else atomicAdd(&count[key >> shift & 255u], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        int i = 255;
        for (; i > 0; --i) {
          const u64 here = by_mass ? mass[i] : count[i];
          if (here >= rest && here > 0) break;
          rest -= here;
        }
        found.key = prefix << 8 | (uint32_t)i, found.rest = rest;
      }
      __syncthreads();
      prefix = found.key, rest = found.rest;
      __syncthreads();
    }
    if (by_mass) {
      const u64 w = row.weight(prefix);
      rest = w ? (rest + w - 1) / w : 1;
    }
    found.key = prefix, found.rest = max(rest, 1ull);  // (by all threads alike)
    __syncthreads();
  };
  // Of the tokens with key > last, and the first `ties` of those with last: their weights' sum.
  uint32_t last = 1;
  u64 ties = there;
  auto sum_kept = [&] {
    u64 sum = 0, equal = 0;
    for (int i = tid; i < a.vocab; i += kThreads) {
      const uint32_t key = key_at(i);
      if (key > last) sum += row.weight(key);
      else if (key == last) ++equal;
    }
    sum = block_reduce(sum, scratch, add);
    equal = block_reduce(equal, scratch, add);
    ties = min(ties, equal);
    return sum + (ties ? ties * row.weight(last) : 0);
  };
  const int top_k = a.top_k ? a.top_k[b] : 0;
  const float top_p = a.top_p ? a.top_p[b] : 1.f, min_p = a.min_p ? a.min_p[b] : 0.f;
  if (top_k >= 1 && top_k < there) {
    select(false, top_k);
    last = found.key, ties = found.rest;
  }
  if (top_p < 1.f) {
    const u64 target = top_p > 0.f ? part_of(top_p, sum_kept(), true) : 0;
    if (target > 0) {
      select(true, target);
      last = found.key, ties = found.rest;
    } else {
      last = top_key, ties = 1;
    }
  }
  if (min_p > 1.f) {
    last = top_key, ties = 1;
  } else if (min_p > 0.f) {
    const float least = row.m == INFINITY ? row.m : __double2float_ru((double)row.m + log((double)min_p) * (double)temperature);
    const uint32_t key = min(key_of(least), top_key);
    if (key > last) last = key, ties = there;
  }
  const u64 sum = sum_kept();

  // the draw: tiles of kThreads ids in order
  const float u = a.uniform[b];
  const u64 target = u >= 1.f ? sum : (u > 0.f ? part_of(u, sum, false) : 0) + 1;
  u64 before = 0, equal_before = 0, kept = 0;
  __shared__ int chosen;
  __shared__ uint32_t chosen_key;
  if (tid == 0) chosen = -1;
  for (int i0 = 0; i0 < a.vocab; i0 += kThreads) {
    const uint32_t key = i0 + tid < a.vocab ? key_at(i0 + tid) : 0u;
    auto scan = [&](u64 v, u64& total) {  // the sum of v over the threads up to this one
      u64 x = v;
#pragma unroll
      for (int y = 1; y < 32; y <<= 1) {
        const u64 t = __shfl_up_sync(0xffffffffu, x, y);
        if (lane >= y) x += t;
      }
      __syncthreads();
      if (lane == 31) scratch[warp] = x;
      __syncthreads();
      total = 0;
      u64 below = 0;
      for (int w = 0; w < kWarps; ++w) {
        if (w == warp) below = total;
        total += scratch[w];
      }
      return below + x;
    };
    u64 total;
    const u64 rank = scan(key == last && key, total) + equal_before;
    equal_before += total;
    const bool in = key > last || (key == last && key && rank <= ties);
    const u64 w = in ? row.weight(key) : 0;
    const u64 upto = scan(w, total) + before;
    if (w && upto >= target && upto - w < target) chosen = i0 + tid, chosen_key = key;
    before += total;
    scan(in, total);
    kept += total;
  }
  __syncthreads();
  answer(chosen, tid == 0 ? (float)log((double)row.weight(chosen_key) / (double)sum) : 0.f, (int)kept);
}

}  // namespace
}  // namespace pgs

using namespace pgs;

extern "C" int gpt_sample_token(const gpt_sample_token_args* a, void* cuda_stream) {
  clear_call_error();
  if (!a) return call_error(GPT_ERR_INVALID_ARG, "args must be non-NULL");
  if (a->dtype != GPT_DTYPE_FP32 && a->dtype != GPT_DTYPE_BF16)
    return call_error(GPT_ERR_INVALID_ARG, "dtype must be GPT_DTYPE_FP32 or GPT_DTYPE_BF16");
  if (a->rows < 0 || a->vocab < 1) return call_error(GPT_ERR_INVALID_ARG, "rows must not be negative, vocab must be positive");
  if (a->vocab > (1 << 30)) return call_error(GPT_ERR_UNSUPPORTED, "vocab must not exceed 2^30");
  if (a->rows == 0) return GPT_OK;
  if (!a->token && !a->logprob && !a->kept) return call_error(GPT_ERR_INVALID_ARG, "token, logprob and kept are all NULL");
  if (!a->logits || !a->uniform) return call_error(GPT_ERR_INVALID_ARG, "logits and uniform must be non-NULL");
  if (reinterpret_cast<uintptr_t>(a->logits) % elem_size(a->dtype))
    return call_error(GPT_ERR_INVALID_ARG, "logits must lie on their elements' boundaries");
  if (a->rows > 1 && a->logits_stride != 0 && a->logits_stride < a->vocab)
    return call_error(GPT_ERR_INVALID_ARG, "a row stride is smaller than its row");
  SampleParams p;
  p.a = *a;
  p.unit = 48;
  while (((int64_t)a->vocab << p.unit) < 0 || ((int64_t)a->vocab << p.unit) >> p.unit != a->vocab) --p.unit;
  const cudaStream_t st = (cudaStream_t)cuda_stream;
  return launch_after("gpt_sample_token", a->dtype == GPT_DTYPE_BF16 ? sample_token_kernel<__nv_bfloat16> : sample_token_kernel<float>,
                      dim3(a->rows), kThreads, 0, 0, st, p);
}
