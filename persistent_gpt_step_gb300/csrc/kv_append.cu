// kv_append.cu — gpt_kv_append: keys and values of new tokens into a paged
// cache, keys and queries rotated on the way.
//
// Pair i of a head turns by t = p base^(-2i/R) at position p.  In turns,
// t / 2pi = p f with f = base^(-2i/R) / 2pi computed on the host in double and
// passed as two floats f_hi + f_lo.  p is split into a multiple of 2^16 and the
// rest, both exact floats; fma gives what the rounded products with f_hi leave
// over, whole turns drop out of every term exactly, and sincospi needs no further
// range reduction.  Errors in turns: f's double products 2^-49 p f, f_lo's rounding
// 2^-50 p f, and the roundings of the sums, 2^-26 each: 2^-23 below position 2^24.
// From there on the product p f_lo has whole turns as well: 2^-18 up to 2^31.  (The
// fp32 product p base^(-2i/R) would be off by 2^-25 p.)
#include <cmath>

#include "decode_ops.h"

namespace pgs {
namespace {

constexpr int kMaxPairs = 64;  // head_dim <= 128
constexpr int kMaxTokens = 8;  // of a block

struct AppendParams {
  gpt_paged_cache c;
  gpt_kv_append_args a;
  float f_hi[kMaxPairs], f_lo[kMaxPairs];
  int32_t share;  // threads of a token are the block's >> share
};

__device__ __forceinline__ float part_turn(float x) { return x - rintf(x); }

__device__ __forceinline__ void pair_angle(const AppendParams& p, int i, int pos, float* cs, float* sn) {
  const float hi = (float)(pos & ~0xffff), lo = (float)(pos & 0xffff);
  const float f = p.f_hi[i], a = hi * f, b = lo * f;
  const float rest = part_turn(fmaf(hi, f, -a)) + fmaf(lo, f, -b) + (float)pos * p.f_lo[i];
  const float t = part_turn(part_turn(a) + part_turn(b)) + rest;
  sincospif(2.0f * t, sn, cs);
}

// Bound: HBM (every element is read and written once).  A block has one token, or up to
// 8 where these are small, each with a part of its threads.  A token's
// sines and cosines are computed once for all of its heads, a pair a thread: with a
// thread's own four pairs instead 32,768 tokens of 32 + 8 + 8 heads of 128 took 165 us
// (the sincospi), without any rotation 120; now 127, 6.3 TB/s.  A thread has one
// 16-byte piece of the head, and every kThreads / pieces-th row of the token's q, k and
// v heads, kUnroll of them in flight.
template <typename T, int kThreads, int kUnroll, bool kShared>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kN = Piece<T>::kN;
  __shared__ __align__(16) float2 turns[kShared ? kMaxTokens : 1][kMaxPairs];  // cosine, sine
  const gpt_paged_cache& c = p.c;
  const gpt_kv_append_args& a = p.a;
  after_stream();
  const int share = kShared ? p.share : 0, threads = kThreads >> share;
  const int tid = threadIdx.x % threads, sub = threadIdx.x / threads;
  float2* turn = turns[sub];
  const int64_t n = ((int64_t)blockIdx.x << share) + sub;
  const int s = kShared && n >= a.n_tokens ? -1 : a.seq ? a.seq[n] : (int)n;
  if (!kShared && s < 0) return;
  const int pieces = c.head_dim / kN, groups = threads / pieces;
  const int group = tid / pieces, e = tid % pieces * kN;
  const int rows = a.n_head + 2 * c.n_kv_head;  // q heads, k heads, v heads
  uint4 u[kUnroll];
  auto load = [&](int row0) {
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      int row = row0 + i * groups;
      if (group >= groups || row >= rows) continue;
      const T* from;
      if (row < a.n_head) from = (const T*)a.q + n * a.q_row + row * a.q_head;
      else if ((row -= a.n_head) < c.n_kv_head) from = (const T*)a.k + n * a.k_row + row * a.k_head;
      else from = (const T*)a.v + n * a.v_row + (row - c.n_kv_head) * a.v_head;
      u[i] = __ldcs(reinterpret_cast<const uint4*>(from + e));
    }
  };
  int pos = 0, page = -1;
  if (s >= 0) {  // not padding
    pos = a.positions[n];
    load(group);  // under way while the page is looked up
    const bool bad_seq = s >= c.n_seq;
    const bool bad_pos = pos < 0 || pos >= c.max_pages * c.page_size;
    if (!bad_seq && !bad_pos) page = c.page_table[s * c.table_stride + pos / c.page_size];
    for (int i = tid; i < a.rope_dims / 2; i += threads) {
      pair_angle(p, i, pos, &turn[i].x, &turn[i].y);
      if (!kShared) break;  // at most 64 pairs
    }
    if (page < 0 || page >= c.n_pages) {
      if (tid == 0) set_status(a.status, bad_seq ? GPT_STATUS_BAD_SEQ : bad_pos ? GPT_STATUS_BAD_POS : GPT_STATUS_BAD_PAGE);
      page = -1;
      if (!kShared) return;
    }
  }
  __syncthreads();
  if (kShared && page < 0) return;
  const int64_t slot = page * c.page_stride + (pos % c.page_size) * c.slot_stride;
  for (int row0 = group; group < groups && row0 < rows; row0 += kUnroll * groups) {
    if (row0 > group) load(row0);
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      int row = row0 + i * groups;
      if (row >= rows) break;
      if (row < a.n_head + c.n_kv_head && e < a.rope_dims) {
        float x[kN];
        Piece<T>::unpack(u[i], x);
#pragma unroll
        for (int j = 0; j < kN / 2; ++j)
          if (e + 2 * j < a.rope_dims) {
            const float2 t = turn[e / 2 + j];
            const float x0 = x[2 * j], x1 = x[2 * j + 1];
            x[2 * j] = x0 * t.x - x1 * t.y;
            x[2 * j + 1] = x0 * t.y + x1 * t.x;
          }
        u[i] = Piece<T>::pack(x);
      }
      T* to;
      if (row < a.n_head) to = (T*)a.q_out + n * a.qo_row + row * a.qo_head;
      else if ((row -= a.n_head) < c.n_kv_head) to = (T*)c.k + slot + row * c.head_stride;
      else to = (T*)c.v + slot + (row - c.n_kv_head) * c.head_stride;
      *reinterpret_cast<uint4*>(to + e) = u[i];
    }
  }
}

}  // namespace
}  // namespace pgs

using namespace pgs;

extern "C" int gpt_kv_append(const gpt_paged_cache* c, const gpt_kv_append_args* a, void* cuda_stream) {
  clear_call_error();
  if (const int rc = check_cache(c)) return rc;
  if (!a) return call_error(GPT_ERR_INVALID_ARG, "args must be non-NULL");
  const int es = elem_size(c->dtype);
  if (a->n_tokens < 0 || a->n_head < 0) return call_error(GPT_ERR_INVALID_ARG, "n_tokens and n_head must not be negative");
  if (a->rope_dims < 0 || a->rope_dims > c->head_dim || (a->rope_dims & 1))
    return call_error(GPT_ERR_INVALID_ARG, "rope_dims %d: even, from 0 to head_dim %d", a->rope_dims, c->head_dim);
  if (a->rope_dims > 0 && !(a->rope_base >= 1 && std::isfinite(a->rope_base)))
    return call_error(GPT_ERR_INVALID_ARG, "rope_base must be finite and at least 1");
  if (a->n_head > kMostHeads) return call_error(GPT_ERR_UNSUPPORTED, "n_head %d: at most %d", a->n_head, kMostHeads);
  if (a->n_tokens == 0) return GPT_OK;
  if (c->n_seq == 0) return call_error(GPT_ERR_INVALID_ARG, "the cache has no sequences");
  if (!a->k || !a->v || !a->positions) return call_error(GPT_ERR_INVALID_ARG, "k, v and positions must be non-NULL");
  if (!a->seq && a->n_tokens > c->n_seq)
    return call_error(GPT_ERR_INVALID_ARG, "%d tokens without seq, but %d sequences", a->n_tokens, c->n_seq);
  if (!aligned16(a->k) || !aligned16(a->v) || !stride16(a->k_row, es) || !stride16(a->k_head, es) ||
      !stride16(a->v_row, es) || !stride16(a->v_head, es))
    return call_error(GPT_ERR_INVALID_ARG, "k and v addresses and strides must be multiples of 16 bytes");
  if ((a->n_head > 0) != (a->q != nullptr) || (a->n_head > 0) != (a->q_out != nullptr))
    return call_error(GPT_ERR_INVALID_ARG, "q and q_out go with n_head > 0, and only with it");
  if (a->n_head > 0 && (!aligned16(a->q) || !aligned16(a->q_out) || !stride16(a->q_row, es) || !stride16(a->q_head, es) ||
                        !stride16(a->qo_row, es) || !stride16(a->qo_head, es)))
    return call_error(GPT_ERR_INVALID_ARG, "q and q_out addresses and strides must be multiples of 16 bytes");
  if (!apart({{c->page_stride, c->n_pages}, {c->slot_stride, c->page_size}, {c->head_stride, c->n_kv_head}}, c->head_dim) ||
      (a->n_head > 0 && !apart({{a->qo_row, a->n_tokens}, {a->qo_head, a->n_head}}, c->head_dim)))
    return call_error(GPT_ERR_INVALID_ARG, "strides of the cache or q_out are smaller than a head or the dimensions inside");
  if (a->n_head > 0 && a->q_out == a->q &&
      ((a->n_tokens > 1 && a->qo_row != a->q_row) || (a->n_head > 1 && a->qo_head != a->q_head)))
    return call_error(GPT_ERR_INVALID_ARG, "q_out that is q needs its strides");
  AppendParams p = {};
  p.c = *c;
  p.a = *a;
  if (a->rope_dims > 0) {
    double f[kMaxPairs] = {1.0 / 6.283185307179586476925};  // base^(-2i/R) / 2pi, at most six products each
    const int pairs = a->rope_dims / 2;
    for (int n = 1; n < pairs; n *= 2) {
      const double step = std::pow(a->rope_base, -2.0 * n / a->rope_dims);
      for (int i = n; i < pairs && i < 2 * n; ++i) f[i] = f[i - n] * step;
    }
    for (int i = 0; i < pairs; ++i) p.f_hi[i] = (float)f[i], p.f_lo[i] = (float)(f[i] - (double)p.f_hi[i]);
  }
  const cudaStream_t st = (cudaStream_t)cuda_stream;
  // Few tokens: more threads each, for the latency (256 tokens of 48 heads of 128: 3.8
  // us with 256 threads, 4.4 with 128); many: fewer, for the throughput (32,768: 129 us
  // with 128, 149 with 256).  608: four blocks on each of the GPU's 152 SMs, here and below.
  const bool few = a->n_tokens <= 608;
  // Small tokens: as many to a block as its threads keep in flight and as leave four
  // blocks an SM (20,471 tokens of 2 + 1 + 1 heads of 96 8.0 us, one to a block 26; 7,880
  // of 16 + 4 + 4 of 32 5.1 and 11.4; 16,384 of 12 + 12 + 12 of 64 31.6 and 36.8; with
  // half as many in flight 43).  Its own kernel, for the registers: with a variable share
  // the large tokens above take 136 us.
  const int pieces = c->head_dim * es / 16, work = (a->n_head + 2 * c->n_kv_head) * pieces;
  p.share = 0;
  while (!few && (1 << p.share) < kMaxTokens && (work << (p.share + 1)) <= 128 * 6 && (128 >> (p.share + 1)) >= pieces &&
         (a->n_tokens >> (p.share + 1)) >= 608)
    ++p.share;
  const dim3 grid((unsigned)(((int64_t)a->n_tokens + (1 << p.share) - 1) >> p.share));
  auto launch = [&](auto few_kernel, auto many_kernel, auto shared_kernel) {
    return launch_after("gpt_kv_append", few ? few_kernel : p.share ? shared_kernel : many_kernel, grid, few ? 256 : 128, 0, 0, st, p);
  };
  if (c->dtype == GPT_DTYPE_BF16)
    return launch(kv_append_kernel<__nv_bfloat16, 256, 3, false>, kv_append_kernel<__nv_bfloat16, 128, 6, false>,
                  kv_append_kernel<__nv_bfloat16, 128, 6, true>);
  return launch(kv_append_kernel<float, 256, 3, false>, kv_append_kernel<float, 128, 6, false>, kv_append_kernel<float, 128, 6, true>);
}
