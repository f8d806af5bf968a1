// decode_attention.cu — gpt_decode_attention: attention of one new token of
// every sequence over its pages of keys and values.
#include <cmath>

#include "decode_ops.h"

namespace pgs {
namespace {

constexpr int kWarps = 4;

struct DecodeParams {
  gpt_paged_cache c;
  gpt_decode_attention_args a;
};

// exp(x - m) for x <= m; nothing from x = -infinity, whatever m is.
__device__ __forceinline__ float weight(float x, float m) { return x == -INFINITY ? 0.f : __expf(x - m); }

// One block per (sequence, query head); a warp per key in turn, one running
// softmax (max m, sum l, weighted values o) per warp, the warps joined at the end.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) decode_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int kN = Piece<T>::kN;
  const gpt_paged_cache& c = p.c;
  const gpt_decode_attention_args& a = p.a;
  const int64_t s = blockIdx.y;
  const int h = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t head = (int64_t)(h / (a.n_head / c.n_kv_head)) * c.head_stride;
  int len = a.lens[s];
  const int most = c.max_pages * c.page_size;
  if (len < 0 || len > most) {
    if (threadIdx.x == 0) set_status(a.status, GPT_STATUS_BAD_POS);
    len = len < 0 ? 0 : most;
  }
  const bool mine = lane * kN < c.head_dim;  // head_dim <= 128: one piece per lane
  float q[kN], o[kN], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < kN; ++i) q[i] = o[i] = 0.f;
  if (mine)
    Piece<T>::unpack(*reinterpret_cast<const uint4*>((const T*)a.q + s * a.q_row + h * a.q_head + lane * kN), q);
  for (int j = warp; j < len; j += kWarps) {
    const int page = c.page_table[s * c.table_stride + j / c.page_size];
    if (page < 0 || page >= c.n_pages) {
      if (lane == 0) set_status(a.status, GPT_STATUS_BAD_PAGE);
      continue;
    }
    const int64_t at = page * c.page_stride + (j % c.page_size) * c.slot_stride + head + lane * kN;
    float x[kN], z = 0.f;
    if (mine) {
      Piece<T>::unpack(*reinterpret_cast<const uint4*>((const T*)c.k + at), x);
#pragma unroll
      for (int i = 0; i < kN; ++i) z += q[i] * x[i];
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) z += __shfl_xor_sync(0xffffffffu, z, w);
    z *= a.scale;
    const float top = fmaxf(m, z), keep = weight(m, top), e = weight(z, top);
    m = top;
    l = l * keep + e;
    if (mine) {
      Piece<T>::unpack(*reinterpret_cast<const uint4*>((const T*)c.v + at), x);
#pragma unroll
      for (int i = 0; i < kN; ++i) o[i] = o[i] * keep + e * x[i];
    }
  }
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][128];
  if (lane == 0) sm[warp] = m, sl[warp] = l;
  if (mine)
#pragma unroll
    for (int i = 0; i < kN; ++i) so[warp][lane * kN + i] = o[i];
  __syncthreads();
  if (warp == 0) {
    float top = sm[0], total = 0.f;
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sm[w]);
#pragma unroll
    for (int i = 0; i < kN; ++i) o[i] = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      const float keep = weight(sm[w], top);
      total += sl[w] * keep;
      if (mine)
#pragma unroll
        for (int i = 0; i < kN; ++i) o[i] += so[w][lane * kN + i] * keep;
    }
    if (mine) {
#pragma unroll
      for (int i = 0; i < kN; ++i) o[i] = total == 0.f ? 0.f : o[i] / total;
      *reinterpret_cast<uint4*>((T*)a.out + s * a.out_row + h * a.out_head + lane * kN) = Piece<T>::pack(o);
    }
    if (lane == 0 && a.lse) a.lse[s * a.n_head + h] = total == 0.f ? -INFINITY : top + logf(total);
  }
}

int check_args(const gpt_paged_cache* c, int32_t n_head) {
  if (const int rc = check_cache(c)) return rc;
  if (n_head < 1 || n_head % c->n_kv_head)
    return call_error(GPT_ERR_INVALID_ARG, "n_head %d must be a multiple of n_kv_head %d", n_head, c->n_kv_head);
  return GPT_OK;
}

}  // namespace
}  // namespace pgs

using namespace pgs;

extern "C" size_t gpt_decode_attention_workspace(const gpt_paged_cache* c, int32_t n_head) {
  clear_call_error();
  return 0;
}

extern "C" int gpt_decode_attention(const gpt_paged_cache* c, const gpt_decode_attention_args* a, void* cuda_stream) {
  clear_call_error();
  if (!a) return call_error(GPT_ERR_INVALID_ARG, "args must be non-NULL");
  if (const int rc = check_args(c, a->n_head)) return rc;
  if (c->n_seq == 0) return GPT_OK;
  const int es = elem_size(c->dtype);
  if (!a->q || !a->out || !a->lens) return call_error(GPT_ERR_INVALID_ARG, "q, out and lens must be non-NULL");
  if (!aligned16(a->q) || !aligned16(a->out) || !stride16(a->q_row, es) || !stride16(a->q_head, es) ||
      !stride16(a->out_row, es) || !stride16(a->out_head, es))
    return call_error(GPT_ERR_INVALID_ARG, "q and out addresses and strides must be multiples of 16 bytes");
  if (!std::isfinite(a->scale)) return call_error(GPT_ERR_INVALID_ARG, "scale must be finite");
  if (c->n_seq > 65535) return call_error(GPT_ERR_UNSUPPORTED, "at most 65535 sequences");
  const DecodeParams p{*c, *a};
  const dim3 grid(a->n_head, c->n_seq);
  const cudaStream_t st = (cudaStream_t)cuda_stream;
  if (c->dtype == GPT_DTYPE_BF16) decode_kernel<__nv_bfloat16><<<grid, kWarps * 32, 0, st>>>(p);
  else decode_kernel<float><<<grid, kWarps * 32, 0, st>>>(p);
  return check_launch("gpt_decode_attention");
}
