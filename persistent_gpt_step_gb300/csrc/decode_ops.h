// decode_ops.h — what the operators of a batched decode step (kv_append.cu,
// decode_attention.cu, next_token.cu) share: error texts, argument checks, the
// device view of a paged cache and element conversions.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "../../include/gpt.h"

namespace pgs {

// Sets the calling thread's handle-less error text (gpt_last_error(NULL)) and returns code.
int call_error(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
void clear_call_error();

inline int elem_size(int32_t dtype) { return dtype == GPT_DTYPE_BF16 ? 2 : 4; }

// A base address on a 16-byte boundary.
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
// A stride (elements of es bytes) that keeps 16-byte alignment and is not negative.
inline bool stride16(int64_t s, int es) { return s >= 0 && (s * es) % 16 == 0; }
// A written dimension: its stride and its entries.
struct Dim { int64_t stride, n; };
// No two indices of these dimensions of rows of `width` name one element: from the smallest
// stride on, each is at least what the dimensions before it take up.  (Doubles: exact up to
// 2^53 elements.)
inline bool apart(std::initializer_list<Dim> dims, int64_t width) {
  Dim d[3];
  size_t n = 0;
  for (const Dim& x : dims)
    if (x.n > 1) d[n++] = x;
  std::sort(d, d + n, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  double extent = (double)width;
  for (size_t i = 0; i < n; ++i) {
    if ((double)d[i].stride < extent) return false;
    extent += (double)d[i].stride * (double)(d[i].n - 1);
  }
  return true;
}
constexpr int kMostHeads = 1 << 16;  // head counts and their products stay in 32 bits

// GPT_OK, or the refusal of a cache that the header does not allow.
inline int check_cache(const gpt_paged_cache* c) {
  if (!c) return call_error(GPT_ERR_INVALID_ARG, "cache must be non-NULL");
  if (c->dtype != GPT_DTYPE_FP32 && c->dtype != GPT_DTYPE_BF16)
    return call_error(GPT_ERR_INVALID_ARG, "cache dtype must be GPT_DTYPE_FP32 or GPT_DTYPE_BF16");
  if (c->n_pages < 1 || c->page_size < 1 || c->n_seq < 0 || c->max_pages < 1 || c->n_kv_head < 1 || c->head_dim < 1)
    return call_error(GPT_ERR_INVALID_ARG, "cache sizes must be positive");
  const int es = elem_size(c->dtype);
  if (c->n_kv_head > kMostHeads) return call_error(GPT_ERR_UNSUPPORTED, "n_kv_head %d: at most %d", c->n_kv_head, kMostHeads);
  if (c->head_dim > 128 || (c->head_dim * es) % 16)
    return call_error(GPT_ERR_UNSUPPORTED, "head_dim %d: a multiple of 16 bytes, at most 128 elements", c->head_dim);
  if ((int64_t)c->max_pages * c->page_size > INT32_MAX - 4096)  // tiles that end past the last position still count in 32 bits
    return call_error(GPT_ERR_UNSUPPORTED, "max_pages * page_size must stay 4096 below 2^31 for 32 bits");
  if (c->n_seq == 0) return GPT_OK;
  if (!c->k || !c->v || !c->page_table) return call_error(GPT_ERR_INVALID_ARG, "cache pointers must be non-NULL");
  if (!aligned16(c->k) || !aligned16(c->v) || !stride16(c->page_stride, es) || !stride16(c->slot_stride, es) ||
      !stride16(c->head_stride, es))
    return call_error(GPT_ERR_INVALID_ARG, "cache addresses and strides must be multiples of 16 bytes");
  if (c->table_stride < c->max_pages && c->table_stride != 0 && c->n_seq > 1)
    return call_error(GPT_ERR_INVALID_ARG, "table_stride is smaller than max_pages");
  return GPT_OK;
}

// What a CUDA call of ours returned; its error does not stay for the caller's next cudaGetLastError.
inline int check_cuda(const char* what, cudaError_t e) {
  if (e == cudaSuccess) return GPT_OK;
  cudaGetLastError();
  return call_error(GPT_ERR_CUDA, "%s: launch failed: %s", what, cudaGetErrorString(e));
}

#ifdef __CUDACC__
// Launches an operator's kernel with programmatic stream serialization: its blocks may
// take their places while the kernel before it in the stream ends, and wait in
// after_stream() for that kernel's completion.  `cluster` blocks to a cluster, if not 0.
template <typename... P>
inline int launch_after(const char* what, void (*kernel)(P...), dim3 grid, int threads, int smem, int cluster, cudaStream_t st,
                        std::common_type_t<P>... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid, cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = smem, cfg.stream = st;
  cfg.attrs = attr, cfg.numAttrs = cluster ? 2 : 1;
  return check_cuda(what, cudaLaunchKernelEx(&cfg, kernel, args...));
}
// Every thread's first statement, before any access to memory that another kernel
// writes or reads.  The kernels do not let their successors in early themselves: with
// that, the successor's blocks crowd the SMs that are done first (next token of 33 rows
// 20.7 us instead of 14.4; 16.5 without any of this).
__device__ __forceinline__ void after_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void set_status(uint32_t* status, uint32_t bit) {
  if (status) atomicOr(status, bit);
}

// A 16-byte piece of a row as floats, and back (one rounding).
template <typename T> struct Piece;
template <> struct Piece<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const uint4& u, float* x) {
    x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <> struct Piece<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& u, float* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
#endif

}  // namespace pgs
