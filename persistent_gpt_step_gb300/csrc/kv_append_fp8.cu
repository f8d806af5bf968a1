// kv_append_fp8.cu — gpt_kv_append_fp8: keys and values of new tokens into a paged
// cache of e4m3 numbers with a scale for each page and key head, keys and queries
// rotated on the way (rotary.h).
//
// A run: the new rows of one page.  Its scale needs the largest magnitude of all of them
// before the first number is written, so one block has a run's rows of one key head and
// side (keys or values), holds them in registers between the two passes, and owns the
// scale: no atomics on global memory, no second kernel.  The scale comes from the
// magnitudes before the rotation, which turns each pair by at most sqrt 2: it is then
// exact, the same however sines are rounded, and no number reaches 448.
// Bound: HBM (rows read once, numbers and rotated queries written once).
#include "rotary.h"

namespace pgs {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxStrip = 64;   // rows of a block's strip
constexpr int kStage = 1024;    // starts in shared memory
constexpr int kHeld = 8;        // 16-byte pieces that a thread holds
constexpr int kQueryHeld = 4;
constexpr int kMaxTokens = 8;   // of a block of query rows
constexpr int kNoRun = 255;

struct AppendParams {
  gpt_fp8_cache c;
  gpt_kv_append_fp8_args a;
  RotaryRates rates;
  int32_t strip;      // rows of a strip; a block has the runs that begin in one
  int32_t kv_blocks;  // strips x key heads x 2; the blocks behind them have query rows
  int32_t share;      // threads of a token of query rows are the block's >> share
};

// Where a row belongs.
struct Row {
  int seq, pos;       // seq < 0: nowhere
  int first, end;     // rows of its sequence
};

// Every step-th entry of starts, in shared memory.
__device__ __forceinline__ int stage_step(const AppendParams& p) { return (p.c.pages.n_seq + kStage) / kStage; }
__device__ __forceinline__ void stage_starts(const AppendParams& p, int* stage) {
  if (!p.a.starts) return;
  const int step = stage_step(p);
  for (int64_t i = threadIdx.x; i * step <= p.c.pages.n_seq; i += blockDim.x) stage[i] = p.a.starts[i * step];
}

__device__ __forceinline__ Row find_row(const AppendParams& p, const int* stage, int row, bool report) {
  const int n_seq = p.c.pages.n_seq;
  Row r{-1, 0, row, row + 1};
  int s = row;
  if (p.a.starts) {
    const int step = stage_step(p);
    int lo = 0, hi = n_seq / step + 1;  // the last entry at or before the row is in [lo - 1, hi - 1]
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (stage[mid] <= row) lo = mid + 1;
      else hi = mid;
    }
    if (lo == 0) return r;
    if (step > 1) {
      const int64_t from = (int64_t)(lo - 1) * step;
      int64_t a = from + 1, b = min(from + step, (int64_t)n_seq + 1);
      while (a < b) {
        const int64_t mid = (a + b) >> 1;
        if (p.a.starts[mid] <= row) a = mid + 1;
        else b = mid;
      }
      lo = (int)a;
    }
    s = lo - 1;
    if (s >= n_seq) return r;
    r.first = step > 1 ? p.a.starts[s] : stage[s];
    r.end = step > 1 ? p.a.starts[s + 1] : stage[s + 1];
    if (r.first < 0 || r.end > p.a.n_tokens || r.end <= row) {
      if (report) set_status(p.a.status, GPT_STATUS_BAD_SEQ);
      return r;
    }
  }
  const int before = p.a.before[s];
  if (before < 0) return r;
  const int64_t pos = (int64_t)before + (row - r.first);
  if (pos >= (int64_t)p.c.pages.max_pages * p.c.pages.page_size) {
    if (report) set_status(p.a.status, GPT_STATUS_BAD_POS);
    return r;
  }
  r.seq = s, r.pos = (int)pos;
  return r;
}

__device__ __forceinline__ int page_of(const AppendParams& p, const Row& r, bool report) {
  const gpt_paged_cache& c = p.c.pages;
  const int page = c.page_table[r.seq * c.table_stride + r.pos / c.page_size];
  if (page >= 0 && page < c.n_pages) return page;
  if (report) set_status(p.a.status, GPT_STATUS_BAD_PAGE);
  return -1;
}

// The scale that brings `top` to 2^7 up to 2^8.
__device__ __forceinline__ float scale_for(float top) {
  const int exponent = top >= 0x1p-119f ? (int)(__float_as_uint(top) >> 23) - 127 : -119;
  return __uint_as_float((uint32_t)(exponent - 7 + 127) << 23);
}

// Two numbers, rounded to nearest; what is not finite is NaN.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b) {
  uint16_t u;
  a = fabsf(a) <= 448.f ? a : NAN, b = fabsf(b) <= 448.f ? b : NAN;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(u) : "f"(b), "f"(a));
  return u;
}
__device__ __forceinline__ void unpack_e4m3(uint32_t u, float* x) {  // two
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)u));
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(x[0]), "=f"(x[1]) : "r"(h));
}

template <typename T>
__device__ __forceinline__ float largest(const uint4& u) {
  float x[Piece<T>::kN], m = 0.f;
  Piece<T>::unpack(u, x);
#pragma unroll
  for (int i = 0; i < Piece<T>::kN; ++i) m = fabsf(x[i]) < INFINITY ? fmaxf(m, fabsf(x[i])) : m;
  return m;
}

// Rotates the pairs of a piece whose first element is e of a head at position pos.
template <int N>
__device__ __forceinline__ void turn_piece(const AppendParams& p, float* x, int e, int pos) {
#pragma unroll
  for (int j = 0; j < N / 2; ++j)
    if (e + 2 * j < p.a.rope_dims) {
      float cs, sn;
      pair_angle(p.rates, e / 2 + j, pos, &cs, &sn);
      const float x0 = x[2 * j], x1 = x[2 * j + 1];
      x[2 * j] = x0 * cs - x1 * sn;
      x[2 * j + 1] = x0 * sn + x1 * cs;
    }
}

struct Run {
  int begin, end;   // rows
  int page, slot;   // of the first row; page < 0: skipped
  int pos;          // of the first row
  uint32_t top;     // largest magnitude, as bits
  float old;        // the scale that was there
  float inv, ratio; // 1 / scale, old / scale
};

template <typename T>
__device__ __forceinline__ void append_runs(const AppendParams& p, int* stage) {
  constexpr int kN = Piece<T>::kN;
  __shared__ Run runs[kMaxStrip];
  __shared__ uint8_t run_of[kMaxStrip];
  __shared__ uint32_t begins[2];
  __shared__ int rescale;
  const gpt_paged_cache& c = p.c.pages;
  const gpt_kv_append_fp8_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31;
  const int unit = blockIdx.x, sides = 2 * c.n_kv_head;
  const int strip0 = unit / sides * p.strip, side = unit % sides & 1, head = unit % sides >> 1;
  const bool report = unit % sides == 0;
  if (tid == 0) rescale = 0;
  Row r{-1, 0, 0, 0};
  if (tid < p.strip && strip0 + tid < a.n_tokens) r = find_row(p, stage, strip0 + tid, report);
  const int slot = r.pos % c.page_size;
  const bool begin = r.seq >= 0 && (strip0 + tid == r.first || slot == 0);
  if (tid < kMaxStrip) {
    const uint32_t mask = __ballot_sync(0xffffffffu, begin);
    if (lane == 0) begins[tid >> 5] = mask;
  }
  __syncthreads();
  const uint64_t mask = begins[0] | (uint64_t)begins[1] << 32;
  if (mask == 0) return;
  const int n_runs = __popcll(mask);
  float* scales = (side ? p.c.v_scale : p.c.k_scale) + head * p.c.scale_head;
  if (tid < kMaxStrip) {
    int mine = kNoRun;
    if (r.seq >= 0) {
      const int at = tid - min(slot, strip0 + tid - r.first);  // where its run begins
      if (at >= 0 && (mask >> at) & 1u) mine = __popcll(mask & ((1ull << at) - 1ull));
    }
    run_of[tid] = (uint8_t)mine;
    if (begin) {
      Run& x = runs[mine];
      x.begin = strip0 + tid, x.end = (int)min((int64_t)r.end, (int64_t)strip0 + tid + c.page_size - slot);
      x.page = page_of(p, r, report), x.slot = slot, x.pos = r.pos, x.top = 0;
      x.old = x.page >= 0 && slot > 0 ? scales[x.page * p.c.scale_page] : 0.f;
    }
  }
  __syncthreads();
  const int first = runs[0].begin, end = runs[n_runs - 1].end;
  const int pieces = c.head_dim / kN, per_pass = kThreads / pieces, window = kHeld * per_pass;
  const int group = tid / pieces, e = tid % pieces * kN;
  const T* from = side ? (const T*)a.v + head * a.v_head + e : (const T*)a.k + head * a.k_head + e;
  const int64_t stride = side ? a.v_row : a.k_row;
  auto run_at = [&](int row) {  // of a row that is to be written
    if (row >= end || group >= per_pass) return kNoRun;
    const int x = row - strip0 < p.strip ? run_of[row - strip0] : n_runs - 1;
    return x != kNoRun && runs[x].page >= 0 ? x : kNoRun;
  };
  uint4 u[kHeld];
  auto load = [&](int row0) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int row = row0 + i * per_pass + group;
      if (run_at(row) != kNoRun) u[i] = __ldcs(reinterpret_cast<const uint4*>(from + row * stride));
    }
  };
  for (int row0 = first; row0 < end; row0 += window) {
    load(row0);
    int now = kNoRun;
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int x = run_at(row0 + i * per_pass + group);
      if (x == kNoRun) continue;
      if (x != now) {
        if (now != kNoRun) atomicMax(&runs[now].top, __float_as_uint(top));
        now = x, top = 0.f;
      }
      top = fmaxf(top, largest<T>(u[i]));
    }
    __syncwarp();
    const uint32_t same = __match_any_sync(0xffffffffu, now);
    const uint32_t bits = __reduce_max_sync(same, __float_as_uint(top));
    if (now != kNoRun && lane == __ffs(same) - 1) atomicMax(&runs[now].top, bits);
  }
  __syncthreads();
  if (tid < n_runs && runs[tid].page >= 0) {
    Run& x = runs[tid];
    float scale = scale_for(__uint_as_float(x.top));
    x.ratio = 1.f;
    if (x.slot > 0) {
      scale = fmaxf(scale, x.old);
      if (scale != x.old) x.ratio = x.old / scale, rescale = 1;
    }
    x.inv = 1.f / scale;
    scales[x.page * p.c.scale_page] = scale;
  }
  __syncthreads();
  uint8_t* cache = (uint8_t*)(side ? c.v : c.k) + head * c.head_stride;
  if (rescale)
    for (int x = 0; x < n_runs; ++x) {
      if (runs[x].page < 0 || runs[x].ratio == 1.f) continue;
      const float ratio = runs[x].ratio;
      for (int i = tid; i < runs[x].slot * (c.head_dim / 16); i += kThreads) {
        uint4* at = reinterpret_cast<uint4*>(cache + runs[x].page * c.page_stride + i / (c.head_dim / 16) * c.slot_stride) + i % (c.head_dim / 16);
        uint4 v = *at;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t& w = (&v.x)[j];
          float y[4];
          unpack_e4m3(w & 0xffffu, y), unpack_e4m3(w >> 16, y + 2);
          w = pack_e4m3(y[0] * ratio, y[1] * ratio) | pack_e4m3(y[2] * ratio, y[3] * ratio) << 16;
        }
        *at = v;
      }
    }
  for (int row0 = first; row0 < end; row0 += window) {
    if (end - first > window) load(row0);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int row = row0 + i * per_pass + group, x = run_at(row);
      if (x == kNoRun) continue;
      const int into = row - runs[x].begin;
      float y[kN];
      Piece<T>::unpack(u[i], y);
#pragma unroll
      for (int j = 0; j < kN; ++j) y[j] *= runs[x].inv;
      if (side == 0) turn_piece<kN>(p, y, e, runs[x].pos + into);
      uint32_t w[kN / 4];
#pragma unroll
      for (int j = 0; j < kN / 4; ++j) w[j] = pack_e4m3(y[4 * j], y[4 * j + 1]) | pack_e4m3(y[4 * j + 2], y[4 * j + 3]) << 16;
      uint8_t* to = cache + runs[x].page * c.page_stride + (runs[x].slot + into) * c.slot_stride + e;
      if constexpr (kN == 8) *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
      else *reinterpret_cast<uint32_t*>(to) = w[0];
    }
  }
}

// Query rows: as kv_append_kernel's, a token's sines and cosines once for all of its heads.
template <typename T>
__device__ __forceinline__ void turn_queries(const AppendParams& p, const int* stage) {
  constexpr int kN = Piece<T>::kN;
  __shared__ __align__(16) float2 turns[kMaxTokens][kMaxPairs];  // cosine, sine
  const gpt_kv_append_fp8_args& a = p.a;
  const int threads = kThreads >> p.share, tid = threadIdx.x % threads, sub = threadIdx.x / threads;
  const int64_t n = ((int64_t)(blockIdx.x - p.kv_blocks) << p.share) + sub;
  Row r{-1, 0, 0, 0};
  if (n < a.n_tokens) r = find_row(p, stage, (int)n, false);
  if (r.seq >= 0 && page_of(p, r, false) < 0) r.seq = -1;
  if (r.seq >= 0)
    for (int i = tid; i < a.rope_dims / 2; i += threads) pair_angle(p.rates, i, r.pos, &turns[sub][i].x, &turns[sub][i].y);
  __syncthreads();
  if (r.seq < 0) return;
  const int pieces = p.c.pages.head_dim / kN, groups = threads / pieces, group = tid / pieces, e = tid % pieces * kN;
  if (group >= groups) return;
  const T* from = (const T*)a.q + n * a.q_row + e;
  T* to = (T*)a.q_out + n * a.qo_row + e;
  for (int h0 = group; h0 < a.n_head; h0 += kQueryHeld * groups) {
    uint4 u[kQueryHeld];
#pragma unroll
    for (int i = 0; i < kQueryHeld; ++i)
      if (h0 + i * groups < a.n_head) u[i] = __ldcs(reinterpret_cast<const uint4*>(from + (h0 + i * groups) * a.q_head));
#pragma unroll
    for (int i = 0; i < kQueryHeld; ++i) {
      if (h0 + i * groups >= a.n_head) break;
      if (e < a.rope_dims) {
        float x[kN];
        Piece<T>::unpack(u[i], x);
#pragma unroll
        for (int j = 0; j < kN / 2; ++j)
          if (e + 2 * j < a.rope_dims) {
            const float2 t = turns[sub][e / 2 + j];
            const float x0 = x[2 * j], x1 = x[2 * j + 1];
            x[2 * j] = x0 * t.x - x1 * t.y;
            x[2 * j + 1] = x0 * t.y + x1 * t.x;
          }
        u[i] = Piece<T>::pack(x);
      }
      *reinterpret_cast<uint4*>(to + (h0 + i * groups) * a.qo_head) = u[i];
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 3) kv_append_fp8_kernel(const __grid_constant__ AppendParams p) {
  __shared__ int stage[kStage];
  after_stream();
  stage_starts(p, stage);
  if (blockIdx.x == 0 && p.a.starts)
    for (int i = threadIdx.x; i < p.c.pages.n_seq; i += kThreads)
      if (p.a.starts[i] > p.a.starts[i + 1] || p.a.starts[i] < 0 || p.a.starts[i + 1] > p.a.n_tokens) set_status(p.a.status, GPT_STATUS_BAD_SEQ);
  __syncthreads();
  if (blockIdx.x < p.kv_blocks) append_runs<T>(p, stage);
  else turn_queries<T>(p, stage);
}

}  // namespace
}  // namespace pgs

using namespace pgs;

extern "C" int gpt_kv_append_fp8(const gpt_fp8_cache* cache, const gpt_kv_append_fp8_args* a, void* cuda_stream) {
  clear_call_error();
  if (const int rc = check_cache(cache, true)) return rc;
  if (!a) return call_error(GPT_ERR_INVALID_ARG, "args must be non-NULL");
  const gpt_paged_cache* c = &cache->pages;
  const int es = elem_size(c->dtype);
  if (a->n_tokens < 0 || a->n_head < 0) return call_error(GPT_ERR_INVALID_ARG, "n_tokens and n_head must not be negative");
  if (a->rope_dims < 0 || a->rope_dims > c->head_dim || (a->rope_dims & 1))
    return call_error(GPT_ERR_INVALID_ARG, "rope_dims %d: even, from 0 to head_dim %d", a->rope_dims, c->head_dim);
  if (a->rope_dims > 0 && !(a->rope_base >= 1 && std::isfinite(a->rope_base)))
    return call_error(GPT_ERR_INVALID_ARG, "rope_base must be finite and at least 1");
  if (a->n_head > kMostHeads) return call_error(GPT_ERR_UNSUPPORTED, "n_head %d: at most %d", a->n_head, kMostHeads);
  if (a->n_tokens > (1 << 30)) return call_error(GPT_ERR_UNSUPPORTED, "n_tokens %d: at most 2^30", a->n_tokens);
  if (a->n_tokens == 0) return GPT_OK;
  if (c->n_seq == 0) return call_error(GPT_ERR_INVALID_ARG, "the cache has no sequences");
  if (!a->k || !a->v || !a->before) return call_error(GPT_ERR_INVALID_ARG, "k, v and before must be non-NULL");
  if (cache->k_scale == cache->v_scale) return call_error(GPT_ERR_INVALID_ARG, "k_scale must not be v_scale");
  if (!a->starts && a->n_tokens > c->n_seq)
    return call_error(GPT_ERR_INVALID_ARG, "%d tokens without starts, but %d sequences", a->n_tokens, c->n_seq);
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
  p.c = *cache;
  p.a = *a;
  if (a->rope_dims > 0) set_rates(&p.rates, a->rope_base, a->rope_dims);
  p.strip = a->n_tokens <= 4096 ? 16 : kMaxStrip;
  const int64_t kv_blocks = ((int64_t)a->n_tokens + p.strip - 1) / p.strip * 2 * c->n_kv_head;
  p.share = 0;
  const int pieces = c->head_dim * es / 16;
  while ((1 << p.share) < kMaxTokens && a->n_head * pieces << (p.share + 1) <= kThreads * kQueryHeld && kThreads >> (p.share + 1) >= pieces &&
         a->n_tokens >> (p.share + 1) >= 608)
    ++p.share;
  const int64_t q_blocks = a->n_head > 0 ? ((int64_t)a->n_tokens + (1 << p.share) - 1) >> p.share : 0;
  if (kv_blocks + q_blocks > INT32_MAX) return call_error(GPT_ERR_UNSUPPORTED, "n_tokens x n_kv_head is too large for one call");
  p.kv_blocks = (int32_t)kv_blocks;
  const dim3 grid((unsigned)(kv_blocks + q_blocks));
  const cudaStream_t st = (cudaStream_t)cuda_stream;
  return launch_after("gpt_kv_append_fp8", c->dtype == GPT_DTYPE_BF16 ? kv_append_fp8_kernel<__nv_bfloat16> : kv_append_fp8_kernel<float>, grid,
                      kThreads, 0, 0, st, p);
}
