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
constexpr int kQueryHeld = 4;   // 16-byte pieces of queries that a thread has under way
constexpr int kMaxTokens = 8;   // of a block of query rows
constexpr int kNoRun = 255;

struct AppendParams {
  gpt_fp8_cache c;
  gpt_kv_append_fp8_args a;
  RotaryRates rates;
  int32_t strip;      // rows of a strip; a block has the runs that begin in one
  int32_t heads;      // key heads of a block
  int32_t kv_blocks;  // strips x groups of key heads x 2; the blocks behind them have query rows
  int32_t tokens;     // of a block of query rows
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

// Two numbers, rounded to nearest; with kOdd what is not finite is NaN.
template <bool kOdd>
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b) {
  uint16_t u;
  if (kOdd) a = fabsf(a) <= 448.f ? a : NAN, b = fabsf(b) <= 448.f ? b : NAN;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(u) : "f"(b), "f"(a));
  return u;
}
__device__ __forceinline__ void unpack_e4m3(uint32_t u, float* x) {  // two
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)u));
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(x[0]), "=f"(x[1]) : "r"(h));
}

// The largest finite magnitude of a piece, as bits; *odd: there is one that is not finite.
__device__ __forceinline__ uint32_t largest(const uint4& u, float, bool* odd) {
  const uint32_t w[4] = {u.x & 0x7fffffffu, u.y & 0x7fffffffu, u.z & 0x7fffffffu, u.w & 0x7fffffffu};
  uint32_t m = max(max(w[0], w[1]), max(w[2], w[3]));
  if (__builtin_expect(m >= 0x7f800000u, 0)) {
    *odd = true, m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = w[i] < 0x7f800000u ? max(m, w[i]) : m;
  }
  return m;
}
__device__ __forceinline__ uint32_t largest(const uint4& u, __nv_bfloat16, bool* odd) {
  const uint32_t w[4] = {u.x & 0x7fff7fffu, u.y & 0x7fff7fffu, u.z & 0x7fff7fffu, u.w & 0x7fff7fffu};
  const uint32_t two = __vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3]));
  uint32_t m = max(two & 0xffffu, two >> 16);
  if (__builtin_expect(m >= 0x7f80u, 0)) {
    *odd = true, m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = w[i] & 0xffffu, hi = w[i] >> 16;
      m = lo < 0x7f80u ? max(m, lo) : m, m = hi < 0x7f80u ? max(m, hi) : m;
    }
  }
  return m << 16;
}

// Cosine and sine of the pairs of a piece whose first element is e of a head at position pos.
template <int N>
__device__ __forceinline__ void piece_angles(const AppendParams& p, int e, int pos, float2* turn) {
#pragma unroll
  for (int j = 0; j < N / 2; ++j) {
    turn[j] = make_float2(1.f, 0.f);
    if (e + 2 * j < p.a.rope_dims) pair_angle(p.rates, e / 2 + j, pos, &turn[j].x, &turn[j].y);
  }
}
template <int N>
__device__ __forceinline__ void turn_piece(float* x, const float2* turn) {
#pragma unroll
  for (int j = 0; j < N / 2; ++j) {
    const float x0 = x[2 * j], x1 = x[2 * j + 1];
    x[2 * j] = x0 * turn[j].x - x1 * turn[j].y;
    x[2 * j + 1] = x0 * turn[j].y + x1 * turn[j].x;
  }
}

struct Run {
  int begin, end;   // rows
  int page, slot;   // of the first row; page < 0: skipped
  int pos;          // of the first row
};

// A block has a group of key heads, one after the other, of one side.  A thread has the same
// rows and elements of each, so that it computes its sines and cosines once (of 8 heads of
// 128 in 32,768 tokens each: as many instructions as all the rest).
template <typename T>
__device__ __forceinline__ void append_runs(const AppendParams& p, int* stage) {
  constexpr int kN = Piece<T>::kN, kHeld = 32 / kN;  // pieces that a thread holds: 32 elements
  __shared__ Run runs[kMaxStrip];
  __shared__ uint8_t run_of[kMaxStrip];
  __shared__ uint32_t begins[2];
  // of a head, in turns: largest magnitudes (as bits), 1 / scale, old scale / scale, whether one is not 1
  __shared__ uint32_t tops[2][kMaxStrip];
  __shared__ float inv[2][kMaxStrip], ratio[2][kMaxStrip];
  __shared__ int rescale[2];
  const gpt_paged_cache& c = p.c.pages;
  const gpt_kv_append_fp8_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31;
  const int groups = (c.n_kv_head + p.heads - 1) / p.heads, unit = blockIdx.x, sides = 2 * groups;
  const int strip0 = unit / sides * p.strip, side = unit % sides & 1, head0 = (unit % sides >> 1) * p.heads;
  const int head1 = min(head0 + p.heads, c.n_kv_head);
  const bool report = unit % sides == 0;
  if (tid < 2) rescale[tid] = 0;
  if (tid < 2 * kMaxStrip) tops[tid / kMaxStrip][tid % kMaxStrip] = 0;
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
      x.page = page_of(p, r, report), x.slot = slot, x.pos = r.pos;
    }
  }
  __syncthreads();
  const int first = runs[0].begin, end = runs[n_runs - 1].end;
  const int pieces = c.head_dim / kN, per_pass = kThreads / pieces, window = kHeld * per_pass;
  const int group = tid / pieces, e = tid % pieces * kN;
  const bool turns = side == 0 && e < a.rope_dims;
  const T* from = (side ? (const T*)a.v : (const T*)a.k) + e;
  const int64_t stride = side ? a.v_row : a.k_row, head_step = side ? a.v_head : a.k_head;
  float* scales = side ? p.c.v_scale : p.c.k_scale;
  uint8_t* cache = (uint8_t*)(side ? c.v : c.k);

  uint4 u[kHeld];
  int x[kHeld];          // run of a held row, kNoRun: not to be written
  float2 turn[kHeld][kN / 2];
  auto hold = [&](int row0) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int row = row0 + i * per_pass + group;
      x[i] = kNoRun;
      if (row < end && group < per_pass) {
        x[i] = row - strip0 < p.strip ? run_of[row - strip0] : n_runs - 1;
        if (x[i] != kNoRun && runs[x[i]].page < 0) x[i] = kNoRun;
      }
    }
  };
  auto load = [&](int row0, int head) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (x[i] != kNoRun) u[i] = __ldcs(reinterpret_cast<const uint4*>(from + head * head_step + (row0 + i * per_pass + group) * stride));
  };
  auto angles = [&](int row0) {
    if (turns)
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (x[i] != kNoRun) piece_angles<kN>(p, e, runs[x[i]].pos + (row0 + i * per_pass + group - runs[x[i]].begin), turn[i]);
  };
  bool odd = false;
  auto look = [&](uint32_t* top) {  // the held rows' largest magnitudes
    int now = kNoRun;
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      if (x[i] == kNoRun) continue;
      if (x[i] != now) {
        if (now != kNoRun) atomicMax(&top[now], most);
        now = x[i], most = 0;
      }
      most = max(most, largest(u[i], T(), &odd));
    }
    __syncwarp();
    const uint32_t same = __match_any_sync(0xffffffffu, now);
    most = __reduce_max_sync(same, most);
    if (now != kNoRun && lane == __ffs(same) - 1) atomicMax(&top[now], most);
  };
  auto settle = [&](int turn_, int head) {  // the scales
    if (tid == 0) rescale[turn_ ^ 1] = 0;
    if (tid < n_runs && runs[tid].page >= 0) {
      float* at = scales + runs[tid].page * p.c.scale_page + head * p.c.scale_head;
      float scale = scale_for(__uint_as_float(tops[turn_][tid])), share = 1.f;
      if (runs[tid].slot > 0) {
        const float old = *at;
        scale = fmaxf(scale, old);
        if (scale != old) share = old / scale, rescale[turn_] = 1;
      }
      *at = scale;
      inv[turn_][tid] = 1.f / scale, ratio[turn_][tid] = share;
      tops[turn_ ^ 1][tid] = 0;
    }
  };
  auto bring = [&](int turn_, int head) {  // the numbers before the new ones, to a larger scale
    for (int y = 0; y < n_runs; ++y) {
      const float by = ratio[turn_][y];
      if (runs[y].page < 0 || by == 1.f) continue;
      const int each = c.head_dim / 16;
      for (int i = tid; i < runs[y].slot * each; i += kThreads) {
        uint4* at = reinterpret_cast<uint4*>(cache + head * c.head_stride + runs[y].page * c.page_stride + i / each * c.slot_stride) + i % each;
        uint4 v = *at;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t& w = (&v.x)[j];
          float z[4];
          unpack_e4m3(w & 0xffffu, z), unpack_e4m3(w >> 16, z + 2);
          w = pack_e4m3<true>(z[0] * by, z[1] * by) | pack_e4m3<true>(z[2] * by, z[3] * by) << 16;
        }
        *at = v;
      }
    }
  };
  auto write = [&](int row0, int turn_, int head) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      if (x[i] == kNoRun) continue;
      const Run& run = runs[x[i]];
      const float by = inv[turn_][x[i]];
      float y[kN];
      Piece<T>::unpack(u[i], y);
#pragma unroll
      for (int j = 0; j < kN; ++j) y[j] *= by;
      if (turns) turn_piece<kN>(y, turn[i]);
      uint32_t w[kN / 4];
      if (__builtin_expect(odd, 0)) {
#pragma unroll
        for (int j = 0; j < kN / 4; ++j) w[j] = pack_e4m3<true>(y[4 * j], y[4 * j + 1]) | pack_e4m3<true>(y[4 * j + 2], y[4 * j + 3]) << 16;
      } else {
#pragma unroll
        for (int j = 0; j < kN / 4; ++j) w[j] = pack_e4m3<false>(y[4 * j], y[4 * j + 1]) | pack_e4m3<false>(y[4 * j + 2], y[4 * j + 3]) << 16;
      }
      uint8_t* to = cache + head * c.head_stride + run.page * c.page_stride + (run.slot + (row0 + i * per_pass + group - run.begin)) * c.slot_stride + e;
      if constexpr (kN == 8) *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
      else *reinterpret_cast<uint32_t*>(to) = w[0];
    }
  };
  const bool once = end - first <= window;
  if (once) hold(first), load(first, head0), angles(first);
#pragma unroll 1
  for (int head = head0; head < head1; ++head) {
    const int t = (head - head0) & 1;
    if (once) {
      if (head > head0) load(first, head);
      look(tops[t]);
    } else {
      for (int row0 = first; row0 < end; row0 += window) hold(row0), load(row0, head), look(tops[t]);
    }
    __syncthreads();
    settle(t, head);
    __syncthreads();
    if (rescale[t]) bring(t, head);
    if (once) {
      write(first, t, head);
    } else {
      for (int row0 = first; row0 < end; row0 += window) hold(row0), load(row0, head), angles(row0), write(row0, t, head);
    }
  }
}

// Query rows: a token's sines and cosines once for all of its heads.
template <typename T>
__device__ __forceinline__ void turn_queries(const AppendParams& p, const int* stage) {
  constexpr int kN = Piece<T>::kN;
  __shared__ __align__(16) float2 turns[kMaxTokens][kMaxPairs];  // cosine, sine
  __shared__ int positions[kMaxTokens];                          // -1: left out
  const gpt_kv_append_fp8_args& a = p.a;
  const int tid = threadIdx.x, n0 = (blockIdx.x - p.kv_blocks) * p.tokens, n = min(p.tokens, a.n_tokens - n0);
  if (tid < n) {
    const Row r = find_row(p, stage, n0 + tid, false);
    positions[tid] = r.seq >= 0 && page_of(p, r, false) >= 0 ? r.pos : -1;
  }
  __syncthreads();
  const int pairs = a.rope_dims / 2;
  for (int i = tid; i < n * kMaxPairs; i += kThreads)
    if (i % kMaxPairs < pairs && positions[i / kMaxPairs] >= 0)
      pair_angle(p.rates, i % kMaxPairs, positions[i / kMaxPairs], &turns[i / kMaxPairs][i % kMaxPairs].x, &turns[i / kMaxPairs][i % kMaxPairs].y);
  __syncthreads();
  const int pieces = p.c.pages.head_dim / kN, groups = kThreads / pieces, group = tid / pieces, e = tid % pieces * kN;
  if (group >= groups) return;
  const T* from = (const T*)a.q + (int64_t)n0 * a.q_row + e;
  T* to = (T*)a.q_out + (int64_t)n0 * a.qo_row + e;
  const int rows = n * a.n_head;
  for (int row0 = group; row0 < rows; row0 += kQueryHeld * groups) {
    uint4 u[kQueryHeld];
    int token[kQueryHeld], head[kQueryHeld];
#pragma unroll
    for (int i = 0; i < kQueryHeld; ++i) {
      const int row = row0 + i * groups;
      token[i] = row / a.n_head, head[i] = row % a.n_head;
      if (row >= rows || positions[token[i]] < 0) token[i] = -1;
      else u[i] = __ldcs(reinterpret_cast<const uint4*>(from + token[i] * a.q_row + head[i] * a.q_head));
    }
#pragma unroll
    for (int i = 0; i < kQueryHeld; ++i) {
      if (token[i] < 0) continue;
      if (e < a.rope_dims) {
        float x[kN];
        Piece<T>::unpack(u[i], x);
#pragma unroll
        for (int j = 0; j < kN / 2; ++j)
          if (e + 2 * j < a.rope_dims) {
            const float2 t = turns[token[i]][e / 2 + j];
            const float x0 = x[2 * j], x1 = x[2 * j + 1];
            x[2 * j] = x0 * t.x - x1 * t.y;
            x[2 * j + 1] = x0 * t.y + x1 * t.x;
          }
        u[i] = Piece<T>::pack(x);
      }
      *reinterpret_cast<uint4*>(to + token[i] * a.qo_row + head[i] * a.qo_head) = u[i];
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
  // Rows of a strip: as many as leave two units a block and SM (the window of a block's registers
  // is 64 rows of 128), 16 at least; then heads of a block.
  const auto units = [&](int rows) { return ((int64_t)a->n_tokens + rows - 1) / rows * 2 * c->n_kv_head; };
  p.strip = kMaxStrip;
  while (p.strip > 16 && units(p.strip) < 608) p.strip /= 2;
  p.heads = (int32_t)std::max<int64_t>(1, std::min<int64_t>(c->n_kv_head, units(p.strip) / 1216));
  const int64_t kv_blocks = units(p.strip) / c->n_kv_head * ((c->n_kv_head + p.heads - 1) / p.heads);
  p.tokens = std::max(1, std::min(kMaxTokens, a->n_tokens / 1216));
  const int64_t q_blocks = a->n_head > 0 ? ((int64_t)a->n_tokens + p.tokens - 1) / p.tokens : 0;
  if (kv_blocks + q_blocks > INT32_MAX) return call_error(GPT_ERR_UNSUPPORTED, "n_tokens x n_kv_head is too large for one call");
  p.kv_blocks = (int32_t)kv_blocks;
  const dim3 grid((unsigned)(kv_blocks + q_blocks));
  const cudaStream_t st = (cudaStream_t)cuda_stream;
  return launch_after("gpt_kv_append_fp8", c->dtype == GPT_DTYPE_BF16 ? kv_append_fp8_kernel<__nv_bfloat16> : kv_append_fp8_kernel<float>, grid,
                      kThreads, 0, 0, st, p);
}
