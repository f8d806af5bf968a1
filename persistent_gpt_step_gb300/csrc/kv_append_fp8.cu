// kv_append_fp8.cu — gpt_kv_append_fp8: keys and values of new tokens into a paged
// cache of e4m3 numbers with a scale for each page and key head, keys and queries
// rotated on the way (rotary.h).
//
// A run: the new rows of one page.  Its scale needs the largest magnitude of all of them
// before the first number is written, so one warp has a run's rows of one key head and
// side (keys or values), reads them twice (the second time from L2) and owns the scale: no
// atomics on global memory, no barrier between the two passes, no second kernel.  The
// scale comes from the magnitudes before the rotation, which turns each pair by at most
// sqrt 2: it is then exact, the same however sines are rounded, and no number reaches 448.
// Bound: HBM (rows read once, numbers and rotated queries written once): 32,768 tokens of 32 + 8 + 8
// heads of 128 in bf16 131 us, 5.6 TB/s; a few thousand tokens by the chain of loads and the sines
// (4,095 of 12 + 12 + 12 of 64 in fp32 16.8 us, 3.4 TB/s).  Pages of hundreds of slots and more leave few
// warps at work: 32,768 tokens of 4 sequences take 132 us in pages of 64, 210 of 512, 1,025 of 4,096.
#include "rotary.h"

namespace pgs {
namespace {

// Of a block, a head each; two such blocks fit an SM.  (4,095 tokens of 12 + 12 + 12 heads of 64 in fp32: 16.4 us, with 4,
// 8 and 16 at the same warps of an SM 23.0, 20.0, 25.0; 8 heads of 128: 130.5 with 8 or 12, 164 with 4.)
constexpr int kMostWarps = 12;
constexpr int kMaxStrip = 64;    // rows of a block's strip, and of the table of sines and cosines
constexpr int kStage = 1024;     // starts in shared memory
// 16-byte pieces that a thread has under way: 32,768 tokens of 32 + 8 + 8 heads of 128 132 us, with 4 140, with 16
// 175 (8,192 of 16 + 16 + 16 of 64 33 32 60); of queries 132, 137 and 217.
constexpr int kUnder = 8, kQueryUnder = 8;
constexpr int kNoRun = 255;

struct AppendParams {
  gpt_fp8_cache c;
  gpt_kv_append_fp8_args a;
  RotaryRates rates;
  int32_t strip;      // rows of a strip; a block has the runs that begin in one
  int32_t groups;     // of key heads: a block has one,
  int32_t warps;      // a warp for each head
  int32_t kv_blocks;  // strips x groups x 2; the others have query rows
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

// A scale that a page had may be any number, where ours are powers of two.  What is multiplied or divided by one that is
// not goes to 24 bits first, of which the last is set, on the right side, where anything is left: the rounding to 4 bits
// is then that of the exact product or quotient.
__device__ __forceinline__ bool uneven(float scale) { return __float_as_uint(scale) & 0x7fffffu; }
__device__ __forceinline__ float times(float x, float by) {
  const float y = __fmul_rz(x, by);
  return __fmaf_rn(x, by, -y) != 0.f ? __uint_as_float(__float_as_uint(y) | 1u) : y;
}
__device__ __forceinline__ float over(float x, float by) {  // 1 <= by < 2
  const float inverse = __fdividef(1.f, by);
  float y = x * inverse;
  y = __fmaf_rn(__fmaf_rn(-y, by, x), inverse, y);  // to half a unit and a little
  const float rest = __fmaf_rn(-y, by, x);
  const uint32_t b = __float_as_uint(y);
  return rest != 0.f && y != 0.f && !(b & 1u) ? __uint_as_float(b + ((__float_as_uint(rest) ^ b) >> 31 ? ~0u : 1u)) : y;
}
// 1 / scale without its fraction, a power of two; the fraction, in [1, 2).
__device__ __forceinline__ float whole_inverse(float scale) { return 1.f / __uint_as_float(__float_as_uint(scale) & 0x7f800000u); }
__device__ __forceinline__ float fraction(float scale) { return __uint_as_float((__float_as_uint(scale) & 0x7fffffu) | 0x3f800000u); }

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

// The numbers of a page's first slots, of one head, times `by`: by `threads` threads, the first of them 0.  (Not inlined:
// 32,768 tokens 131.0 us, 133.6 so, for the registers.)
__device__ __noinline__ void bring_numbers(const gpt_paged_cache& c, uint8_t* page, int slots, float by, int thread, int threads) {
  const int each = c.head_dim / 16, beside = threads / each, sub = thread / each;  // (slots x each can pass 32 bits)
  for (int slot = sub; sub < beside && slot < slots; slot += beside) {
    uint4* at = reinterpret_cast<uint4*>(page + slot * c.slot_stride) + thread % each;
    uint4 v = *at;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t& w = (&v.x)[j];
      float x[4];
      unpack_e4m3(w & 0xffffu, x), unpack_e4m3(w >> 16, x + 2);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = times(x[k], by);
      w = pack_e4m3<true>(x[0], x[1]) | pack_e4m3<true>(x[2], x[3]) << 16;
    }
    *at = v;
  }
}

struct Run {
  int begin, end;   // rows
  int page, slot;   // of the first row; page < 0: skipped
  int pos;          // of the first row
};

// A block's strip of rows, of a group of heads and one side: the runs that begin in it.
template <typename T>
__device__ __forceinline__ void append_runs(const AppendParams& p, const RotaryRates& rates, const int* stage, float2* turns, int unit) {
  constexpr int kN = Piece<T>::kN;
  __shared__ Run runs[kMaxStrip];
  __shared__ uint8_t run_of[kMaxStrip];
  __shared__ int many;
  // of a warp's head: largest magnitudes (as bits), then the scales' fractions; 1 / scale without these
  __shared__ uint32_t tops[kMostWarps][kMaxStrip];
  __shared__ float invs[kMostWarps][kMaxStrip];
  const gpt_paged_cache& c = p.c.pages;
  const gpt_kv_append_fp8_args& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, sides = 2 * p.groups;
  const int strip0 = unit / sides * p.strip, side = unit % sides & 1, head = (unit % sides >> 1) * p.warps + warp;
  const bool report = unit % sides == 0;
  // the runs, by the first warp
  if (warp == 0) {
    uint64_t mask = 0;
    Row r[2];
    int slot[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = lane + 32 * k;
      r[k] = Row{-1, 0, 0, 0};
      if (i < p.strip && strip0 + i < a.n_tokens) r[k] = find_row(p, stage, strip0 + i, report);
      slot[k] = r[k].pos % c.page_size;
      mask |= (uint64_t)__ballot_sync(0xffffffffu, r[k].seq >= 0 && (strip0 + i == r[k].first || slot[k] == 0)) << (32 * k);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = lane + 32 * k;
      int mine = kNoRun;
      const int at = i - min(slot[k], strip0 + i - r[k].first);  // where its run begins
      // (Where starts decrease, a row can be another sequence's than the one before it, whose run would take it past the page.)
      const int seq0 = __shfl_sync(0xffffffffu, r[0].seq, at & 31), seq1 = __shfl_sync(0xffffffffu, r[1].seq, at & 31);
      if (r[k].seq >= 0 && at >= 0 && (mask >> at) & 1u && (at < 32 ? seq0 : seq1) == r[k].seq) mine = __popcll(mask & ((1ull << at) - 1ull));
      run_of[i] = (uint8_t)mine;
      if ((mask >> i) & 1u) {
        Run& x = runs[mine];
        x.begin = strip0 + i, x.end = (int)min((int64_t)r[k].end, (int64_t)strip0 + i + c.page_size - slot[k]);
        x.page = page_of(p, r[k], report), x.slot = slot[k], x.pos = r[k].pos;
      }
    }
    if (lane == 0) many = __popcll(mask);
  }
  __syncthreads();
  const int n_runs = many;
  if (n_runs == 0) return;
  const int first = runs[0].begin, end = runs[n_runs - 1].end;
  const bool works = warp < p.warps && head < c.n_kv_head;
  auto run_at = [&](int row) {  // of a row below `end`, kNoRun: not to be written
    const int x = n_runs == 1 ? 0 : row - strip0 < p.strip ? run_of[row - strip0] : n_runs - 1;
    return x != kNoRun && runs[x].page >= 0 ? x : kNoRun;
  };

  // A lane has a piece of every `side by side`-th row.
  const int pieces = c.head_dim / kN, beside = 32 / pieces, sub = lane / pieces, e = (sub < beside ? lane % pieces : pieces - 1) * kN;
  const int64_t stride = side ? a.v_row : a.k_row;
  const T* from = (side ? (const T*)a.v + head * a.v_head : (const T*)a.k + head * a.k_head) + e;
  bool odd = false;
  uint4 u[kUnder];
  auto load = [&](int row0, int stop) {
#pragma unroll
    for (int i = 0; i < kUnder; ++i) {
      const int row = row0 + i * beside + sub;
      u[i] = make_uint4(0u, 0u, 0u, 0u);
      if (sub < beside && row < stop && run_at(row) != kNoRun) u[i] = __ldcg(reinterpret_cast<const uint4*>(from + row * stride));
    }
  };
  // Runs of eight rows and more on the average: one after the other, rows past the end as the last
  // one again (and lanes past the pieces of a load as the last ones), so that nothing is conditional.
  const bool runs_long = end - first >= 8 * n_runs;
  const int sub_of = min(sub, beside - 1);
  auto load_run = [&](const T* at, int row0, int last) {
    const bool half = row0 + kUnder / 2 * beside > last;
#pragma unroll
    for (int i = 0; i < kUnder; ++i)
      if (i < kUnder / 2 || !half) u[i] = __ldcg(reinterpret_cast<const uint4*>(at + min(row0 + i * beside + sub_of, last) * stride));
  };
  if (works) {
    // the first pass: magnitudes
    if (runs_long) {
#pragma unroll 1
      for (int y = 0; y < n_runs; ++y) {
        if (runs[y].page < 0) continue;
        uint32_t top = 0;
        const int last = runs[y].end - 1;
#pragma unroll 1
        for (int row0 = runs[y].begin; row0 <= last; row0 += kUnder * beside) {
          load_run(from, row0, last);
#pragma unroll
          for (int i = 0; i < kUnder; ++i)
            if (i < kUnder / 2 || row0 + kUnder / 2 * beside <= last) top = max(top, largest(u[i], T(), &odd));
        }
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) tops[warp][y] = top;
      }
    } else {
      for (int i = lane; i < n_runs; i += 32) tops[warp][i] = 0;
      __syncwarp();
      const uint32_t same = __match_any_sync(0xffffffffu, sub);
      for (int row0 = first; row0 < end; row0 += kUnder * beside) {
        load(row0, end);
#pragma unroll
        for (int i = 0; i < kUnder; ++i) {
          const int row = row0 + i * beside + sub;
          const uint32_t top = __reduce_max_sync(same, largest(u[i], T(), &odd));
          if (sub < beside && e == 0 && row < end && top) {
            const int x = run_at(row);
            if (x != kNoRun) atomicMax(&tops[warp][x], top);
          }
        }
      }
    }
    odd = __any_sync(0xffffffffu, odd);
    __syncwarp();
    // scales; the numbers before the new ones are brought to a larger one
    float* scales = (side ? p.c.v_scale : p.c.k_scale) + head * p.c.scale_head;
    uint8_t* cache = (uint8_t*)(side ? c.v : c.k) + head * c.head_stride;
    bool other = false;  // a scale is no power of two
    for (int y0 = 0; y0 < n_runs; y0 += 32) {
      const int y = y0 + lane;
      float share = 1.f;
      if (y < n_runs && runs[y].page >= 0) {
        float* at = scales + runs[y].page * p.c.scale_page;
        float scale = scale_for(__uint_as_float(tops[warp][y]));
        if (runs[y].slot > 0) {
          const float old = *at;
          scale = fmaxf(scale, old);
          if (scale != old) share = old / scale;
        }
        *at = scale;
        invs[warp][y] = whole_inverse(scale);
        tops[warp][y] = __float_as_uint(fraction(scale));
        other |= uneven(scale);
      }
      for (uint32_t left = __ballot_sync(0xffffffffu, share != 1.f); left; left &= left - 1) {
        const int z = y0 + __ffs(left) - 1;
        const float by = __shfl_sync(0xffffffffu, share, z - y0);
        bring_numbers(c, cache + runs[z].page * c.page_stride, runs[z].slot, by, lane, 32);
      }
    }
    odd |= __any_sync(0xffffffffu, other);
    __syncwarp();
  }
  // the second pass, 64 rows at a time: sines and cosines by the block, numbers by the warps
  const int pairs = side == 0 ? a.rope_dims / 2 : 0;
  uint8_t* cache = (uint8_t*)(side ? c.v : c.k) + head * c.head_stride + e;
  for (int chunk = first; chunk < end; chunk += kMaxStrip) {
    const int stop = min(end, chunk + kMaxStrip);
    if (pairs > 0) {
      __syncthreads();
      for (int i = tid; i < (stop - chunk) * kMaxPairs; i += blockDim.x) {
        const int row = chunk + i / kMaxPairs, pair = i % kMaxPairs, x = run_at(row);
        turns[i] = make_float2(1.f, 0.f);
        if (pair < pairs && x != kNoRun) pair_angle_fine(rates, pair, runs[x].pos + (row - runs[x].begin), &turns[i].x, &turns[i].y);
      }
      __syncthreads();
    }
    if (!works) continue;
    if (runs_long && !odd) {
#pragma unroll 1
      for (int y = 0; y < n_runs; ++y) {
        if (runs[y].page < 0) continue;
        const int last = min(runs[y].end, stop) - 1;
        const float by = invs[warp][y];
        uint8_t* to = cache + runs[y].page * c.page_stride + (int64_t)(runs[y].slot - runs[y].begin) * c.slot_stride;
#pragma unroll 1
        for (int row0 = max(runs[y].begin, chunk); row0 <= last; row0 += kUnder * beside) {
          load_run(from, row0, last);
#pragma unroll
          for (int i = 0; i < kUnder; ++i) {
            if (i == kUnder / 2 && row0 + kUnder / 2 * beside > last) break;
            const int row = min(row0 + i * beside + sub_of, last);
            float x[kN];
            Piece<T>::unpack(u[i], x);
#pragma unroll
            for (int j = 0; j < kN; j += 2) {
              const float2 z = mul(Pair(x[j], x[j + 1]), Pair(by)).both();
              x[j] = z.x, x[j + 1] = z.y;
            }
            if (pairs > 0) {
              const float4* turn = reinterpret_cast<const float4*>(turns + (row - chunk) * kMaxPairs + e / 2);
#pragma unroll
              for (int j = 0; j < kN / 4; ++j) {
                const float4 t = turn[j];
                const float a0 = x[4 * j], a1 = x[4 * j + 1], b0 = x[4 * j + 2], b1 = x[4 * j + 3];
                x[4 * j] = a0 * t.x - a1 * t.y, x[4 * j + 1] = a0 * t.y + a1 * t.x;
                x[4 * j + 2] = b0 * t.z - b1 * t.w, x[4 * j + 3] = b0 * t.w + b1 * t.z;
              }
            }
            uint32_t w[kN / 4];
#pragma unroll
            for (int j = 0; j < kN / 4; ++j) w[j] = pack_e4m3<false>(x[4 * j], x[4 * j + 1]) | pack_e4m3<false>(x[4 * j + 2], x[4 * j + 3]) << 16;
            if constexpr (kN == 8) *reinterpret_cast<uint2*>(to + row * c.slot_stride) = make_uint2(w[0], w[1]);
            else *reinterpret_cast<uint32_t*>(to + row * c.slot_stride) = w[0];
          }
        }
      }
      continue;
    }
    for (int row0 = chunk; row0 < stop; row0 += kUnder * beside) {
      load(row0, stop);
#pragma unroll
      for (int i = 0; i < kUnder; ++i) {
        const int row = row0 + i * beside + sub;
        if (sub >= beside || row >= stop) continue;
        const int x = run_at(row);
        if (x == kNoRun) continue;
        const float by = invs[warp][x];
        float y[kN];
        Piece<T>::unpack(u[i], y);
#pragma unroll
        for (int j = 0; j < kN; j += 2) {
          const float2 z = mul(Pair(y[j], y[j + 1]), Pair(by)).both();
          y[j] = z.x, y[j + 1] = z.y;
        }
        if (e / 2 < pairs) {
          const float2* turn = turns + (row - chunk) * kMaxPairs + e / 2;
#pragma unroll
          for (int j = 0; j < kN / 2; ++j)
            if (e / 2 + j < pairs) {
              const float2 t = turn[j];
              const float x0 = y[2 * j], x1 = y[2 * j + 1];
              y[2 * j] = x0 * t.x - x1 * t.y;
              y[2 * j + 1] = x0 * t.y + x1 * t.x;
            }
        }
        uint32_t w[kN / 4];
        if (__builtin_expect(odd, 0)) {
          const float part = __uint_as_float(tops[warp][x]);
          if (part != 1.f)
#pragma unroll
            for (int j = 0; j < kN; ++j) y[j] = over(y[j], part);
#pragma unroll
          for (int j = 0; j < kN / 4; ++j) w[j] = pack_e4m3<true>(y[4 * j], y[4 * j + 1]) | pack_e4m3<true>(y[4 * j + 2], y[4 * j + 3]) << 16;
        } else {
#pragma unroll
          for (int j = 0; j < kN / 4; ++j) w[j] = pack_e4m3<false>(y[4 * j], y[4 * j + 1]) | pack_e4m3<false>(y[4 * j + 2], y[4 * j + 3]) << 16;
        }
        uint8_t* to = cache + runs[x].page * c.page_stride + (runs[x].slot + (row - runs[x].begin)) * c.slot_stride;
        if constexpr (kN == 8) *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t*>(to) = w[0];
      }
    }
  }
}

// Query rows: a thread has a piece of every head of a token, for which it computes the sines and
// cosines once.
template <typename T>
__device__ __forceinline__ void turn_queries(const AppendParams& p, const RotaryRates& rates, const int* stage, int block) {
  constexpr int kN = Piece<T>::kN;
  const gpt_kv_append_fp8_args& a = p.a;
  const int pieces = p.c.pages.head_dim / kN, group = threadIdx.x / pieces, e = threadIdx.x % pieces * kN;
  const int64_t n = (int64_t)block * p.tokens + group;
  if (group >= p.tokens || n >= a.n_tokens) return;
  const T* from = (const T*)a.q + n * a.q_row + e;
  T* to = (T*)a.q_out + n * a.qo_row + e;
  uint4 u[kQueryUnder];
  auto load = [&](int head) {
#pragma unroll
    for (int i = 0; i < kQueryUnder; ++i)
      if (head + i < a.n_head) u[i] = __ldcs(reinterpret_cast<const uint4*>(from + (head + i) * a.q_head));
  };
  const Row r = find_row(p, stage, (int)n, false);
  if (r.seq < 0) return;
  load(0);  // under way while the page is looked up
  if (page_of(p, r, false) < 0) return;
  float2 turn[kN / 2];
#pragma unroll
  for (int j = 0; j < kN / 2; ++j)
    if (e + 2 * j < a.rope_dims) pair_angle_fine(rates, e / 2 + j, r.pos, &turn[j].x, &turn[j].y);
  const bool all = e + kN <= a.rope_dims;
#pragma unroll 1
  for (int head = 0; head < a.n_head; head += kQueryUnder) {
    if (head > 0) load(head);
#pragma unroll
    for (int i = 0; i < kQueryUnder; ++i) {
      if (head + i >= a.n_head) break;
      if (e < a.rope_dims) {
        float x[kN];
        Piece<T>::unpack(u[i], x);
#pragma unroll
        for (int j = 0; j < kN / 2; ++j)
          if (all || e + 2 * j < a.rope_dims) {
            const float x0 = x[2 * j], x1 = x[2 * j + 1];
            x[2 * j] = x0 * turn[j].x - x1 * turn[j].y;
            x[2 * j + 1] = x0 * turn[j].y + x1 * turn[j].x;
          }
        u[i] = Piece<T>::pack(x);
      }
      *reinterpret_cast<uint4*>(to + (head + i) * a.qo_head) = u[i];
    }
  }
}

// What blocks of both kinds begin with.
__device__ __forceinline__ void begin_block(const AppendParams& p, RotaryRates& rates, int* stage) {
  // (rates are read by threads' own pairs: from the parameters one after the other)
  for (int i = threadIdx.x; i < kMaxPairs; i += blockDim.x) rates.hi[i] = p.rates.hi[i], rates.lo[i] = p.rates.lo[i];
  after_stream();
  stage_starts(p, stage);
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kMostWarps * 32, 2) kv_append_fp8_kernel(const __grid_constant__ AppendParams p) {
  extern __shared__ __align__(16) float2 turns[];  // [kMaxStrip][kMaxPairs] cosine, sine
  __shared__ int stage[kStage];
  __shared__ RotaryRates rates;
  begin_block(p, rates, stage);
  if (blockIdx.x == 0 && p.a.starts)
    for (int i = threadIdx.x; i < p.c.pages.n_seq; i += blockDim.x)
      if (p.a.starts[i] > p.a.starts[i + 1] || p.a.starts[i] < 0 || p.a.starts[i + 1] > p.a.n_tokens) set_status(p.a.status, GPT_STATUS_BAD_SEQ);
  // The longer blocks first.  (In even turns 20,000 tokens of 4 + 1 + 1 heads of 96 take 42.6 us for 29.1, 8,192 of
  // 16 + 16 + 16 of 64 33.4 for 30.0, 32,768 of 32 + 8 + 8 of 128 131.9 for 130.3.)
  if ((int)blockIdx.x < p.kv_blocks) append_runs<T>(p, rates, stage, turns, blockIdx.x);
  else turn_queries<T>(p, rates, stage, blockIdx.x - p.kv_blocks);
}

// One new token of each sequence (no starts): every run is a row.  A block has a token, a warp
// the pieces of as many heads as fit, each element once in registers.
template <typename T, int kThreads, int kUnroll>
__global__ void __launch_bounds__(kThreads) kv_append_fp8_step_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kN = Piece<T>::kN;
  __shared__ __align__(16) float2 turns[kMaxPairs];  // cosine, sine
  const gpt_paged_cache& c = p.c.pages;
  const gpt_kv_append_fp8_args& a = p.a;
  after_stream();
  const int tid = threadIdx.x, lane = tid & 31, pieces = c.head_dim / kN, beside = 32 / pieces, sub = lane / pieces;
  const int group = sub < beside ? (tid >> 5) * beside + sub : 1 << 30, groups = kThreads / 32 * beside, e = lane % pieces * kN;
  const int64_t n = blockIdx.x;
  const int rows = a.n_head + 2 * c.n_kv_head;  // q heads, k heads, v heads
  uint4 u[kUnroll];
  auto load = [&](int row0) {
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      int row = row0 + i * groups;
      if (row >= rows) continue;
      const T* from;
      if (row < a.n_head) from = (const T*)a.q + n * a.q_row + row * a.q_head;
      else if ((row -= a.n_head) < c.n_kv_head) from = (const T*)a.k + n * a.k_row + row * a.k_head;
      else from = (const T*)a.v + n * a.v_row + (row - c.n_kv_head) * a.v_head;
      u[i] = __ldcs(reinterpret_cast<const uint4*>(from + e));
    }
  };
  const Row r = find_row(p, nullptr, (int)n, tid == 0);
  if (r.seq < 0) return;
  load(group);  // under way while the page is looked up
  const int page = page_of(p, r, tid == 0), slot = r.pos % c.page_size;
  for (int i = tid; i < kMaxPairs; i += kThreads) {
    turns[i] = make_float2(1.f, 0.f);
    if (i < a.rope_dims / 2) pair_angle_fine(p.rates, i, r.pos, &turns[i].x, &turns[i].y);
  }
  if (page < 0) return;
  __syncthreads();
  const uint32_t same = __match_any_sync(0xffffffffu, sub);
  const int64_t scale_at = page * p.c.scale_page, at = page * c.page_stride;
  const int passes = (rows + kUnroll * groups - 1) / (kUnroll * groups);
  for (int pass = 0, row0 = group; pass < passes; ++pass, row0 += kUnroll * groups) {
    if (pass > 0) load(row0);
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      int row = row0 + i * groups;
      const bool there = row < rows, query = row < a.n_head;
      if (!__any_sync(0xffffffffu, there)) break;
      bool odd = false;
      const uint32_t top = __reduce_max_sync(same, there && !query ? largest(u[i], T(), &odd) : 0u);
      if (!there) continue;
      float x[kN], by = 1.f, part = 1.f;
      Piece<T>::unpack(u[i], x);
      const bool key = !query && (row -= a.n_head) < c.n_kv_head, value = !query && !key;
      if (value) row -= c.n_kv_head;
      uint8_t* numbers = (uint8_t*)(key ? c.k : c.v) + row * c.head_stride + at;
      if (!query) {
        float* scales = (key ? p.c.k_scale : p.c.v_scale) + scale_at + row * p.c.scale_head;
        float scale = scale_for(__uint_as_float(top));
        if (slot > 0) {
          const float old = *scales;
          __syncwarp(same);
          scale = fmaxf(scale, old);
          if (scale != old) bring_numbers(c, numbers, slot, old / scale, lane % pieces, pieces);
        }
        if (e == 0) *scales = scale;
        by = whole_inverse(scale), part = fraction(scale);
#pragma unroll
        for (int j = 0; j < kN; ++j) x[j] *= by;
      }
      if (!value && e < a.rope_dims)
#pragma unroll
        for (int j = 0; j < kN / 2; ++j)
          if (e + 2 * j < a.rope_dims) {
            const float2 t = turns[e / 2 + j];
            const float x0 = x[2 * j], x1 = x[2 * j + 1];
            x[2 * j] = x0 * t.x - x1 * t.y;
            x[2 * j + 1] = x0 * t.y + x1 * t.x;
          }
      if (query) {
        *reinterpret_cast<uint4*>((T*)a.q_out + n * a.qo_row + row * a.qo_head + e) = e < a.rope_dims ? Piece<T>::pack(x) : u[i];
      } else {
        if (part != 1.f)
#pragma unroll
          for (int j = 0; j < kN; ++j) x[j] = over(x[j], part);
        uint32_t w[kN / 4];
#pragma unroll
        for (int j = 0; j < kN / 4; ++j) w[j] = pack_e4m3<true>(x[4 * j], x[4 * j + 1]) | pack_e4m3<true>(x[4 * j + 2], x[4 * j + 3]) << 16;
        uint8_t* to = numbers + slot * c.slot_stride + e;
        if constexpr (kN == 8) *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t*>(to) = w[0];
      }
    }
  }
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
  const cudaStream_t st = (cudaStream_t)cuda_stream;
  const bool bf16 = c->dtype == GPT_DTYPE_BF16;
  if (!a->starts) {
    // A wide block for a token, all under way at once, while four fit an SM; then narrow ones, that take turns (32 + 8 + 8
    // heads of 128 in bf16, 256 600 1,000 2,000 4,000 tokens: 5.1 6.1 10.1 18.0 32.8 us and 7.1 7.9 9.4 16.7 31.6).
    const bool few = a->n_tokens <= 4 * 152;
    const auto kernel = bf16 ? (few ? kv_append_fp8_step_kernel<__nv_bfloat16, 256, 6> : kv_append_fp8_step_kernel<__nv_bfloat16, 128, 3>)
                             : (few ? kv_append_fp8_step_kernel<float, 256, 6> : kv_append_fp8_step_kernel<float, 128, 3>);
    return launch_after("gpt_kv_append_fp8", kernel, dim3((unsigned)a->n_tokens), few ? 256 : 128, 0, 0, st, p);
  }
  p.groups = (c->n_kv_head + kMostWarps - 1) / kMostWarps;
  p.warps = (c->n_kv_head + p.groups - 1) / p.groups;
  // Rows of a strip: about a page, 32 at least, where there are blocks enough (8,192 tokens of 16
  // heads of 64 in pages of 16: 33.5 us, in strips of 16 38.6, of 64 36.4; 2,000 of 8 heads of 128
  // in pages of 128: 30.4 in strips of 16, 37.7 of 64).
  const auto units = [&](int rows) { return ((int64_t)a->n_tokens + rows - 1) / rows * 2 * p.groups; };
  p.strip = 16;
  while (p.strip < std::min(kMaxStrip, std::max(32, c->page_size)) && units(2 * p.strip) >= 304) p.strip *= 2;
  const int64_t kv_blocks = units(p.strip);
  const int threads = 32 * std::max(p.warps, 4);
  p.tokens = threads / (c->head_dim * es / 16);
  const int64_t q_blocks = a->n_head > 0 ? ((int64_t)a->n_tokens + p.tokens - 1) / p.tokens : 0;
  if (kv_blocks + q_blocks > INT32_MAX) return call_error(GPT_ERR_UNSUPPORTED, "n_tokens x n_kv_head is too large for one call");
  p.kv_blocks = (int32_t)kv_blocks;
  const auto kernel = bf16 ? kv_append_fp8_kernel<__nv_bfloat16> : kv_append_fp8_kernel<float>;
  const int turns = a->rope_dims ? kMaxStrip * kMaxPairs * (int)sizeof(float2) : 0;
  return launch_after("gpt_kv_append_fp8", kernel, dim3((unsigned)(kv_blocks + q_blocks)), threads, turns, 0, st, p);
}
