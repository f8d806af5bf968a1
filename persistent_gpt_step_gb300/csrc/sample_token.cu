// sample_token.cu — gpt_sample_token: a token drawn from a row of logits with
// temperature, top-k, top-p and min-p, from a given number.
//
// Weights are integers: w = round(2^U exp((z - m) / T)), U such that a row's sum fits 64
// bits.  Sums of integers are the same in any order, so every limit (a count or a sum over
// the tokens above one) and the draw itself (a running sum by id) are exact, whatever
// threads add.  All three limits keep a prefix of the tokens in order of falling z, then
// rising id; with the composite key (z's order, ~id) of a token, which is its own, the kept
// tokens are those at or above the last kept one's.
//
// Rows without limits need one pass and no exact sum of all weights: their sums in fp32, good to
// 2^-21, name the token unless the number falls that near a border between two; only then
// the weights are summed as integers.
//
// A row is the work of a cluster of blocks, each with a range of its ids, each warp with a
// part of that.  The logits are read again in each pass (from L2; nothing is written):
//  1. the largest z;
//  2. for a limit, counts (and weights) in 1,024 bins of equal width below it, of which one
//     holds the limit's last token;
//  3. what lies in that bin, or, where it is few, all above its end, into a list that the
//     first block sorts: where the list holds all, it draws from it;
//  4. otherwise the weights of the kept tokens, a sum for each warp, then the warp's range in
//     which the number falls, a token after the other.
#include <cooperative_groups.h>

#include <cmath>

#include "decode_ops.h"

namespace pgs {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlocks = 8;        // of a cluster at most
constexpr int kBins = 1024;
constexpr int kList = 1024;
constexpr int kTable = 1024;
constexpr int kPieces = 8;        // of a warp's range, where sums are in fp32
using u64 = unsigned long long;

struct SampleParams {
  gpt_sample_token_args a;
  int32_t unit;               // U
  u64 coarse[32], fine[32];   // 2^62 2^(i/32), 2^63 2^(i/1024)
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// Ascends with z; 0: no token.  Both zeros are one value.
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);
  return z > -INFINITY ? (b >> 31 ? ~b : b | 0x80000000u) : 0u;
}
__device__ __forceinline__ float value_of(uint32_t key) { return __uint_as_float(key >> 31 ? key & 0x7fffffffu : ~key); }
__device__ __forceinline__ u64 composite(float z, int id) {
  const uint32_t key = key_of(z);
  return key ? (u64)key << 32 | ~(uint32_t)id : 0ull;
}
__device__ __forceinline__ int id_of(u64 comp) { return (int)~(uint32_t)comp; }

// 2^U exp((z - m) / T) to 2^-42 of itself and half a unit, in fp32 and integer
// operations: y = (z - m) c, c = log2 e / T, is kept in two floats (z - m and the product with
// their rounding errors, from halves of z and m, so that nothing overflows), split into
// J / 1024 + r with |r| <= 2^-11; 2^r - 1 = L r + (L r)^2 / 2 + (L r)^3 / 6 with L = ln 2 in
// two floats (the next term is below 2^-50), as an integer in units of 2^-42, and
// 2^(J mod 1024 / 1024) from a table of 62 bits.
struct Weigher {
  const u64* table;
  float mh, c_hi, c_lo;
  int unit;
  bool infinite;  // m is
  __device__ __forceinline__ u64 operator()(float z) const {
    constexpr double kLn2 = 0.69314718055994530942, kUp = 4398046511104.0;  // 2^42
    constexpr float kL = (float)kLn2, kL42 = (float)(kL * kUp), kRest42 = (float)((kLn2 - (double)kL) * kUp);
    constexpr float kC2 = (float)(kLn2 * kLn2 / 2 * kUp), kC3 = (float)(kLn2 * kLn2 * kLn2 / 6 * kUp);
    constexpr float kMagic = 12288.f;  // 1.5 2^13: sums with it are multiples of 2^-10
    if (infinite) return z == INFINITY ? 1ull << unit : 0ull;
    const float zh = __fmul_rn(z, 0.5f), s = __fsub_rn(zh, mh), t = __fsub_rn(s, zh);
    const float e = __fsub_rn(__fsub_rn(zh, __fsub_rn(s, t)), __fadd_rn(mh, t));
    const float p = __fmul_rn(s, c_hi);
    if (!(p > -64.f)) return 0ull;
    const float up = __fadd_rn(p, kMagic), r = __fsub_rn(p, __fsub_rn(up, kMagic));
    const float low = __fmaf_rn(s, c_lo, __fmaf_rn(e, c_hi, __fmaf_rn(s, c_hi, -p)));
    const int J = (int)(__float_as_uint(up) - __float_as_uint(kMagic));
    const float a = __fmul_rn(r, kL42);
    const float rest = __fmaf_rn(__fmul_rn(r, r), __fmaf_rn(r, kC3, kC2), __fmaf_rn(r, kRest42, __fmaf_rn(low, kL42, __fmaf_rn(r, kL42, -a))));
    const int more = __float2int_rn(a) + __float2int_rn(rest);
    const u64 base = table[J & (kTable - 1)];
    const u64 w = base + (u64)(((int64_t)more * (int)(base >> 32)) >> 10);
    const int shift = 61 - unit - (J >> 10);
    return shift < 64 ? ((w >> shift) + 1) >> 1 : 0ull;
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
// The first of the running sums that the number u falls under, as the least such sum.
__device__ __forceinline__ u64 goal_of(float u, u64 sum) { return u >= 1.f ? sum : (u > 0.f ? part_of(u, sum, false) : 0) + 1; }

// Eight logits of a row from a boundary of their size on.
__device__ __forceinline__ void load8(const float* z, float* x) {
  asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
               : "l"(z) : "memory");
}
__device__ __forceinline__ void load8(const __nv_bfloat16* z, float* x) {
  uint4 u;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(z) : "memory");
  Piece<__nv_bfloat16>::unpack(u, x);
}

// 2^n, 0 and the largest power where that is too small or large.
__device__ __forceinline__ float power(int n) { return __uint_as_float((uint32_t)min(max(n + 127, 0), 254) << 23); }

// A sum of 2^(c z) over a thread's tokens, as (sum + rest) 2^ref.
// c z is split into an integer and a fraction of at most 1/2 (a product with c in two floats: good
// to 2^-25), powers of the integer part are exact, and of the rounded sums of eight only the three
// roundings inside are not carried along.  Together with ex2.approx (2^-22): 2^-21.
struct FastSum {
  float c_hi, c_lo, inv_c;
  float sum, rest, top;
  float low, high;   // z outside change nothing, or need another ref
  int ref, missing;  // missing: of the units, what is no token
  bool bad;          // too large for the split
  __device__ __forceinline__ void start(float hi, float lo) {
    c_hi = hi, c_lo = lo, inv_c = 1.f / hi;
    clear(), missing = 0, top = -INFINITY, bad = false;
  }
  __device__ __forceinline__ void clear() { sum = rest = 0.f, low = high = -INFINITY, ref = -(1 << 24); }
  __device__ __forceinline__ void add(const float* x) {
    float m = x[0], all = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) m = fmaxf(m, x[i]), all += x[i];
    if (!(all > -INFINITY))
#pragma unroll
      for (int i = 0; i < 8; ++i) missing += !(x[i] > -INFINITY);
    if (!(m > low)) return;
    top = fmaxf(top, m);
    if (m > high) {
      const float at = m * c_hi;
      if (!(fabsf(at) < 0x1p21f)) {
        bad = true;
        return;
      }
      const int now = __float2int_rn(at);
      const float keep = power(ref - now);
      sum *= keep, rest *= keep, ref = now;
      low = (float)(now - 100) * inv_c, high = (float)(now + 40) * inv_c;
    }
    constexpr float kMagic = 12582912.f;  // 1.5 2^23
    const int less = __float_as_int(kMagic) + ref;
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float z = fmaxf(x[i], low), up = __fmaf_rn(z, c_hi, kMagic), n = __fsub_rn(up, kMagic);
      const float r = __fmaf_rn(z, c_lo, __fmaf_rn(z, c_hi, -n));
      float f;
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(f) : "f"(r));
      w[i] = __int_as_float(__float_as_int(f) + ((__float_as_int(up) - less) << 23));
    }
#pragma unroll
    for (int k = 1; k < 8; k *= 2)
#pragma unroll
      for (int i = 0; i < 8; i += 2 * k) w[i] += w[i + k];
    two_sum(w[0], 0.f);
  }
  __device__ __forceinline__ void two_sum(float v, float more) {  // sum + rest += v + more, exactly but for the rests' roundings
    const float s = __fadd_rn(sum, v), t = __fsub_rn(s, sum);
    rest = __fadd_rn(rest, __fadd_rn(more, __fadd_rn(__fsub_rn(sum, __fsub_rn(s, t)), __fsub_rn(v, t))));
    sum = s;
  }
  // The warp's sum in every lane, with one ref.
  __device__ __forceinline__ void join_warp() {
    const int all = __reduce_max_sync(0xffffffffu, ref);
    const float keep = power(ref - all);
    sum *= keep, rest *= keep, ref = all;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) {
      const float v = __shfl_xor_sync(0xffffffffu, sum, x), more = __shfl_xor_sync(0xffffffffu, rest, x);
      two_sum(v, more);
    }
  }
};

template <typename T>
struct RowView {
  const T* z;
  int vocab, shift;  // unit w: ids 8 w - shift ..
  __device__ __forceinline__ void load(int w, float* x) const {
    const int64_t id = (int64_t)w * 8 - shift;
    if (id >= 0 && id + 8 <= vocab) {
      load8(z + id, x);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = id + i >= 0 && id + i < vocab ? to_float(z[id + i]) : -INFINITY;
    }
  }
  // f(8 logits, the first's id) for units w0 + first, w0 + first + step, ... below w1, two of them under way.
  template <typename F>
  __device__ __forceinline__ void each(int w0, int w1, int first, int step, F f) const {
    float x[2][8];
    int w = w0 + first;
    if (w < w1) load(w, x[0]);
    for (; w < w1; w += 2 * step) {
      if (w + step < w1) load(w + step, x[1]);
      f(x[0], w * 8 - shift);
      if (w + step >= w1) break;
      if (w + 2 * step < w1) load(w + 2 * step, x[0]);
      f(x[1], (w + step) * 8 - shift);
    }
  }
};

struct Shared {
  u64 table[kTable];
  union {
    struct { u64 mass[kBins]; uint32_t count[kBins]; } bins;
    u64 weights[kList];
  };
  u64 list[kList];
  u64 scratch[kWarps], parts[kWarps];
  struct { float sum, rest; int ref; u64 upto; } pieces[kWarps * kPieces];  // of the warps' ranges
  struct { u64 before, below, under; int piece; } fast;  // where the number falls
  double drop;
  u64 slots[2][3][kBlocks];  // values of the cluster's blocks, in turns
  struct { u64 before; uint32_t bin, count; int way; } found;  // (the first block's)
  uint32_t listed;
  int chosen;
};

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) v += __shfl_xor_sync(0xffffffffu, v, x);
  return v;
}
__device__ __forceinline__ u64 warp_max(u64 v) {
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, x));
  return v;
}
// The sum of v over the block's threads up to this one.
__device__ __forceinline__ u64 block_scan(u64 v, u64* scratch, u64* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int y = 1; y < 32; y <<= 1) {
    const u64 t = __shfl_up_sync(0xffffffffu, v, y);
    if (lane >= y) v += t;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = v;
  __syncthreads();
  u64 sum = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) v += sum;
    sum += scratch[w];
  }
  *total = sum;
  return v;
}
// Sorts the first n in falling order; what lies behind them up to a power of two is written over.
__device__ __forceinline__ void sort_falling(u64* x, int n) {
  int m = 2;
  while (m < n) m *= 2;
  for (int i = n + threadIdx.x; i < m; i += kThreads) x[i] = 0;
  for (int k = 2; k <= m; k *= 2)
    for (int j = k / 2; j > 0; j /= 2) {
      __syncthreads();
      for (int i = threadIdx.x; i < m / 2; i += kThreads) {
        const int a = (i & ~(j - 1)) * 2 + (i & (j - 1)), b = a + j;
        const u64 u = x[a], v = x[b];
        if ((u < v) == !(a & k)) x[a] = v, x[b] = u;
      }
    }
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 3) sample_token_kernel(const __grid_constant__ SampleParams p) {
  __shared__ Shared sm;
  cg::cluster_group cluster = cg::this_cluster();
  const gpt_sample_token_args& a = p.a;
  const int blocks = cluster.num_blocks(), part = cluster.block_rank();
  after_stream();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t b = blockIdx.x / blocks;
  RowView<T> row;
  row.z = (const T*)a.logits + b * a.logits_stride, row.vocab = a.vocab;
  row.shift = (int)((reinterpret_cast<uintptr_t>(row.z) / sizeof(T)) & 7);
  const int units = (int)(((int64_t)a.vocab + row.shift + 7) / 8);
  const int b0 = (int)((int64_t)part * units / blocks), b1 = (int)((int64_t)(part + 1) * units / blocks);
  const int w0 = b0 + (int)((int64_t)warp * (b1 - b0) / kWarps), w1 = b0 + (int)((int64_t)(warp + 1) * (b1 - b0) / kWarps);
  const float temperature = a.temperature ? a.temperature[b] : 1.f, u = a.uniform[b];
  const int top_k = a.top_k ? a.top_k[b] : 0;
  const float top_p = a.top_p ? a.top_p[b] : 1.f, min_p = a.min_p ? a.min_p[b] : 0.f;

  // A value of each block to all of them; what the cluster's blocks wrote before is visible after it.
  int turn = 0;
  auto share = [&](u64 x, u64 y, u64 z) {  // by all threads of the block alike
    if (tid < blocks) {
      u64(*to)[kBlocks] = cluster.map_shared_rank(sm.slots[turn & 1], tid);
      to[0][part] = x, to[1][part] = y, to[2][part] = z;
    }
    if (blocks > 1) cluster.sync();
    else __syncthreads();
    return sm.slots[turn++ & 1];
  };
  auto block_sum = [&](u64 v) {
    v = warp_sum(v);
    __syncthreads();
    if (lane == 0) sm.scratch[warp] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += sm.scratch[w];
    return v;
  };
  auto answer = [&](int token, float logprob, int kept) {
    if (a.token) a.token[b] = token;
    if (a.logprob) a.logprob[b] = logprob;
    if (a.kept) a.kept[b] = kept;
  };
  if (blocks > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");

  auto make_table = [&] {
    for (int i = tid; i < kTable; i += kThreads) sm.table[i] = __umul64hi(p.coarse[i >> 5], p.fine[i & 31]) << 1;
  };
  auto log_of = [&](float w, float sum) { return logf(__fdiv_rn(w, sum)); };
  // c = log2 e / T in two floats
  float c_hi = 0.f, c_lo = 0.f;
  if (temperature < INFINITY) {
    constexpr double kLog2e = 1.442695040888963407;
    constexpr float kHi = (float)kLog2e, kLo = (float)(kLog2e - (double)kHi);
    const float t = fmaxf(temperature, 0x1p-126f);
    c_hi = __fdiv_rn(kHi, t), c_lo = __fdiv_rn(__fadd_rn(__fmaf_rn(-c_hi, t, kHi), kLo), t);
  }
  Weigher weight;
  weight.table = sm.table, weight.unit = p.unit;
  auto set_top = [&](float m) { weight.mh = 0.5f * m, weight.c_hi = 2.f * c_hi, weight.c_lo = 2.f * c_lo, weight.infinite = m == INFINITY; };

  u64 best = 0;
  const bool limits = (top_k >= 1 && top_k < a.vocab) || top_p < 1.f || min_p > 0.f;
  if (temperature > 0.f && !limits && c_hi > 1e-30f) {
    FastSum f;
    f.start(c_hi, c_lo);
    const int steps = (w1 - w0 + 31) / 32, each = (steps + 2 * kPieces - 1) / (2 * kPieces) * 64;  // units of a piece
    {
      float x[2][8];
      if (w0 + lane < w1) row.load(w0 + lane, x[0]);
      for (int i = 0; i < kPieces; ++i) {
        const int end = min(w1, w0 + (i + 1) * each);
        f.clear();
        for (int w = w0 + i * each + lane; w < end; w += 64) {
          if (w + 32 < w1) row.load(w + 32, x[1]);
          f.add(x[0]);
          if (w + 64 < w1) row.load(w + 64, x[0]);
          if (w + 32 < end) f.add(x[1]);
        }
        __syncwarp();
        f.join_warp();
        auto& piece = sm.pieces[warp * kPieces + i];
        if (lane == 0) piece.sum = f.sum, piece.rest = f.rest, piece.ref = f.ref;
      }
    }
    const uint32_t gone = __reduce_add_sync(0xffffffffu, f.missing), bad = __any_sync(0xffffffffu, f.bad);
    const u64 top = warp_max(composite(f.top, 0));
    if (lane == 0) sm.scratch[warp] = top, sm.parts[warp] = (u64)bad << 32 | gone;
    __syncthreads();
    u64 first = 0, flags = 0, sum = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) first = max(first, sm.scratch[i]), flags += sm.parts[i];
    // the pieces as integers, in units of 2^(1 - U) of 2^mine: with the largest weight about 1
    const int mine = first && flags >> 32 == 0 ? __float2int_rn(value_of((uint32_t)(first >> 32)) * c_hi) : -(1 << 22);
    if (warp == 0) {
      auto whole = [&](const auto& piece) {
        const int up = piece.ref - mine + p.unit - 1;  // in two factors: up to 2^48 and more down than a float goes
        const float a = power(min(up, 0)), b = power(max(up, 0));
        return (u64)(__float2ll_rn(piece.sum * a * b) + __float2ll_rn(piece.rest * a * b));
      };
      const u64 v0 = whole(sm.pieces[2 * lane]), v1 = whole(sm.pieces[2 * lane + 1]);
      u64 upto = v0 + v1;
#pragma unroll
      for (int y = 1; y < 32; y <<= 1) {
        const u64 t = __shfl_up_sync(0xffffffffu, upto, y);
        if (lane >= y) upto += t;
      }
      sm.pieces[2 * lane].upto = upto - v1, sm.pieces[2 * lane + 1].upto = upto;
      sum = __shfl_sync(0xffffffffu, upto, 31);
    }
    if (blocks > 1) asm volatile("barrier.cluster.wait;" ::: "memory");
    const u64(*got)[kBlocks] = share(sum, (u64)(uint32_t)mine << 32 | (uint32_t)(first >> 32), flags);  // (by the first warp's threads)
    uint32_t top_key = 0;
    int ref = -(1 << 22);
    flags = 0;
    for (int i = 0; i < blocks; ++i) top_key = max(top_key, (uint32_t)got[1][i]), ref = max(ref, (int)(got[1][i] >> 32)), flags += got[2][i];
    if (top_key == 0) {
      if (part == 0 && tid == 0) answer(-1, -INFINITY, 0);
      return;
    }
    const float m = value_of(top_key);
    set_top(m);
    int accepted = 0;
    if (flags >> 32 == 0) {
      auto moved = [&](u64 v, int from) { return ref - from < 64 ? v >> (ref - from) : 0ull; };
      u64 all = 0, before = 0;
      for (int i = 0; i < blocks; ++i) {
        if (i == part) before = all;
        all += moved(got[0][i], (int)(got[1][i] >> 32));
      }
      // The piece in which the number falls, surely: each sum is off by 2^-21 of itself and
      // some units.
      if (tid == 0) sm.fast.piece = -1;
      __syncthreads();
      const u64 goal = u >= 1.f ? all : u > 0.f ? part_of(u, all, false) : 0;
      if (tid < kWarps * kPieces) {
        const u64 from = before + (tid ? moved(sm.pieces[tid - 1].upto, mine) : 0), to = before + moved(sm.pieces[tid].upto, mine);
        const u64 off = ((from + goal) >> 21) + 256;
        if (goal >= from + off) {
          const u64 local = goal - from;
          const u64 off_to = ((to + goal) >> 21) + 256;
          if (to > goal + off_to) sm.fast.piece = tid, sm.fast.before = from, sm.fast.below = local - min(local, off), sm.fast.under = local + off;
        }
      }
      __syncthreads();
      const int piece = sm.fast.piece;
      if (piece >= 0) {
        make_table();
        __syncthreads();
        const int s = b0 + (int)((int64_t)(piece / kPieces) * (b1 - b0) / kWarps), e = b0 + (int)((int64_t)(piece / kPieces + 1) * (b1 - b0) / kWarps);
        const int piece_units = ((e - s + 31) / 32 + 2 * kPieces - 1) / (2 * kPieces) * 64;
        const int s0 = s + piece % kPieces * piece_units, s1 = min(e, s0 + piece_units);
        const int per = (s1 - s0 + kThreads - 1) / kThreads, t0 = min(s1, s0 + tid * per), t1 = min(s1, t0 + per);
        u64 own = 0, total;
        row.each(t0, t1, 0, 1, [&](const float* x, int) {
#pragma unroll
          for (int i = 0; i < 8; ++i) own += weight(x[i]);
        });
        u64 upto = block_scan(own, sm.scratch, &total) - own;
        // from these sums' units to the weights', 2^-U of 2^(c m): to 2^-20
        const float up = exp2f(1.f - fmaf(m, c_lo, fmaf(m, c_hi, -(float)ref)));
        const u64 below = (u64)((float)sm.fast.below * up * (1.f - 0x1p-20f)), under = (u64)((float)sm.fast.under * up * (1.f + 0x1p-20f)) + 1;
        if (upto <= below && upto + own > under)
          row.each(t0, t1, 0, 1, [&](const float* x, int id) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const u64 w = weight(x[i]);
              if (upto <= below && upto + w > under) {
                answer(id + i, log_of((float)w, (float)all * up), units * 8 - (int)flags);
                accepted = 1;
              }
              upto += w;
            }
          });
      }
      accepted = __syncthreads_or(accepted);
    }
    const u64(*verdict)[kBlocks] = share(accepted, 0, 0);
    for (int i = 0; i < blocks; ++i) accepted |= (int)verdict[0][i];
    if (accepted) return;
    make_table();
    __syncthreads();
  } else {
  // 1. the first token in order
  {
    // (doubles are slow: by one warp, while the logits are under way)
    if (min_p > 0.f && min_p <= 1.f && warp == kWarps - 1) sm.drop = log((double)min_p) * (double)temperature;
    float top = -INFINITY;
    int at = 0;
    row.each(w0, w1, lane, 32, [&](const float* x, int id) {
      float m = x[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) m = fmaxf(m, x[i]);
      if (m > top) {
        top = m;
#pragma unroll
        for (int i = 7; i >= 0; --i)
          if (x[i] == m) at = id + i;
      }
    });
    best = warp_max(composite(top, at));
    if (lane == 0) sm.scratch[warp] = best;
    make_table();
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) best = max(best, sm.scratch[w]);
    if (blocks > 1) asm volatile("barrier.cluster.wait;" ::: "memory");
    const u64(*got)[kBlocks] = share(best, 0, 0);
    for (int i = 0; i < blocks; ++i) best = max(best, got[0][i]);
  }
  if (best == 0 || !(temperature > 0.f)) {
    if (part == 0 && tid == 0) best == 0 ? answer(-1, -INFINITY, 0) : answer(id_of(best), 0.f, 1);
    return;
  }
  set_top(value_of((uint32_t)(best >> 32)));
  }
  const float m = 2.f * weight.mh;
  // what min_p keeps
  u64 least = 1;
  if (min_p > 1.f) {
    least = best;
  } else if (min_p > 0.f) {
    const float from = m == INFINITY ? m : __double2float_ru((double)m + sm.drop);
    least = min((u64)key_of(from) << 32, best);
    if (least == 0) least = 1;
  }

  // Bins of equal width from m down; the last one goes on to the end.
  const float per_bin = kBins / (32.f * fmaxf(1.f, fminf(temperature, 1e30f)));
  auto bin_of = [&](float z) { return (int)fminf((m - z) * per_bin, (float)(kBins - 1)); };
  auto push = [&](u64 comp) {
    uint32_t* listed = cluster.map_shared_rank(&sm.listed, 0);
    const uint32_t at = atomicAdd(listed, 1u);
    if (at < kList) cluster.map_shared_rank(sm.list, 0)[at] = comp;
  };

  // By the first block: the draw among the list's first n, in falling order, whose weights are in sm.weights.
  auto draw_from_list = [&](int n, u64 sum) {
    const u64 goal = goal_of(u, sum);
    u64* by_id = sm.list;
    u64 comps[kList / kThreads];
#pragma unroll
    for (int i = 0; i < kList / kThreads; ++i) comps[i] = tid + i * kThreads < n ? sm.list[tid + i * kThreads] : 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kList / kThreads; ++i)  // rising ids: falling ~id
      if (tid + i * kThreads < n) by_id[tid + i * kThreads] = (u64)(uint32_t)comps[i] << 32 | (uint32_t)(tid + i * kThreads);
    __syncthreads();
    sort_falling(by_id, n);
    const int each = (n + kThreads - 1) / kThreads;
    u64 mine = 0, total;
    for (int i = tid * each; i < min(n, (tid + 1) * each); ++i) mine += sm.weights[(uint32_t)by_id[i]];
    u64 upto = block_scan(mine, sm.scratch, &total) - mine;
    for (int i = tid * each; i < min(n, (tid + 1) * each); ++i) {
      const u64 w = sm.weights[(uint32_t)by_id[i]];
      if (upto < goal && upto + w >= goal) answer((int)~(uint32_t)(by_id[i] >> 32), log_of((float)w, (float)sum), n);
      upto += w;
    }
  };
  // By the first block: the list sorted, weights of its first n, and their sum.
  auto weigh_list = [&](int n) {
    u64 sum = 0;
    for (int i = tid; i < n; i += kThreads) {
      const u64 w = weight(value_of((uint32_t)(sm.list[i] >> 32)));
      sm.weights[i] = w, sum += w;
    }
    return block_sum(sum);
  };
  // How many of the list's first n, whose weights are in sm.weights, it takes for a sum of at least `goal`.
  auto fewest = [&](int n, u64 goal) {
    const int each = (n + kThreads - 1) / kThreads;
    u64 mine = 0, total;
    for (int i = tid * each; i < min(n, (tid + 1) * each); ++i) mine += sm.weights[i];
    u64 upto = block_scan(mine, sm.scratch, &total) - mine;
    for (int i = tid * each; i < min(n, (tid + 1) * each); ++i) {
      if (upto < goal && upto + sm.weights[i] >= goal) sm.chosen = i + 1;
      upto += sm.weights[i];
    }
    __syncthreads();
    return sm.chosen;
  };

  // The last token of the prefix of `target` tokens, or of the fewest whose weights sum to at
  // least that, among those at or above `floor`.  0: the row is done (all that counts was in
  // the list).  kMass: target is top_p of all weights; kCount: `floor` where there are not as many.
  enum { kCount, kMass };
  enum { kBin, kWhole, kNoLimit };
  auto select = [&](int by, u64 target, u64 floor) -> u64 {
    u64 lo = 0, hi = 0;  // of the composite keys that are left, after the first round
    int shift = -1, bin = 0;
    u64 before = 0;
    for (int round = 0;; ++round) {
      for (int i = tid; i < kBins; i += kThreads) sm.bins.mass[i] = 0, sm.bins.count[i] = 0;
      if (tid == 0) sm.listed = 0;
      __syncthreads();
      auto place = [&](float z, u64 comp) {  // the bin, -1: none
        if (comp < floor) return -1;
        if (shift < 0) return bin_of(z);
        return comp >= lo && comp <= hi ? (int)((hi - comp) >> shift) : -1;
      };
      row.each(w0, w1, lane, 32, [&](const float* x, int id) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int at = place(x[i], composite(x[i], id + i));
          if (at < 0) continue;
          atomicAdd(&sm.bins.count[at], 1u);
          if (by == kMass) atomicAdd(&sm.bins.mass[at], weight(x[i]));
        }
      });
      __syncthreads();
      if (blocks > 1) {
        cluster.sync();  // the first block's bins have been cleared and filled
        if (part > 0)
          for (int i = tid; i < kBins; i += kThreads) {
            if (sm.bins.count[i]) atomicAdd(cluster.map_shared_rank(sm.bins.count, 0) + i, sm.bins.count[i]);
            if (sm.bins.mass[i]) atomicAdd(cluster.map_shared_rank(sm.bins.mass, 0) + i, sm.bins.mass[i]);
          }
        cluster.sync();
      }
      if (part == 0) {
        constexpr int kPer = kBins / kThreads;
        u64 mass = 0, count = 0, all_mass, all_count;
#pragma unroll
        for (int i = 0; i < kPer; ++i) mass += sm.bins.mass[tid * kPer + i], count += sm.bins.count[tid * kPer + i];
        u64 mass_to = block_scan(mass, sm.scratch, &all_mass) - mass;
        u64 count_to = block_scan(count, sm.scratch, &all_count) - count;
        if (round == 0 && by == kMass) target = max(part_of(top_p, all_mass, true), 1ull);
        if (tid == 0) sm.found.way = round == 0 && by == kCount && target >= all_count ? kNoLimit : kBin;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const u64 here = by == kMass ? sm.bins.mass[tid * kPer + i] : sm.bins.count[tid * kPer + i];
          const u64 to = before + (by == kMass ? mass_to : count_to);
          if (to < target && to + here >= target) {
            sm.found.bin = tid * kPer + i, sm.found.before = to, sm.found.count = sm.bins.count[tid * kPer + i];
            if (round == 0 && sm.found.way == kBin && count_to + sm.found.count <= kList) sm.found.way = kWhole;
          }
          mass_to += sm.bins.mass[tid * kPer + i], count_to += sm.bins.count[tid * kPer + i];
        }
        __syncthreads();
      }
      // the choice, to all blocks: the bin, and whether the list takes all above its end
      const u64(*got)[kBlocks] = share((u64)sm.found.bin << 32 | sm.found.count, sm.found.way, sm.found.before);
      if (got[1][0] == kNoLimit) return floor;
      bin = (int)(got[0][0] >> 32), before = got[2][0];
      const bool take_all = got[1][0] == kWhole;
      const uint32_t count = (uint32_t)got[0][0];
      u64 low = ~0ull, high = 0;
      row.each(w0, w1, lane, 32, [&](const float* x, int id) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const u64 comp = composite(x[i], id + i);
          const int at = place(x[i], comp);
          if (at < 0 || (take_all ? at > bin : at != bin)) continue;
          if (take_all || count <= kList) push(comp);
          else low = min(low, comp), high = max(high, comp);
        }
      });
      if (!take_all && count > kList) {  // once more, in this bin
        low = ~warp_max(~low), high = warp_max(high);
        __syncthreads();
        if (lane == 0) sm.parts[warp] = low, sm.scratch[warp] = high;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) low = min(low, sm.parts[w]), high = max(high, sm.scratch[w]);
        const u64(*ends)[kBlocks] = share(low, high, 0);
        for (int i = 0; i < blocks; ++i) low = min(low, ends[0][i]), high = max(high, ends[1][i]);
        lo = low, hi = high, shift = 0;
        while ((hi - lo) >> shift >= kBins) ++shift;
        continue;
      }
      if (blocks > 1) cluster.sync();
      else __syncthreads();
      u64 last = 0;
      if (part == 0) {
        const int n = (int)sm.listed;
        sort_falling(sm.list, n);
        if (!take_all) {
          if (by == kCount) {
            last = sm.list[target - before - 1];
          } else {
            weigh_list(n);
            last = sm.list[fewest(n, target - before) - 1];
          }
        } else {
          int keep = n;
          if (by == kCount) keep = (int)target;
          u64 sum = weigh_list(keep);
          if (by == kMass) keep = fewest(keep, target);
          else if (top_p < 1.f) keep = fewest(keep, max(top_p > 0.f ? part_of(top_p, sum, true) : 0, 1ull));
          int above = 0;  // min_p
          for (int i = tid; i < keep; i += kThreads) above += sm.list[i] >= least;
          keep = (int)block_sum(above);
          sum = 0;
          for (int i = tid; i < keep; i += kThreads) sum += sm.weights[i];
          draw_from_list(keep, block_sum(sum));
        }
      }
      if (take_all) return 0;
      return share(last, 0, 0)[0][0];
    }
  };

  u64 last = 1;  // the kept tokens are those at or above it
  if (top_k >= 1 && top_k < a.vocab) {
    last = top_k == 1 ? best : select(kCount, top_k, 1);
    if (last == 0) return;
  }
  if (top_p <= 0.f) {
    last = best;
  } else if (top_p < 1.f && last != best) {
    last = select(kMass, 0, last);
    if (last == 0) return;
  }
  last = max(last, least);

  // 4. the kept tokens' weights
  u64 sum = 0, kept = 0;
  row.each(w0, w1, lane, 32, [&](const float* x, int id) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (composite(x[i], id + i) >= last) sum += weight(x[i]), ++kept;
  });
  sum = warp_sum(sum), kept = warp_sum(kept);
  __syncthreads();
  if (lane == 0) sm.parts[warp] = sum, sm.scratch[warp] = kept;
  __syncthreads();
  sum = kept = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) sum += sm.parts[w], kept += sm.scratch[w];
  const u64(*got)[kBlocks] = share(sum, kept, 0);
  u64 before = 0;
  sum = kept = 0;
  for (int i = 0; i < blocks; ++i) {
    if (i == part) before = sum;
    sum += got[0][i], kept += got[1][i];
  }
  const u64 goal = goal_of(u, sum);
  if (before >= goal || before + got[0][part] < goal) return;  // another block's
  int w = 0;
  while (before + sm.parts[w] < goal) before += sm.parts[w++];
  const int s0 = b0 + (int)((int64_t)w * (b1 - b0) / kWarps), s1 = b0 + (int)((int64_t)(w + 1) * (b1 - b0) / kWarps);
  const int each = (s1 - s0 + kThreads - 1) / kThreads;  // units of a thread, side by side
  auto weigh = [&](const float* x, int id, int i) { return composite(x[i], id + i) >= last ? weight(x[i]) : 0ull; };
  u64 mine = 0, total;
  const int t0 = min(s1, s0 + tid * each), t1 = min(s1, t0 + each);
  row.each(t0, t1, 0, 1, [&](const float* x, int id) {
#pragma unroll
    for (int i = 0; i < 8; ++i) mine += weigh(x, id, i);
  });
  u64 upto = before + block_scan(mine, sm.scratch, &total) - mine;
  if (upto >= goal || upto + mine < goal) return;
  row.each(t0, t1, 0, 1, [&](const float* x, int id) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const u64 w = weigh(x, id, i);
      if (upto < goal && upto + w >= goal) answer(id + i, log_of((float)w, (float)sum), (int)kept);
      upto += w;
    }
  });
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
  while ((int64_t)a->vocab > (int64_t)1 << (63 - p.unit)) --p.unit;
  static const struct Powers {
    u64 coarse[32], fine[32];
    Powers() {
      for (int i = 0; i < 32; ++i) {
        coarse[i] = (u64)std::llroundl(std::exp2l(62.0L + i / 32.0L));
        fine[i] = (u64)std::exp2l(63.0L + i / 1024.0L);
      }
    }
  } powers;
  std::copy(powers.coarse, powers.coarse + 32, p.coarse);
  std::copy(powers.fine, powers.fine + 32, p.fine);
  int blocks = 1;
  while (blocks < kBlocks && a->vocab / (2 * blocks) >= 512 && (int64_t)a->rows * 2 * blocks <= 608) blocks *= 2;
  if ((int64_t)a->rows * blocks > INT32_MAX) return call_error(GPT_ERR_UNSUPPORTED, "too many rows");
  const cudaStream_t st = (cudaStream_t)cuda_stream;
  return launch_after("gpt_sample_token", a->dtype == GPT_DTYPE_BF16 ? sample_token_kernel<__nv_bfloat16> : sample_token_kernel<float>,
                      dim3(a->rows * blocks), kThreads, 0, blocks, st, p);
}
