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
// A row is the work of a cluster of blocks, each with a range of its ids, each warp with a
// part of that.  Nothing is written; the logits are read again (from L2) where a row needs
// more than one pass:
//  - without limits: one pass of sums in fp32, good to 2^-21, names the token unless the number
//    falls that near a border between two; only then the weights are summed as integers;
//  - with top_k, or min_p alone: a first pass takes the largest logit of each thread.  The n-th
//    largest of these has at least n tokens at or above it, so that the tokens at or above its bin
//    (1,024 of equal width below the row's largest) hold the first top_k.  A second pass lists
//    them; the first block takes the limits and draws from the list, by counting for each entry
//    what lies before it;
//  - with top_p alone: by_sums;
//  - where a list does not hold what it must: slow_row, bins of counts and sums of all tokens, as
//    many rounds as it takes, then the sums of the kept ones by warp.
// Bound: a few rows by the chain of phases, each with a barrier of the cluster (0.7 us): 1 row of 12,288 7.5 us without
// limits, 12 with top_k, 64 of 50,304 14.5 and 22; with top_p alone by passes over the row (14 and 40).  Many rows by
// instructions: 512 of 131,072 in fp32 without limits 90 us, 3.0 TB/s, 25 instructions a token; in bf16 79; with top_p
// alone 296.  Lists that overflow are finished by one block: 1 row of 131,072 with a top_k of 900 to 2,000 takes 160 to
// 220 us (of 200 19, of 5,000, where all blocks stay, 50), with a min_p that keeps 20,000 97.
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
constexpr int kShares = 2048;     // bins of by_sums
constexpr int kList = 1024;
// Entries of a list that are compared with one another, one a thread; longer ones go through bins.  (Rows of
// 12,288 with a top_k of up to 200: 13.6 us, and 17.6 through bins; 512 of 131,072: 119 and 133.)
constexpr int kShort = kThreads;
constexpr int kTable = 1024;
constexpr int kPieces = 2;        // of a warp's range, where sums are in fp32 (with 4 a row of 131,072 10.4 us, 9.7 so)
using u64 = unsigned long long;

struct SampleParams {
  gpt_sample_token_args a;
  int32_t unit;               // U
  u64 coarse[32], fine[32];   // 2^62 2^(i/32), 2^63 2^(i/1024)
};

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
    u64 w[2];
    two(z, -INFINITY, w);
    return w[0];
  }
  __device__ __forceinline__ void eight(const float* x, u64* w) const {
#pragma unroll
    for (int i = 0; i < 8; i += 2) two(x[i], x[i + 1], w + i);
  }
  __device__ __forceinline__ void two(float z0, float z1, u64* w) const {
    constexpr double kLn2 = 0.69314718055994530942, kUp = 4398046511104.0;  // 2^42
    constexpr float kL = (float)kLn2, kL42 = (float)(kL * kUp), kRest42 = (float)((kLn2 - (double)kL) * kUp);
    constexpr float kC2 = (float)(kLn2 * kLn2 / 2 * kUp), kC3 = (float)(kLn2 * kLn2 * kLn2 / 6 * kUp);
    constexpr float kMagic = 12288.f;  // 1.5 2^13: sums with it are multiples of 2^-10
    const Pair half(0.5f), minus(-1.f), top(mh), hi(c_hi), z(z0, z1);
    // s + e = (z - m) / 2
    const Pair s = fma(z, half, Pair(-mh)), t = fma(z, Pair(-0.5f), s);
    const Pair e = fma(add(top, t), minus, fma(z, half, fma(s, minus, t)));
    const float2 q = mul(s, hi).both();
    const Pair p(fmaxf(q.x, -100.f), fmaxf(q.y, -100.f));  // (NaN too) nothing is left of 2^-100
    const Pair up = add(p, Pair(kMagic)), r = add(p, fma(up, minus, Pair(kMagic)));
    const Pair low = fma(s, Pair(c_lo), fma(e, hi, fma(s, hi, mul(s, Pair(-c_hi)))));
    const Pair a = mul(r, Pair(kL42)), a_low = fma(r, Pair(kL42), mul(r, Pair(-kL42)));
    const Pair rest = fma(mul(r, r), fma(r, Pair(kC3), Pair(kC2)), fma(r, Pair(kRest42), fma(low, Pair(kL42), a_low)));
    const float2 up2 = up.both(), a2 = a.both(), rest2 = rest.both();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int J = (int)(__float_as_uint(i ? up2.y : up2.x) - __float_as_uint(kMagic));
      const int more = __float2int_rn(i ? a2.y : a2.x) + __float2int_rn(i ? rest2.y : rest2.x);
      const u64 base = table[J & (kTable - 1)];
      const u64 v = base + (u64)(((int64_t)more * (int)(base >> 32)) >> 10);
      const u64 rounded = ((v >> min(61 - unit - (J >> 10), 63)) + 1) >> 1;
      w[i] = infinite ? ((i ? z1 : z0) == INFINITY ? 1ull << unit : 0ull) : rounded;
    }
  }
};

// The least integer that is at least f x, the largest that is at most f x, for 0 <= f < 1.
__device__ __noinline__ u64 part_of(float f, u64 x, bool up) {
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

// Eight logits as loaded from a boundary of their size on, unpacked where they are used.
template <typename T> struct Unit;
template <> struct Unit<float> {
  float x[8];
  __device__ __forceinline__ void load(const float* z) {
    asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
                 : "l"(z));
  }
  __device__ __forceinline__ void set(int i, const float* z, bool there) { x[i] = there ? *z : -INFINITY; }
  __device__ __forceinline__ const float* values(float*) const { return x; }
};
template <> struct Unit<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* z) {
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(z));
  }
  __device__ __forceinline__ void set(int i, const __nv_bfloat16* z, bool there) {
    const uint32_t bits = there ? *reinterpret_cast<const uint16_t*>(z) : 0xff80u;
    uint32_t& w = (&u.x)[i / 2];
    w = i & 1 ? w | bits << 16 : bits;
  }
  __device__ __forceinline__ const float* values(float* to) const {
    Piece<__nv_bfloat16>::unpack(u, to);
    return to;
  }
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}
// Of eight; without NaN, if one is a number.
__device__ __forceinline__ float max_of(const float* x) { return max3(max3(x[0], x[1], x[2]), max3(x[3], x[4], x[5]), fmaxf(x[6], x[7])); }

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
    const float m = max_of(x);
    Pair all(x[0], x[1]);
#pragma unroll
    for (int i = 2; i < 8; i += 2) all = pgs::add(all, Pair(x[i], x[i + 1]));
    const float2 sums = all.both();
    if (!(sums.x + sums.y > -INFINITY))
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
    // up = c z to the next integer, over a number whose low bits are -ref: its own low bits are the exponent
    const float magic = 12582912.f - (float)ref;  // 1.5 2^23
    Pair w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Pair z(fmaxf(x[2 * i], low), fmaxf(x[2 * i + 1], low)), hi(c_hi);
      const Pair up = fma(z, hi, Pair(magic));
      const float2 r = fma(z, Pair(c_lo), fma(z, hi, fma(up, Pair(-1.f), Pair(magic)))).both(), n = up.both();
      float f, g;
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(f) : "f"(r.x));
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(g) : "f"(r.y));
      w[i] = Pair(__int_as_float(__float_as_int(f) + (__float_as_int(n.x) << 23)), __int_as_float(__float_as_int(g) + (__float_as_int(n.y) << 23)));
    }
    const float2 v = pgs::add(pgs::add(w[0], w[1]), pgs::add(w[2], w[3])).both();
    two_sum(v.x + v.y, 0.f);
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
#pragma unroll 1
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
  __device__ __forceinline__ void load(int w, Unit<T>& x) const {
    const int64_t id = (int64_t)w * 8 - shift;
    if (id >= 0 && id + 8 <= vocab) {
      x.load(z + id);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x.set(i, z + id + i, id + i >= 0 && id + i < vocab);
    }
  }
  // f(8 logits, the first's id) for units w0 + lane, w0 + lane + 32, ... below w1, kAhead more under
  // way.  Code that runs once or twice costs its instructions' way from memory (61 % of the waits,
  // with four copies of each f): one copy of a long f, the next unit under way; a few of a short one.
  template <int kAhead = 1, typename F>
  __device__ __forceinline__ void each(int w0, int w1, F f) const {
    Unit<T> x[kAhead];
    int w = w0 + (threadIdx.x & 31);
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (w + 32 * i < w1) load(w + 32 * i, x[i]);
#pragma unroll 1
    for (; w < w1; w += 32 * kAhead) {
      if constexpr (kAhead == 1) {
        Unit<T> next;
        float y[8];
        if (w + 32 < w1) load(w + 32, next);
        f(x[0].values(y), w * 8 - shift);
        x[0] = next;
      } else {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (w + 32 * i < w1) {
            float y[8];
            f(x[i].values(y), (w + 32 * i) * 8 - shift);
          }
          if (w + 32 * (kAhead + i) < w1) load(w + 32 * (kAhead + i), x[i]);
        }
      }
    }
  }
};

// The tokens at or above a composite key (of 1: all of them).
struct Kept {
  float z;
  int id;
  __device__ __forceinline__ explicit Kept(u64 last) : z(last > 1 ? value_of((uint32_t)(last >> 32)) : -INFINITY), id(last > 1 ? id_of(last) : INT32_MIN) {}  // (not what a unit holds before the row's first token)
  __device__ __forceinline__ bool has(float x, int i) const { return x > z || (x == z && i <= id); }
  __device__ __forceinline__ bool none(const float* x) const {  // of eight
    return !(max_of(x) >= z);
  }
};

struct Shared {
  u64 table[kTable];
  union {
    struct { u64 mass[kBins]; uint32_t count[kBins]; } bins;
    u64 weights[kList];  // of the entries of `all`
    ulonglong2 entries[kShort];
    uint32_t share[kShares];  // of a bin's weights, in units of its first
  };
  union {
    float maxima[kBlocks * kThreads];  // of the cluster's threads (in the first block)
    u64 all[kList];                    // its blocks' lists, side by side (in the first block)
  };
  u64 list[kList];                     // of this block
  u64 scratch[kWarps], parts[kWarps];
  struct { float sum, rest; int ref; u64 upto; } pieces[kWarps * kPieces];  // of the warps' ranges
  u64 slots[2][3][kBlocks];            // values of the cluster's blocks, in turns
  union {
    struct { u64 before, below, under; int piece; } fast;       // where the number falls
    struct { u64 before, all; uint32_t bin, count; int way; } found;  // (the first block's)
    struct { int low, high; uint32_t upto; } ends;                     // (the first block's)
  };
  u64 ends_of[kWarps][2], counts[kWarps];
  u64 sums[kThreads];
  struct { u64 before; int bin; } crossed;
  double drop;
  uint32_t listed, gathered, base;
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
__device__ __noinline__ u64 block_scan(u64 v, u64* scratch, u64* total) {
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
#pragma unroll 4
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) v += sum;
    sum += scratch[w];
  }
  *total = sum;
  return v;
}
// Adds to a sum in shared memory, a word and its carry after the other: atomics of 64 bits go round there for
// each thread that meets another (131,072 equal logits with top_p 884 us; the limits of a list of them 20 us, 4 so).
__device__ __forceinline__ void add64(u64* sum, u64 w) {
  uint32_t* word = reinterpret_cast<uint32_t*>(sum);
  const uint32_t low = (uint32_t)w;
  uint32_t high = (uint32_t)(w >> 32);
  if (low && atomicAdd(word, low) > ~low) ++high;
  if (high) atomicAdd(word + 1, high);
}
// Of the n entries of sm.all at or above `floor`, in falling order or (kById) by rising ids: the one at
// which the running sum of their weights (kCount: of ones) reaches `goal`, which it does.  The range of
// their keys is cut in 256 bins, and that of the bin where that happens again, until it holds one.
// By all threads of the block.
enum { kCount, kMass, kById };
__device__ __noinline__ int cross(Shared& sm, int n, int by, u64 goal, u64 floor) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  static_assert(kThreads == 256, "a bin each");
  auto key_of_entry = [&](u64 comp) { return by == kById ? (u64) ~(uint32_t)comp : ~comp; };
  u64 lo = 0, hi = ~0ull, before = 0;
  while (true) {
    u64 first = ~0ull, last = 0;
#pragma unroll 1
    for (int i = tid; i < n; i += kThreads) {
      const u64 comp = sm.all[i], key = key_of_entry(comp);
      if (comp >= floor && key >= lo && key <= hi) first = min(first, key), last = max(last, key);
    }
    first = ~warp_max(~first), last = warp_max(last);
    if (lane == 0) sm.ends_of[warp][0] = first, sm.ends_of[warp][1] = last;
    sm.sums[tid] = 0;
    __syncthreads();
    lo = ~0ull, hi = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) lo = min(lo, sm.ends_of[w][0]), hi = max(hi, sm.ends_of[w][1]);
    if (lo == hi) break;
    const int shift = max(0, 56 - __clzll((long long)(hi - lo)));
#pragma unroll 1
    for (int i = tid; i < n; i += kThreads) {
      const u64 comp = sm.all[i], key = key_of_entry(comp);
      if (comp >= floor && key >= lo && key <= hi) add64(&sm.sums[(key - lo) >> shift], by == kCount ? 1 : sm.weights[i]);
    }
    __syncthreads();
    u64 total;
    const u64 here = sm.sums[tid], to = before + block_scan(here, sm.scratch, &total) - here;
    if (to < goal && to + here >= goal) sm.crossed.before = to, sm.crossed.bin = tid;
    __syncthreads();
    before = sm.crossed.before;
    lo += (u64)sm.crossed.bin << shift, hi = lo + (1ull << shift) - 1;
  }
  for (int i = tid; i < n; i += kThreads)
    if (sm.all[i] >= floor && key_of_entry(sm.all[i]) == lo) sm.chosen = i;
  __syncthreads();
  return sm.chosen;
}

template <typename T>
__device__ __noinline__ bool finish_long(const SampleParams& p, Shared& sm, int n, u64 best, u64 whole, float m, int top_k);

// What a thread knows of its row.
template <typename T>
struct Sampler {
  const SampleParams& p;
  const gpt_sample_token_args& a;
  Shared& sm;
  cg::cluster_group cluster;
  RowView<T> row;
  int tid, lane, warp;
  int blocks, part, home;     // of the row; the first block's rank in the cluster
  int units, b0, b1, w0, w1;  // of the row; the block's and the warp's
  int64_t b;
  float u, temperature, top_p, min_p, c_hi, c_lo;
  int top_k;
  int turn;
  Weigher weight;

  // alone: the block does the whole row by itself
  __device__ __forceinline__ Sampler(const SampleParams& params, Shared& shared, bool alone) : p(params), a(params.a), sm(shared), cluster(cg::this_cluster()) {
    tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    blocks = cluster.num_blocks(), part = cluster.block_rank(), home = 0, turn = 0;
    int log_blocks = 31 - __clz(blocks);  // (a power of two)
    b = blockIdx.x >> log_blocks;
    if (alone) home = part, blocks = 1, part = 0, log_blocks = 0;
    row.z = (const T*)a.logits + b * a.logits_stride, row.vocab = a.vocab;
    row.shift = (int)((reinterpret_cast<uintptr_t>(row.z) / sizeof(T)) & 7);
    units = (int)(((int64_t)a.vocab + row.shift + 7) / 8);
    b0 = (int)((int64_t)part * units >> log_blocks), b1 = (int)((int64_t)(part + 1) * units >> log_blocks);
    w0 = warp_begin(warp), w1 = warp_begin(warp + 1);
    u = a.uniform[b], temperature = a.temperature ? a.temperature[b] : 1.f;
    top_k = a.top_k ? a.top_k[b] : 0;
    if (top_k < 1 || top_k >= a.vocab) top_k = 0;
    top_p = a.top_p ? a.top_p[b] : 1.f, min_p = a.min_p ? a.min_p[b] : 0.f;
    // c = log2 e / T in two floats
    c_hi = c_lo = 0.f;
    if (temperature < INFINITY) {
      constexpr double kLog2e = 1.442695040888963407;
      constexpr float kHi = (float)kLog2e, kLo = (float)(kLog2e - (double)kHi);
      const float t = fmaxf(temperature, 0x1p-126f);
      c_hi = __fdiv_rn(kHi, t), c_lo = __fdiv_rn(__fadd_rn(__fmaf_rn(-c_hi, t, kHi), kLo), t);
    }
    weight.table = sm.table, weight.unit = p.unit;
  }
  __device__ __forceinline__ int warp_begin(int w) const { return b0 + (int)((int64_t)w * (b1 - b0) / kWarps); }
  __device__ __forceinline__ void set_top(float m) {
    weight.mh = 0.5f * m, weight.c_hi = 2.f * c_hi, weight.c_lo = 2.f * c_lo, weight.infinite = m == INFINITY;
  }
  __device__ __forceinline__ float top() const { return 2.f * weight.mh; }

  // A value of each block to all of them; what the cluster's blocks wrote before is visible after it.
  __device__ __forceinline__ const u64 (*share(u64 x, u64 y, u64 z))[kBlocks] {  // (the first warp's threads' values)
    if (tid < blocks) {
      u64(*to)[kBlocks] = cluster.map_shared_rank(sm.slots[turn & 1], home + tid);
      to[0][part] = x, to[1][part] = y, to[2][part] = z;
    }
    sync_all();
    return sm.slots[turn++ & 1];
  }
  __device__ __forceinline__ void sync_all() {
    if (blocks > 1) cluster.sync();
    else __syncthreads();
  }
  __device__ __forceinline__ u64 block_sum(u64 v) {
    v = warp_sum(v);
    __syncthreads();
    if (lane == 0) sm.scratch[warp] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += sm.scratch[w];
    return v;
  }
  __device__ __forceinline__ void answer(int token, float logprob, int kept) {
    if (a.token) a.token[b] = token;
    if (a.logprob) a.logprob[b] = logprob;
    if (a.kept) a.kept[b] = kept;
  }
  // The log probability of token `id`, of weight w, from a sum in the same units.  A weight of few units is rounded by much
  // of itself: there its logit gives it.
  __device__ __forceinline__ float log_of(u64 w, float sum, int id) const {
    float part = (float)w, log_w = 0.f;
    if (w < 1u << 22) part = (float)(1ull << weight.unit), log_w = fmaf(0.5f, (float)row.z[id], -weight.mh) * weight.c_hi * 0.693147181f;
    return log_w + logf(__fdiv_rn(part, fmaxf(sum, part)));  // (a sum in fp32 can lie below the one weight in it)
  }

  // Bins of equal width from the largest logit down; the last one goes on to the end.
  __device__ __forceinline__ float per_bin() const { return kBins / (32.f * fmaxf(1.f, fminf(temperature, 1e30f))); }
  __device__ __forceinline__ int bin_of(float z, float each) const { return (int)fminf((top() - z) * each, (float)(kBins - 1)); }

  // The least composite key that min_p keeps.
  __device__ __forceinline__ u64 least(u64 best) const {
    if (min_p > 1.f) return best;
    if (!(min_p > 0.f)) return 1;
    const uint32_t key = key_of(top() == INFINITY ? INFINITY : __double2float_ru((double)top() + sm.drop));
    return key ? min((u64)key << 32 | 0x80000000u, best) : 1;  // (any id)
  }

  // A pass that lists the tokens that f names (f(eight logits, the first's id, name)), then all
  // blocks' lists in the first block's sm.all, sm.gathered of them; those behind kList are lost.
  template <typename F>
  __device__ __forceinline__ void gather(F f) {
    if (tid == 0) sm.listed = 0;
    __syncthreads();
    row.each(w0, w1, [&](const float* x, int id) {
      f(x, id, [&](float z, int i) {
        const uint32_t at = atomicAdd(&sm.listed, 1u);
        if (at < kList) sm.list[at] = composite(z, i);
      });
    });
    __syncthreads();
    const uint32_t n = sm.listed;
    if (tid == 0 && n) sm.base = atomicAdd(cluster.map_shared_rank(&sm.gathered, home), n);
    __syncthreads();
    u64* all = cluster.map_shared_rank(sm.all, home);
    for (uint32_t i = tid; i < min(n, (uint32_t)kList); i += kThreads)
      if (sm.base + i < kList) all[sm.base + i] = sm.list[i];
  }

  // By the first block, of the n <= kShort entries of sm.all: the limits, and the draw among what
  // they keep.  whole: the sum of all tokens' weights, for top_p alone; false: the entries do not reach it.
  __device__ __forceinline__ bool finish_short(int n, u64 best, u64 whole) {
    const u64 mine = tid < n ? sm.all[tid] : 0, from = least(best);
    u64 w = tid < n ? weight(value_of((uint32_t)(mine >> 32))) : 0;
    ulonglong2* entries = sm.entries;
    if (tid < n) entries[tid] = make_ulonglong2(mine, w);
    __syncthreads();
    u64 above = 0;
    int rank = 0;
    if (tid < n) {
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        const ulonglong2 x = entries[i];
        if (x.x > mine) ++rank, above += x.y;
      }
    }
    bool keep = tid < n && mine >= from && (top_k == 0 || rank < top_k);
    if (top_p < 1.f) {
      const u64 sum = block_sum(tid < n && (top_k == 0 || rank < top_k) ? w : 0);
      const u64 goal = max(top_p > 0.f ? part_of(top_p, top_k ? sum : whole, true) : 0, 1ull);
      if (sum < goal) return false;
      keep = keep && above < goal;
    }
    if (!keep) w = 0;
    const u64 sum = block_sum(w);
    const int kept = __syncthreads_count(keep);
    // the kept ones alone, side by side: the first of them in order
    if (keep) entries[rank] = make_ulonglong2(mine, w);
    __syncthreads();
    const u64 goal = goal_of(u, sum);
    u64 upto = 0;
    if (w) {
#pragma unroll 4
      for (int i = 0; i < kept; ++i) {
        const ulonglong2 x = entries[i];
        if ((uint32_t)x.x > (uint32_t)mine) upto += x.y;  // a smaller id
      }
    }
    if (w && upto < goal && upto + w >= goal) answer(id_of(mine), log_of(w, (float)sum, id_of(mine)), kept);
    return true;
  }

  // The weights of a unit below w1, of the tokens at or above the limit.  (One load: one by one, the
  // eight waited for memory each, 3 us of a row's 8.)
  __device__ __forceinline__ void weigh_unit(int w, int w1, const Kept& limit, u64* v) const {
    Unit<T> x;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0;
    if (w >= w1) return;
    row.load(w, x);
    const float* z = x.values(y);
    weight.eight(z, v);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!limit.has(z[i], w * 8 - row.shift + i)) v[i] = 0;
  }

  // Weights of the n entries of sm.all, and their sum.
  __device__ __forceinline__ u64 weigh_list(int n) {
    u64 sum = 0;
    for (int i = tid; i < n; i += kThreads) {
      const u64 w = weight(value_of((uint32_t)(sm.all[i] >> 32)));
      sm.weights[i] = w, sum += w;
    }
    return block_sum(sum);
  }
  __device__ __forceinline__ bool finish(int n, u64 best, u64 whole) { return n <= kShort ? finish_short(n, best, whole) : finish_long<T>(p, sm, n, best, whole, top(), top_k); }

  // Units of a piece of a warp's range: whole steps.
  static constexpr int kStep = 32;
  static __device__ __forceinline__ int piece_units(int range) { return ((range + kStep - 1) / kStep + kPieces - 1) / kPieces * kStep; }

  // What is left to slow_row: nothing, or the row, by all blocks or by this one alone.
  enum { kDone, kTogether, kAlone, kDrawn };

  // Rows without limits.  (A block alone took 45 us for the 131,072 integers of a row: all of them stay
  // until the number's token is known.)
  __device__ __forceinline__ int without_limits() {
    FastSum f;
    f.start(c_hi, c_lo);
    const int each = piece_units(w1 - w0);
    {
      constexpr int kTurns = sizeof(T) == 2 ? 2 : 1;  // (512 rows of 131,072 in bf16 80 us, one at a time 86; in fp32 92 both)
      Unit<T> x;
      if (w0 + lane < w1) row.load(w0 + lane, x);
#pragma unroll 1
      for (int k = 0; k < kPieces; ++k) {
        const int end = min(w1, w0 + (k + 1) * each);
        f.clear();
#pragma unroll(kTurns)
        for (int w = w0 + k * each + lane; w < end; w += 32) {
          Unit<T> next;
          float y[8];
          if (w + 32 < w1) row.load(w + 32, next);
          f.add(x.values(y));
          x = next;
        }
        __syncwarp();
        if (w0 + k * each < w1) f.join_warp();
        auto& piece = sm.pieces[warp * kPieces + k];
        if (lane == 0) piece.sum = f.sum, piece.rest = f.rest, piece.ref = f.ref;
      }
    }
    const uint32_t gone = __reduce_add_sync(0xffffffffu, f.missing), bad = __any_sync(0xffffffffu, f.bad);
    const uint32_t key = __reduce_max_sync(0xffffffffu, key_of(f.top));
    if (lane == 0) sm.scratch[warp] = key, sm.parts[warp] = (u64)bad << 32 | gone;
    __syncthreads();
    u64 first = 0, flags = 0, sum = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) first = max(first, sm.scratch[i]), flags += sm.parts[i];
    // the pieces as integers, in units of 2^(1 - U) of 2^mine: with the largest weight about 1
    const int mine = first && flags >> 32 == 0 ? __float2int_rn(value_of((uint32_t)first) * c_hi) : -(1 << 22);
    if (warp == 0) {
      auto whole = [&](const auto& piece) {
        const int up = piece.ref - mine + weight.unit - 1;  // in two factors: up to 2^48 and more, down to nothing
        const float x = power(min(up, 0)), y = power(max(up, 0));
        return (u64)(__float2ll_rn(piece.sum * x * y) + __float2ll_rn(piece.rest * x * y));
      };
      static_assert(kWarps * kPieces <= 32, "a lane each");
      u64 upto = lane < kWarps * kPieces ? whole(sm.pieces[lane]) : 0;
#pragma unroll
      for (int y = 1; y < 32; y <<= 1) {
        const u64 t = __shfl_up_sync(0xffffffffu, upto, y);
        if (lane >= y) upto += t;
      }
      if (lane < kWarps * kPieces) sm.pieces[lane].upto = upto;
      sum = __shfl_sync(0xffffffffu, upto, 31);
    }
    if (blocks > 1) asm volatile("barrier.cluster.wait;" ::: "memory");
    const u64(*got)[kBlocks] = share(sum, (u64)(uint32_t)mine << 32 | (uint32_t)first, flags);
    uint32_t top_key = 0;
    int ref = -(1 << 22);
    flags = 0;
#pragma unroll 1
    for (int i = 0; i < blocks; ++i) top_key = max(top_key, (uint32_t)got[1][i]), ref = max(ref, (int)(got[1][i] >> 32)), flags += got[2][i];
    if (top_key == 0) {
      if (part == 0 && tid == 0) answer(-1, -INFINITY, 0);
      return kDone;
    }
    const float m = value_of(top_key);
    set_top(m);
    if (flags >> 32) return kTogether;
    int accepted = 0;
    auto moved = [&](u64 v, int from) { return ref - from < 64 ? v >> (ref - from) : 0ull; };
    u64 all = 0, before = 0;
#pragma unroll 1
    for (int i = 0; i < blocks; ++i) {
      if (i == part) before = all;
      all += moved(got[0][i], (int)(got[1][i] >> 32));
    }
    const u64 goal = u >= 1.f ? all : u > 0.f ? part_of(u, all, false) : 0;
    // The piece in which the number falls, surely.  Sums are off by 2^-21 of themselves and some units: one
    // from the row's start, S, less the number's share u of the whole one, W, by
    // |(1 - u) dS - u d(W - S)| <= 2^-21 ((1 - u) S + u (W - S)); the weights as integers by half a unit each.
    auto off_by = [&](u64 from) {
      return (u64)(((float)from * (1.f - u) + (float)(all - min(from, all)) * u) * (0x1p-21f * (1.f + 0x1p-18f))) + 256 + a.vocab;
    };
    if (tid == 0) sm.fast.piece = -1;
    __syncthreads();
    if (tid < kWarps * kPieces) {
      const u64 from = before + (tid ? moved(sm.pieces[tid - 1].upto, mine) : 0), to = before + moved(sm.pieces[tid].upto, mine);
      const u64 off = off_by(from), off_to = off_by(to);
      if (u < 1.f && goal >= from + off && to > goal + off_to)
        sm.fast.piece = tid, sm.fast.below = goal - from - off, sm.fast.under = goal - from + max(off, off_to);
    }
    __syncthreads();
    const int piece = sm.fast.piece;
    if (piece >= 0) {
      // its tokens one after the other, 2,048 at a time
      const int s = warp_begin(piece / kPieces), e = warp_begin(piece / kPieces + 1);
      const int s0 = s + piece % kPieces * piece_units(e - s), s1 = min(e, s0 + piece_units(e - s));
      // from these sums' units to the weights', 2^-U of 2^(c m): to 2^-20
      const float up = exp2f(1.f - fmaf(m, c_lo, fmaf(m, c_hi, -(float)ref)));
      const u64 below = (u64)((float)sm.fast.below * up * (1.f - 0x1p-20f)), under = (u64)((float)sm.fast.under * up * (1.f + 0x1p-20f)) + 1;
      u64 upto = 0;
#pragma unroll 1
      for (int w = s0; w < s1; w += kThreads) {
        u64 v[8], own = 0, total;
        weigh_unit(w + tid, s1, Kept(1), v);
#pragma unroll
        for (int i = 0; i < 8; ++i) own += v[i];
        u64 at = upto + block_scan(own, sm.scratch, &total) - own;
        if (at <= below && at + own > under)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (at <= below && at + v[i] > under) {
              answer((w + tid) * 8 - row.shift + i, log_of(v[i], (float)all * up, (w + tid) * 8 - row.shift + i), units * 8 - (int)flags);
              accepted = 1;
            }
            at += v[i];
          }
        upto += total;
      }
    }
    accepted = __syncthreads_or(accepted);
    const u64(*verdict)[kBlocks] = share(accepted, 0, 0);
#pragma unroll 1
    for (int i = 0; i < blocks; ++i) accepted |= (int)verdict[0][i];
    return accepted ? kDone : kTogether;
  }

  // 1. of the other rows: the first token in order, and each thread's largest logit.
  __device__ __forceinline__ u64 first_token() {
    float m = -INFINITY;
    int at = 0;
    row.template each<2>(w0, w1, [&](const float* x, int id) {
      const float y = max_of(x);
      if (y > m) {
        m = y;
#pragma unroll
        for (int i = 7; i >= 0; --i)
          if (x[i] == y) at = id + i;
      }
    });
    u64 best = warp_max(composite(m, at));
    if (lane == 0) sm.scratch[warp] = best;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) best = max(best, sm.scratch[w]);
    if (blocks > 1) asm volatile("barrier.cluster.wait;" ::: "memory");
    cluster.map_shared_rank(sm.maxima, home)[part * kThreads + tid] = m;
    const u64(*got)[kBlocks] = share(best, 0, 0);
#pragma unroll 1
    for (int i = 0; i < blocks; ++i) best = max(best, got[0][i]);
    return best;
  }

  // Rows with limits by a list of the largest logits.
  __device__ __forceinline__ int by_list(u64 best) {
    const float each = per_bin();
    int bin = kBins;
    if (top_k) {
      const int n = top_k;
      int way = 0;
      if (part == 0) {
        for (int i = tid; i < kBins; i += kThreads) sm.bins.count[i] = 0;
        if (tid == 0) sm.chosen = kBins;
        __syncthreads();
        for (int i = tid; i < blocks * kThreads; i += kThreads)
          if (sm.maxima[i] > -INFINITY) atomicAdd(&sm.bins.count[bin_of(sm.maxima[i], each)], 1u);
        __syncthreads();
        constexpr int kPer = kBins / kThreads;
        u64 count = 0, total;
#pragma unroll
        for (int i = 0; i < kPer; ++i) count += sm.bins.count[tid * kPer + i];
        u64 to = block_scan(count, sm.scratch, &total) - count;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (to < n && to + sm.bins.count[tid * kPer + i] >= n) sm.chosen = tid * kPer + i;
          to += sm.bins.count[tid * kPer + i];
        }
        __syncthreads();
        way = sm.chosen;
      }
      bin = (int)share(way, 0, 0)[0][0];
      if (bin >= kBins - 1 && blocks * kThreads < a.vocab) return kTogether;  // (fewer threads than vocab: the last bin holds any number)
    }
    const Kept limit(top_k ? 1 : least(best));
    gather([&](const float* x, int id, auto name) {
      const float m = max_of(x);
      if (!(m >= limit.z) || bin_of(m, each) > bin) return;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (limit.has(x[i], id + i) && bin_of(x[i], each) <= bin) name(x[i], id + i);
    });
    sync_all();
    if (part > 0) return kDone;
    return sm.gathered <= kList && finish((int)sm.gathered, best, 0) ? kDone : kAlone;
  }

  // Rows with top_p alone, or with min_p: bins of 1/64 of a power of two of weight, in each the
  // sum of the weights in units of the bin's first (one addition a token, in 32 bits), name the
  // bins in which the limit's last token can lie.  A second pass lists these, or, where they are few,
  // all above their end, and sums all weights, and those above, as integers.
  // kDone; or, with *last the last token that top_p keeps or 1, what is left: kTogether, or kDrawn, the
  // draw alone.
  __device__ __forceinline__ int by_sums(u64 best, u64* last_kept) {
    constexpr float kSpan = 32.f;
    const float each = kShares / kSpan * c_hi;  // bins of a logit
    const int bits = min(14, 31 - (32 - __clz(a.vocab - 1)));
    if (!(each > 1e-3f && each < 1e30f) || bits < 8) return kTogether;
    for (int i = tid; i < kShares; i += kThreads) sm.share[i] = 0;
    __syncthreads();
    const float m = top(), one = (float)(1 << bits);
    row.each(w0, w1, [&](const float* x, int) {
      int at[8];
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = (m - x[i]) * each, n = floorf(y);  // (NaN where x is)
        at[i] = n < (float)(kShares - 1) ? (int)n : -1;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(v[i]) : "f"((n - y) * (kSpan / kShares)));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (at[i] >= 0) atomicAdd(&sm.share[at[i]], (uint32_t)__float2int_rn(v[i] * one));
    });
    sync_all();
    if (blocks > 1) {
      if (part > 0)
        for (int i = tid; i < kShares; i += kThreads)
          if (sm.share[i]) atomicAdd(cluster.map_shared_rank(sm.share, 0) + i, sm.share[i]);
      cluster.sync();
    }
    u64 ends = 0, way = 0;
    if (part == 0) {
      constexpr int kPer = kShares / kThreads;
      if (tid == 0) sm.ends.low = kShares - 1, sm.ends.high = kShares - 1, sm.ends.upto = ~0u;
      u64 mass = 0, count = 0, all, total;
      auto here = [&](int i) { return (u64)((float)sm.share[i] * exp2f(20.f - i * (kSpan / kShares))); };
#pragma unroll 1
      for (int i = 0; i < kPer; ++i) mass += here(tid * kPer + i), count += sm.share[tid * kPer + i];
      u64 mass_to = block_scan(mass, sm.scratch, &all) - mass;
      u64 count_to = block_scan(count, sm.scratch, &total) - count;
      // In units of 2^-bits: a sum of bins is off by 0.51 of itself (a rounding of half a unit of at least
      // 0.98), so is the whole one, and what lies below the bins, 2^-32 of the first token each, is at most
      // 0.5 of it.  ex2 and the roundings here are below 0.1, up to 2^14.
      const float goal = top_p * (float)all, off = goal * 2.f / one;
      const u64 goal_lo = (u64)fmaxf(goal - off, 0.f), goal_hi = (u64)(goal + off) + 64;
#pragma unroll 1
      for (int i = 0; i < kPer; ++i) {
        const u64 next = mass_to + here(tid * kPer + i), count_next = count_to + sm.share[tid * kPer + i];
        if (mass_to <= goal_lo && next > goal_lo) sm.ends.low = tid * kPer + i;
        if (mass_to <= goal_hi && next > goal_hi) sm.ends.high = tid * kPer + i, sm.ends.upto = (uint32_t)(count_next * 17 >> (bits + 4));
        mass_to = next, count_to = count_next;
      }
      __syncthreads();
      ends = (u64)sm.ends.low << 32 | sm.ends.high;
      // (the tokens, from above: each is more than 0.98 of its bin's first.  A list of more is slower than the
      // rows' sums, 14 us and 10; but a min_p above the bins would need them all again)
      way = sm.ends.upto <= (min_p > 0.f ? kList : kShort);
    }
    const u64(*choice)[kBlocks] = share(ends, way, 0);
    const int low = choice[1][0] ? 0 : (int)(choice[0][0] >> 32), high = (int)(uint32_t)choice[0][0];
    u64 whole = 0, above = 0;
    uint32_t many = 0;
    gather([&](const float* x, int id, auto name) {
      u64 w[8];
      int at[8];
      weight.eight(x, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) at[i] = (int)fminf((m - x[i]) * each, (float)(kShares - 1));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        whole += w[i];
        if (at[i] < low) above += w[i], ++many;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (x[i] > -INFINITY && at[i] >= low && at[i] <= high) name(x[i], id + i);
    });
    above = warp_sum(above), many = __reduce_add_sync(0xffffffffu, many);
    if (lane == 0) sm.parts[warp] = above, sm.counts[warp] = many;
    whole = block_sum(whole), above = block_sum(lane == 0 ? above : 0);
    const u64(*got)[kBlocks] = share(whole, above, 0);
    whole = above = 0;
#pragma unroll 1
    for (int i = 0; i < blocks; ++i) whole += got[0][i], above += got[1][i];
    u64 last = 1;
    if (part == 0 && sm.gathered <= kList) {
      const int n = (int)sm.gathered;
      if (low == 0) {
        last = finish(n, best, whole) ? 0 : 1;
      } else {
        const u64 goal = max(part_of(top_p, whole, true), 1ull);
        if (above < goal && above + weigh_list(n) >= goal) last = sm.all[cross(sm, n, kMass, goal - above, 1)];
      }
    }
    last = share(last, 0, 0)[0][0];
    if (last == 0) return kDone;
    *last_kept = last;
    if (last == 1 || least(best) > last) return kTogether;  // (a stricter min_p cuts what lies above the bins)
    // what the limit keeps of this block's part of the list, to the sums of what lies above
    for (uint32_t i = tid; i < sm.listed; i += kThreads) {
      const u64 comp = sm.list[i];
      if (comp < last) continue;
      const int at = (id_of(comp) + row.shift) / 8;
      int w = 0;
      while (w < kWarps - 1 && at >= warp_begin(w + 1)) ++w;
      add64(&sm.parts[w], weight(value_of((uint32_t)(comp >> 32)))), add64(&sm.counts[w], 1);
    }
    __syncthreads();
    return kDrawn;
  }
};

// As finish_short, for up to kList entries.
template <typename T>
__device__ __noinline__ bool finish_long(const SampleParams& p, Shared& sm, int n, u64 best, u64 whole, float m, int top_k) {
  Sampler<T> s(p, sm, true);
  s.set_top(m);
  u64 sum = s.weigh_list(n), kept, from = 1;
  auto sum_from = [&] {
    sum = kept = 0;
    for (int i = s.tid; i < n; i += kThreads)
      if (sm.all[i] >= from) sum += sm.weights[i], ++kept;
    sum = s.block_sum(sum), kept = s.block_sum(kept);
  };
  if (top_k && top_k < n) from = sm.all[cross(sm, n, kCount, top_k, 1)], sum_from();
  if (s.top_p < 1.f) {
    const u64 goal = max(s.top_p > 0.f ? part_of(s.top_p, top_k ? sum : whole, true) : 0, 1ull);
    if (sum < goal) return false;
    from = sm.all[cross(sm, n, kMass, goal, from)];
  }
  from = max(from, s.least(best));
  sum_from();
  const int i = cross(sm, n, kById, goal_of(s.u, sum), from);
  if (s.tid == 0) s.answer(id_of(sm.all[i]), s.log_of(sm.weights[i], (float)sum, id_of(sm.all[i])), (int)kept);
  return true;
}

// The draw, where sm.parts and sm.counts have the sums of the weights, and the numbers, of the kept
// tokens of each warp's range.
template <typename T>
__device__ __noinline__ void draw_row(const SampleParams& p, Shared& sm, bool alone, int turn, float m, u64 last) {
  Sampler<T> s(p, sm, alone);
  s.turn = turn;
  s.set_top(m);
  const Kept limit(last);
  u64 sum = 0, kept = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) sum += sm.parts[w], kept += sm.counts[w];
  const u64(*got)[kBlocks] = s.share(sum, kept, 0);
  u64 before = 0;
  sum = kept = 0;
#pragma unroll 1
  for (int i = 0; i < s.blocks; ++i) {
    if (i == s.part) before = sum;
    sum += got[0][i], kept += got[1][i];
  }
  const u64 goal = goal_of(s.u, sum);
  if (before >= goal || before + got[0][s.part] < goal) return;  // another block's
  int w = 0;
  while (before + sm.parts[w] < goal) before += sm.parts[w++];
  // the warp's tokens one after the other, 2,048 at a time
  const int s0 = s.warp_begin(w), s1 = s.warp_begin(w + 1);
  for (int v = s0; v < s1; v += kThreads) {
    u64 y[8], own = 0, total;
    s.weigh_unit(v + s.tid, s1, limit, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) own += y[i];
    u64 upto = before + block_scan(own, sm.scratch, &total) - own;
    if (upto < goal && upto + own >= goal)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (upto < goal && upto + y[i] >= goal) s.answer((v + s.tid) * 8 - s.row.shift + i, s.log_of(y[i], (float)sum, (v + s.tid) * 8 - s.row.shift + i), (int)kept);
        upto += y[i];
      }
    before += total;
    if (before >= goal) return;
  }
}

// Any row whose first token is known (without limits: whose largest logit is): rounds of bins for
// each limit, where `last`, from which on tokens are kept, is not known yet (1), then the sums of the
// kept tokens.
template <typename T>
__device__ __noinline__ void slow_row(const SampleParams& p, Shared& sm, bool alone, int turn, u64 best, float m, u64 last) {
  Sampler<T> s(p, sm, alone);
  s.turn = turn;
  s.set_top(m);
  const Weigher weight = s.weight;
  const auto& row = s.row;
  const int tid = s.tid, lane = s.lane, warp = s.warp, blocks = s.blocks, part = s.part, w0 = s.w0, w1 = s.w1;
  const float each = s.per_bin();

  // The last token of the prefix of `target` tokens, or (kMass) of the fewest whose weights sum
  // to top_p of the sum of all, among those at or above `floor`; `floor` where there are not as many.
  // 0: the row is done (all that counts was in the list).
  enum { kBin, kWhole, kNoLimit };
  auto select = [&](int by, u64 target, u64 floor) -> u64 {
    u64 lo = 0, hi = 0;  // of the composite keys that are left, after the first round
    int shift = -1, bin = 0;
    u64 before = 0;
    for (int round = 0;; ++round) {
      __syncthreads();
      for (int i = tid; i < kBins; i += kThreads) sm.bins.mass[i] = 0, sm.bins.count[i] = 0;
      if (tid == 0) sm.gathered = 0;
      __syncthreads();
      const Kept from(floor);
      auto place = [&](float z, int id) {  // the bin, -1: none
        if (!from.has(z, id)) return -1;
        if (shift < 0) return s.bin_of(z, each);
        const u64 comp = composite(z, id);
        return comp >= lo && comp <= hi ? (int)((hi - comp) >> shift) : -1;
      };
      row.each(w0, w1, [&](const float* x, int id) {
        if (from.none(x)) return;
        int at[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) at[i] = place(x[i], id + i);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (at[i] >= 0) atomicAdd(&sm.bins.count[at[i]], 1u);
        if (by == kMass) {
          u64 w[8];
          weight.eight(x, w);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (at[i] >= 0 && w[i]) add64(&sm.bins.mass[at[i]], w[i]);
        }
      });
      s.sync_all();  // (the first block's bins have been cleared and filled)
      if (blocks > 1) {
        if (part > 0)
          for (int i = tid; i < kBins; i += kThreads) {
            if (sm.bins.count[i]) atomicAdd(s.cluster.map_shared_rank(sm.bins.count, 0) + i, sm.bins.count[i]);
            if (sm.bins.mass[i]) atomicAdd(s.cluster.map_shared_rank(sm.bins.mass, 0) + i, sm.bins.mass[i]);
          }
        s.cluster.sync();
      }
      if (part == 0) {
        constexpr int kPer = kBins / kThreads;
        u64 mass = 0, count = 0, all_mass, all_count;
#pragma unroll
        for (int i = 0; i < kPer; ++i) mass += sm.bins.mass[tid * kPer + i], count += sm.bins.count[tid * kPer + i];
        u64 mass_to = block_scan(mass, sm.scratch, &all_mass) - mass;
        u64 count_to = block_scan(count, sm.scratch, &all_count) - count;
        if (round == 0 && by == kMass) target = max(part_of(s.top_p, all_mass, true), 1ull);
        if (tid == 0) sm.found.all = all_mass, sm.found.way = round == 0 && by == kCount && target >= all_count ? kNoLimit : kBin;
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
      const u64(*got)[kBlocks] = s.share((u64)sm.found.bin << 32 | sm.found.count, sm.found.way, sm.found.before);
      if (got[1][0] == kNoLimit) return floor;
      bin = (int)(got[0][0] >> 32), before = got[2][0];
      const bool take_all = got[1][0] == kWhole;
      if (!take_all && (uint32_t)got[0][0] > kList) {  // once more, in this bin
        u64 low = ~0ull, high = 0;
        row.each(w0, w1, [&](const float* x, int id) {
          if (from.none(x)) return;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (place(x[i], id + i) == bin) low = min(low, composite(x[i], id + i)), high = max(high, composite(x[i], id + i));
        });
        low = ~warp_max(~low), high = warp_max(high);
        __syncthreads();
        if (lane == 0) sm.parts[warp] = low, sm.scratch[warp] = high;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) low = min(low, sm.parts[w]), high = max(high, sm.scratch[w]);
        const u64(*ends)[kBlocks] = s.share(low, high, 0);
#pragma unroll 1
        for (int i = 0; i < blocks; ++i) low = min(low, ends[0][i]), high = max(high, ends[1][i]);
        lo = low, hi = high, shift = 0;
        while ((hi - lo) >> shift >= kBins) ++shift;
        continue;
      }
      s.gather([&](const float* x, int id, auto name) {
        if (from.none(x)) return;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int at = place(x[i], id + i);
          if (at >= 0 && (take_all ? at <= bin : at == bin)) name(x[i], id + i);
        }
      });
      s.sync_all();
      u64 last = 0;
      if (part == 0) {
        const int n = (int)sm.gathered;
        if (take_all) {
          // (top_p of the tokens at or above `floor`, which top_k has cut: the list is of these alone)
          s.top_k = by == kCount ? s.top_k : 0;
          s.finish(n, best, sm.found.all);
        } else {
          if (by == kMass) s.weigh_list(n);
          last = sm.all[cross(sm, n, by, target - before, 1)];
        }
      }
      if (take_all) return 0;
      return s.share(last, 0, 0)[0][0];
    }
  };

  if (last == 1 && s.top_k) {
    last = select(kCount, s.top_k, 1);
    if (last == 0) return;
  }
  if ((last == 1 || s.top_k) && s.top_p < 1.f) {
    last = select(kMass, 0, last);
    if (last == 0) return;
  }
  last = max(last, s.least(best));

  // the kept tokens' weights
  const Kept limit(last);
  auto weigh = [&](const float* x, int id, u64* w) {  // eight, 0 for those that are not kept; how many are
    int n = 0;
    weight.eight(x, w);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (limit.has(x[i], id + i)) ++n;
      else w[i] = 0;
    return n;
  };
  u64 sum = 0, kept = 0;
  row.each(w0, w1, [&](const float* x, int id) {
    if (limit.none(x)) return;
    u64 w[8];
    kept += weigh(x, id, w);
    sum += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
  });
  sum = warp_sum(sum), kept = warp_sum(kept);
  __syncthreads();
  if (lane == 0) sm.parts[warp] = sum, sm.counts[warp] = kept;
  __syncthreads();
  draw_row<T>(p, sm, alone, s.turn, m, last);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) sample_token_kernel(const __grid_constant__ SampleParams p) {
  __shared__ Shared sm;
  // what needs nothing of the stream before
  const u64 fine = p.fine[threadIdx.x & 31];
  for (int i = threadIdx.x; i < kTable; i += kThreads) sm.table[i] = __umul64hi(p.coarse[i >> 5], fine) << 1;
  if (threadIdx.x == 0) sm.gathered = 0;
  __syncthreads();
  after_stream();
  Sampler<T> s(p, sm, false);
  if (s.blocks > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");  // waited for before another block's memory is touched
  u64 best = 0, last = 1;
  int left = Sampler<T>::kTogether;
  if (s.temperature > 0.f && s.top_k == 0 && !(s.top_p < 1.f) && !(s.min_p > 0.f) && s.c_hi > 1e-30f) {
    left = s.without_limits();
  } else {
    // (doubles are slow: by one warp, while the logits are under way)
    if (s.min_p > 0.f && s.min_p <= 1.f && s.warp == kWarps - 1) sm.drop = log((double)s.min_p) * (double)s.temperature;
    best = s.first_token();
    if (best == 0 || !(s.temperature > 0.f) || s.top_k == 1 || s.top_p <= 0.f || s.min_p > 1.f) {
      if (s.part == 0 && s.tid == 0) best == 0 ? s.answer(-1, -INFINITY, 0) : s.answer(id_of(best), 0.f, 1);
      return;
    }
    s.set_top(value_of((uint32_t)(best >> 32)));
    if (s.top_k || (s.min_p > 0.f && !(s.top_p < 1.f))) {
      left = s.by_list(best);
    } else if (s.top_p < 1.f) {
      left = s.by_sums(best, &last);
    }
  }
  if (left == Sampler<T>::kDone) return;
  if (left == Sampler<T>::kDrawn) return draw_row<T>(p, sm, false, s.turn, s.top(), last);
  slow_row<T>(p, sm, left == Sampler<T>::kAlone, s.turn, best, s.top(), last);
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
  // Blocks of a row: as long as all are resident at once, three an SM, or each still has 32,768 tokens, and
  // never with fewer than 512.  Blocks of 1, 2, 4, 8, us: 33 rows of 49,999 with top_p 71 48 35 32; 64 of 50,304
  // 72 49 41 43; 200 of them 97 74 84 103, without limits 25 21 31 45; 512 of 32,000 without limits 32 37
  // 55 88; 512 of 131,072 with top_k 118 128 118 145; 1 of 12,288 with it 21 16 14 14.
  int blocks = 1;
  while (blocks < kBlocks && a->vocab / (2 * blocks) >= 512 && ((int64_t)a->rows * 2 * blocks <= 456 || a->vocab / (2 * blocks) >= 32768)) blocks *= 2;
  if ((int64_t)a->rows * blocks > INT32_MAX) return call_error(GPT_ERR_UNSUPPORTED, "too many rows");
  const cudaStream_t st = (cudaStream_t)cuda_stream;
  return launch_after("gpt_sample_token", a->dtype == GPT_DTYPE_BF16 ? sample_token_kernel<__nv_bfloat16> : sample_token_kernel<float>,
                      dim3(a->rows * blocks), kThreads, 0, blocks, st, p);
}
