// decode_attention.cuh — the kernels of gpt_decode_attention: attention of one new
// token of every sequence over its pages of keys and values.
//
// Mathematics: with z_j = scale q.k_j, any set of keys reduces to (m, l, o) =
// (reference m, sum 2^(z_j - m), sum 2^(z_j - m) v_j), and sets join by bringing
// them to a common m; the output is o / l, the lse m + log l.  Scores are kept in
// base 2 (scale log2 e folded in).
//
// Bound: every key and value is read once, 4 FLOP per element and query head, so
// HBM bandwidth is the limit at any usual number of query heads per key head.
// The kernel therefore keeps loads in flight and does as little as possible
// between them:
//  - Work is cut by keys, not by rows: the 16-key tiles of all (sequence, key
//    head) rows are one line, of which every warp of a one-wave grid takes an equal
//    part, whatever the lengths are (the host does not know them).  Rows inside one
//    warp's part are finished from its registers; a row cut by part boundaries
//    leaves (m, l, o) pieces in shared memory, which the block joins once at its
//    end, and one cut by block boundaries pieces in the workspace, which a second
//    kernel joins.  (Rows of few tiles a warp do without the line: decode_row_kernel.)
//  - Each warp reads its keys and values from global memory straight into the
//    operand registers of its products; no barrier until the warp's part is done.
//    The values of a step are requested before its keys are used and the next
//    step's keys before its values are used: 4 KB of each, 16 warps an SM.
//  - bf16: 16 keys at a time through mma.m16n8k16, keys (or the 16 value dims) as
//    the 16-row operand and up to 8 query heads as its 8 columns.  An operand's
//    16-byte pieces serve as they are: the order of the contraction index is free
//    for the scores (the query is laid out to match) and the order of the output
//    dims for the values.  The probabilities enter as two bf16 parts (p = hi + lo,
//    2^-17 of p left over), so that their rounding does not show beside the
//    output's own.
//  - fp32: fused multiply-adds, four lanes to a key for the scores, a lane to
//    four dims for the values.
// Measured (HBM copy 6.7 TB/s): 64 sequences of 17 to 8,192 keys, 32 query over 8 key
// heads of 128, bf16, 175 us (6.1 TB/s); 131,071 keys of one sequence 94 us (5.7); 200
// sequences of 1 to 1,024 keys, 16 heads of 64, 80 us (5.2).
#pragma once
#include <cooperative_groups.h>

#include <type_traits>

#include "decode_attention.h"

namespace pgs {
namespace {

namespace cg = cooperative_groups;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^(x - m) for x <= m; nothing from x = -infinity, whatever m is.
__device__ __forceinline__ float weight(float x, float m) { return x == -INFINITY ? 0.f : exp2_fast(x - m); }

__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 u;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p));
  return u;
}
// Two neighbouring 16-byte pieces in one load, on a 32-byte boundary.
__device__ __forceinline__ void load32(const void* p, uint4& a, uint4& b) {
  asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w) : "l"(p));
}
__device__ __forceinline__ uint4 load16_if(const void* p, bool ok) {
  uint4 u = make_uint4(0u, 0u, 0u, 0u);
  if (ok) asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p));
  return u;
}

// Length of a sequence, cut to what its table can name.
__device__ __forceinline__ int seq_len(const DecodeParams& p, int s, bool report) {
  const int len = p.a.lens[s], most = p.c.max_pages * p.c.page_size;
  if (len >= 0 && len <= most) return len;
  if (report) set_status(p.a.status, GPT_STATUS_BAD_POS);
  return len < 0 ? 0 : most;
}

// Where a warp's keys are.  kFast (pages of whole 8-key groups, everything within
// 64 GB): lane i holds the offset, in 16 bytes, of group i of the next 32, one division
// and one table entry a group; rows of a group are slot_stride apart.  Otherwise a lane
// holds the offset, in elements, of its own key of the step, one of each a key.  Table
// entries are read one round ahead.  kNoKey: no such key, or a bad page.  kLast: groups
// past the end are the last one again instead.
template <bool kFast, int kKeys, bool kLast = false>
struct Walk {
  using Off = std::conditional_t<kFast, uint32_t, int64_t>;
  static constexpr Off kNoKey = (Off)-1;
  const DecodeParams& p;
  const int32_t* table;
  Off head, off;
  int next, end, page, at;

  __device__ __forceinline__ Walk(const DecodeParams& p_, int s, int h, int k0, int k1)
      : p(p_), table(p_.c.page_table + s * p_.c.table_stride), end(k1), at(0) {
    const int lane = threadIdx.x & 31;
    head = kFast ? h * p.head16 : h * p.c.head_stride;
    next = k0 + (kFast ? lane * 8 : lane & (kKeys - 1));
    page = fetch();
  }
  __device__ __forceinline__ int here() const { return kLast ? min(next, (end - 1) & ~7) : next; }
  __device__ __forceinline__ int fetch() const {
    if (!kLast && next >= end) return -1;
    const int id = table[here() / p.c.page_size];
    if (id >= 0 && id < p.c.n_pages) return id;
    set_status(p.a.status, GPT_STATUS_BAD_PAGE);
    return -1;
  }
  __device__ __forceinline__ void turn() {
    if constexpr (kFast) off = page < 0 ? kNoKey : page * p.page16 + (here() % p.c.page_size) * p.slot16 + head;
    else off = page < 0 ? kNoKey : page * p.c.page_stride + (next % p.c.page_size) * p.c.slot_stride + head;
    next += kFast ? 256 : kKeys;
    page = fetch();
  }
  // kFast: offset of the next group of 8 keys.
  __device__ __forceinline__ Off group() {
    const Off x = __shfl_sync(0xffffffffu, off, at);
    if (++at == 32) turn(), at = 0;
    return x;
  }
};

// A group's address (its first slot's); one that is not there reads the pool's first slots.
template <typename T>
__device__ __forceinline__ const T* group_at(const T* base, uint32_t off) {
  return reinterpret_cast<const T*>(reinterpret_cast<const char*>(base) + (off == ~0u ? 0ull : (unsigned long long)off * 16));
}

// A piece of a row in shared memory: (m, l) of each head, then their o rows from left_o on.
__host__ __device__ constexpr int left_o(int heads) { return (2 * heads + 3) / 4 * 4; }
__host__ __device__ constexpr int left_floats(int heads, int dp) { return left_o(heads) + heads * dp; }

__device__ __forceinline__ void store_lse(const DecodeParams& p, int s, int hq, float m, float total) {
  if (p.a.lse) p.a.lse[(int64_t)s * p.a.n_head + hq] = total == 0.f ? -INFINITY : m * kLn2 + logf(total);
}

__device__ __forceinline__ void store4(float* to, const float* x) { *reinterpret_cast<float4*>(to) = make_float4(x[0], x[1], x[2], x[3]); }
__device__ __forceinline__ void store4(__nv_bfloat16* to, const float* x) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
  *reinterpret_cast<uint2*>(to) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void load4(const float* from, float* x) {
  const float4 y = *reinterpret_cast<const float4*>(from);
  x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* from, float* x) {
  const uint2 y = *reinterpret_cast<const uint2*>(from);
  x[0] = __uint_as_float(y.x << 16), x[1] = __uint_as_float(y.x & 0xffff0000u);
  x[2] = __uint_as_float(y.y << 16), x[3] = __uint_as_float(y.y & 0xffff0000u);
}
__device__ __forceinline__ bool finite4(const float* x) { return x[0] * 0.f + x[1] * 0.f + (x[2] * 0.f + x[3] * 0.f) == 0.f; }

// Results that are not finite.  A value of infinity or NaN at a key that counts belongs in
// the result however small the key's weight is, and one at a key with a score of -infinity
// does not; the products make NaN of both where a weight, or the low part of one, is zero (or
// negative) beside an infinity.  Weights of up to 2^8, and sums of many, also overflow where
// the result does not.  So a head whose results are not all finite is computed once more by
// a block, key by key, with weights of at most 2^-31 (whose sum over a row is at most 1).
// 131,071 keys take 5 ms.
constexpr int kCarefulFloats = kWarps * 130;
__device__ __forceinline__ float scaled(float x, float f) { return x * 0.f == 0.f ? x * f : x; }
__device__ __forceinline__ float with_value(float x, float w, float v) { return v * 0.f == 0.f ? fmaf(w, v, x) : x + v; }

// Query head hq, which reads key head h, of sequence s, by all threads of a block, if what
// is there is not finite.
template <typename T>
__device__ __noinline__ void careful_head(const DecodeParams& p, int s, int h, int hq, float* scratch) {
  constexpr int kAtOnce = 16 / sizeof(T);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = p.c.head_dim, e = lane * 4, len = seq_len(p, s, false);
  T* out = (T*)p.a.out + s * p.a.out_row + hq * p.a.out_head + e;
  float q[4] = {0.f, 0.f, 0.f, 0.f}, o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
  __syncthreads();
  if (e < d) load4(out, o);
  if (__all_sync(0xffffffffu, finite4(o))) return;
  if (p.a.lse && isnan(p.a.lse[(int64_t)s * p.a.n_head + hq])) return;  // of NaN or infinite scores: everything is NaN
  const int32_t* table = p.c.page_table + s * p.c.table_stride;
  const T *kb = (const T*)p.c.k + h * p.c.head_stride + e, *vb = (const T*)p.c.v + h * p.c.head_stride + e;
  if (e < d) load4((const T*)p.a.q + s * p.a.q_row + hq * p.a.q_head + e, q);
  o[0] = o[1] = o[2] = o[3] = 0.f;
  for (int64_t k = warp * 32; k < len; k += kWarps * 32) {
    int64_t at = -1;  // in elements; -1: no such key, or a bad page
    if (k + lane < len) {
      const int id = table[(int)(k + lane) / p.c.page_size];
      if (id >= 0 && id < p.c.n_pages) at = id * p.c.page_stride + ((int)(k + lane) % p.c.page_size) * p.c.slot_stride;
    }
    for (int j0 = 0; j0 < 32; j0 += kAtOnce) {
      float x[kAtOnce][4], v[kAtOnce][4], z[kAtOnce], top = m;
      bool there[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int64_t from = __shfl_sync(0xffffffffu, at, j0 + j);
        there[j] = from >= 0;
        x[j][0] = x[j][1] = x[j][2] = x[j][3] = v[j][0] = v[j][1] = v[j][2] = v[j][3] = 0.f;
        if (there[j] && e < d) load4(kb + from, x[j]), load4(vb + from, v[j]);
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        z[j] = fmaf(x[j][3], q[3], fmaf(x[j][2], q[2], fmaf(x[j][1], q[1], x[j][0] * q[0])));
#pragma unroll
        for (int y = 16; y > 0; y >>= 1) z[j] += __shfl_xor_sync(0xffffffffu, z[j], y);
        z[j] = there[j] ? z[j] * p.scale2 : -INFINITY;
        top = fmaxf(top, z[j]);
      }
      const float keep = weight(m, top);
      m = top;
      l *= keep;
#pragma unroll
      for (int u = 0; u < 4; ++u) o[u] = scaled(o[u], keep);
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        if (z[j] == -INFINITY) continue;
        const float w = weight(z[j], m);
        l += w;
#pragma unroll
        for (int u = 0; u < 4; ++u) o[u] = with_value(o[u], w * 0x1p-31f, v[j][u]);
      }
    }
  }
  float* mine = scratch + warp * 130;
  if (lane == 0) mine[128] = m, mine[129] = l;
#pragma unroll
  for (int u = 0; u < 4; ++u) mine[lane * 4 + u] = o[u];
  __syncthreads();
  if (warp > 0) return;
  for (int w = 0; w < kWarps; ++w) m = fmaxf(m, scratch[w * 130 + 128]);
  l = o[0] = o[1] = o[2] = o[3] = 0.f;
  for (int w = 0; w < kWarps; ++w) {
    const float keep = weight(scratch[w * 130 + 128], m);
    l += scratch[w * 130 + 129] * keep;
#pragma unroll
    for (int u = 0; u < 4; ++u) o[u] = with_value(o[u], keep, scratch[w * 130 + lane * 4 + u]);
  }
  const float inv = l == 0.f ? 0.f : 1.0f / (l * 0x1p-31f);
#pragma unroll
  for (int u = 0; u < 4; ++u) o[u] = l * 0.f == 0.f ? scaled(o[u], inv) : NAN;  // NaN of NaN or infinite scores
  if (e < d) store4(out, o);
  if (lane == 0) store_lse(p, s, hq, m, l);
}

// A warp's part of a row: keys [k0, k1) of sequence s for key head h, query heads
// hq .. hq + n; left: where its piece goes, or null to finish the row.
struct Part {
  int s, h, hq, n, k0, k1;
  float* left;
};

// ---- bf16 ---------------------------------------------------------------------

__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// kMode: query heads of a row.  4: up to 4, columns 4..7 of the scores repeat them, so
// that one product takes hi from columns 0..3 and lo from 4..7; 8, 16: up to that
// many, hi and lo in products of their own.
template <int kMode, int DP_, bool kFast, bool kExact>
struct Bf16Path {
  using T = __nv_bfloat16;
  static constexpr int NT = kMode == 16 ? 2 : 1, DP = DP_, kHeads = kMode;
  static constexpr int kBlocks = kMode == 16 ? 1 : 2;  // of an SM
  // A unit of the line is a step, of 32 keys in heads up to 64, where a row's start counts
  // as one of them (200 sequences of 1 to 1,024 keys, 16 heads of 64: 87.4 us with 0, 80.2
  // with 1, 81.7 with 2, 83.2 with 3, 87.9 with 6).
  static constexpr int kUnit = 16 * (128 / DP_), kUnitStart = DP_ == 64 ? 1 : kStart;
  static constexpr bool kTwice = kMode == 4;
  static constexpr int KG = 128 / DP;           // 16-key groups of a step: 32 registers of keys, 32 of values
  // Heads of 65 to 127: no keys are read past the last step, and none of the pool's first
  // slots in place of groups past the end (104 sequences of 13 to 878 keys, 8 heads of 96,
  // 38.3 us instead of 43.8; 10 of 2,596 to 18,383, 6 over 2 heads of 80, 26.2 instead of
  // 35.8).  Elsewhere the conditions cost more than such reads: 111 to 233 sequences of 32
  // over 8 heads of 128 2 %, 64 of 12 heads of 32 2.5 %.
  static constexpr bool kEdge = kFast && !kExact && DP == 128;
  static constexpr int kQuery = NT * (DP / 32) * 128;  // a warp's queries: a 16-byte piece per lane, tile and 32 dims

  // Dims of a lane's piece i of a key or query: lane c has 16 of every 64, in two pieces
  // for one load (4,096 keys of 8 heads of 128 12.6 us, with 16-byte loads 13.5).
  static __device__ __forceinline__ int piece_dim(int i, int c) { return i / 2 * 64 + c * 16 + i % 2 * 8; }

  // Lane (r, c): query head r of a tile, its pieces.
  static __device__ __forceinline__ void stage_query(const DecodeParams& p, float* mine, const Part& w) {
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < DP / 32; ++i) {
        const int qh = kTwice ? r & 3 : t * 8 + r;
        reinterpret_cast<uint4*>(mine)[(t * (DP / 32) + i) * 32 + lane] =
            load16_if((const T*)p.a.q + w.s * p.a.q_row + (w.hq + qh) * p.a.q_head + piece_dim(i, c),
                      qh < w.n && piece_dim(i, c) < p.c.head_dim);
      }
  }

  static __device__ __forceinline__ void run(const DecodeParams& p, float* mine, const Part& w) {
    const int k0 = w.k0, k1 = w.k1;
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const int d = p.c.head_dim;
    const int64_t row = p.c.slot_stride;
    const T* kb = (const T*)p.c.k + (kFast ? r * row : 0);
    const T* vb = (const T*)p.c.v + r * 8 + (kFast ? 2 * c * row : 0);
    const uint4* query = reinterpret_cast<const uint4*>(mine) + lane;
    float o[NT][DP / 64][4][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t][0] = m[t][1] = -INFINITY, l[t][0] = l[t][1] = 0.f;
#pragma unroll
      for (int b = 0; b < DP / 64; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[t][b][i / 4][i % 4] = 0.f;
    }
    uint4 kr[KG][2][DP / 32], vr[KG][4][DP / 64];
    using Keys = Walk<kFast, 16 * KG, kEdge>;
    Keys walk(p, w.s, w.h, k0, k1);
    typename Keys::Off off[KG][2];  // of the step's groups of 8 (kFast); off[0][0]: of the lane's key
    auto advance = [&] {
      if constexpr (kFast) {
#pragma unroll
        for (int g = 0; g < KG; ++g) off[g][0] = walk.group(), off[g][1] = walk.group();
      } else {
        off[0][0] = walk.off;
        walk.turn();
      }
    };
    auto load_keys = [&] {
#pragma unroll
      for (int g = 0; g < KG; ++g)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if constexpr (kFast) {
            const T* at = group_at(kb, off[g][u]);
#pragma unroll
            for (int i = 0; i < DP / 32; i += 2)
              if constexpr (kExact) load32(at + piece_dim(i, c), kr[g][u][i], kr[g][u][i + 1]);
              else kr[g][u][i] = load16_if(at + piece_dim(i, c), piece_dim(i, c) < d), kr[g][u][i + 1] = load16_if(at + piece_dim(i + 1, c), piece_dim(i + 1, c) < d);
          } else {
            const int64_t at = __shfl_sync(0xffffffffu, off[0][0], g * 16 + u * 8 + r);
#pragma unroll
            for (int i = 0; i < DP / 32; ++i) kr[g][u][i] = load16_if(kb + at + piece_dim(i, c), at >= 0 && piece_dim(i, c) < d);
          }
    };
    stage_query(p, mine, w);
    walk.turn();
    advance();
    load_keys();
    for (int k = k0; k < k1; k += 16 * KG) {
      // the step's values
      uint32_t there = 0xffffffffu;  // keys that count
#pragma unroll
      for (int g = 0; g < KG; ++g)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if constexpr (kFast) {
            const T* at = group_at(vb, off[g][u >> 1]) + (u & 1) * row;
#pragma unroll
            for (int b = 0; b < DP / 64; ++b) vr[g][u][b] = kExact ? load16(at + b * 64) : load16_if(at + b * 64, b * 64 + r * 8 < d);
            if ((u & 1) && off[g][u >> 1] == ~0u) there &= ~(0xffu << (g * 16 + (u >> 1) * 8));
          } else {
            const int64_t at = __shfl_sync(0xffffffffu, off[0][0], g * 16 + (u >> 1) * 8 + 2 * c + (u & 1));
#pragma unroll
            for (int b = 0; b < DP / 64; ++b) vr[g][u][b] = load16_if(vb + at + b * 64, at >= 0 && b * 64 + r * 8 < d);
          }
      if constexpr (kFast) {
        if (k1 - k < 16 * KG) there &= (1u << (k1 - k)) - 1u;
      } else {
        there = __ballot_sync(0xffffffffu, off[0][0] >= 0);
      }
      advance();
      // scores: 16 keys x 8 heads a tile
      float z[KG][NT][4];
#pragma unroll
      for (int g = 0; g < KG; ++g)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) z[g][t][i] = 0.f;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < DP / 32; ++i) {
          const uint4 q = query[(t * (DP / 32) + i) * 32];
#pragma unroll
          for (int g = 0; g < KG; ++g) {
            mma16816(z[g][t], kr[g][0][i].x, kr[g][1][i].x, kr[g][0][i].y, kr[g][1][i].y, q.x, q.y);
            mma16816(z[g][t], kr[g][0][i].z, kr[g][1][i].z, kr[g][0][i].w, kr[g][1][i].w, q.z, q.w);
          }
        }
      if (!kEdge || k + 16 * KG < k1) load_keys();
#pragma unroll
      for (int g = 0; g < KG; ++g)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) z[g][t][i] *= p.scale2;
      if (__builtin_expect(there != 0xffffffffu >> (32 - 16 * KG) && there != 0xffffffffu, 0)) {
#pragma unroll
        for (int g = 0; g < KG; ++g) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!((there >> (g * 16 + (i >> 1) * 8 + r)) & 1u)) z[g][t][i] = -INFINITY;
          if constexpr (kFast)  // what such a slot holds may be NaN
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (!((there >> (g * 16 + (u >> 1) * 8 + 2 * c + (u & 1))) & 1u))
#pragma unroll
                for (int b = 0; b < DP / 64; ++b) vr[g][u][b] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      // softmax: the reference of a head moves only when a score passes it by 2^8
      bool move = false;
#pragma unroll
      for (int g = 0; g < KG; ++g)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          move |= fmaxf(z[g][t][0], z[g][t][2]) > m[t][0] + 8.f || fmaxf(z[g][t][1], z[g][t][3]) > m[t][1] + 8.f;
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = m[t][e];
#pragma unroll
            for (int g = 0; g < KG; ++g) top = fmaxf(top, fmaxf(z[g][t][e], z[g][t][e + 2]));
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            const float keep = weight(m[t][e], top);
            m[t][e] = top;
            l[t][e] *= keep;
#pragma unroll
            for (int b = 0; b < DP / 64; ++b)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[t][b][i][e] *= keep, o[t][b][i][e + 2] *= keep;
          }
      }
#pragma unroll
      for (int g = 0; g < KG; ++g)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float m0 = m[t][0] == -INFINITY ? 0.f : m[t][0], m1 = m[t][1] == -INFINITY ? 0.f : m[t][1];
          const float p0 = exp2_fast(z[g][t][0] - m0), p1 = exp2_fast(z[g][t][1] - m1);
          const float p2 = exp2_fast(z[g][t][2] - m0), p3 = exp2_fast(z[g][t][3] - m1);
          l[t][0] += p0 + p2, l[t][1] += p1 + p3;
          uint32_t ha = pack2(p0, p1), hb = pack2(p2, p3);
          const uint32_t la = pack2(p0 - __uint_as_float(ha << 16), p1 - __uint_as_float(ha & 0xffff0000u));
          const uint32_t lb = pack2(p2 - __uint_as_float(hb << 16), p3 - __uint_as_float(hb & 0xffff0000u));
          if (kTwice) ha = c < 2 ? ha : la, hb = c < 2 ? hb : lb;
          const uint32_t h0 = transpose8(ha), h1 = transpose8(hb);
          uint32_t l0, l1;
          if (!kTwice) l0 = transpose8(la), l1 = transpose8(lb);
#pragma unroll
          for (int b = 0; b < DP / 64; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t va = (&vr[g][0][b].x)[i], vc = (&vr[g][1][b].x)[i], ve = (&vr[g][2][b].x)[i], vg = (&vr[g][3][b].x)[i];
              const uint32_t a0 = __byte_perm(va, vc, 0x5410), a1 = __byte_perm(va, vc, 0x7632);
              const uint32_t a2 = __byte_perm(ve, vg, 0x5410), a3 = __byte_perm(ve, vg, 0x7632);
              mma16816(o[t][b][i], a0, a1, a2, a3, h0, h1);
              if (!kTwice) mma16816(o[t][b][i], a0, a1, a2, a3, l0, l1);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int qh = t * 8 + 2 * c + e;
        float total = l[t][e];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) total += __shfl_xor_sync(0xffffffffu, total, x);
        if (kTwice)
#pragma unroll
          for (int b = 0; b < DP / 64; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              o[t][b][i][e] += __shfl_xor_sync(0xffffffffu, o[t][b][i][e], 2);
              o[t][b][i][e + 2] += __shfl_xor_sync(0xffffffffu, o[t][b][i][e + 2], 2);
            }
        if (qh >= w.n) continue;
        if (w.left) {
          if (r == 0) w.left[2 * qh] = m[t][e], w.left[2 * qh + 1] = total;
#pragma unroll
          for (int b = 0; b < DP / 64; ++b) {
            float4* to = reinterpret_cast<float4*>(w.left + left_o(kHeads) + qh * DP + b * 64 + r * 8);
            to[0] = make_float4(o[t][b][0][e], o[t][b][0][e + 2], o[t][b][1][e], o[t][b][1][e + 2]);
            to[1] = make_float4(o[t][b][2][e], o[t][b][2][e + 2], o[t][b][3][e], o[t][b][3][e + 2]);
          }
        } else {
          const float inv = total == 0.f ? 0.f : 1.0f / total;
          T* to = (T*)p.a.out + w.s * p.a.out_row + (w.hq + qh) * p.a.out_head + r * 8;
#pragma unroll
          for (int b = 0; b < DP / 64; ++b)
            if (kExact || b * 64 + r * 8 < d)
              *reinterpret_cast<uint4*>(to + b * 64) = make_uint4(pack2(o[t][b][0][e] * inv, o[t][b][0][e + 2] * inv), pack2(o[t][b][1][e] * inv, o[t][b][1][e + 2] * inv),
                                                                  pack2(o[t][b][2][e] * inv, o[t][b][2][e + 2] * inv), pack2(o[t][b][3][e] * inv, o[t][b][3][e + 2] * inv));
          if (r == 0) store_lse(p, w.s, w.hq + qh, m[t][e], total);
        }
      }
  }
};

// ---- fp32 ---------------------------------------------------------------------

template <int GH_, int DP_, bool kFast, bool kExact>
struct Fp32Path {
  using T = float;
  static constexpr int DP = DP_, kHeads = GH_, kUnit = kTile, kUnitStart = kStart;
  // With 8 heads the reads of the queries in shared memory bound it: twice the keys of a
  // step use each, with the registers of a block alone on its SM.
  static constexpr int kBlocks = GH_ == 8 ? 1 : 2;
  static constexpr int KG = (GH_ == 8 ? 256 : 128) / DP;  // 8-key groups of a step: 32 registers of keys, 32 of values (64 each)
  static constexpr int kKeys = 8 * KG;
  static constexpr uint32_t kAll = 0xffffffffu >> (32 - kKeys);
  static constexpr int kLanes = DP / 4;          // lanes to a row of values
  static constexpr int kRows = 32 / kLanes;      // rows of values a load covers
  // Dims of a lane's piece i of a key: in heads up to 64 lane c has 8 of every 32, in two
  // pieces for one load; in larger ones 4 of every 16 (the wide loads' register groups
  // spill there: 16 over 8 heads of 128, 48.7 us instead of 42.9).
  static constexpr bool kPairs = DP == 64;
  static __device__ __forceinline__ int piece_dim(int i, int c) { return kPairs ? i / 2 * 32 + c * 8 + i % 2 * 4 : i * 16 + c * 4; }
  static constexpr int kQuery = kHeads * DP + kKeys * kHeads;  // a warp's queries and probabilities

  static __device__ __forceinline__ void stage_query(const DecodeParams& p, float* mine, const Part& w) {
    __syncwarp();
    // 16 bytes a lane, all of them under way at once (an element at a time 8 sequences of
    // up to 105 keys, 16 over 4 heads of 80, 9.3 us instead of 7.1)
    constexpr int kPieces = kHeads * DP / 4;
    uint4 u[(kPieces + 31) / 32];
#pragma unroll
    for (int k = 0; k < (kPieces + 31) / 32; ++k) {
      const int i = ((threadIdx.x & 31) + k * 32) * 4, qh = i / DP, e = i % DP;
      u[k] = load16_if((const float*)p.a.q + w.s * p.a.q_row + (w.hq + qh) * p.a.q_head + e, qh < w.n && e < p.c.head_dim);
    }
#pragma unroll
    for (int k = 0; k < (kPieces + 31) / 32; ++k) {
      const int i = (threadIdx.x & 31) + k * 32;
      if (i < kPieces) reinterpret_cast<uint4*>(mine)[i] = u[k];
    }
    __syncwarp();
  }

  static __device__ __forceinline__ void run(const DecodeParams& p, float* mine, const Part& w) {
    const int k0 = w.k0, k1 = w.k1;
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const int d = p.c.head_dim;
    const int64_t row = p.c.slot_stride;
    const int vd = (lane % kLanes) * 4, vrow = lane / kLanes;
    const float* kb = (const float*)p.c.k + (kFast ? r * row : 0);
    const float* vb = (const float*)p.c.v + vd + (kFast ? vrow * row : 0);
    const float* sq = mine;
    float* sp = mine + kHeads * DP;  // [key][head]
    float m[kHeads], l[kHeads];
    float4 o[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) m[i] = -INFINITY, l[i] = 0.f, o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    uint4 kr[KG][DP / 16], vr[kKeys / kRows];
    Walk<kFast, kKeys> walk(p, w.s, w.h, k0, k1);
    typename Walk<kFast, kKeys>::Off off[KG];  // of the step's groups of 8 (kFast); off[0]: of the lane's key
    auto advance = [&] {
      if constexpr (kFast) {
#pragma unroll
        for (int g = 0; g < KG; ++g) off[g] = walk.group();
      } else {
        off[0] = walk.off;
        walk.turn();
      }
    };
    auto load_keys = [&] {
#pragma unroll
      for (int g = 0; g < KG; ++g)
        if constexpr (kFast) {
          const float* at = group_at(kb, off[g]);
#pragma unroll
          for (int i = 0; i < DP / 16; i += 2)
            if constexpr (kExact && kPairs) load32(at + piece_dim(i, c), kr[g][i], kr[g][i + 1]);
            else if constexpr (kExact) kr[g][i] = load16(at + piece_dim(i, c)), kr[g][i + 1] = load16(at + piece_dim(i + 1, c));
            else kr[g][i] = load16_if(at + piece_dim(i, c), piece_dim(i, c) < d), kr[g][i + 1] = load16_if(at + piece_dim(i + 1, c), piece_dim(i + 1, c) < d);
        } else {
          const int64_t at = __shfl_sync(0xffffffffu, off[0], g * 8 + r);
#pragma unroll
          for (int i = 0; i < DP / 16; ++i) kr[g][i] = load16_if(kb + at + piece_dim(i, c), at >= 0 && piece_dim(i, c) < d);
        }
    };
    stage_query(p, mine, w);
    walk.turn();
    advance();
    load_keys();
    for (int k = k0; k < k1; k += kKeys) {
      uint32_t there = kAll;  // keys that count
      if constexpr (kFast) {
#pragma unroll
        for (int g = 0; g < KG; ++g) {
          const float* at = group_at(vb, off[g]);
#pragma unroll
          for (int i = 0; i < 8 / kRows; ++i)
            vr[g * (8 / kRows) + i] = kExact ? load16(at + i * kRows * row) : load16_if(at + i * kRows * row, vd < d);
          if (off[g] == ~0u) there &= ~(0xffu << (g * 8));
        }
        if (k1 - k < kKeys) there &= (1u << (k1 - k)) - 1u;
        if (there != kAll)  // what a slot that does not count holds may be NaN
#pragma unroll
          for (int i = 0; i < kKeys / kRows; ++i)
            if (!((there >> (i * kRows + vrow)) & 1u)) vr[i] = make_uint4(0u, 0u, 0u, 0u);
      } else {
#pragma unroll
        for (int i = 0; i < kKeys / kRows; ++i) {
          const int64_t at = __shfl_sync(0xffffffffu, off[0], i * kRows + vrow);
          vr[i] = load16_if(vb + at, at >= 0 && vd < d);
        }
        there = __ballot_sync(0xffffffffu, off[0] >= 0);
      }
      advance();
      float z[KG][kHeads];
#pragma unroll
      for (int i = 0; i < kHeads; ++i) {
#pragma unroll
        for (int g = 0; g < KG; ++g) z[g][i] = 0.f;
#pragma unroll
        for (int b = 0; b < DP / 16; ++b) {
          const float4 x = *reinterpret_cast<const float4*>(sq + i * DP + piece_dim(b, c));
#pragma unroll
          for (int g = 0; g < KG; ++g) {
            const uint4 u = kr[g][b];
            z[g][i] = fmaf(x.x, __uint_as_float(u.x), z[g][i]);
            z[g][i] = fmaf(x.y, __uint_as_float(u.y), z[g][i]);
            z[g][i] = fmaf(x.z, __uint_as_float(u.z), z[g][i]);
            z[g][i] = fmaf(x.w, __uint_as_float(u.w), z[g][i]);
          }
        }
      }
      // (keys past the last step left out: 177 sequences of 32 to 52 keys, 16 heads of 128,
      // 28.4 us instead of 29.7)
      if (!kFast || k + kKeys < k1) load_keys();
      bool move = false;
#pragma unroll
      for (int g = 0; g < KG; ++g) {
        const bool ok = (there >> (g * 8 + r)) & 1u;
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
          z[g][i] += __shfl_xor_sync(0xffffffffu, z[g][i], 1);
          z[g][i] += __shfl_xor_sync(0xffffffffu, z[g][i], 2);
          z[g][i] = ok ? z[g][i] * p.scale2 : -INFINITY;
          move |= z[g][i] > m[i] + 8.f;
        }
      }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
          float top = m[i];
#pragma unroll
          for (int g = 0; g < KG; ++g) top = fmaxf(top, z[g][i]);
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
          const float keep = weight(m[i], top);
          m[i] = top;
          l[i] *= keep;
          o[i].x *= keep, o[i].y *= keep, o[i].z *= keep, o[i].w *= keep;
        }
      }
      __syncwarp();  // the last step's probabilities have been read
#pragma unroll
      for (int g = 0; g < KG; ++g)
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
          const float e = exp2_fast(z[g][i] - (m[i] == -INFINITY ? 0.f : m[i]));
          l[i] += e;
          if ((i & 3) == c) sp[(g * 8 + r) * kHeads + i] = e;
        }
      __syncwarp();
#pragma unroll
      for (int j = 0; j < kKeys / kRows; ++j) {
        const float* e = sp + (j * kRows + vrow) * kHeads;
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
          o[i].x = fmaf(e[i], __uint_as_float(vr[j].x), o[i].x);
          o[i].y = fmaf(e[i], __uint_as_float(vr[j].y), o[i].y);
          o[i].z = fmaf(e[i], __uint_as_float(vr[j].z), o[i].z);
          o[i].w = fmaf(e[i], __uint_as_float(vr[j].w), o[i].w);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
#pragma unroll
      for (int x = kLanes; x < 32; x <<= 1) {
        o[i].x += __shfl_xor_sync(0xffffffffu, o[i].x, x);
        o[i].y += __shfl_xor_sync(0xffffffffu, o[i].y, x);
        o[i].z += __shfl_xor_sync(0xffffffffu, o[i].z, x);
        o[i].w += __shfl_xor_sync(0xffffffffu, o[i].w, x);
      }
      if (i >= w.n) continue;
      if (w.left) {
        if (lane == 0) w.left[2 * i] = m[i], w.left[2 * i + 1] = l[i];
        if (vrow == 0) *reinterpret_cast<float4*>(w.left + left_o(kHeads) + i * DP + vd) = o[i];
      } else {
        const float inv = l[i] == 0.f ? 0.f : 1.0f / l[i];
        if (vrow == 0 && (kExact || vd < d))
          *reinterpret_cast<float4*>((float*)p.a.out + w.s * p.a.out_row + (w.hq + i) * p.a.out_head + vd) =
              make_float4(o[i].x * inv, o[i].y * inv, o[i].z * inv, o[i].w * inv);
        if (lane == 0) store_lse(p, w.s, w.hq + i, m[i], l[i]);
      }
    }
  }
};

// ---- the kernels --------------------------------------------------------------

template <class P>
__global__ void __launch_bounds__(kWarps * 32, P::kBlocks) decode_kernel(const __grid_constant__ DecodeParams p) {
  using T = typename P::T;
  constexpr int kLeft = left_floats(P::kHeads, P::DP);
  extern __shared__ __align__(16) float sm[];  // [kWarps][2] pieces, [kWarps] queries
  __shared__ struct { int s, row, valid, ends, tiles; } info[kWarps][2];  // a team's pieces: that continues a row, that begins one
  after_stream();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n_seq = p.c.n_seq, d = p.c.head_dim;
  const int blk = blockIdx.x, blocks = gridDim.x;
  const int teams = kWarps / p.team, team = warp / p.team, hl = warp % p.team;
  if (hl == 0 && lane < 2) info[team][lane].valid = 0;  // by the warp that sets it: no block barrier before the join
  __syncwarp();
  if (tid == 0) p.meta[blk].seq = -1;

  // The line of work: for every row its start (as long as P::kUnitStart tiles), then its
  // tiles.  Every warp looks at the sequences for itself, 256 at a time, 8 a lane.
  constexpr int kLook = 8;
  int keys[kLook];          // of the lane's sequences
  int64_t before, total;    // units before them among those looked at, and of all of these
  auto look_at = [&](int s0) {
    int64_t sum = 0;
#pragma unroll
    for (int i = 0; i < kLook; ++i) {
      const int s = s0 + lane * kLook + i;
      keys[i] = s < n_seq ? seq_len(p, s, tid == lane && blk == 0) : 0;
    }
#pragma unroll
    for (int i = 0; i < kLook; ++i) sum += keys[i] > 0 ? (keys[i] + P::kUnit - 1) / P::kUnit + P::kUnitStart : 0;
    sum *= p.rows;
    before = sum;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, before, x);
      if (lane >= x) before += y;
    }
    total = __shfl_sync(0xffffffffu, before, 31);
    before -= sum;
  };
  int64_t units = 0;
  for (int s0 = 0; s0 < n_seq; s0 += 32 * kLook) look_at(s0), units += total;
  const int64_t active = min((int64_t)blocks * teams, units), gt = (int64_t)blk * teams + team;
  auto cut = [&](int64_t i) {  // where part i of the line begins
    return (uint64_t)(i * units) >> 32 ? i * units / active : (int64_t)((uint32_t)(i * units) / (uint32_t)active);
  };
  const int64_t begin = gt < active ? cut(gt) : 0, end = gt < active ? cut(gt + 1) : 0;

  auto empty_rows = [&] {  // sequences of no keys
    for (int s = blk; s < n_seq; s += blocks)
      if (seq_len(p, s, false) == 0) {
        const float zero[4] = {0.f, 0.f, 0.f, 0.f};
        for (int i = tid; i < p.a.n_head * (d / 4); i += kWarps * 32)
          store4((T*)p.a.out + s * p.a.out_row + i / (d / 4) * p.a.out_head + i % (d / 4) * 4, zero);
        for (int h = tid; h < p.a.n_head; h += kWarps * 32) store_lse(p, s, h, 0.f, 0.f);
      }
  };
  if ((int64_t)blk * teams >= active) return empty_rows();

  // the sequence that the team begins in, its keys and the units of it before that
  int s = 0, len = 0;
  int64_t into = 0, base = 0;
  for (int s0 = 0; s0 < n_seq; s0 += 32 * kLook) {
    if (n_seq > 32 * kLook) look_at(s0);
    if (begin >= base && begin < base + total) {
      const int owner = 31 - __clz(__ballot_sync(0xffffffffu, base + before <= begin));  // the last lane at or before `begin`
      int64_t at = begin - base - before;
#pragma unroll
      for (int i = 0; i < kLook; ++i) {
        const int64_t here = keys[i] > 0 ? (int64_t)((keys[i] + P::kUnit - 1) / P::kUnit + P::kUnitStart) * p.rows : 0;
        if (at >= 0 && at < here) s = s0 + lane * kLook + i, len = keys[i], into = at;
        at -= here;
      }
      s = __shfl_sync(0xffffffffu, s, owner), len = __shfl_sync(0xffffffffu, len, owner);
      into = __shfl_sync(0xffffffffu, into, owner);
      break;
    }
    base += total;
  }

  float* mine = sm + kWarps * 2 * kLeft + warp * P::kQuery;
  int64_t left = end - begin;
  if (left > 0) {
    int tiles = (len + P::kUnit - 1) / P::kUnit;
    int row, at;  // units of the row before the team's
    if (into >> 32) row = (int)(into / (tiles + P::kUnitStart)), at = (int)(into % (tiles + P::kUnitStart));
    else row = (uint32_t)into / (uint32_t)(tiles + P::kUnitStart), at = (uint32_t)into % (uint32_t)(tiles + P::kUnitStart);
    while (true) {
      const int stop = (int)min((int64_t)(tiles + P::kUnitStart), at + left);
      const int t0 = max(at - P::kUnitStart, 0), t1 = max(stop - P::kUnitStart, 0);
      const bool whole = t0 == 0 && t1 == tiles;
      Part w;
      w.s = s, w.h = row / p.chunks * p.team + hl;
      w.hq = w.h * p.group + row % p.chunks * p.chunk, w.n = min(p.chunk, (w.h + 1) * p.group - w.hq);
      w.k0 = t0 * P::kUnit, w.k1 = min(len, t1 * P::kUnit);
      w.left = whole ? nullptr : sm + (warp * 2 + (t0 == 0)) * kLeft;
      if (t1 > t0) P::run(p, mine, w);
      if (t1 > t0 && !whole && hl == 0 && lane == 0) {
        auto& f = info[team][t0 == 0];
        f.s = s, f.row = row, f.valid = 1, f.ends = t1 == tiles, f.tiles = tiles - t1;
      }
      left -= stop - at;
      if (left == 0) break;
      at = 0;
      if (++row == p.rows) {
        row = 0;
        do len = seq_len(p, ++s, false); while (len == 0);
        tiles = (len + P::kUnit - 1) / P::kUnit;
      }
    }
  }
  __syncthreads();

  // Join the pieces of each row: one that begins a row or comes from the block
  // before, then the next teams' continuations.  Piece 2 t + b: of team t.
  uint32_t valid, ends;
  {
    const bool there = lane < 2 * teams && info[(lane & 15) >> 1][lane & 1].valid;
    valid = __ballot_sync(0xffffffffu, there);
    ends = __ballot_sync(0xffffffffu, there && info[(lane & 15) >> 1][lane & 1].ends);
  }
  while (valid) {
    const int j = __ffs(valid) - 1;
    int last = j;  // pieces j, then 2 (j / 2 + 1), ... last
    while (!((ends >> last) & 1u) && (valid >> ((last | 1) + 1)) & 1u) last = (last | 1) + 1;
    valid &= ~((2u << last) - 1u);
    const int ps = info[j >> 1][j & 1].s, row = info[j >> 1][j & 1].row;
    const bool begins = j & 1, done = begins && (ends >> last) & 1u;
    const int first = row % p.chunks * p.chunk, n = min(p.chunk, p.group - first);
    const int64_t slot = 2 * blk + begins;
    for (int i = tid; i < p.team * p.chunk * (d / 4); i += kWarps * 32) {
      const int e = i % (d / 4) * 4, qh = i / (d / 4) % p.chunk, g = i / (d / 4) / p.chunk;
      if (qh >= n) continue;
      float top = -INFINITY, sum = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
      auto piece = [&](int k) { return sm + (((k >> 1) * p.team + g) * 2 + (k & 1)) * kLeft; };
      for (int k = j; k <= last; k = (k | 1) + 1) top = fmaxf(top, piece(k)[2 * qh]);
      for (int k = j; k <= last; k = (k | 1) + 1) {
        const float* from = piece(k);
        const float keep = weight(from[2 * qh], top);
        sum += from[2 * qh + 1] * keep;
        const float4 y = *reinterpret_cast<const float4*>(from + left_o(P::kHeads) + qh * P::DP + e);
        x[0] += y.x * keep, x[1] += y.y * keep, x[2] += y.z * keep, x[3] += y.w * keep;
      }
      if (done) {
        const int hq = (row / p.chunks * p.team + g) * p.group + first + qh;
        const float inv = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] *= inv;
        store4((T*)p.a.out + ps * p.a.out_row + hq * p.a.out_head + e, x);
        if (e == 0) store_lse(p, ps, hq, top, sum);
      } else {
        const int64_t at = (slot * p.team + g) * p.chunk + qh;
        if (e == 0) p.piece_ml[2 * at] = top, p.piece_ml[2 * at + 1] = sum;
        store4(p.piece_o + at * d + e, x);
      }
    }
    if (begins && !done && tid == 0) {  // the row goes on in later blocks: which team ends it?
      const int64_t stop = cut((int64_t)blk * teams + (j >> 1) + 1) + info[j >> 1][1].tiles;
      int64_t to = (int64_t)((float)stop * (float)active / (float)units);  // then exactly: begins before stop, the next does not
      while ((to + 1) * units < stop * active) ++to;
      while (to * units >= stop * active) --to;
      p.meta[blk] = Meta{ps, row, (int)to / teams, 0};
    }
  }
  empty_rows();
}

// The query heads of this block's rows in decode_row_kernel, once more.
template <typename T>
__device__ __noinline__ void careful_rows(const DecodeParams& p, float* scratch) {
  const int64_t row0 = (int64_t)(blockIdx.x / cg::this_cluster().num_blocks()) * p.pack, all = (int64_t)p.c.n_seq * p.rows;
  for (int i = 0; i < p.pack * p.chunk && row0 + i / p.chunk < all; ++i) {
    const int row = (int)((row0 + i / p.chunk) % p.rows), h = row / p.chunks, hq = h * p.group + row % p.chunks * p.chunk + i % p.chunk;
    if (hq < (h + 1) * p.group) careful_head<T>(p, (int)((row0 + i / p.chunk) / p.rows), h, hq, scratch);
  }
}

// Few or short rows: a cluster of blocks per row, or a block for `pack` rows, the keys
// of a row in equal parts over its warps; these are joined in shared memory, blocks
// through each other's.  One launch, no line of work to look up, no workspace.
template <class P>
__global__ void __launch_bounds__(kWarps * 32, P::kBlocks) decode_row_kernel(const __grid_constant__ DecodeParams p) {
  using T = typename P::T;
  constexpr int kLeft = left_floats(P::kHeads, P::DP);
  extern __shared__ __align__(16) float sm[];  // [kWarps] pieces, the block's piece, [kWarps] queries
  __shared__ int infinite;  // a result of the block's, or in the first block of the cluster's, is not finite
  cg::cluster_group cluster = cg::this_cluster();
  const int blocks = cluster.num_blocks(), rank = cluster.block_rank();
  after_stream();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, d = p.c.head_dim;
  if (tid == 0) infinite = 0;
  const int each = kWarps / p.pack;  // warps of a row
  const int64_t row0 = (int64_t)(blockIdx.x / blocks) * p.pack, all = (int64_t)p.c.n_seq * p.rows;
  auto part_of = [&](int64_t r) {  // sequence and heads of a row
    Part w;
    w.s = (int)r / p.rows, w.h = (int)r % p.rows / p.chunks;
    w.hq = w.h * p.group + (int)r % p.rows % p.chunks * p.chunk, w.n = min(p.chunk, (w.h + 1) * p.group - w.hq);
    return w;
  };
  if (warp < each * p.pack && row0 + warp / each < all) {
    Part w = part_of(row0 + warp / each);
    const int len = seq_len(p, w.s, true), tiles = (len + kTile - 1) / kTile;
    const int part = rank * each + warp % each, parts = blocks * each;
    w.k0 = (int)((int64_t)part * tiles / parts) * kTile, w.k1 = min(len, (int)((int64_t)(part + 1) * tiles / parts) * kTile);
    w.left = sm + warp * kLeft;
    if (w.k0 < w.k1) P::run(p, sm + (kWarps + 1) * kLeft + warp * P::kQuery, w);
    else if (lane < w.n) w.left[2 * lane] = -INFINITY, w.left[2 * lane + 1] = 0.f;
  }
  __syncthreads();
  // (m, l, o) of one head and four dims over n pieces, those without keys left out
  auto join = [&](int qh, int e, int n, auto piece, float& top, float& sum, float* x) {
    top = -INFINITY, sum = 0.f, x[0] = x[1] = x[2] = x[3] = 0.f;
    for (int k = 0; k < n; ++k) top = fmaxf(top, piece(k)[2 * qh]);
    for (int k = 0; k < n; ++k) {
      const float* from = piece(k);
      if (from[2 * qh + 1] == 0.f) continue;
      const float keep = weight(from[2 * qh], top);
      sum += from[2 * qh + 1] * keep;
      const float4 y = *reinterpret_cast<const float4*>(from + left_o(P::kHeads) + qh * P::DP + e);
      x[0] += y.x * keep, x[1] += y.y * keep, x[2] += y.z * keep, x[3] += y.w * keep;
    }
  };
  auto finish = [&](const Part& w, int qh, int e, float top, float sum, float* x) {
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] *= inv;
    store4((T*)p.a.out + w.s * p.a.out_row + (w.hq + qh) * p.a.out_head + e, x);
    if (e == 0) store_lse(p, w.s, w.hq + qh, top, sum);
    if (!finite4(x) && sum * 0.f == 0.f) *cluster.map_shared_rank(&infinite, 0) = 1;
  };
  float top, sum, x[4];
  float* whole = sm + kWarps * kLeft;
  for (int i = tid; i < p.pack * p.chunk * (d / 4); i += kWarps * 32) {
    const int e = i % (d / 4) * 4, qh = i / (d / 4) % p.chunk, g = i / (d / 4) / p.chunk;
    if (row0 + g >= all) break;
    const Part w = part_of(row0 + g);
    if (qh >= w.n) continue;
    join(qh, e, each, [&](int k) { return sm + (g * each + k) * kLeft; }, top, sum, x);
    if (blocks == 1) {
      finish(w, qh, e, top, sum, x);
    } else {
      if (e == 0) whole[2 * qh] = top, whole[2 * qh + 1] = sum;
      store4(whole + left_o(P::kHeads) + qh * P::DP + e, x);
    }
  }
  if (blocks == 1) {
    __syncthreads();
  } else {
    cluster.sync();
    const Part w = part_of(row0);
    for (int i = rank * kWarps * 32 + tid; i < w.n * (d / 4); i += blocks * kWarps * 32) {
      const int e = i % (d / 4) * 4, qh = i / (d / 4);
      join(qh, e, blocks, [&](int k) { return (const float*)cluster.map_shared_rank(whole, k); }, top, sum, x);
      finish(w, qh, e, top, sum, x);
    }
    cluster.sync();  // a block's memory stays until the others have read it
  }
  if (infinite) careful_rows<T>(p, sm);
}

// A row that several blocks worked on: the pieces of its blocks, joined.  Block
// (b, y): the row begun in block b, its query heads from join_heads y on; the warps
// share the heads and, where these are fewer, the pieces.  The last y: look_at_heads.
template <typename T>
__device__ __forceinline__ void join_row(const DecodeParams& p, float* scratch) {
  __shared__ float sm_ml[kWarps][2], sm_o[kWarps][128];
  __shared__ int again[kWarps];  // heads whose results are not finite, or -1
  const int blk = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = p.c.head_dim;
  const Meta mt = p.meta[blk];
  if (mt.seq < 0) return;
  const int first = mt.row % p.chunks * p.chunk, n = min(p.chunk, p.group - first), pieces = mt.last - blk + 1;
  const int heads = min(p.join_heads, p.team * n - p.join_heads * (int)blockIdx.y);
  if (heads <= 0) return;
  const int share = pieces > 2 ? kWarps / heads : 1;  // warps of a head
  const int i = p.join_heads * blockIdx.y + warp / share, sub = warp % share, g = i / n, qh = i % n;
  const bool mine = warp / share < heads;
  float top = -INFINITY, total = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
  if (mine) {
    const int e = min(lane * 4, d - 4);
    auto at = [&](int j) { return ((int64_t)(j == 0 ? 2 * blk + 1 : 2 * (blk + j)) * p.team + g) * p.chunk + qh; };
    for (int j0 = sub; j0 < pieces; j0 += 32 * share) {  // a piece per lane at a time
      float2 ml = make_float2(-INFINITY, 0.f);
      if (j0 + lane * share < pieces) ml = *reinterpret_cast<const float2*>(p.piece_ml + 2 * at(j0 + lane * share));
      float best = fmaxf(top, ml.x);
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, w));
      const float keep = weight(top, best), factor = weight(ml.x, best);
      float sum = ml.y * factor;
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      total = total * keep + sum;
      top = best;
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] *= keep;
      const int count = min(32, (pieces - j0 + share - 1) / share);
      for (int j = 0; j < count; j += 8) {
        float4 y[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) y[u] = *reinterpret_cast<const float4*>(p.piece_o + at(j0 + min(j + u, count - 1) * share) * d + e);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float f = __shfl_sync(0xffffffffu, factor, (j + u) & 31);
          if (j + u < count) x[0] += y[u].x * f, x[1] += y[u].y * f, x[2] += y[u].z * f, x[3] += y[u].w * f;
        }
      }
    }
  }
  if (share > 1) {  // the first warp of a head adds the others'
    if (lane == 0) sm_ml[warp][0] = top, sm_ml[warp][1] = total;
    store4(&sm_o[warp][lane * 4], x);
    __syncthreads();
  }
  const bool ends = mine && sub == 0;
  if (share > 1 && ends) {
    float best = top;
    for (int w = 1; w < share; ++w) best = fmaxf(best, sm_ml[warp + w][0]);
    const float keep = weight(top, best);
    total *= keep;
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] *= keep;
    for (int w = 1; w < share; ++w) {
      const float f = weight(sm_ml[warp + w][0], best);
      total += sm_ml[warp + w][1] * f;
      const float4 y = *reinterpret_cast<const float4*>(&sm_o[warp + w][lane * 4]);
      x[0] += y.x * f, x[1] += y.y * f, x[2] += y.z * f, x[3] += y.w * f;
    }
    top = best;
  }
  int infinite = -1;
  if (ends) {
    const int hq = (mt.row / p.chunks * p.team + g) * p.group + first + qh;
    const float inv = total == 0.f ? 0.f : 1.0f / total;
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] *= inv;
    if (lane * 4 < d) store4((T*)p.a.out + mt.seq * p.a.out_row + hq * p.a.out_head + lane * 4, x);
    if (lane == 0) store_lse(p, mt.seq, hq, top, total);
    if (!__all_sync(0xffffffffu, finite4(x))) infinite = hq;
  }
  if (lane == 0) again[warp] = infinite;
  if (__syncthreads_and(infinite < 0)) return;
  for (int w = 0; w < kWarps; ++w)
    if (again[w] >= 0) careful_head<T>(p, mt.seq, again[w] / p.group, again[w], scratch);
}

// The heads that the line kernel ended itself, looked at for results that are not finite.
template <typename T>
__device__ __forceinline__ void look_at_heads(const DecodeParams& p, float* scratch) {
  constexpr int kAtOnce = 4;
  __shared__ uint32_t found[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = p.c.head_dim, e = min(lane * 4, d - 4);
  const int64_t heads = (int64_t)p.c.n_seq * p.a.n_head, warps = (int64_t)gridDim.x * kWarps;
  auto sequence = [&](int64_t at) { return at >> 32 ? (int)(at / p.a.n_head) : (int)((uint32_t)at / (uint32_t)p.a.n_head); };
  for (int64_t head0 = (int64_t)blockIdx.x * kWarps; head0 < heads; head0 += kAtOnce * warps) {
    float x[kAtOnce][4];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int64_t at = min(head0 + warp + i * warps, heads - 1);
      const int s = sequence(at);
      load4((const T*)p.a.out + s * p.a.out_row + (at - (int64_t)s * p.a.n_head) * p.a.out_head + e, x[i]);
    }
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) bits |= !finite4(x[i]) && head0 + warp + i * warps < heads ? 1u << i : 0u;
    if (__syncthreads_and(bits == 0)) continue;
    bits = __reduce_or_sync(0xffffffffu, bits);
    if (lane == 0) found[warp] = bits;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w)
      for (uint32_t b = found[w]; b; b &= b - 1) {
        const int64_t at = head0 + w + (__ffs(b) - 1) * warps;
        const int s = sequence(at), hq = (int)(at - (int64_t)s * p.a.n_head), h = hq / p.group;
        bool joined = false;  // in another block, which looks at what it has written itself
        for (int i = lane; i < gridDim.x; i += 32)
          joined |= p.meta[i].seq == s && p.meta[i].row == h / p.team * p.chunks + hq % p.group / p.chunk;
        if (!__any_sync(0xffffffffu, joined)) careful_head<T>(p, s, h, hq, scratch);
      }
    __syncthreads();
  }
}

// Looking at the heads here takes 0.2 to 1.3 us (200 sequences of 1 to 1,024 keys, 16 heads of
// 64, 81.8 us with it and 80.4 without; 131,071 keys 93.1 and 92.3); in the line kernel, where
// a row ends, it takes as much, and with heads of 96 5 us (104 sequences of 13 to 878 keys, 8
// heads, 42.7, here 38.2).
template <typename T>
__global__ void __launch_bounds__(kWarps * 32, 3) decode_join_kernel(const __grid_constant__ DecodeParams p) {
  __shared__ float scratch[kCarefulFloats];
  after_stream();
  if (blockIdx.y + 1 < gridDim.y) join_row<T>(p, scratch);
  else look_at_heads<T>(p, scratch);
}

template <class P>
int launch(const DecodeParams& p, const Plan& pl, cudaStream_t st) {
  constexpr int kLeft = left_floats(P::kHeads, P::DP);
  constexpr int kRowBytes = ((kWarps + 1) * kLeft + kWarps * P::kQuery) * 4, kLineBytes = kWarps * (2 * kLeft + P::kQuery) * 4;
  static_assert(kRowBytes >= kCarefulFloats * 4, "careful_head's scratch");
  static thread_local int ready = -1;  // device whose shared-memory limits have been raised
  int dev = -1;
  cudaGetDevice(&dev);
  if (ready != dev) {
    cudaError_t e = cudaFuncSetAttribute(decode_row_kernel<P>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowBytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(decode_kernel<P>, cudaFuncAttributeMaxDynamicSharedMemorySize, kLineBytes);
    if (const int rc = check_cuda("gpt_decode_attention", e)) return rc;
    ready = dev;
  }
  if (pl.cluster) {
    const dim3 grid((unsigned)(((int64_t)p.c.n_seq * p.rows + pl.pack - 1) / pl.pack * pl.cluster));
    return launch_after("gpt_decode_attention", decode_row_kernel<P>, grid, kWarps * 32, kRowBytes, pl.cluster, st, p);
  }
  if (const int rc = launch_after("gpt_decode_attention", decode_kernel<P>, dim3(pl.blocks), kWarps * 32, kLineBytes, 0, st, p)) return rc;
  const dim3 grid(pl.blocks, (pl.team * pl.chunk + pl.join_heads - 1) / pl.join_heads + 1);
  return launch_after("gpt_decode_attention (join)", decode_join_kernel<typename P::T>, grid, kWarps * 32, 0, 0, st, p);
}

// The launch for a head size of at most DP: the fast forms need pages of whole 8-key
// groups within 64 GB, the exact one also heads of exactly DP, keys on 32-byte boundaries.
template <template <int, int, bool, bool> class Path, int N, int DP>
int launch_form(const DecodeParams& p, const Plan& pl, cudaStream_t st) {
  if (!pl.fast) return launch<Path<N, DP, false, false>>(p, pl, st);
  return pl.exact ? launch<Path<N, DP, true, true>>(p, pl, st) : launch<Path<N, DP, true, false>>(p, pl, st);
}

}  // namespace
}  // namespace pgs
