// decode_fp8.cuh — attention of one new token over a cache in 8 bits: the part of a
// row that a warp does, for the kernels of decode_attention.cuh.
//
// Keys and values are e4m3 numbers, a scale each per page and head.  A number is exact in
// fp16, so both products are mma.m16n8k16 on fp16 with fp32 sums:
//  - scores: 16 keys x 8 query heads, four dims of a lane to a product as they lie in
//    memory; the key scale of a page multiplies the score.  A query is brought below 2^15 by
//    a power of two of its own (what falls under 2^-25 there is 2^-39 of its largest): bf16
//    queries are then exact, fp32 ones enter as two fp16 parts (2^-23).
//  - values: the weights, each times the value scale of its page, enter as two fp16 parts (2^-22
//    left over) below 2^15.  Scales may lie further apart than fp16 reaches, and a key of the
//    largest weight in a page of a small one, so that these products have a reference of their
//    own beside the weights' (7 under the maximum): an integer, 10 under a bound of their largest
//    that is at most two above it.  What brings weights from one to the other is a power of two,
//    rounded down, so that what falls under fp16's smallest number is 2^-32 of the largest product.
// Bound: HBM, half the bytes of a bf16 cache, and the instructions beside it: 328 for 16 keys of 128
// dims, of these 69 conversions, 16 products and 95 on integers, and 1,900 for a row's start and end
// (64 ragged sequences of 32 over 8 heads of 128 104 us, 5.2 TB/s; 131,071 keys 61 us, 4.4 TB/s;
// 200 sequences of 16 heads of 64 48 us, 4.4 TB/s).  With 8 query heads to a key head 73 us (64 ragged
// sequences of 32 over 4 heads of 128, floor 40; for fp32 results 81); pages that are not of whole
// 8-key groups 78 us (64 of up to 4,096 keys, 32 over 8 heads, pages of 5; floor 40).
#pragma once
#include "decode_attention.cuh"

namespace pgs {
namespace {

__device__ __forceinline__ void mma16816_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The four numbers of a word as fp16 pairs.
__device__ __forceinline__ void to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h;}" : "=r"(lo), "=r"(hi) : "r"(w));
}
__device__ __forceinline__ uint32_t pack2_f16(float lo, float hi) {
  uint32_t u;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(hi), "f"(lo));
  return u;
}
__device__ __forceinline__ float2 unpack2_f16(uint32_t u) {
  float2 x;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}" : "=f"(x.x), "=f"(x.y) : "r"(u));
  return x;
}
// What two numbers leave over of their fp16 parts.
__device__ __forceinline__ uint32_t rest2_f16(float lo, float hi, uint32_t parts) {
  const float2 x = unpack2_f16(parts);
  return pack2_f16(lo - x.x, hi - x.y);
}
// The same, nothing of an infinity.
__device__ __forceinline__ uint32_t finite_rest2_f16(float lo, float hi, uint32_t parts) {
  const float2 x = unpack2_f16(parts);
  return pack2_f16(fabsf(x.x) == INFINITY ? 0.f : lo - x.x, fabsf(x.y) == INFINITY ? 0.f : hi - x.y);
}
__device__ __forceinline__ uint2 load8(const void* p) {
  uint2 u;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(u.x), "=r"(u.y) : "l"(p));
  return u;
}

__device__ __forceinline__ float power2(int n) { return __uint_as_float((uint32_t)(n + 127) << 23); }
__device__ __forceinline__ float power2_inverse(float x) { return __uint_as_float((254u << 23) - __float_as_uint(x)); }  // of a power of two
// log2 of a scale is below this (0: -126).
__device__ __forceinline__ float log2_above(float scale) { return (float)((int)(__float_as_uint(scale) >> 23) - 126); }

// As Walk, with the scales of each group's (or key's) page: table entries are read two
// rounds ahead and looked at one round ahead, when the scales are read.
template <bool kFast, int kKeys>
struct ScaledWalk {
  using Off = std::conditional_t<kFast, uint32_t, int64_t>;
  static constexpr Off kNoKey = (Off)-1;
  static constexpr int kRound = kFast ? 256 : kKeys;  // keys
  const DecodeParams& p;
  const int32_t* table;
  const float *ks_at, *vs_at;  // of the head
  Off head, off;
  float ks, vs, ks1, vs1;
  int at1, page1, page2, end, lane_at;

  __device__ __forceinline__ ScaledWalk(const DecodeParams& p_, int s, int h, int k0, int k1)
      : p(p_), table(p_.c.page_table + s * p_.c.table_stride), ks_at(p_.k_scale + h * p_.scale_head), vs_at(p_.v_scale + h * p_.scale_head),
        end(k1), lane_at(0) {
    const int lane = threadIdx.x & 31;
    head = kFast ? h * p.head16 : h * p.c.head_stride;
    at1 = k0 + (kFast ? lane * 8 : lane & (kKeys - 1));
    page1 = checked(entry(at1));
    scales();
    page2 = entry(at1 + kRound);
  }
  __device__ __forceinline__ int entry(int at) const { return at < end ? table[at / p.c.page_size] : -1; }
  __device__ __forceinline__ int checked(int id) const {  // the entry of at1
    if (id >= 0 && id < p.c.n_pages) return id;
    if (at1 < end) set_status(p.a.status, GPT_STATUS_BAD_PAGE);
    return -1;
  }
  __device__ __forceinline__ void scales() {
    ks1 = vs1 = 0.f;
    if (page1 >= 0) ks1 = __ldg(ks_at + page1 * p.scale_page), vs1 = __ldg(vs_at + page1 * p.scale_page);
  }
  // kFast: the offset of the lane's group of the next round.
  __device__ __forceinline__ Off next() const { return page1 < 0 ? kNoKey : page1 * p.page16 + (at1 % p.c.page_size) * p.slot16 + head; }
  __device__ __forceinline__ void turn() {
    if constexpr (kFast) off = next();
    else off = page1 < 0 ? kNoKey : page1 * p.c.page_stride + (at1 % p.c.page_size) * p.c.slot_stride + head;
    ks = ks1, vs = vs1;
    at1 += kRound, page1 = checked(page2);
    scales();
    page2 = entry(at1 + kRound);
  }
  // kFast: the next group of 8 keys.
  __device__ __forceinline__ void group(Off& o, float& k, float& v) {
    o = __shfl_sync(0xffffffffu, off, lane_at), k = __shfl_sync(0xffffffffu, ks, lane_at), v = __shfl_sync(0xffffffffu, vs, lane_at);
    if (++lane_at == 32) turn(), lane_at = 0;
  }
};

// kMode: query heads of a row, 16 of them in two tiles.  With 4, columns 4..7 of the products take
// the low parts of weights and fp32 queries (and bf16 ones once more); otherwise products of their own do.
template <typename T_, int kMode, int DP_, bool kFast, bool kExact>
struct Fp8Path {
  using T = T_;
  using Cache = E4m3;
  static constexpr bool kFull = std::is_same_v<T, float>;
  static constexpr int NT = kMode == 16 ? 2 : 1, DP = DP_, kHeads = kMode;
  static constexpr bool kTwice = kMode == 4;
  static constexpr int kParts = kFull && !kTwice ? 2 : 1;  // of a query, a product each
  static constexpr int kBlocks = kMode == 16 ? 1 : 2;      // of an SM
  // 16-key groups of a step: two of 128 dims leave too few registers (64 ragged sequences of 32 over 8 heads 144 us for 121),
  // two of 64 are as long as one of those (200 sequences of 16 heads 48.2 us and 49.0, 32 of 14 over 2 heads 16.1 and 17.2).
  static constexpr int KG = DP_ == 128 ? 1 : 2, kKeys = 16 * KG, kUnit = kKeys;
  // A row's start, in units: 104 ragged sequences of 8 heads of 96 28.7 us with 2, 27.2 with 3, 27.0 with 4, 27.5 with 6;
  // 200 of 16 heads of 64 (of 32 keys a unit) 48.1 48.2 49.0 49.3, 2 of up to 60,000 and 12 heads 40.8 39.2 38.1 39.7.
  static constexpr int kUnitStart = DP_ == 128 ? 4 : 3;
  static constexpr int KP = DP / 64;                       // a lane's 16-byte pieces of a key
  static constexpr int VW = DP / 32;                       // a lane's words of a value
  static constexpr int kQuery = NT * kParts * KP * 256;    // a warp's queries: 32 bytes per lane, tile, part and piece

  // Dims of a lane's piece i of a key or query; those of its part of a value begin at r * 4 VW.
  static __device__ __forceinline__ int piece_dim(int i, int c) { return c * 16 * KP + i * 16; }

  // Lane (r, c): query head r of a tile, its pieces, in fp16, eight words for each; put(part, piece,
  // half, four words).  Returns 2^e of the head, by which its scores are to be multiplied.
  template <typename Put>
  static __device__ __forceinline__ float read_query(const DecodeParams& p, const Part& w, int t, Put put) {
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const int qh = kTwice ? r & 3 : t * 8 + r;
    constexpr int kN = Piece<T>::kN, kLoads = 16 / kN;
    uint4 u[KP][kLoads];
#pragma unroll
    for (int i = 0; i < KP; ++i)
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
        u[i][j] = load16_if((const T*)p.a.q + w.s * p.a.q_row + (w.hq + qh) * p.a.q_head + piece_dim(i, c) + j * kN,
                            qh < w.n && piece_dim(i, c) < p.c.head_dim);
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < KP; ++i)
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        float x[kN];
        Piece<T>::unpack(u[i][j], x);
#pragma unroll
        for (int k = 0; k < kN; ++k) top = fabsf(x[k]) < INFINITY ? fmaxf(top, fabsf(x[k])) : top;
      }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int e = max((int)(__float_as_uint(top) >> 23) - 127 - 14, -126);  // top 2^-e is below 2^15
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
    for (int i = 0; i < KP; ++i)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float x[8];
#pragma unroll
        for (int k = 0; k < 8 / kN; ++k) Piece<T>::unpack(u[i][half * (8 / kN) + k], x + k * kN);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] *= down;
        uint32_t h[4], l[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          h[k] = pack2_f16(x[2 * k], x[2 * k + 1]);
          if (kFull) l[k] = finite_rest2_f16(x[2 * k], x[2 * k + 1], h[k]);
          if (kFull && kTwice && r >= 4) h[k] = l[k];
        }
        put(0, i, half, make_uint4(h[0], h[1], h[2], h[3]));
        if (kParts == 2) put(1, i, half, make_uint4(l[0], l[1], l[2], l[3]));
      }
    return __uint_as_float((uint32_t)(e + 127) << 23);
  }
  static __device__ __forceinline__ float stage_query(const DecodeParams& p, uint4* query, const Part& w, int t) {
    return read_query(p, w, t, [&](int part, int i, int half, uint4 x) { query[(((t * kParts + part) * KP + i) * 2 + half) * 32] = x; });
  }
  template <int N>
  static __device__ __forceinline__ float query_registers(const DecodeParams& p, uint32_t (&q)[N][8], const Part& w) {
    return read_query(p, w, 0, [&](int, int i, int half, uint4 x) {
      q[i][4 * half] = x.x, q[i][4 * half + 1] = x.y, q[i][4 * half + 2] = x.z, q[i][4 * half + 3] = x.w;
    });
  }

  // What a weight is multiplied by; finite, so that nothing is left of a weight of zero.
  static __device__ __forceinline__ float bring(float scale, float rate) { return fminf(scale * rate, 0x1.fffffep127f); }

  // New references of a column from its largest score, and bound of a product's log2, best and best_w of
  // a lane; m, mw, rate, l and o as in run.
  static __device__ __forceinline__ void move(float best, float best_w, float& m, float& mw, float& rate, float& l, float (&o)[VW][2][4], int e) {
    best = fmaxf(best, m + 7.f), best_w = fmaxf(best_w, mw + 10.f);
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, x));
      best_w = fmaxf(best_w, __shfl_xor_sync(0xffffffffu, best_w, x));
    }
    best -= 7.f, best_w = ceilf(best_w) - 10.f;
    const float keep = weight(m, best), n = fminf(fmaxf(floorf(best - best_w), -126.f), 126.f);
    const int more = (int)n - ((int)(__float_as_uint(rate) >> 23) - 127);
    const float keep_w = keep * power2(more / 2) * power2(more - more / 2);
    m = best, mw = best_w, rate = power2((int)n);
    l *= keep;
#pragma unroll
    for (int b = 0; b < VW; ++b)
#pragma unroll
      for (int i = 0; i < 2; ++i) o[b][i][e] *= keep_w, o[b][i][e + 2] *= keep_w;
  }

  // What lane (r, c) has of query head qh: reference, sum of weights, its dims of their values' sum.
  static __device__ __forceinline__ void finish(const DecodeParams& p, const Part& w, int qh, float m, float total, float (&y)[VW][4]) {
    const int r = (threadIdx.x & 31) >> 2;
    if (qh >= w.n) return;
    if (w.left) {
      if (r == 0) w.left[2 * qh] = m, w.left[2 * qh + 1] = total;
      float* to = w.left + left_o(kHeads) + qh * DP + r * 4 * VW;
#pragma unroll
      for (int b = 0; b < VW; ++b) store4(to + 4 * b, y[b]);
    } else {
      const float inv = total == 0.f ? 0.f : 1.0f / total;
      T* to = (T*)p.a.out + w.s * p.a.out_row + (w.hq + qh) * p.a.out_head + r * 4 * VW;
#pragma unroll
      for (int b = 0; b < VW; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) y[b][i] *= inv;
      if (kExact || r * 4 * VW < p.c.head_dim)
#pragma unroll
        for (int b = 0; b < VW; ++b) store4(to + 4 * b, y[b]);
      if (r == 0) store_lse(p, w.s, w.hq + qh, m, total);
    }
  }

  static __device__ __forceinline__ void run(const DecodeParams& p, float* mine, const Part& w) {
    const int k0 = w.k0, k1 = w.k1;
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const int d = p.c.head_dim;
    const int64_t row = p.c.slot_stride;
    const uint8_t* kb = (const uint8_t*)p.c.k + (kFast ? r * row : 0);
    const uint8_t* vb = (const uint8_t*)p.c.v + r * 4 * VW + (kFast ? 2 * c * row : 0);
    uint4* query = reinterpret_cast<uint4*>(mine) + lane;
    // m, mw: references of the weights, and of their products with scales; rate: 2^(m - mw), rounded down to a power of two
    float o[NT][VW][2][4], m[NT][2], mw[NT][2], rate[NT][2], l[NT][2], factor[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t][0] = m[t][1] = mw[t][0] = mw[t][1] = -INFINITY, rate[t][0] = rate[t][1] = 1.f, l[t][0] = l[t][1] = 0.f;
#pragma unroll
      for (int b = 0; b < VW; ++b)
#pragma unroll
        for (int i = 0; i < 8; ++i) o[t][b][i / 4][i % 4] = 0.f;
    }
    uint4 kr[KG][2][KP];
    uint32_t vr[KG][4][VW];
    using Keys = ScaledWalk<kFast, kKeys>;
    Keys walk(p, w.s, w.h, k0, k1);
    // Of the step's groups of 8: offsets, scales.  Without kFast: off[0][0] of the lane's key,
    // the scales of key g * 16 + u * 8 + r.
    typename Keys::Off off[KG][2];
    float ks[KG][2], vs[KG][2];
    auto advance = [&] {
      if constexpr (kFast) {
#pragma unroll
        for (int g = 0; g < KG; ++g)
#pragma unroll
          for (int u = 0; u < 2; ++u) walk.group(off[g][u], ks[g][u], vs[g][u]);
      } else {
        off[0][0] = walk.off;
#pragma unroll
        for (int g = 0; g < KG; ++g)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            ks[g][u] = __shfl_sync(0xffffffffu, walk.ks, g * 16 + u * 8 + r);
            vs[g][u] = __shfl_sync(0xffffffffu, walk.vs, g * 16 + u * 8 + r);
          }
      }
    };
    auto load_keys = [&] {
#pragma unroll
      for (int g = 0; g < KG; ++g)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if constexpr (kFast) {
            const uint8_t* at = group_at(kb, off[g][u]);
            if constexpr (kExact && KP == 2) load32(at + piece_dim(0, c), kr[g][u][0], kr[g][u][KP - 1]);
            else
#pragma unroll
              for (int i = 0; i < KP; ++i) kr[g][u][i] = kExact ? load16(at + piece_dim(i, c)) : load16_if(at + piece_dim(i, c), piece_dim(i, c) < d);
          } else {
            const int64_t at = __shfl_sync(0xffffffffu, off[0][0], g * 16 + u * 8 + r);
#pragma unroll
            for (int i = 0; i < KP; ++i) kr[g][u][i] = load16_if(kb + at + piece_dim(i, c), at >= 0 && piece_dim(i, c) < d);
          }
    };
    auto load_value = [&](const uint8_t* at, bool ok, uint32_t* to) {
      if constexpr (VW == 4) {
        const uint4 u = kExact ? load16(at) : load16_if(at, ok && r * 16 < d);
        to[0] = u.x, to[1] = u.y, to[2] = u.z, to[3] = u.w;
      } else {
        const uint2 u = kExact || (ok && r * 8 < d) ? load8(at) : make_uint2(0u, 0u);
        to[0] = u.x, to[1] = u.y;
      }
    };
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float up = stage_query(p, query, w, t);
      factor[t][0] = __shfl_sync(0xffffffffu, up, 8 * c);
      factor[t][1] = __shfl_sync(0xffffffffu, up, 8 * c + 4);
    }
    walk.turn();
    advance();
    if constexpr (!kFast) walk.turn();
    load_keys();
    for (int k = k0; k < k1; k += kKeys) {
      uint32_t there = 0xffffffffu;  // keys that count
#pragma unroll
      for (int g = 0; g < KG; ++g)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if constexpr (kFast) {
            load_value(group_at(vb, off[g][u >> 1]) + (u & 1) * row, true, vr[g][u]);
            if ((u & 1) && off[g][u >> 1] == ~0u) there &= ~(0xffu << (g * 16 + (u >> 1) * 8));
          } else {
            const int64_t at = __shfl_sync(0xffffffffu, off[0][0], g * 16 + (u >> 1) * 8 + 2 * c + (u & 1));
            load_value(vb + at, at >= 0, vr[g][u]);
          }
      if constexpr (kFast) {
        if (k1 - k < kKeys) there &= (1u << (k1 - k)) - 1u;
      } else {
        there = __ballot_sync(0xffffffffu, off[0][0] >= 0);
      }
      // the step's scales, and the largest of the values'
      float key_scale[KG][2], value_scale[KG][2], top = 0.f;
#pragma unroll
      for (int g = 0; g < KG; ++g)
#pragma unroll
        for (int u = 0; u < 2; ++u) key_scale[g][u] = ks[g][u], value_scale[g][u] = vs[g][u], top = fmaxf(top, vs[g][u]);
      advance();
      // scores: 16 keys x 8 columns a tile
      float z[KG][NT][4];
#pragma unroll
      for (int g = 0; g < KG; ++g)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) z[g][t][i] = 0.f;
#pragma unroll
      for (int i = 0; i < KP; ++i)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint4 q[NT][kParts];
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int x = 0; x < kParts; ++x) q[t][x] = query[(((t * kParts + x) * KP + i) * 2 + half) * 32];
#pragma unroll
          for (int g = 0; g < KG; ++g)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint32_t a0, a1, a2, a3;
              to_f16((&kr[g][0][i].x)[half * 2 + j], a0, a2);
              to_f16((&kr[g][1][i].x)[half * 2 + j], a1, a3);
#pragma unroll
              for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int x = 0; x < kParts; ++x) mma16816_f16(z[g][t], a0, a1, a2, a3, j ? q[t][x].z : q[t][x].x, j ? q[t][x].w : q[t][x].y);
            }
        }
      load_keys();
#pragma unroll
      for (int g = 0; g < KG; ++g)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (kFull && kTwice) z[g][t][i] += __shfl_xor_sync(0xffffffffu, z[g][t][i], 2);
            z[g][t][i] *= factor[t][i & 1] * key_scale[g][i >> 1] * p.scale2;
          }
      if (__builtin_expect(there != 0xffffffffu, 0)) {
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
                for (int b = 0; b < VW; ++b) vr[g][u][b] = 0u;
        }
      }
      // softmax: the references of a head move only when a weight, or its product with a scale, could pass 2^15
      bool move = false;
      const float above = log2_above(top);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float most = fminf(m[t][e], mw[t][e] - above) + 15.f;
#pragma unroll
          for (int g = 0; g < KG; ++g) move |= fmaxf(z[g][t][e], z[g][t][e + 2]) > most;
        }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float best = -INFINITY, best_w = -INFINITY;
#pragma unroll
            for (int g = 0; g < KG; ++g) {
              best = fmaxf(best, fmaxf(z[g][t][e], z[g][t][e + 2]));
              best_w = fmaxf(best_w, fmaxf(z[g][t][e] + log2_above(value_scale[g][0]), z[g][t][e + 2] + log2_above(value_scale[g][1])));
            }
            Fp8Path::move(best, best_w, m[t][e], mw[t][e], rate[t][e], l[t][e], o[t], e);
          }
      }
#pragma unroll
      for (int g = 0; g < KG; ++g) {
        uint32_t h0[NT], h1[NT], l0[NT], l1[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float m0 = fmaxf(m[t][0], -0x1.fffffep127f), m1 = fmaxf(m[t][1], -0x1.fffffep127f);
          float p0 = exp2_fast(z[g][t][0] - m0), p1 = exp2_fast(z[g][t][1] - m1);
          float p2 = exp2_fast(z[g][t][2] - m0), p3 = exp2_fast(z[g][t][3] - m1);
          l[t][0] += p0 + p2, l[t][1] += p1 + p3;
          p0 *= bring(value_scale[g][0], rate[t][0]), p1 *= bring(value_scale[g][0], rate[t][1]);
          p2 *= bring(value_scale[g][1], rate[t][0]), p3 *= bring(value_scale[g][1], rate[t][1]);
          uint32_t ha = pack2_f16(p0, p1), hb = pack2_f16(p2, p3);
          const uint32_t la = rest2_f16(p0, p1, ha), lb = rest2_f16(p2, p3, hb);
          if (kTwice) ha = c < 2 ? ha : la, hb = c < 2 ? hb : lb;
          h0[t] = transpose8(ha), h1[t] = transpose8(hb);
          if (!kTwice) l0[t] = transpose8(la), l1[t] = transpose8(lb);
        }
#pragma unroll
        for (int b = 0; b < VW; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t a0, a1, a2, a3;
            to_f16(__byte_perm(vr[g][0][b], vr[g][1][b], i ? 0x7362 : 0x5140), a0, a1);
            to_f16(__byte_perm(vr[g][2][b], vr[g][3][b], i ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              mma16816_f16(o[t][b][i], a0, a1, a2, a3, h0[t], h1[t]);
              if (!kTwice) mma16816_f16(o[t][b][i], a0, a1, a2, a3, l0[t], l1[t]);
            }
          }
      }
      // (At the end: next to the step's other loads it waits for them.  64 sequences in pages of 5 slots 78 us for 86.)
      if constexpr (!kFast) walk.turn();
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int qh = t * 8 + 2 * c + e;
        float total = l[t][e];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) total += __shfl_xor_sync(0xffffffffu, total, x);
        float y[VW][4];
#pragma unroll
        for (int b = 0; b < VW; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y[b][i] = o[t][b][i >> 1][e + 2 * (i & 1)];
            if (kTwice) y[b][i] += __shfl_xor_sync(0xffffffffu, y[b][i], 2);
            y[b][i] *= power2_inverse(rate[t][e]);
          }
        finish(p, w, qh, m[t][e], total, y);
      }
  }
};

// Up to 4 query heads, pages of whole 8-key groups: the same through shared memory.  The
// registers of a step's keys and values are all that a warp has under way above, and it waits
// for memory most of its time (long_scoreboard 6.2 of 10.6 clocks an instruction).  Here the next
// step's are on their way into a ring of two stages while a step is at work, and the one's after it
// as soon as its own are in registers: 8 KB a warp.  A stage's 16-byte pieces lie so that
// neighbouring rows' are in other banks.  The queries stay in registers.
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ uint4 shared16(uint32_t at) {
  uint4 u;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(at));
  return u;
}
__device__ __forceinline__ uint2 shared8(uint32_t at) {
  uint2 u;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(u.x), "=r"(u.y) : "r"(at));
  return u;
}

// 64 ragged sequences of 32 over 8 heads of 128 104 us (117 without the ring), 200 of 16 heads of 64 48 (61), 131,071 keys
// 61 (67).
// kSame: pages of whole 16-key groups, one scale for each of these (300 ragged sequences of 8 heads of 128 93.3 us, 94.1
// with two, 64 of 32 over 8 104.5 and 105.2).
template <typename T_, int DP_, bool kExact, bool kSame>
struct Fp8Ring {
  using T = T_;
  using Cache = E4m3;
  using Path = Fp8Path<T, 4, DP_, true, kExact>;
  static constexpr bool kFull = std::is_same_v<T, float>;
  static constexpr int DP = DP_, kHeads = 4, kBlocks = 2;
  static constexpr int KP = Path::KP, VW = Path::VW, KG = Path::KG, kKeys = Path::kKeys, kUnit = kKeys, kUnitStart = Path::kUnitStart;
  static constexpr int kGroups = 2 * KG;                    // groups of 8 keys of a step
  static constexpr int kStages = 2, kSide = kKeys * DP;     // bytes of a stage's keys
  static constexpr int kQuery = kStages * 2 * kSide / 4;

  static __device__ __forceinline__ void run(const DecodeParams& p, float* mine, const Part& w) {
    const int k1 = w.k1;
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const int d = p.c.head_dim;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(mine);
    __syncwarp();  // the last part's reads of it
    if (!kExact)
      for (int i = lane; i < kQuery / 4; i += 32) reinterpret_cast<uint4*>(mine)[i] = make_uint4(0u, 0u, 0u, 0u);  // dims from d on
    // A lane's pieces: copies (row and 16 bytes of it), operands of the products.
    constexpr int kPer = DP / 16;                                // pieces of a row
    const int row = lane / kPer, piece = lane % kPer;            // of the first copy; the other is 4 rows further
    const uint32_t to = ring + (DP == 128 ? row * 128 + (piece ^ row) * 16
                                          : (row >> 1) * 128 + (((row & 1) * 4 + piece) ^ (((row >> 1) & 3) * 2)) * 16);
    const uint32_t to4 = ring + (row + 4) * 128 + (piece ^ (row + 4)) * 16;  // DP 128
    const bool copies = kExact || piece * 16 < d;
    const int64_t from = (int64_t)row * p.c.slot_stride + piece * 16;
    const uint8_t *key_from = (const uint8_t*)p.c.k + from, *value_from = (const uint8_t*)p.c.v + from;
    const uint32_t key0 = ring + (DP == 128 ? r * 128 + ((2 * c) ^ r) * 16 : (r >> 1) * 128 + (((r & 1) * 4 + c) ^ (((r >> 1) & 3) * 2)) * 16);
    const uint32_t key1 = ring + r * 128 + ((2 * c + 1) ^ r) * 16;      // DP 128: the second 16 of its 32 dims
    const uint32_t val0 = ring + kSide + (DP == 128 ? 2 * c * 128 + (r ^ (2 * c)) * 16 : c * 128 + ((r >> 1) ^ (c * 2)) * 16 + (r & 1) * 8);
    const uint32_t val1 = ring + kSide + (DP == 128 ? (2 * c + 1) * 128 + (r ^ (2 * c + 1)) * 16 : c * 128 + ((4 + (r >> 1)) ^ (c * 2)) * 16 + (r & 1) * 8);

    float o[VW][2][4], m[2], mw[2], rate[2], l[2], factor[2];
    m[0] = m[1] = mw[0] = mw[1] = -INFINITY, rate[0] = rate[1] = 1.f, l[0] = l[1] = 0.f;
#pragma unroll
    for (int b = 0; b < VW; ++b)
#pragma unroll
      for (int i = 0; i < 8; ++i) o[b][i / 4][i % 4] = 0.f;
    // Rounds of 32 groups, one a lane: offsets (in 16 bytes) and scales of this one, offsets of the
    // next, of which groups are there, a bit each.
    using Keys = ScaledWalk<true, kKeys>;
    Keys walk(p, w.s, w.h, w.k0, k1);
    uint32_t valid, valid_next = __ballot_sync(0xffffffffu, walk.page1 >= 0), next = walk.next();
    auto turn = [&] {
      valid = valid_next;
      walk.turn();
      valid_next = __ballot_sync(0xffffffffu, walk.page1 >= 0), next = walk.next();
    };
    turn();
    __syncwarp();
    // Copies of the step whose first group is the j-th from the round's start.
    auto copy = [&](int j, uint32_t stage) {
      const uint32_t offs = j < 32 ? walk.off : next, there = (j < 32 ? valid : valid_next) >> (j & 31);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const uint32_t off = __shfl_sync(0xffffffffu, offs, (j + g) & 31);
        if (!((there >> g) & 1u) || !copies) continue;
        const uint8_t *key = key_from + (unsigned long long)off * 16, *value = value_from + (unsigned long long)off * 16;
        copy16(to + stage + g * 8 * DP, key), copy16(to + stage + g * 8 * DP + kSide, value);
        if constexpr (DP == 128) {
          copy16(to4 + stage + g * 8 * DP, key + 4 * p.c.slot_stride);
          copy16(to4 + stage + g * 8 * DP + kSide, value + 4 * p.c.slot_stride);
        }
      }
    };
    auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
    copy(0, 0), commit();
    int left = k1 - w.k0;  // keys
    if (left > kKeys) copy(kGroups, 2 * kSide);
    commit();
    // queries
    uint32_t q[KP][8];
    {
      const float up = Path::template query_registers<KP>(p, q, w);
      factor[0] = __shfl_sync(0xffffffffu, up, 8 * c);
      factor[1] = __shfl_sync(0xffffffffu, up, 8 * c + 4);
    }
    uint32_t stage = 0;
#pragma unroll 1
    for (int j = 0; left > 0; left -= kKeys, stage ^= 2 * kSide) {
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncwarp();
      uint4 kr[KG][2][KP];
      uint32_t vr[KG][4][VW];
#pragma unroll
      for (int g = 0; g < KG; ++g)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          constexpr int kGroup = 8 * DP;
          kr[g][u][0] = shared16(key0 + stage + (g * 2 + u) * kGroup);
          if (KP == 2) kr[g][u][KP - 1] = shared16(key1 + stage + (g * 2 + u) * kGroup);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if constexpr (VW == 4) {
              const uint4 v = shared16((x ? val1 : val0) + stage + (g * 2 + u) * kGroup);
              vr[g][2 * u + x][0] = v.x, vr[g][2 * u + x][1] = v.y, vr[g][2 * u + x][2] = v.z, vr[g][2 * u + x][3] = v.w;
            } else {
              const uint2 v = shared8((x ? val1 : val0) + stage + (g * 2 + u) * kGroup);
              vr[g][2 * u + x][0] = v.x, vr[g][2 * u + x][1] = v.y;
            }
          }
        }
      __syncwarp();
      if (left > 2 * kKeys) copy(j + 2 * kGroups, stage);
      commit();
      // the step's groups: scales, and which keys count
      float ks[KG][2], vs[KG][2], top = 0.f;
#pragma unroll
      for (int g = 0; g < KG; ++g)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (kSame && u == 1) {
            ks[g][1] = ks[g][0], vs[g][1] = vs[g][0];
          } else {
            ks[g][u] = __shfl_sync(0xffffffffu, walk.ks, j + 2 * g + u) * p.scale2, vs[g][u] = __shfl_sync(0xffffffffu, walk.vs, j + 2 * g + u);
            top = fmaxf(top, vs[g][u]);
          }
        }
      const bool whole = left >= kKeys && (valid >> j & ((1u << kGroups) - 1u)) == (1u << kGroups) - 1u;
      uint32_t there = 0xffffffffu;
      if (!whole) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
          if (!((valid >> (j + g)) & 1u)) there &= ~(0xffu << (8 * g));
        if (left < kKeys) there &= (1u << left) - 1u;
      }
      j += kGroups;
      if (j == 32) turn(), j = 0;
      // scores
      float z[KG][4];
#pragma unroll
      for (int g = 0; g < KG; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) z[g][i] = 0.f;
#pragma unroll
      for (int i = 0; i < KP; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int g = 0; g < KG; ++g) {
            uint32_t a0, a1, a2, a3;
            to_f16((&kr[g][0][i].x)[j], a0, a2);
            to_f16((&kr[g][1][i].x)[j], a1, a3);
            mma16816_f16(z[g], a0, a1, a2, a3, q[i][2 * j], q[i][2 * j + 1]);
          }
#pragma unroll
      for (int g = 0; g < KG; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (kFull) z[g][i] += __shfl_xor_sync(0xffffffffu, z[g][i], 2);
          z[g][i] *= factor[i & 1] * ks[g][i >> 1];
        }
      if (__builtin_expect(!whole, 0)) {
#pragma unroll
        for (int g = 0; g < KG; ++g) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!((there >> (g * 16 + (i >> 1) * 8 + r)) & 1u)) z[g][i] = -INFINITY;
#pragma unroll
          for (int u = 0; u < 4; ++u)  // what such a slot holds may be NaN
            if (!((there >> (g * 16 + (u >> 1) * 8 + 2 * c + (u & 1))) & 1u))
#pragma unroll
              for (int b = 0; b < VW; ++b) vr[g][u][b] = 0u;
        }
      }
      // softmax: as above
      bool move = false;
      const float above = log2_above(top);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float most = fminf(m[e], mw[e] - above) + 15.f;
#pragma unroll
        for (int g = 0; g < KG; ++g) move |= fmaxf(z[g][e], z[g][e + 2]) > most;
      }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float best = -INFINITY, best_w = -INFINITY;
#pragma unroll
          for (int g = 0; g < KG; ++g) {
            best = fmaxf(best, fmaxf(z[g][e], z[g][e + 2]));
            best_w = fmaxf(best_w, fmaxf(z[g][e] + log2_above(vs[g][0]), z[g][e + 2] + log2_above(vs[g][1])));
          }
          Path::move(best, best_w, m[e], mw[e], rate[e], l[e], o, e);
        }
      }
      const float m0 = fmaxf(m[0], -0x1.fffffep127f), m1 = fmaxf(m[1], -0x1.fffffep127f);
#pragma unroll
      for (int g = 0; g < KG; ++g) {
        float p0 = exp2_fast(z[g][0] - m0), p1 = exp2_fast(z[g][1] - m1);
        float p2 = exp2_fast(z[g][2] - m0), p3 = exp2_fast(z[g][3] - m1);
        l[0] += p0 + p2, l[1] += p1 + p3;
        p0 *= Path::bring(vs[g][0], rate[0]), p1 *= Path::bring(vs[g][0], rate[1]);
        p2 *= Path::bring(vs[g][1], rate[0]), p3 *= Path::bring(vs[g][1], rate[1]);
        const uint32_t ha = pack2_f16(p0, p1), hb = pack2_f16(p2, p3);
        const uint32_t la = rest2_f16(p0, p1, ha), lb = rest2_f16(p2, p3, hb);
        const uint32_t h0 = transpose8(c < 2 ? ha : la), h1 = transpose8(c < 2 ? hb : lb);
#pragma unroll
        for (int b = 0; b < VW; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t a0, a1, a2, a3;
            to_f16(__byte_perm(vr[g][0][b], vr[g][1][b], i ? 0x7362 : 0x5140), a0, a1);
            to_f16(__byte_perm(vr[g][2][b], vr[g][3][b], i ? 0x7362 : 0x5140), a2, a3);
            mma16816_f16(o[b][i], a0, a1, a2, a3, h0, h1);
          }
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int qh = 2 * c + e;
      float total = l[e];
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) total += __shfl_xor_sync(0xffffffffu, total, x);
      float y[VW][4];
#pragma unroll
      for (int b = 0; b < VW; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[b][i] = o[b][i >> 1][e + 2 * (i & 1)];
          y[b][i] += __shfl_xor_sync(0xffffffffu, y[b][i], 2);
          y[b][i] *= power2_inverse(rate[e]);
        }
      Path::finish(p, w, qh, m[e], total, y);
    }
  }
};

template <typename T, int N, int DP>
int launch_fp8(const DecodeParams& p, const Plan& pl, cudaStream_t st) {
  if (!pl.fast) return launch<Fp8Path<T, N, DP, false, false>>(p, pl, st);
  if constexpr (N == 4) {
    if (p.c.head_dim != DP) return launch<Fp8Ring<T, DP, false, false>>(p, pl, st);
    return p.c.page_size % 16 == 0 ? launch<Fp8Ring<T, DP, true, true>>(p, pl, st) : launch<Fp8Ring<T, DP, true, false>>(p, pl, st);
  }
  else return pl.exact ? launch<Fp8Path<T, N, DP, true, true>>(p, pl, st) : launch<Fp8Path<T, N, DP, true, false>>(p, pl, st);
}

}  // namespace
}  // namespace pgs
