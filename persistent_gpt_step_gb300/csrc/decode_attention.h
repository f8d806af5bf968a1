// decode_attention.h — what the host side of gpt_decode_attention and its kernels
// share; the kernels are compiled by type and head size, a translation unit each.
#pragma once
#include "decode_ops.h"

namespace pgs {

constexpr int kWarps = 8;      // of a block
constexpr int kTile = 16;      // keys of a unit of work
// What the start of a row costs a warp, in tiles (the first loads' latencies and the
// row's end): without it warps with many short rows end last.  In tables of 8,192
// positions, 200 sequences of 1 to 512 keys, 8 heads of 128 in fp32: 75.1 us with 0, 73.3
// with 1, 73.2 with 2, 74.3 with 4, 75.6 with 8; 256 of 1 to 256 keys, 8 over 4 heads of
// 128 in bf16: 27.5, 24.1, 24.5, 25.9, 27.1; 16 of 500 to 4,000, 32 over 4 heads of 128 in
// fp32: 43.6, 41.4, 39.3, 39.6, 39.3.
constexpr int kStart = 2;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct Meta { int32_t seq, row, last, pad; };  // a row begun in this block and ended in block `last`

struct DecodeParams {
  gpt_paged_cache c;
  gpt_decode_attention_args a;
  int32_t group;     // query heads per key head
  int32_t chunk;     // query heads of a row
  int32_t chunks;    // rows of one key head
  int32_t team;      // warps that take the same keys, a key head each
  int32_t pack;      // rows of a block (decode_row_kernel)
  int32_t rows;      // rows (of `team` key heads) of one sequence
  int32_t join_heads;  // query heads of a block of the second kernel, 1 to 8
  uint32_t page16, slot16, head16;  // the cache's strides in 16 bytes (fast forms)
  float scale2;      // scale log2 e
  Meta* meta;        // [blocks]
  float *piece_ml, *piece_o;  // [blocks][2][team chunk][2], [...][head_dim]
};

struct Plan {
  int blocks;          // of the line's grid
  int chunk, chunks;   // query heads of a row, rows of a key head
  int team;            // warps that take the same keys
  int cluster, pack;   // decode_row_kernel: blocks of a row, rows of a block (one is 1); 0: the line
  int join_heads;      // query heads of a block of the second kernel
  bool fast;           // pages of whole 8-key groups, offsets in 16 bytes within 32 bits
  bool exact;          // fast, heads of 64 or 128, keys on 32-byte boundaries
  size_t ml_at, o_at, bytes;  // the workspace: pieces' (m, l), their o, its size
};

// Launches for head sizes up to 64 and 128.
int decode_bf16_64(const DecodeParams& p, const Plan& pl, cudaStream_t st);
int decode_bf16_128(const DecodeParams& p, const Plan& pl, cudaStream_t st);
int decode_fp32_64(const DecodeParams& p, const Plan& pl, cudaStream_t st);
int decode_fp32_128(const DecodeParams& p, const Plan& pl, cudaStream_t st);

}  // namespace pgs
