// decode_attention.cu — gpt_decode_attention and gpt_decode_attention_fp8: argument
// checks, the choice of a kernel and its grid, the workspace.
#include <algorithm>
#include <cmath>

#include "decode_attention.h"

namespace pgs {
namespace {

int check_heads(const gpt_paged_cache* c, int32_t n_head) {
  if (n_head < 1 || n_head % c->n_kv_head)
    return call_error(GPT_ERR_INVALID_ARG, "n_head %d must be a multiple of n_kv_head %d", n_head, c->n_kv_head);
  if (n_head > kMostHeads) return call_error(GPT_ERR_UNSUPPORTED, "n_head %d: at most %d", n_head, kMostHeads);
  return GPT_OK;
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 152;
  }
  return sms;
}

// Blocks of the grid, query heads of a row, and the workspace; es: bytes of an element of
// the cache.
Plan make_plan(const gpt_paged_cache* c, int32_t n_head, int es) {
  Plan pl;
  const int group = n_head / c->n_kv_head;
  pl.chunk = group <= 8 ? group : c->dtype == GPT_DTYPE_BF16 ? (group < 16 ? group : 16) : 8;
  pl.chunks = (group + pl.chunk - 1) / pl.chunk;
  pl.blocks = sm_count() * (pl.chunk > (c->dtype == GPT_DTYPE_BF16 || es == 1 ? 8 : 4) ? 1 : 2);  // as the kernels' kBlocks
  const double span = ((double)(c->n_pages - 1) * c->page_stride + (double)(c->page_size - 1) * c->slot_stride +
                       (double)(c->n_kv_head - 1) * c->head_stride + c->head_dim) * es;
  pl.fast = c->page_size % 8 == 0 && span < 16.0 * 0xffffffffu;
  pl.exact = pl.fast && c->head_dim % 64 == 0 && reinterpret_cast<uintptr_t>(c->k) % 32 == 0 && c->page_stride * es % 32 == 0 &&
             c->slot_stride * es % 32 == 0 && c->head_stride * es % 32 == 0;
  // Teams: warps that read the same keys' neighbouring heads keep DRAM pages open
  // where a head's row is short (200 sequences of 16 heads of 64: 86 us with teams of
  // 1, 81 with 4, 82 with 8); but a row of a team is cut into that many more pieces
  // (one sequence of 131,071 keys and 8 heads: 93 us with 1, 98 with 2, 105 with 4).
  // So: up to 4, as long as a row does not have more than 16 pieces.
  const int64_t tiles = ((int64_t)c->max_pages * c->page_size + kTile - 1) / kTile, rows = (int64_t)c->n_kv_head * pl.chunks * c->n_seq;
  const int64_t used = std::min<int64_t>(pl.blocks, (rows * (tiles + kStart) + kWarps - 1) / kWarps);
  pl.team = 1;
  while (pl.team < 4 && c->n_kv_head % (2 * pl.team) == 0 && used * 2 * pl.team <= 16 * rows) pl.team *= 2;
  // Rows of few tiles a warp take decode_row_kernel: no line to look up, no second
  // kernel.  Up to a block per row at once: a cluster of blocks for each (one sequence
  // of 513 keys, 12 heads of 64 in fp32 6.8 us, the line and its join 9.8; 4,096 keys
  // of 8 heads of 128 11.8 and 19.4; 304 rows of 2,048 keys of 64 33 and 38), but a few
  // rows in clusters of 8 leave half the GPU idle (16,000 keys of 8 heads of 128 33.7
  // and 25.0).  More rows: as many to a block as all run at once, down to a warp for a
  // row (768 rows of 512 keys of 64 25.1 and 29.8, 2,400 of 128 20.4 and 29.2), then in
  // several waves (8,192 rows of 1 to 128 44 and 53).  With more tiles a warp the spread
  // of lengths weighs more than the line's few us (768 rows of 1 to 1,024 36 and 31),
  // with longer rows of keys earlier (heads of 128: 768 rows of 1 to 512 34 and 30).
  pl.cluster = 0, pl.pack = 1;
  const int deep = c->head_dim * es <= 128 ? 16 : 12;
  if (rows <= pl.blocks) {
    const int64_t most = std::min<int64_t>(8, pl.blocks / rows);
    if (tiles <= (most == 8 && 16 * rows < pl.blocks ? 8 : deep) * most * kWarps) pl.cluster = (int)std::min<int64_t>(most, (tiles + kWarps - 1) / kWarps);
  } else {
    while (pl.pack < kWarps && (rows + pl.pack - 1) / pl.pack > pl.blocks) pl.pack = pl.pack == 4 ? kWarps : pl.pack + 1;
    const bool waves = (rows + pl.pack - 1) / pl.pack > pl.blocks;
    if (rows <= (1 << 28) && tiles <= (waves && deep == 12 ? 8 : deep) * (kWarps / pl.pack)) pl.cluster = 1;
  }
  if (pl.cluster) {
    pl.team = pl.join_heads = 1, pl.bytes = 0;
    return pl;
  }
  // Pieces of a row, about: the more, the fewer heads for a block of the second kernel.
  const int64_t pieces = used * pl.team / rows;
  pl.join_heads = pieces > 32 ? 1 : pieces > 16 ? 2 : pieces > 8 ? 4 : 8;
  const size_t records = (size_t)pl.blocks * 2 * pl.team * pl.chunk;
  pl.ml_at = (pl.blocks * sizeof(Meta) + 15) / 16 * 16;
  pl.o_at = (pl.ml_at + records * 8 + 15) / 16 * 16;
  pl.bytes = pl.o_at + records * c->head_dim * 4;
  return pl;
}

// Both entries: over a cache of dtype's elements, or over one in 8 bits with these scales.
int attend(const gpt_paged_cache* c, const gpt_fp8_cache* scales, const gpt_decode_attention_args* a, cudaStream_t st) {
  if (const int rc = check_heads(c, a->n_head)) return rc;
  if (c->n_seq == 0) return GPT_OK;
  const int es = elem_size(c->dtype), cache_es = scales ? 1 : es;
  if (!a->q || !a->out || !a->lens) return call_error(GPT_ERR_INVALID_ARG, "q, out and lens must be non-NULL");
  if (!aligned16(a->q) || !aligned16(a->out) || !stride16(a->q_row, es) || !stride16(a->q_head, es) ||
      !stride16(a->out_row, es) || !stride16(a->out_head, es))
    return call_error(GPT_ERR_INVALID_ARG, "q and out addresses and strides must be multiples of 16 bytes");
  if (a->out == a->q) return call_error(GPT_ERR_INVALID_ARG, "out must not be q");
  if (!apart({{a->out_row, c->n_seq}, {a->out_head, a->n_head}}, c->head_dim))
    return call_error(GPT_ERR_INVALID_ARG, "strides of out are smaller than a head or the dimension inside");
  if (!std::isfinite(a->scale * kLog2e)) return call_error(GPT_ERR_INVALID_ARG, "scale must be finite");
  const Plan pl = make_plan(c, a->n_head, cache_es);
  if (pl.bytes && (!a->workspace || a->workspace_bytes < pl.bytes || !aligned16(a->workspace)))
    return call_error(GPT_ERR_INVALID_ARG, "workspace: %zu bytes on a 16-byte boundary", pl.bytes);
  DecodeParams p = {};
  p.c = *c;
  p.a = *a;
  p.group = a->n_head / c->n_kv_head;
  p.chunk = pl.chunk, p.chunks = pl.chunks, p.team = pl.team, p.pack = pl.pack, p.join_heads = pl.join_heads;
  p.rows = c->n_kv_head / pl.team * pl.chunks;
  if (scales) p.k_scale = scales->k_scale, p.v_scale = scales->v_scale, p.scale_page = scales->scale_page, p.scale_head = scales->scale_head;
  if (pl.fast) {
    p.page16 = (uint32_t)(c->page_stride * cache_es / 16), p.slot16 = (uint32_t)(c->slot_stride * cache_es / 16);
    p.head16 = (uint32_t)(c->head_stride * cache_es / 16);
  }
  p.scale2 = a->scale * kLog2e;
  p.meta = (Meta*)a->workspace;
  p.piece_ml = (float*)((char*)a->workspace + pl.ml_at);
  p.piece_o = (float*)((char*)a->workspace + pl.o_at);
  const bool wide = c->head_dim > 64, bf16 = c->dtype == GPT_DTYPE_BF16;
  if (scales && bf16) return wide ? decode_fp8_bf16_128(p, pl, st) : decode_fp8_bf16_64(p, pl, st);
  if (scales) return wide ? decode_fp8_fp32_128(p, pl, st) : decode_fp8_fp32_64(p, pl, st);
  if (bf16) return wide ? decode_bf16_128(p, pl, st) : decode_bf16_64(p, pl, st);
  return wide ? decode_fp32_128(p, pl, st) : decode_fp32_64(p, pl, st);
}

}  // namespace
}  // namespace pgs

using namespace pgs;

extern "C" size_t gpt_decode_attention_workspace(const gpt_paged_cache* c, int32_t n_head) {
  clear_call_error();
  if (check_cache(c) != GPT_OK || check_heads(c, n_head) != GPT_OK || c->n_seq == 0) return 0;
  return make_plan(c, n_head, elem_size(c->dtype)).bytes;
}

extern "C" int gpt_decode_attention(const gpt_paged_cache* c, const gpt_decode_attention_args* a, void* cuda_stream) {
  clear_call_error();
  if (!a) return call_error(GPT_ERR_INVALID_ARG, "args must be non-NULL");
  if (const int rc = check_cache(c)) return rc;
  return attend(c, nullptr, a, (cudaStream_t)cuda_stream);
}

extern "C" size_t gpt_decode_attention_fp8_workspace(const gpt_fp8_cache* c, int32_t n_head) {
  clear_call_error();
  if (check_cache(c, false) != GPT_OK || check_heads(&c->pages, n_head) != GPT_OK || c->pages.n_seq == 0) return 0;
  return make_plan(&c->pages, n_head, 1).bytes;
}

extern "C" int gpt_decode_attention_fp8(const gpt_fp8_cache* c, const gpt_decode_attention_args* a, void* cuda_stream) {
  clear_call_error();
  if (!a) return call_error(GPT_ERR_INVALID_ARG, "args must be non-NULL");
  if (const int rc = check_cache(c, false)) return rc;
  return attend(&c->pages, c, a, (cudaStream_t)cuda_stream);
}
