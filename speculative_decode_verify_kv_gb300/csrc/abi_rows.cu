// abi_rows.cu -- the C ABI's packed-row calls (include/trtv.h): staging with
// norm and rotation, prompt attention, tree attention and tree commit.  Host
// code only: argument checks and launches; nothing is allocated, synchronised
// or read from the device, so every call can be captured into a CUDA graph.
#include <algorithm>
#include <cmath>

#include "host.h"
#include "launch.h"
#include "rows.cuh"

namespace trtv {
namespace {

constexpr int kMaxBatch = 2048;   // the requests' scan lies in shared memory
constexpr int kMaxTreeTokens = 128;
constexpr int kMaxHeads = 65536;  // a token's row is indexed by 32 bits
constexpr float kMinScale = 5.421011e-20f;  // 2^-64
// stream-K charge of an item in positions, what switching items costs (us).
// 256-row items, at 128 / 256 / 384 / 512: 8 prompts of up to 4000 tokens 501 / 460 /
// 461 / 471, of head_dim 64 394 / 373 / 382 / 391, one of 16384 of head_dim 64 1167 /
// 1142 / 1148 / 1155.  E4M3, at 256 / 384 / 512 / 640: 8 prompts 699 / 624 / 601 / 612,
// one of 16384 1783 / 1671 / 1625 / 1633, 4 chunks over 2-12 k positions 146.4 / 143.7 /
// 142.1 / 142.5.  One tile, at 64 / 128 / 256: 64 trees of 16 nodes 113.2 / 110.5 /
// 109.8 (head_dim 64 74.6 / 73.0 / 69.6), but little work is cut best at 128: one tree
// of 8 over 900 positions 14.0 / 13.4 / 15.0 (head_dim 64 12.1 / 11.1 / 12.5), three over
// 700-1500 17.0 / 15.6 / 16.1.  E4M3, at 64 / 128 / 256 / 384: 64 trees 113.1 / 110.8 /
// 105.8 / 100.7, one over 700 14.4 / 14.5 / 15.0 / 14.4, one over 16000 30.0 at each.
constexpr int kRowsSetupTwo = 256, kRowsSetupTwoFp8 = 512, kRowsSetupOne = 128, kRowsSetupOneFp8 = 256;

// Geometry checks shared by the packed-row calls.
trtv_status rows_geom(const trtv_geom* g, const int32_t* indptr, int32_t num_tokens, RowsGeom* r) {
  if (g == nullptr) return TRTV_ERR_INVALID_ARG;
  if (g->batch < 1 || g->qo_len < 1 || g->num_q_heads < 1 || g->num_kv_heads < 1 ||
      g->num_q_heads % g->num_kv_heads != 0 || g->max_pages_per_req < 1 || g->num_slots < 1 || g->slot_stride < 2 ||
      g->num_ctas < 0 || g->num_ctas > kMaxCombineParts)
    return TRTV_ERR_INVALID_ARG;
  if (g->kv_dtype != TRTV_BF16 && g->kv_dtype != TRTV_FP8_E4M3) return TRTV_ERR_INVALID_ARG;
  if (!(g->sm_scale > 0.f) || !(g->k_scale > 0.f) || !std::isfinite(g->sm_scale) || !std::isfinite(g->k_scale) ||
      !std::isfinite(g->v_scale))
    return TRTV_ERR_INVALID_ARG;
  // (a scale that vanishes in binary32 would turn a masked score of minus infinity into NaN)
  if (!(g->sm_scale * g->k_scale >= kMinScale) || !std::isfinite(g->sm_scale * g->k_scale)) return TRTV_ERR_INVALID_ARG;
  if (g->head_dim != 64 && g->head_dim != 128) return TRTV_ERR_UNSUPPORTED;
  if (g->kv_dtype == TRTV_FP8_E4M3 && g->head_dim != 128) return TRTV_ERR_UNSUPPORTED;
  if (g->batch > kMaxBatch || g->num_q_heads > kMaxHeads || g->num_q_heads / g->num_kv_heads > 128)
    return TRTV_ERR_UNSUPPORTED;
  // cache positions are 32-bit, and the pool is addressed by 32-bit rows
  if (g->max_pages_per_req > (1 << 23)) return TRTV_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(g->num_slots) * g->slot_stride * kGroups * g->num_kv_heads * kSub >= (int64_t{1} << 31))
    return TRTV_ERR_UNSUPPORTED;
  if (num_tokens < 0) return TRTV_ERR_INVALID_ARG;
  if (indptr == nullptr && static_cast<int64_t>(g->batch) * g->qo_len > num_tokens) return TRTV_ERR_INVALID_ARG;
  if (!aligned(indptr, 4)) return TRTV_ERR_INVALID_ARG;
  r->indptr = indptr;
  r->batch = g->batch;
  r->qo_len = g->qo_len;
  r->num_tokens = num_tokens;
  r->num_q_heads = g->num_q_heads;
  r->num_kv_heads = g->num_kv_heads;
  r->group = g->num_q_heads / g->num_kv_heads;
  r->max_pages = g->max_pages_per_req;
  r->num_slots = g->num_slots;
  r->slot_stride = g->slot_stride;
  return TRTV_OK;
}

trtv_status rows_device(RowsGeom* r, const int32_t* page_table, const int32_t* kv_lens) {
  if (page_table == nullptr || kv_lens == nullptr || !aligned(page_table, 4) || !aligned(kv_lens, 4))
    return TRTV_ERR_INVALID_ARG;
  r->page_table = page_table;
  r->kv_lens = kv_lens;
  r->err = err_word();
  return r->err == nullptr ? TRTV_ERR_CUDA : TRTV_OK;
}

// What one attention call needs besides its pointers.
struct RowsPlan {
  bool two;            // 256-row items
  int num_ctas;
  size_t ws_o, ws_lse, ws_splits, ws_cont, ws_total;
};

// 256-row items where a request can fill more than one 128-row tile: its tiles
// share each page's bytes and the two softmax groups have a tile each.
// Otherwise the groups take a tile's pages in turn.
bool rows_plan(const trtv_geom* g, const RowsGeom& r, RowsPlan* pl) {
  const int tile_toks = kRowsTile / r.group;
  pl->two = g->qo_len > tile_toks;
  pl->num_ctas = g->num_ctas > 0 ? g->num_ctas : sm_count();
  if (pl->num_ctas <= 0) return false;
  const size_t rows = pl->two ? 2 * kRowsTile : kRowsTile, pieces = 2 * static_cast<size_t>(pl->num_ctas);
  size_t off = 0;
  pl->ws_o = off;
  off = align_up(off + pieces * rows * g->head_dim * sizeof(float), 256);
  pl->ws_lse = off;
  off = align_up(off + pieces * rows * sizeof(float), 256);
  pl->ws_splits = off;
  off = align_up(off + pl->num_ctas * sizeof(RowsSplit), 256);
  pl->ws_cont = off;
  off = align_up(off + pl->num_ctas * sizeof(int), 256);
  pl->ws_total = off;
  return true;
}

// Shared memory: Q (one or two tiles), the page ring, E4M3: the codes' ring, the
// groups' exchange, the pieces, the requests' scan and its 32 warp totals,
// barriers.  The ring takes what is left, at most kMaxStages pages.
constexpr int kMaxStages = 8;
bool rows_smem(const trtv_geom* g, const RowsPlan& pl, RowsAttnParams* p, size_t* bytes) {
  const bool fp8 = g->kv_dtype == TRTV_FP8_E4M3;
  const size_t tile = static_cast<size_t>(kRowsTile) * g->head_dim * 2, raw = static_cast<size_t>(kRowsTile) * g->head_dim;
  const size_t scan = align_up((static_cast<size_t>(g->batch) + 1 + 32) * sizeof(int64_t), 16);
  const size_t ml = pl.two ? 0 : 2 * kRowsTile * 2 * sizeof(float);
  const size_t bars = (4 * kMaxStages + 32) * sizeof(uint64_t), pieces = 4 * 48;
  const size_t q = (pl.two ? 2 : 1) * tile;
  const size_t fixed = q + ml + pieces + scan + bars + kAlignSlack;
  if (fp8) {
    // four converted tiles and three stages of codes where they fit (one-tile
    // items, 64 trees of 16 nodes: 7 % faster than three and five), else three;
    // what is left holds codes in flight
    if (fixed + 2 * raw + 3 * tile > kSmemOptin) return false;
    p->nst = fixed + 3 * raw + 4 * tile <= kSmemOptin ? 4 : 3;
    p->nraw = static_cast<int>(std::min<size_t>((kSmemOptin - fixed - p->nst * tile) / raw, kMaxStages));
  } else {
    if (fixed + 3 * tile > kSmemOptin) return false;
    p->nst = static_cast<int>(std::min<size_t>((kSmemOptin - fixed) / tile, kMaxStages));
    p->nraw = 0;
  }
  const size_t codes = p->nraw * raw;
  size_t off = 0;
  p->off_q = 0;
  off += q;
  p->off_ring = static_cast<int>(off);
  off += p->nst * tile;
  p->off_raw = static_cast<int>(off);
  off += codes;
  p->off_ml = static_cast<int>(off);
  off += ml;
  p->off_pieces = static_cast<int>(off);
  off += pieces;
  p->off_scan = static_cast<int>(off);
  off += scan;
  p->off_bar = static_cast<int>(off);
  off += bars;
  *bytes = off + kAlignSlack;
  return true;
}

// The pool as [sub-pages][KV heads][32 rows][head_dim]: a box is one head's
// 128-byte column block of a whole page.
bool encode_pages(const trtv_geom* g, const void* pool, CUtensorMap* map) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
  if (enc == nullptr) return false;
  const bool fp8 = g->kv_dtype == TRTV_FP8_E4M3;
  const cuuint64_t elem = fp8 ? 1 : 2, D = g->head_dim, Hk = g->num_kv_heads;
  cuuint64_t dims[4] = {D, kSub, Hk, static_cast<cuuint64_t>(g->num_slots) * g->slot_stride * kGroups};
  cuuint64_t strides[3] = {D * elem, kSub * D * elem, Hk * kSub * D * elem};
  cuuint32_t box[4] = {static_cast<cuuint32_t>(128 / elem), kSub, 1, kGroups}, estr[4] = {1, 1, 1, 1};
  return enc(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(pool),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// q as [rows][query heads][head_dim]: a box is one tile's 64-column block (its
// tokens' heads of one group).
bool encode_rows(const trtv_geom* g, const RowsGeom& r, int tile_toks, const void* q, CUtensorMap* map) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
  if (enc == nullptr) return false;
  const cuuint64_t D = g->head_dim, Hq = g->num_q_heads;
  cuuint64_t dims[3] = {D, Hq, static_cast<cuuint64_t>(r.num_tokens)}, strides[2] = {D * 2, Hq * D * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(r.group), static_cast<cuuint32_t>(tile_toks)}, estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

trtv_status rows_attn(const trtv_geom* g, const void* q, const void* pool, const int32_t* page_table,
                      const int32_t* kv_lens, const int32_t* indptr, int32_t num_tokens, const uint32_t* mask,
                      void* out, int32_t out_dtype, void* ws, size_t ws_bytes, void* stream) {
  RowsAttnParams p{};
  trtv_status s = rows_geom(g, indptr, num_tokens, &p.g);
  if (s != TRTV_OK || num_tokens == 0) return s;
  if (q == nullptr || pool == nullptr || out == nullptr) return TRTV_ERR_INVALID_ARG;
  if (out_dtype != TRTV_BF16 && out_dtype != TRTV_F32) return TRTV_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(pool, 16) || !aligned(out, 16) || !aligned(mask, 4)) return TRTV_ERR_INVALID_ARG;
  if (page_table == nullptr || kv_lens == nullptr || !aligned(page_table, 4) || !aligned(kv_lens, 4))
    return TRTV_ERR_INVALID_ARG;
  RowsPlan pl;
  if (!rows_plan(g, p.g, &pl)) return TRTV_ERR_CUDA;
  if (ws == nullptr || !aligned(ws, 256) || ws_bytes < pl.ws_total) return TRTV_ERR_WORKSPACE;
  size_t smem = 0;
  if (!rows_smem(g, pl, &p, &smem)) return TRTV_ERR_UNSUPPORTED;
  if ((s = rows_device(&p.g, page_table, kv_lens)) != TRTV_OK) return s;
  p.tile_toks = kRowsTile / p.g.group;
  p.items = mask != nullptr && pl.two ? (g->qo_len + 2 * p.tile_toks - 1) / (2 * p.tile_toks) : 1;
  if (p.items > pl.num_ctas) p.items = 1;
  CUtensorMap kv_map, q_map;
  if (!encode_pages(g, pool, &kv_map) || !encode_rows(g, p.g, p.tile_toks, q, &q_map)) return TRTV_ERR_CUDA;
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  p.tree_mask = mask;
  p.mask_words = (g->qo_len + 31) / 32;
  p.out = out;
  p.ws_o = reinterpret_cast<float*>(wsb + pl.ws_o);
  p.ws_lse = reinterpret_cast<float*>(wsb + pl.ws_lse);
  p.splits = reinterpret_cast<RowsSplit*>(wsb + pl.ws_splits);
  p.cont = reinterpret_cast<int*>(wsb + pl.ws_cont);
  p.out_f32 = out_dtype == TRTV_F32;
  p.num_ctas = pl.num_ctas;
  const bool fp8 = g->kv_dtype == TRTV_FP8_E4M3;
  p.setup = pl.two ? (fp8 ? kRowsSetupTwoFp8 : kRowsSetupTwo) : fp8 ? kRowsSetupOneFp8 : kRowsSetupOne;
  p.scale_log2 = g->sm_scale * g->k_scale * 1.4426950408889634f;
  p.v_scale = g->v_scale;
  p.wait_ns = wait_limit_ns();
  p.withhold = withheld_pages();
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = fp8 ? launch_rows_attn_fp8(pl.two, kv_map, q_map, p, smem, st)
                      : launch_rows_attn_bf16(g->head_dim, pl.two, kv_map, q_map, p, smem, st);
  if (e == cudaSuccess) e = launch_rows_join(g->head_dim, pl.two, p, st);
  return e == cudaSuccess ? TRTV_OK : TRTV_ERR_CUDA;
}

}  // namespace
}  // namespace trtv

using namespace trtv;

extern "C" {

trtv_status trtv_norm_rope_stage(const trtv_geom* g, const trtv_norm_rope* in, const int32_t* qo_indptr,
                                 int32_t num_tokens, void* q_out, void* kv_pool, const int32_t* page_table,
                                 const int32_t* kv_lens, void* stream) {
  NormRopeParams p{};
  trtv_status s = rows_geom(g, qo_indptr, num_tokens, &p.g);
  if (s != TRTV_OK || num_tokens == 0) return s;
  if (in == nullptr || in->q == nullptr || in->k == nullptr || in->v == nullptr || q_out == nullptr ||
      kv_pool == nullptr)
    return TRTV_ERR_INVALID_ARG;
  const int D = g->head_dim;
  const int64_t qw = static_cast<int64_t>(g->num_q_heads) * D, kw = static_cast<int64_t>(g->num_kv_heads) * D;
  if (in->q_stride < qw || in->k_stride < kw || in->v_stride < kw || in->q_stride % 8 || in->k_stride % 8 ||
      in->v_stride % 8)
    return TRTV_ERR_INVALID_ARG;
  if (in->rot_dim < 0 || in->rot_dim > D || in->rot_dim % 8 != 0 || (in->interleaved != 0 && in->interleaved != 1) ||
      !(in->eps >= 0.f) || !std::isfinite(in->eps))
    return TRTV_ERR_INVALID_ARG;
  if (in->rot_dim > 0 && (in->rope_table == nullptr || in->table_len < 1)) return TRTV_ERR_INVALID_ARG;
  if (in->q == q_out && in->q_stride != qw) return TRTV_ERR_INVALID_ARG;
  if (g->kv_dtype == TRTV_FP8_E4M3 && g->v_scale == 0.f) return TRTV_ERR_INVALID_ARG;   // values are divided by it
  const void* ptrs[] = {in->q, in->k, in->v, in->q_weight, in->k_weight, in->rope_table, q_out, kv_pool};
  for (const void* x : ptrs)
    if (!aligned(x, 16)) return TRTV_ERR_INVALID_ARG;
  if (!aligned(in->positions, 4)) return TRTV_ERR_INVALID_ARG;
  const int heads = g->num_q_heads + 2 * g->num_kv_heads;
  if (static_cast<int64_t>(num_tokens) * heads >= (int64_t{1} << 33)) return TRTV_ERR_UNSUPPORTED;  // grid size
  if ((s = rows_device(&p.g, page_table, kv_lens)) != TRTV_OK) return s;
  p.q = static_cast<const __nv_bfloat16*>(in->q);
  p.k = static_cast<const __nv_bfloat16*>(in->k);
  p.v = static_cast<const __nv_bfloat16*>(in->v);
  p.q_stride = in->q_stride;
  p.k_stride = in->k_stride;
  p.v_stride = in->v_stride;
  p.q_weight = static_cast<const __nv_bfloat16*>(in->q_weight);
  p.k_weight = static_cast<const __nv_bfloat16*>(in->k_weight);
  p.rope = in->rope_table;
  p.positions = in->positions;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.pool = kv_pool;
  p.table_len = in->table_len;
  p.rot_dim = in->rot_dim;
  p.interleaved = in->interleaved;
  p.eps = in->eps;
  p.k_scale = g->k_scale;
  p.v_scale = g->v_scale;
  // A warp takes all of a token's heads where there are tokens enough for 16
  // warps an SM; fewer tokens are spread over more warps, down to one batch of
  // rows each (256 tokens of 40 heads: 24.3 us by itself against 27.1).
  const int sms = sm_count();
  if (sms <= 0) return TRTV_ERR_CUDA;
  const int batch_rows = 512 / D;
  const int64_t want = (16 * static_cast<int64_t>(sms) + num_tokens - 1) / num_tokens;
  const int chunks = static_cast<int>(std::min<int64_t>(want, (heads + batch_rows - 1) / batch_rows));
  p.heads_per_warp = ((heads + chunks - 1) / chunks + batch_rows - 1) / batch_rows * batch_rows;
  p.chunks = (heads + p.heads_per_warp - 1) / p.heads_per_warp;
  const cudaError_t e = launch_norm_rope_stage(D, g->kv_dtype == TRTV_FP8_E4M3, p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? TRTV_OK : TRTV_ERR_CUDA;
}

size_t trtv_workspace_bytes_rows(const trtv_geom* geom) {
  RowsGeom r{};
  RowsPlan pl;
  RowsAttnParams p{};
  size_t smem = 0;
  const int32_t any = 0;  // (rows are not checked: a host pointer that nothing reads)
  if (rows_geom(geom, &any, 0, &r) != TRTV_OK || !rows_plan(geom, r, &pl) || !rows_smem(geom, pl, &p, &smem)) return 0;
  return pl.ws_total;
}

trtv_status trtv_prompt_attn(const trtv_geom* g, const void* q, const void* kv_pool, const int32_t* page_table,
                             const int32_t* kv_lens, const int32_t* qo_indptr, int32_t num_tokens, void* out,
                             int32_t out_dtype, void* workspace, size_t ws_bytes, void* stream) {
  return rows_attn(g, q, kv_pool, page_table, kv_lens, qo_indptr, num_tokens, nullptr, out, out_dtype, workspace,
                   ws_bytes, stream);
}

trtv_status trtv_verify_tree(const trtv_geom* g, const void* q, const void* kv_pool, const int32_t* page_table,
                             const int32_t* kv_lens, const int32_t* qo_indptr, int32_t num_tokens,
                             const uint32_t* tree_mask, void* out, int32_t out_dtype, void* workspace,
                             size_t ws_bytes, void* stream) {
  if (tree_mask == nullptr && num_tokens != 0) return TRTV_ERR_INVALID_ARG;
  if (g != nullptr && g->qo_len > kMaxTreeTokens) return TRTV_ERR_UNSUPPORTED;
  return rows_attn(g, q, kv_pool, page_table, kv_lens, qo_indptr, num_tokens, tree_mask, out, out_dtype, workspace,
                   ws_bytes, stream);
}

trtv_status trtv_tree_commit(const trtv_geom* g, void* kv_pool, const int32_t* page_table, const int32_t* kv_lens,
                             const int32_t* qo_indptr, const int32_t* path, const int32_t* path_len,
                             int32_t max_path, int32_t* new_kv_lens, void* stream) {
  CommitParams p{};
  trtv_status s = rows_geom(g, qo_indptr, 0x7fffffff, &p.g);  // no row-indexed buffer here
  if (s != TRTV_OK) return s;
  if (kv_pool == nullptr || path == nullptr || path_len == nullptr || new_kv_lens == nullptr || max_path < 1)
    return TRTV_ERR_INVALID_ARG;
  if (!aligned(kv_pool, 16) || !aligned(path, 4) || !aligned(path_len, 4) || !aligned(new_kv_lens, 4))
    return TRTV_ERR_INVALID_ARG;
  if (g->qo_len > kMaxTreeTokens) return TRTV_ERR_UNSUPPORTED;
  if ((s = rows_device(&p.g, page_table, kv_lens)) != TRTV_OK) return s;
  p.pool = static_cast<uint8_t*>(kv_pool);
  p.path = path;
  p.path_len = path_len;
  p.new_kv_lens = new_kv_lens;
  p.max_path = max_path;
  p.row_bytes = g->head_dim * (g->kv_dtype == TRTV_FP8_E4M3 ? 1 : 2);
  const cudaError_t e = launch_tree_commit(p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? TRTV_OK : TRTV_ERR_CUDA;
}

}  // extern "C"
