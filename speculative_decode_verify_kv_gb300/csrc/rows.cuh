// rows.cuh -- packed token rows (qo_indptr): which rows a request owns, and
// the launch parameters of the calls that take them.
#pragma once

#include "common.cuh"

namespace trtv {

struct RowsGeom {
  const int32_t* indptr;   // [batch + 1] or null: qo_len rows per request
  const int32_t* kv_lens;
  const int32_t* page_table;
  int* err;
  int batch, qo_len, num_tokens;
  int num_q_heads, num_kv_heads, group;
  int max_pages, num_slots, slot_stride;
};

// Rows row0 .. row0 + n - 1 of request b; n = 0 when it has none, or when its
// qo_indptr entries do not fit (ok = false).
struct RowSpan {
  int row0, n;
  bool ok;
};

__device__ __forceinline__ RowSpan row_span(const RowsGeom& g, int b) {
  if (g.indptr == nullptr) return {b * g.qo_len, g.qo_len, true};
  const int lo = g.indptr[b], hi = g.indptr[b + 1];
  // hi - lo cannot overflow once both lie in [0, num_tokens]
  if (lo < 0 || hi > g.num_tokens || lo > hi || hi - lo > g.qo_len || (b == 0 && lo != 0)) return {0, 0, false};
  return {lo, hi - lo, true};
}

// Flags qo_indptr entries that do not fit; every thread of one CTA calls it.
__device__ __forceinline__ void check_spans(const RowsGeom& g) {
  if (g.indptr == nullptr) return;
  for (int b = threadIdx.x; b < g.batch; b += blockDim.x)
    if (!row_span(g, b).ok) atomicOr(g.err, TRTV_DEVERR_INDPTR);
}

// The request whose rows hold `row` and that request's rows; batch when nobody
// holds it.  The whole warp calls it with one row.  32-ary search (the last b
// with indptr[b] <= row): one coalesced-ish load round per factor of 32 in the
// batch.  Entries out of order can lead the search past the request that holds
// the row, so where the request found does not, every request is looked at,
// unless no entry lies past the row, as for rows behind the last request's
// (staging 2048 requests of one token with 8192 rows behind them 16.1 us, 51 when
// those look at every request; 64 requests of 4 with 16128 rows 10.3 us, 10.0 when
// nothing is looked at).
__device__ __forceinline__ int row_owner(const RowsGeom& g, int row, int lane, RowSpan& span) {
  auto holds = [&](const RowSpan& s) { return s.ok && row >= s.row0 && row < s.row0 + s.n; };
  int lo = 0, hi = g.batch;
  if (g.indptr == nullptr) {
    lo = row / g.qo_len;
    span = row_span(g, lo);
    return min(lo, g.batch);   // equal rows per request, maybe more of them than requests
  }
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, i < hi && g.indptr[i] <= row);
    const int k = m == 0 ? 0 : 31 - __clz(m);
    lo += k * step;
    hi = min(hi, lo + step);
  }
  span = row_span(g, lo);
  if (holds(span)) return lo;
  int top = 0;
#pragma unroll 8
  for (int i = lane; i <= g.batch; i += 32) top = max(top, g.indptr[i]);
  if (__reduce_max_sync(0xffffffffu, top) <= row) return g.batch;
#pragma unroll 1
  for (int b0 = 0; b0 < g.batch; b0 += 32) {
    const unsigned m = __ballot_sync(0xffffffffu, b0 + lane < g.batch && holds(row_span(g, b0 + lane)));
    if (m != 0) {
      lo = b0 + __ffs(m) - 1;
      span = row_span(g, lo);
      return lo;
    }
  }
  return g.batch;
}

// Element offset, inside the pool, of cache position `pos`'s row of KV head 0
// in slot s's K page (V: one buffer further).
__device__ __forceinline__ int64_t cell_offset(const RowsGeom& g, int64_t s, int pos, int D) {
  return (s * g.slot_stride * kGroups + (pos % kPage) / kSub) * g.num_kv_heads * static_cast<int64_t>(kSub) * D +
         static_cast<int64_t>(pos % kSub) * D;
}

struct NormRopeParams {
  RowsGeom g;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t q_stride, k_stride, v_stride;
  const __nv_bfloat16* q_weight;
  const __nv_bfloat16* k_weight;
  const float* rope;
  const int32_t* positions;
  __nv_bfloat16* q_out;
  void* pool;
  int table_len, rot_dim, interleaved;
  int heads_per_warp, chunks;   // heads of a token that one warp takes; warps per token
  float eps, k_scale, v_scale;
};

struct CommitParams {
  RowsGeom g;
  uint8_t* pool;
  const int32_t* path;
  const int32_t* path_len;
  int32_t* new_kv_lens;
  int max_path, row_bytes;  // bytes of one head's row in the cache
};

constexpr int kRowsTile = 128;   // rows of one UMMA tile of the attention

// A row-tile item of the attention that the stream-K split cut: written by the
// CTA that holds its first page, read by the join kernel.
struct __align__(16) RowsSplit {
  int b, h, tok0, n;      // b < 0: none.  tok0: the item's first token of the request, n: the request's tokens
  int row0, c_last, stride, pad;  // the request's first row; the CTA of the item's last page; from one of its CTAs to the next
};

struct RowsAttnParams {
  RowsGeom g;
  const uint32_t* tree_mask;   // [num_tokens, mask_words] or null: the causal bound
  void* out;
  float* ws_o;                 // [2 * num_ctas, rows, D] pieces, each normalised by its own sum
  float* ws_lse;               // [2 * num_ctas, rows] log2 of their sums
  RowsSplit* splits;           // [num_ctas]
  int* cont;                   // [num_ctas] nonzero: the CTA's first piece continues an item that began before it
  int mask_words, out_f32, num_ctas;
  int tile_toks;               // tokens of a 128-row tile: 128 / group
  int items;                   // trees: 256-row items that the largest has per KV head; else 1
  int nst, nraw;               // page stages in shared memory; FP8: stages of raw codes
  int off_q, off_ring, off_raw, off_ml, off_pieces, off_scan, off_bar;   // shared memory, from the 1024-aligned base
  int setup;                   // what starting an item costs, in positions
  float scale_log2, v_scale;   // sm_scale * k_scale * log2(e)
  uint64_t wait_ns;
  int withhold;
};

// two: 256 rows (two tiles) per item, else 128 rows whose pages two softmax
// groups take in turn
cudaError_t launch_rows_attn_bf16(int head_dim, bool two, const CUtensorMap& kv_map, const CUtensorMap& q_map,
                                  const RowsAttnParams& p, size_t smem, cudaStream_t st);
cudaError_t launch_rows_attn_fp8(bool two, const CUtensorMap& kv_map, const CUtensorMap& q_map,
                                 const RowsAttnParams& p, size_t smem, cudaStream_t st);
cudaError_t launch_rows_join(int head_dim, bool two, const RowsAttnParams& p, cudaStream_t st);
cudaError_t launch_norm_rope_stage(int head_dim, bool fp8, const NormRopeParams& p, cudaStream_t st);
cudaError_t launch_tree_commit(const CommitParams& p, cudaStream_t st);

}  // namespace trtv
