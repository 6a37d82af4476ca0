// rows_attn.cu -- attention of packed token rows over the paged cache:
// prompts (causal) and drafted trees (a bit mask among the new tokens).
#include "launch.h"
#include "rows.cuh"

namespace trtv {

// One warp per (token, query head); lanes over 32 positions for the scores,
// over the head dims for P V.  Online softmax in the log2 domain, binary32.
template <int D, bool FP8>
__global__ void __launch_bounds__(256) rows_attn_kernel(const __grid_constant__ RowsAttnParams p) {
  constexpr int E = D / 32;
  __shared__ float qs[8][D];
  const RowsGeom& g = p.g;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0) check_spans(g);
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 8 + warp;
  if (unit >= static_cast<int64_t>(g.num_tokens) * g.num_q_heads) return;
  const int tok = static_cast<int>(unit / g.num_q_heads), hq = static_cast<int>(unit % g.num_q_heads);
  const int b = row_request(g, tok, lane);
  if (b >= g.batch) return;
  const RowSpan span = row_span(g, b);
  if (!span.ok || tok < span.row0 || tok >= span.row0 + span.n) return;  // nobody's row
  const int n = span.n, t = tok - span.row0, L = g.kv_lens[b], ctx = L - n;
  const bool ok = len_valid(L, n, g.max_pages);
  if (!ok && lane == 0) atomicOr(g.err, TRTV_DEVERR_KV_LEN);
  for (int d = lane; d < D; d += 32) qs[warp][d] = __bfloat162float(p.q[unit * D + d]);
  __syncwarp();
  const int h = hq / g.group;
  const int end = !ok ? 0 : (p.tree_mask != nullptr ? L : ctx + t + 1);
  auto at = [&](int64_t off) -> float {
    if constexpr (FP8) {
      const uint32_t two = e4m3x2_to_f16x2(static_cast<const uint8_t*>(p.pool)[off]);
      return __half2float(__ushort_as_half(static_cast<unsigned short>(two & 0xFFFFu)));
    } else {
      return __bfloat162float(static_cast<const __nv_bfloat16*>(p.pool)[off]);
    }
  };
  float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  const int64_t v_off = static_cast<int64_t>(kGroups) * g.num_kv_heads * kSub * D;
  for (int p0 = 0; p0 < end; p0 += 32) {
    int s = g.page_table[static_cast<int64_t>(b) * g.max_pages + p0 / kPage];
    if (s < 0 || s >= g.num_slots) {
      if (lane == 0) atomicOr(g.err, TRTV_DEVERR_PAGE_ID);
      s = 0;
    }
    const int64_t base = cell_offset(g, s, p0, D) + static_cast<int64_t>(h) * kSub * D;
    const int pos = p0 + lane;
    bool see = pos < end;
    if (p.tree_mask != nullptr && see && pos >= ctx) {
      const int j = pos - ctx;
      see = (p.tree_mask[static_cast<int64_t>(tok) * p.mask_words + j / 32] >> (j % 32)) & 1u;
    }
    float x = -INFINITY;
    if (see) {
      float acc = 0.f;
      for (int d = 0; d < D; ++d) acc += qs[warp][d] * at(base + static_cast<int64_t>(lane) * D + d);
      x = acc * p.scale_log2;
    }
    float mx = x;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
    const float mn = fmaxf(m, mx);
    if (mn == -INFINITY) continue;
    const float al = exp2f(m - mn), w = exp2f(x - mn);
    m = mn;
    l = l * al + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= al;
    for (int i = 0; i < 32; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      if (wi == 0.f) continue;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] += wi * at(base + v_off + static_cast<int64_t>(i) * D + lane + 32 * e);
    }
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
  const float sc = l > 0.f ? p.v_scale / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if (p.out_f32) static_cast<float*>(p.out)[unit * D + lane + 32 * e] = o[e] * sc;
    else static_cast<__nv_bfloat16*>(p.out)[unit * D + lane + 32 * e] = __float2bfloat16(o[e] * sc);
  }
}

cudaError_t launch_rows_attn(int head_dim, bool fp8, const RowsAttnParams& p, cudaStream_t st) {
  const int64_t blocks = (static_cast<int64_t>(p.g.num_tokens) * p.g.num_q_heads + 7) / 8;
  const dim3 grid(static_cast<unsigned>(blocks)), block(256);
  if (fp8) return launch_pdl(rows_attn_kernel<128, true>, grid, block, 0, st, p);
  return head_dim == 64 ? launch_pdl(rows_attn_kernel<64, false>, grid, block, 0, st, p)
                        : launch_pdl(rows_attn_kernel<128, false>, grid, block, 0, st, p);
}

}  // namespace trtv
