// rows_attn_fp8.cu -- prompt and tree attention over E4M3 caches, and the join
// of items cut between CTAs.
#include "launch.h"
#include "rows_attn.cuh"

namespace trtv {

cudaError_t launch_rows_attn_fp8(bool two, const CUtensorMap& kv_map, const CUtensorMap& q_map,
                                 const RowsAttnParams& p, size_t smem, cudaStream_t st) {
  return launch_rows_attn_kind<128, TRTV_FP8_E4M3>(two, kv_map, q_map, p, smem, st);
}

// Joins the pieces o_i (each normalised by its own sum, log2 lse_i) of a cut
// item: o = sum_i 2^(lse_i - M) o_i / sum_i 2^(lse_i - M), M = max lse_i, in
// CTA order, so the result does not depend on timing.  One CTA per (attention
// CTA that holds an item's first page, 16 rows).  Latency bound: after the
// item's record everything is loaded at once, kBatch pieces of two elements a
// thread, CTAs in the item's range that held none of its pages masked by their
// `cont` word (no ranges are computed here).  Nothing past the last piece is
// loaded (items of two pieces, 4 chunks of 300-512 tokens: 120.5 -> 117 us).  Batches
// of two, six CTAs an SM: 115 us, but a tree cut into many pieces 16.5 -> 18.3.
// Few rows (E2M1): up to eight pieces at a time, their weights side by side, two CTAs
// an SM for the registers (one request's decoding over 8000 positions, head_dim 128,
// 16.7 -> 14.8 us, over 60000 23.0 -> 21.3; twelve at a time 15.2 and 22.2).
constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 16;   // (or all of a piece with fewer)

template <int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads, ROWS > 32 ? 4 : 2) rows_join_kernel(const __grid_constant__ RowsAttnParams p) {
  constexpr int JR = ROWS < kJoinRows ? ROWS : kJoinRows;
  constexpr int F4 = D / 4, EL = (JR * F4 + kJoinThreads - 1) / kJoinThreads, kBatch = ROWS > 32 ? 4 : EL == 1 ? 8 : 4;
  const RowsGeom& g = p.g;
  const int c0 = blockIdx.x / (ROWS / JR), chunk = blockIdx.x % (ROWS / JR), tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  // b, h, tok0, n | row0, c_last, stride
  const int4 d0 = __ldcg(reinterpret_cast<const int4*>(p.splits + c0)), d1 = __ldcg(reinterpret_cast<const int4*>(p.splits + c0) + 1);
  if (d0.x < 0) return;
  const int nc = (d1.y - c0) / d1.z + 1;
  float m[EL], l[EL];
  float4 acc[EL];
  int row[EL], tok[EL];
  bool live[EL];
#pragma unroll
  for (int u = 0; u < EL; ++u) {
    row[u] = min(chunk * JR + (u * kJoinThreads + tid) / F4, ROWS - 1);
    const int t = row[u] % kRowsTile / g.group;
    tok[u] = d0.z + (row[u] / kRowsTile) * p.tile_toks + t;
    live[u] = t < p.tile_toks && tok[u] < d0.w && (u * kJoinThreads + tid) / F4 < JR;
    m[u] = -INFINITY;
    l[u] = 0.f;
    acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int i0 = 0; i0 < nc; i0 += kBatch) {
    float x[EL][kBatch];
    float4 v[EL][kBatch];
    bool used[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      used[k] = false;
      if (i0 + k >= nc) continue;   // (the same for the whole CTA)
      const int c = c0 + (i0 + k) * d1.z;
      used[k] = i0 + k == 0 || __ldcg(p.cont + c) != 0;
      const int64_t sl = 2 * static_cast<int64_t>(c) + (i0 + k == 0 ? 1 : 0);   // (an unused slot holds anything)
#pragma unroll
      for (int u = 0; u < EL; ++u) {
        x[u][k] = __ldcg(p.ws_lse + sl * ROWS + row[u]);
        v[u][k] = __ldcg(reinterpret_cast<const float4*>(p.ws_o + (sl * ROWS + row[u]) * D) + tid % F4);
      }
    }
#pragma unroll
    for (int u = 0; u < EL; ++u) {
      if constexpr (ROWS <= 32) {   // (the pieces' weights side by side, not one after the other)
        float mn = m[u];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (used[k]) mn = max_nan(mn, x[u][k]);
        if (mn == -INFINITY) continue;
        const float so = exp2f(m[u] - mn);
        float w[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) w[k] = used[k] ? exp2f(x[u][k] - mn) : 0.f;
        l[u] *= so;
        acc[u] = make_float4(acc[u].x * so, acc[u].y * so, acc[u].z * so, acc[u].w * so);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          if (w[k] == 0.f) continue;   // (what lies there may be anything)
          l[u] += w[k];
          acc[u].x += w[k] * v[u][k].x;
          acc[u].y += w[k] * v[u][k].y;
          acc[u].z += w[k] * v[u][k].z;
          acc[u].w += w[k] * v[u][k].w;
        }
        m[u] = mn;
        continue;
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (!used[k] || x[u][k] == -INFINITY) continue;
        const float mn = fmaxf(m[u], x[u][k]);
        const float so = exp2f(m[u] - mn), w = exp2f(x[u][k] - mn);
        l[u] = l[u] * so + w;
        acc[u].x = acc[u].x * so + w * v[u][k].x;
        acc[u].y = acc[u].y * so + w * v[u][k].y;
        acc[u].z = acc[u].z * so + w * v[u][k].z;
        acc[u].w = acc[u].w * so + w * v[u][k].w;
        m[u] = mn;
      }
    }
  }
#pragma unroll
  for (int u = 0; u < EL; ++u) {
    if (!live[u]) continue;
    const float f = l[u] == 0.f ? 0.f : p.v_scale / l[u];
    const float4 a = make_float4(acc[u].x * f, acc[u].y * f, acc[u].z * f, acc[u].w * f);
    const int64_t o = (static_cast<int64_t>(d1.x + tok[u]) * g.num_q_heads + static_cast<int64_t>(d0.y) * g.group +
                       row[u] % kRowsTile % g.group) * D + 4 * (tid % F4);
    if (p.out_f32)
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o) = a;
    else
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + o) = make_uint2(pack2<false>(a.x, a.y), pack2<false>(a.z, a.w));
  }
}

template <int D>
cudaError_t launch_join_kind(int rows, const RowsAttnParams& p, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(p.num_ctas) * (rows < kJoinRows ? 1 : rows / kJoinRows)), block(kJoinThreads);
  switch (rows) {
    case 8: return launch_pdl(rows_join_kernel<D, 8>, grid, block, 0, st, p);
    case 16: return launch_pdl(rows_join_kernel<D, 16>, grid, block, 0, st, p);
    case 32: return launch_pdl(rows_join_kernel<D, 32>, grid, block, 0, st, p);
    case 128: return launch_pdl(rows_join_kernel<D, 128>, grid, block, 0, st, p);
    default: return launch_pdl(rows_join_kernel<D, 256>, grid, block, 0, st, p);
  }
}

cudaError_t launch_rows_join(int head_dim, int rows, const RowsAttnParams& p, cudaStream_t st) {
  if (p.num_ctas < 2) return cudaSuccess;  // nothing is cut
  return head_dim == 64 ? launch_join_kind<64>(rows, p, st) : launch_join_kind<128>(rows, p, st);
}

}  // namespace trtv
