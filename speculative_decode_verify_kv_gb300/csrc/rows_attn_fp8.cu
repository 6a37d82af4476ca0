// rows_attn_fp8.cu -- prompt and tree attention over E4M3 caches, and the join
// of items cut between CTAs.
#include "launch.h"
#include "rows_attn.cuh"

namespace trtv {

cudaError_t launch_rows_attn_fp8(bool two, const CUtensorMap& kv_map, const CUtensorMap& q_map,
                                 const RowsAttnParams& p, size_t smem, cudaStream_t st) {
  return two ? launch_rows_attn_one<128, true, true>(kv_map, q_map, p, smem, st)
             : launch_rows_attn_one<128, true, false>(kv_map, q_map, p, smem, st);
}

// Joins the pieces o_i (each normalised by its own sum, log2 lse_i) of a cut
// item: o = sum_i 2^(lse_i - M) o_i / sum_i 2^(lse_i - M), M = max lse_i, in
// CTA order, so the result does not depend on timing.  One CTA per (attention
// CTA that holds an item's first page, 32 rows); kBatch pieces' loads in
// flight per thread.
constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 32;

template <int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) rows_join_kernel(const __grid_constant__ RowsAttnParams p) {
  constexpr int F4 = D / 4, EL = kJoinRows * F4 / kJoinThreads, kBatch = 4;
  __shared__ RowsSplit d;
  __shared__ int slots[kMaxCombineParts];
  const RowsGeom& g = p.g;
  const int c0 = blockIdx.x / (ROWS / kJoinRows), chunk = blockIdx.x % (ROWS / kJoinRows), tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  if (tid < static_cast<int>(sizeof(RowsSplit) / 16))
    reinterpret_cast<int4*>(&d)[tid] = __ldcg(reinterpret_cast<const int4*>(p.splits + c0) + tid);
  __syncthreads();
  if (d.b < 0) return;
  const int nc = d.c_last - c0 + 1;
  for (int i = tid; i < nc; i += kJoinThreads) {
    // pages that start in CTA c0 + i's units; a range between two page starts holds none
    const int64_t a = cta_unit_begin(c0 + i, d.W, p.num_ctas) - d.first, e = cta_unit_begin(c0 + i + 1, d.W, p.num_ctas) - d.first;
    const bool used = i == 0 || (a + kPage - 1) / kPage < (e + kPage - 1) / kPage;
    slots[i] = used ? 2 * (c0 + i) + (i == 0 ? 1 : 0) : -1;
  }
  __syncthreads();
  float m[EL], l[EL];
  float4 acc[EL];
  int64_t row[EL];
  bool live[EL];
#pragma unroll
  for (int u = 0; u < EL; ++u) {
    const int r = chunk * kJoinRows + (u * kJoinThreads + tid) / F4, rt = r % kRowsTile, t = rt / g.group;
    const int tok = d.tok0 + (r / kRowsTile) * p.tile_toks + t;
    live[u] = t < p.tile_toks && tok < d.n;
    row[u] = r;
    m[u] = -INFINITY;
    l[u] = 0.f;
    acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int i0 = 0; i0 < nc; i0 += kBatch) {
    float x[EL][kBatch];
    float4 v[EL][kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int64_t sl = i0 + k < nc ? slots[i0 + k] : -1;
#pragma unroll
      for (int u = 0; u < EL; ++u) {
        x[u][k] = -INFINITY;
        if (sl >= 0 && live[u]) {
          x[u][k] = __ldcg(p.ws_lse + sl * ROWS + row[u]);
          v[u][k] = __ldcg(reinterpret_cast<const float4*>(p.ws_o + (sl * ROWS + row[u]) * D) + tid % F4);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < EL; ++u) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (x[u][k] == -INFINITY) continue;
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
    const int rt = static_cast<int>(row[u]) % kRowsTile;
    const int tok = d.tok0 + (static_cast<int>(row[u]) / kRowsTile) * p.tile_toks + rt / g.group;
    const float f = l[u] == 0.f ? 0.f : p.v_scale / l[u];
    const float4 a = make_float4(acc[u].x * f, acc[u].y * f, acc[u].z * f, acc[u].w * f);
    const int64_t o = (static_cast<int64_t>(d.row0 + tok) * g.num_q_heads + static_cast<int64_t>(d.h) * g.group + rt % g.group) * D +
                      4 * (tid % F4);
    if (p.out_f32)
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o) = a;
    else
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + o) = make_uint2(pack2<false>(a.x, a.y), pack2<false>(a.z, a.w));
  }
}

cudaError_t launch_rows_join(int head_dim, bool two, const RowsAttnParams& p, cudaStream_t st) {
  if (p.num_ctas < 2) return cudaSuccess;  // nothing is cut
  const dim3 grid(static_cast<unsigned>(p.num_ctas) * (two ? 256 : 128) / kJoinRows), block(kJoinThreads);
  if (head_dim == 64)
    return two ? launch_pdl(rows_join_kernel<64, 256>, grid, block, 0, st, p)
               : launch_pdl(rows_join_kernel<64, 128>, grid, block, 0, st, p);
  return two ? launch_pdl(rows_join_kernel<128, 256>, grid, block, 0, st, p)
             : launch_pdl(rows_join_kernel<128, 128>, grid, block, 0, st, p);
}

}  // namespace trtv
