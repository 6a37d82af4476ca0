// rows_few.cu -- attention of few rows over E2M1 caches.
#include "launch.h"
#include "rows_few.cuh"

namespace trtv {

template <int D, int MT>
cudaError_t launch_few_one(const CUtensorMap& kv_map, const RowsAttnParams& p, size_t smem, cudaStream_t st) {
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(&rows_few_kernel<D, MT>), smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(rows_few_kernel<D, MT>, dim3(p.num_ctas), dim3(few_threads(D, MT)), smem, st, kv_map, p);
}

cudaError_t launch_rows_few(int head_dim, int mt, const CUtensorMap& kv_map, const RowsAttnParams& p, size_t smem, cudaStream_t st) {
  if (head_dim == 64) return mt == 1 ? launch_few_one<64, 1>(kv_map, p, smem, st) : launch_few_one<64, 2>(kv_map, p, smem, st);
  return mt == 1 ? launch_few_one<128, 1>(kv_map, p, smem, st) : launch_few_one<128, 2>(kv_map, p, smem, st);
}

FewShape few_shape(int head_dim, int mt) { return {few_warps(head_dim, mt), few_q_bytes(head_dim, mt), few_warps(head_dim, mt) * few_tiles(head_dim, mt) * 8 / kPage}; }

}  // namespace trtv
