// rows_few.cu -- attention of few rows over E2M1 caches.
#include "launch.h"
#include "rows_few.cuh"

namespace trtv {

template <int D, int NR>
cudaError_t launch_few_one(const CUtensorMap& kv_map, const RowsAttnParams& p, size_t smem, cudaStream_t st) {
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(&rows_few_kernel<D, NR>), smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(rows_few_kernel<D, NR>, dim3(p.num_ctas), dim3(few_threads(NR)), smem, st, kv_map, p);
}

template <int D>
cudaError_t launch_few_kind(int nr, const CUtensorMap& kv_map, const RowsAttnParams& p, size_t smem, cudaStream_t st) {
  return nr == 1   ? launch_few_one<D, 1>(kv_map, p, smem, st)
         : nr == 2 ? launch_few_one<D, 2>(kv_map, p, smem, st)
                   : launch_few_one<D, 4>(kv_map, p, smem, st);
}

cudaError_t launch_rows_few(int head_dim, int nr, const CUtensorMap& kv_map, const RowsAttnParams& p, size_t smem, cudaStream_t st) {
  return head_dim == 64 ? launch_few_kind<64>(nr, kv_map, p, smem, st) : launch_few_kind<128>(nr, kv_map, p, smem, st);
}

FewShape few_shape(int head_dim, int nr) {
  return {few_warps(nr), few_q_bytes(head_dim, nr), few_warps(nr) * few_tiles(head_dim, nr) * 16 / kPage};
}

}  // namespace trtv
