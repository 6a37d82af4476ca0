// rows_attn_bf16.cu -- prompt and tree attention over bf16 caches.
#include "launch.h"
#include "rows_attn.cuh"

namespace trtv {

cudaError_t launch_rows_attn_bf16(int head_dim, bool two, const CUtensorMap& kv_map, const CUtensorMap& q_map,
                                  const RowsAttnParams& p, size_t smem, cudaStream_t st) {
  return head_dim == 64 ? launch_rows_attn_kind<64, false>(two, kv_map, q_map, p, smem, st)
                        : launch_rows_attn_kind<128, false>(two, kv_map, q_map, p, smem, st);
}

}  // namespace trtv
