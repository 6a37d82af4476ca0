// row_kernels.cu -- the cache writers of the packed-row calls:
//   norm_rope_stage_kernel  per-head RMS norm of queries and keys, rotation,
//                           and the rows' way to q_out and the paged cache
//   tree_commit_kernel      the accepted path's cache rows to the front of
//                           the tree's positions
#include "launch.h"
#include "rows.cuh"

namespace trtv {

// ---------------------------------------------------------------------------
// Norm, rotation, staging.  y = x (mean(x^2) + eps)^(-1/2) w; pairs (y1, y2)
// turn by the table's (c, s): (y1 c - y2 s, y2 c + y1 s).  Sums and products
// in binary32, one rounding where a value is stored (bf16, or E4M3 of the
// binary32 quotient by the cache's scale).
//
// D / 8 lanes hold one head: lane l has the 4 + 4 elements that turn together,
// 4 l .. and rot / 2 + 4 l .. (halves) or 8 l .. and 8 l + 4 .. (interleaved,
// and the dims past rot), so a rotation needs no other lane and a cosine and a
// sine load (float4 each) serve every head of the token.  A warp takes a
// token's heads (q, then k, then v) in batches of kStageRows rows per lane
// group, the next batch's loads out before this one is worked on; what a token
// costs besides (its request, its page, its table row) is loaded once.
// Bound by the bytes: 12 prompts, 72 heads of 128, 1.07 GB: 176 us = 6.1 TB/s,
// 90 % of the copy rate (8 heads a warp and no look-ahead: 294 us; batches of
// 1 / 3 / 4 rows: 203 / 185 / 195 us; blocks of 256 threads: 189 us).  An E4M3
// cache and fewer tokens (9599 of 40 heads, 192 MB): 41.7 us = 68 %.  Seven blocks
// fit on an SM, 4256 tokens are a round of warps, so these take three rounds, the last
// a quarter full: 8512 / 8960 / 9600 / 12768 / 25536 tokens take 34.7 / 40.0 / 41.1 /
// 49.8 / 93.6 us, six full rounds 80 % (pairing chosen at run time: 43.1 us; a branch
// per kind of head instead of selects: 50 us, the rows' latencies no longer overlap).
constexpr int kStageThreads = 128;
constexpr int kStageRows = 2;   // rows in flight per lane group, twice

__device__ __forceinline__ void unpack4(uint2 w, float (&x)[4]) {
  x[0] = __uint_as_float(w.x << 16);
  x[1] = __uint_as_float(w.x & 0xFFFF0000u);
  x[2] = __uint_as_float(w.y << 16);
  x[3] = __uint_as_float(w.y & 0xFFFF0000u);
}

__device__ __forceinline__ uint2 pack4(const float (&x)[4]) {
  return make_uint2(pack2<false>(x[0], x[1]), pack2<false>(x[2], x[3]));
}

__device__ __forceinline__ uint32_t pack4_e4m3(const float (&x)[4], float scale) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0] / scale, x[1] / scale), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2] / scale, x[3] / scale), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

template <int D, bool FP8, bool INTER>
__global__ void __launch_bounds__(kStageThreads) norm_rope_stage_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int LPR = D / 8;         // lanes per row
  constexpr int GPW = 32 / LPR;      // rows a warp holds at a time
  const RowsGeom& g = p.g;
  const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
  const int nq = g.num_q_heads, nqk = nq + g.num_kv_heads, heads = nqk + g.num_kv_heads;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0) check_spans(g);
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kStageThreads / 32) + (threadIdx.x >> 5);
  if (unit / p.chunks >= g.num_tokens) return;
  const int tok = static_cast<int>(unit / p.chunks);
  const int h0 = static_cast<int>(unit % p.chunks) * p.heads_per_warp, h1 = min(heads, h0 + p.heads_per_warp);
  const bool turns = 8 * l < p.rot_dim;
  const bool halves = turns && !INTER;
  const int da = halves ? 4 * l : 8 * l, db = halves ? p.rot_dim / 2 + 4 * l : 8 * l + 4;

  // row h of the token's heads (q, then k, then v): bases such that row h lies h D on
  const __nv_bfloat16* const qs = p.q + tok * p.q_stride;
  const __nv_bfloat16* const ks = p.k + tok * p.k_stride - static_cast<int64_t>(nq) * D;
  const __nv_bfloat16* const vs = p.v + tok * p.v_stride - static_cast<int64_t>(nqk) * D;
  struct Rows {
    uint2 a[kStageRows], b[kStageRows];
  };
  auto load = [&](int h, Rows& x) {
#pragma unroll
    for (int r = 0; r < kStageRows; ++r) {
      const int hr = h + r * GPW + sub;
      x.a[r] = x.b[r] = make_uint2(0, 0);
      if (hr < h1) {
        const __nv_bfloat16* s = (hr < nq ? qs : hr < nqk ? ks : vs) + hr * D;
        x.a[r] = *reinterpret_cast<const uint2*>(s + da);
        x.b[r] = *reinterpret_cast<const uint2*>(s + db);
      }
    }
  };
  Rows cur;
  load(h0, cur);   // before the token's request is known

  RowSpan span;
  const int b = row_owner(g, tok, lane, span);
  if (b >= g.batch) return;   // nobody's row
  const int L = g.kv_lens[b];
  const bool len_ok = len_valid(L, span.n, g.max_pages);
  const int cell = L - span.n + (tok - span.row0);   // >= 0 and below the capacity when len_ok
  const int pos = p.positions != nullptr ? p.positions[tok] : cell;
  const bool pos_ok = p.rot_dim == 0 || (pos >= 0 && pos < p.table_len);
  const bool live = len_ok && pos_ok;
  int slot = -1;
  if (live) {
    slot = g.page_table[static_cast<int64_t>(b) * g.max_pages + cell / kPage];
    if (slot < 0 || slot >= g.num_slots) {
      slot = -1;
      if (lane == 0) atomicOr(g.err, TRTV_DEVERR_PAGE_ID);
    }
  } else if (lane == 0) {
    atomicOr(g.err, len_ok ? TRTV_DEVERR_POSITION : TRTV_DEVERR_KV_LEN);
  }
  float co[4] = {1.f, 1.f, 1.f, 1.f}, si[4] = {0.f, 0.f, 0.f, 0.f};
  if (turns && live) {
    const float* row = p.rope + static_cast<int64_t>(pos) * p.rot_dim + 4 * l;
    const float4 c = *reinterpret_cast<const float4*>(row);
    const float4 s = *reinterpret_cast<const float4*>(row + p.rot_dim / 2);
    co[0] = c.x; co[1] = c.y; co[2] = c.z; co[3] = c.w;
    si[0] = s.x; si[1] = s.y; si[2] = s.z; si[3] = s.w;
  }
  // weights as the heads need them: q's, and from head nq on k's
  uint2 wq[2] = {}, wk[2] = {};
  if (p.q_weight != nullptr) {
    wq[0] = *reinterpret_cast<const uint2*>(p.q_weight + da);
    wq[1] = *reinterpret_cast<const uint2*>(p.q_weight + db);
  }
  if (p.k_weight != nullptr) {
    wk[0] = *reinterpret_cast<const uint2*>(p.k_weight + da);
    wk[1] = *reinterpret_cast<const uint2*>(p.k_weight + db);
  }
  __nv_bfloat16* const qd = p.q_out + static_cast<int64_t>(tok) * nq * D;
  const int64_t kd = cell_offset(g, slot < 0 ? 0 : slot, live ? cell : 0, D) - static_cast<int64_t>(nq) * kSub * D;
  const int64_t vd = kd + static_cast<int64_t>(kGroups - 1) * g.num_kv_heads * kSub * D;   // (one page buffer on, Hk heads later)
  auto process = [&](int h, const Rows& x) {
#pragma unroll
    for (int r = 0; r < kStageRows; ++r) {
      const int hr = h + r * GPW + sub;
      if (h + r * GPW >= h1) break;   // the same for the whole warp
      const bool is_q = hr < nq, is_v = hr >= nqk;
      float a[4], c[4];
      unpack4(x.a[r], a);
      unpack4(x.b[r], c);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) ss += a[i] * a[i] + c[i] * c[i];
#pragma unroll
      for (int o = 1; o < LPR; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (hr >= h1) continue;
      if (!is_v) {
        if ((is_q ? p.q_weight : p.k_weight) != nullptr) {
          const float f = rsqrtf(ss * (1.f / D) + p.eps);
          float wa[4], wc[4];
          unpack4(is_q ? wq[0] : wk[0], wa);
          unpack4(is_q ? wq[1] : wk[1], wc);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a[i] = a[i] * f * wa[i];
            c[i] = c[i] * f * wc[i];
          }
        }
        if (!INTER && turns) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float u = a[i] * co[i] - c[i] * si[i];
            c[i] = c[i] * co[i] + a[i] * si[i];
            a[i] = u;
          }
        } else if (INTER && turns) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float u = a[2 * i] * co[i] - a[2 * i + 1] * si[i];
            a[2 * i + 1] = a[2 * i + 1] * co[i] + a[2 * i] * si[i];
            a[2 * i] = u;
            const float v = c[2 * i] * co[2 + i] - c[2 * i + 1] * si[2 + i];
            c[2 * i + 1] = c[2 * i + 1] * co[2 + i] + c[2 * i] * si[2 + i];
            c[2 * i] = v;
          }
        }
      }
      if (is_q) {
        __nv_bfloat16* dst = qd + hr * D;
        *reinterpret_cast<uint2*>(dst + da) = live ? pack4(a) : make_uint2(0, 0);
        *reinterpret_cast<uint2*>(dst + db) = live ? pack4(c) : make_uint2(0, 0);
      } else if (slot >= 0) {
        const int64_t off = (is_v ? vd : kd) + static_cast<int64_t>(hr) * kSub * D;
        if constexpr (FP8) {
          const float scale = is_v ? p.v_scale : p.k_scale;
          uint8_t* dst = static_cast<uint8_t*>(p.pool) + off;
          *reinterpret_cast<uint32_t*>(dst + da) = pack4_e4m3(a, scale);
          *reinterpret_cast<uint32_t*>(dst + db) = pack4_e4m3(c, scale);
        } else {
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.pool) + off;
          *reinterpret_cast<uint2*>(dst + da) = is_v ? x.a[r] : pack4(a);
          *reinterpret_cast<uint2*>(dst + db) = is_v ? x.b[r] : pack4(c);
        }
      }
    }
  };
  // the next rows' loads go out before this batch is worked on
  for (int h = h0; h < h1; h += kStageRows * GPW) {
    Rows next;
    if (h + kStageRows * GPW < h1) load(h + kStageRows * GPW, next);
    process(h, cur);
    cur = next;
  }
}

cudaError_t launch_norm_rope_stage(int head_dim, bool fp8, const NormRopeParams& p, cudaStream_t st) {
  const int64_t warps = static_cast<int64_t>(p.chunks) * p.g.num_tokens;
  const int64_t blocks = (warps + kStageThreads / 32 - 1) / (kStageThreads / 32);
  const dim3 grid(static_cast<unsigned>(blocks)), block(kStageThreads);
  if (p.interleaved) {
    if (fp8) return launch_pdl(norm_rope_stage_kernel<128, true, true>, grid, block, 0, st, p);
    return head_dim == 64 ? launch_pdl(norm_rope_stage_kernel<64, false, true>, grid, block, 0, st, p)
                          : launch_pdl(norm_rope_stage_kernel<128, false, true>, grid, block, 0, st, p);
  }
  if (fp8) return launch_pdl(norm_rope_stage_kernel<128, true, false>, grid, block, 0, st, p);
  return head_dim == 64 ? launch_pdl(norm_rope_stage_kernel<64, false, false>, grid, block, 0, st, p)
                        : launch_pdl(norm_rope_stage_kernel<128, false, false>, grid, block, 0, st, p);
}

// ---------------------------------------------------------------------------
// Tree commit.  Row i of the tree's cache positions takes row path[i].  The
// path ascends strictly, so path[i] >= i and a thread that owns one 16-byte
// column of all rows may move them in ascending order, kMove rows read before
// they are written: later sources lie at or past the rows written so far.  One
// CTA per request (the lengths may be updated in place); an accepted prefix
// that already lies in place is not moved.  Latency bound: one round of loads
// for the tables, one for the rows.
constexpr int kCommitThreads = 256;
constexpr int kMaxTree = 128;
constexpr int kMove = 8;

__global__ void __launch_bounds__(kCommitThreads) tree_commit_kernel(const __grid_constant__ CommitParams p) {
  __shared__ int64_t src[kMaxTree], dst[kMaxTree];  // 16-byte units, column 0
  __shared__ int bad, first;
  const RowsGeom& g = p.g;
  const int b = blockIdx.x, tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  if (tid == 0) {
    bad = 0;
    first = kMaxTree;
  }
  const RowSpan span = row_span(g, b);
  const int L = g.kv_lens[b], n = span.n, ctx = L - n, k = p.path_len[b];
  __syncthreads();
  if (!span.ok) {
    if (tid == 0) atomicOr(&bad, TRTV_DEVERR_INDPTR);
  } else if (n > 0) {
    if (!len_valid(L, n, g.max_pages)) {
      if (tid == 0) atomicOr(&bad, TRTV_DEVERR_KV_LEN);
    } else if (k < 0 || k > n || k > p.max_path) {
      if (tid == 0) atomicOr(&bad, TRTV_DEVERR_PATH);
    } else {
      const int32_t* table = g.page_table + static_cast<int64_t>(b) * g.max_pages;
      const int32_t* path = p.path + static_cast<int64_t>(b) * p.max_path;
      const int D16 = p.row_bytes / 16;
      for (int j = ctx / kPage + tid; j <= (L - 1) / kPage; j += kCommitThreads)
        if (table[j] < 0 || table[j] >= g.num_slots) atomicOr(&bad, TRTV_DEVERR_PAGE_ID);
      if (tid < k) {
        const int t = path[tid], before = tid > 0 ? path[tid - 1] : -1;
        if (t <= before || t >= n) {
          atomicOr(&bad, TRTV_DEVERR_PATH);
        } else {
          src[tid] = cell_offset(g, table[(ctx + t) / kPage], ctx + t, D16);
          dst[tid] = cell_offset(g, table[(ctx + tid) / kPage], ctx + tid, D16);
          if (t != tid) atomicMin(&first, tid);
        }
      }
    }
  }
  __syncthreads();
  if (tid == 0) {
    const int e = bad;
    if (e != 0) atomicOr(g.err, e);
    p.new_kv_lens[b] = e != 0 || n == 0 ? L : ctx + k;
  }
  if (bad != 0 || n == 0) return;
  const int D16 = p.row_bytes / 16;
  const int64_t page = static_cast<int64_t>(kGroups) * g.num_kv_heads * kSub * D16;
  uint4* pool = reinterpret_cast<uint4*>(p.pool);
  const int cols = 2 * g.num_kv_heads * D16;
  for (int c = tid; c < cols; c += kCommitThreads) {
    const int hv = c / D16;
    const int64_t col = (hv & 1) * page + static_cast<int64_t>(hv >> 1) * kSub * D16 + c % D16;
    for (int i = first; i < k; i += kMove) {
      uint4 v[kMove];
#pragma unroll
      for (int u = 0; u < kMove; ++u)
        if (i + u < k) v[u] = pool[src[i + u] + col];
#pragma unroll
      for (int u = 0; u < kMove; ++u)
        if (i + u < k) pool[dst[i + u] + col] = v[u];
    }
  }
}

cudaError_t launch_tree_commit(const CommitParams& p, cudaStream_t st) {
  return launch_pdl(tree_commit_kernel, dim3(p.g.batch), dim3(kCommitThreads), 0, st, p);
}

}  // namespace trtv
