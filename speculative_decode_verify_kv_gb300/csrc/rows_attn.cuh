// rows_attn.cuh -- attention of packed token rows over the paged cache on the
// tcgen05 tensor cores: prompts (causal) and drafted trees (a bit mask among
// the new tokens).  head_dim 64 or 128, bf16 or E4M3 K/V, any group <= 128.
//
// Work.  A 128-row tile is tile_toks = 128 / G tokens times the G query heads
// of one KV head (row = t G + g), so every K/V byte a CTA loads serves the whole
// group.  An item is a (request, KV head, tokens) with its pages 0 .. np - 1:
//   TWO   256 rows, two tiles that share each page: softmax group s (4 warps,
//         one row per thread) has tile s.  Prompts: bound by the tensor cores.
//   else  one tile of at most 128 rows; softmax group s takes the pages with
//         (page - first) % 2 = s and its own O, joined at the end (both lie in
//         the same TMEM lanes).  Small trees: bound by the K/V bytes.
// One CTA per SM walks a contiguous share of all items' pages (stream-K in
// units of cache positions: a prompt tile's cost is then a quadratic in its
// index, with no rounding to sum, and a page belongs to the CTA that holds its
// first position).  Pieces of an item cut between CTAs are joined by
// rows_join_kernel.
//
// Per page and tile: S = Q K^T (128 x 128, fp32 in TMEM), softmax in registers
// (running maximum, moved only when it rises by more than 2^8; sums in fp32 of
// the unrounded weights), P back over S as 16-bit pairs -- 8 (bf16) or 11 (f16)
// significant bits, the rounding of the second product's operand -- and
// O += P V (fp32 in TMEM).  The issuing warp orders QK of the next page behind
// PV of this one, tile by tile, so one group's softmax runs under the other's
// products; UMMAs complete in order, so S may be overwritten by a QK issued
// after the PV that reads P there, and S ready means the PV before it is done.
//
// E4M3 caches: four warps turn each page's codes into f16 (exact) in the UMMA's
// layout, and each row of Q is scaled by a power of two into f16's range
// (exact for elements within 2^-29 of the row's largest), undone in the logits'
// scale.
//
// Warps: 0-3 and 4-7 softmax groups, 8 page loads, 9 UMMA issue, 10 V pages'
// relay (rows at or past kv_len are zeroed: P is zero there but 0 * NaN is
// not), 11 Q loads, 12-15 (E4M3) conversion.
#pragma once

#include "rows.cuh"
#include "umma.cuh"

namespace trtv {

constexpr float kRowsLazy = 8.0f;   // log2 of how far a row may outgrow its reference maximum

// ---- items ------------------------------------------------------------------

struct RowsItem {
  int b, h, j;        // request, KV head, item index within (b, h)
  int n, ctx, row0, nt;
  int64_t u;          // its first unit (setup, then positions)
  bool valid;
};

struct RowsWalk {
  const RowsAttnParams& p;
  const int64_t* scan;   // [batch + 1] units before each request
  int toks;              // tokens per item
  bool causal;

  __device__ __forceinline__ int64_t cost(const RowsItem& it) const {
    return p.setup + (causal ? static_cast<int64_t>(it.ctx) + static_cast<int64_t>(toks) * (it.j + 1)
                             : static_cast<int64_t>(it.ctx) + it.n);
  }
  // units of the first j items of one KV head
  __device__ __forceinline__ int64_t before(const RowsItem& it, int64_t j) const {
    return causal ? j * (p.setup + static_cast<int64_t>(it.ctx)) + toks * (j * (j + 1) / 2)
                  : j * (p.setup + static_cast<int64_t>(it.ctx) + it.n);
  }
  __device__ __forceinline__ void request(RowsItem& it, int b) const {
    const RowSpan s = row_span(p.g, b);
    it.b = b;
    it.n = s.n;
    it.row0 = s.row0;
    it.ctx = p.g.kv_lens[b] - s.n;
    it.nt = (s.n + toks - 1) / toks;
  }
  // pages that the tokens before `end` of the item's request see
  __device__ __forceinline__ int pages(const RowsItem& it, int end) const {
    return (it.ctx + (causal ? min(end, it.n) : it.n) - 1) / kPage + 1;
  }
  __device__ __forceinline__ int item_pages(const RowsItem& it) const { return pages(it, (it.j + 1) * toks); }

  // the item that holds unit u (u < scan[batch])
  __device__ __forceinline__ RowsItem at(int64_t u) const {
    RowsItem it{};
    int lo = 0, hi = p.g.batch;          // largest b with scan[b] <= u
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (scan[mid] <= u) lo = mid; else hi = mid;
    }
    request(it, lo);
    const int64_t head = (scan[lo + 1] - scan[lo]) / p.g.num_kv_heads;
    it.h = static_cast<int>((u - scan[lo]) / head);
    const int64_t base = scan[lo] + it.h * head, r = u - base;
    int jl = 0, jh = it.nt;              // largest j with before(j) <= r
    while (jh - jl > 1) {
      const int mid = (jl + jh) / 2;
      if (before(it, mid) <= r) jl = mid; else jh = mid;
    }
    it.j = jl;
    it.u = base + before(it, jl);
    it.valid = true;
    return it;
  }
  __device__ __forceinline__ void next(RowsItem& it) const {
    it.u += cost(it);
    if (++it.j < it.nt) return;
    it.j = 0;
    if (++it.h < p.g.num_kv_heads) return;
    it.h = 0;
    int b = it.b + 1;
    while (b < p.g.batch && scan[b + 1] == scan[b]) ++b;
    it.valid = b < p.g.batch;
    if (it.valid) request(it, b);
  }
  // its pages [j0, j1) that lie in units [u0, u1)
  __device__ __forceinline__ void piece(const RowsItem& it, int64_t u0, int64_t u1, int& j0, int& j1) const {
    const int64_t f = it.u + p.setup, np = item_pages(it);
    const int64_t a = u0 > f ? (u0 - f + kPage - 1) / kPage : 0, e = u1 > f ? (u1 - f + kPage - 1) / kPage : 0;
    j0 = static_cast<int>(a < np ? a : np);
    j1 = static_cast<int>(e < np ? e : np);
  }
};

// Units of request b over all its items; 0 when it has none or is left out.
__device__ __forceinline__ int64_t rows_units(const RowsAttnParams& p, int b, int toks, bool causal, bool flag) {
  const RowSpan s = row_span(p.g, b);
  if (!s.ok) {
    if (flag) atomicOr(p.g.err, TRTV_DEVERR_INDPTR);
    return 0;
  }
  if (s.n == 0) return 0;
  const int L = p.g.kv_lens[b];
  if (!len_valid(L, s.n, p.g.max_pages)) {
    if (flag) atomicOr(p.g.err, TRTV_DEVERR_KV_LEN);
    return 0;
  }
  const int64_t nt = (s.n + toks - 1) / toks;
  const int64_t head = causal ? nt * (p.setup + static_cast<int64_t>(L - s.n)) + toks * (nt * (nt + 1) / 2)
                              : nt * (p.setup + static_cast<int64_t>(L));
  return head * p.g.num_kv_heads;
}

// Exclusive scan of the requests' units into scan[0 .. batch]; the whole block.
__device__ __forceinline__ void rows_scan(const RowsAttnParams& p, int toks, bool causal, int64_t* scan,
                                          int64_t* warp_tot) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x, n = p.g.batch;
  const int seg = (n + nthr - 1) / nthr, lo = min(n, tid * seg), hi = min(n, lo + seg);
  int64_t local = 0;
  for (int i = lo; i < hi; ++i) {
    const int64_t c = rows_units(p, i, toks, causal, blockIdx.x == 0);
    scan[i] = c;
    local += c;
  }
  int64_t incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_tot[warp] = incl;
  __syncthreads();
  int64_t run = incl - local;
  for (int w = 0; w < warp; ++w) run += warp_tot[w];
  for (int i = lo; i < hi; ++i) {
    const int64_t c = scan[i];
    scan[i] = run;
    run += c;
  }
  if (tid == nthr - 1) scan[n] = run;
  __syncthreads();
}

// ---- small device helpers -----------------------------------------------------

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// K or V page of one head: 128 positions x 64 columns (128 bytes each) per box
__device__ __forceinline__ void tma_load_page(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int h, int sub) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(0), "r"(h), "r"(sub), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tma_load_q(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int head, int row) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(head), "r"(row), "r"(smem_u32(bar))
      : "memory");
}

// Allowed columns of a page for one row of a tree, as four words: positions
// before the tree all, node i by bit i of m (bits at n and above cleared).
// off = first position of the page minus the tree's first.
__device__ __forceinline__ void tree_window(const uint32_t (&m)[4], int off, uint32_t (&w)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int o = off + 32 * k;
    uint32_t lo = 0, hi = 0;   // words o / 32 and the next, for o >= 0
    if (o <= -32) {
      w[k] = 0xffffffffu;
      continue;
    }
    if (o < 0) {
      w[k] = (m[0] << -o) | ((1u << -o) - 1u);
      continue;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (o / 32 == i) lo = m[i];
      if (o / 32 + 1 == i) hi = m[i];
    }
    w[k] = __funnelshift_r(lo, hi, o & 31);
  }
}

template <int D, bool FP8, bool TWO>
__global__ void __launch_bounds__(FP8 ? 512 : 384, 1)
    rows_attn_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap q_map,
                     const __grid_constant__ RowsAttnParams p) {
  static_assert(D == 64 || D == 128, "head_dim 64 or 128");
  static_assert(!FP8 || D == 128, "E4M3 caches: head_dim 128");
  constexpr int HB = D / 64;                        // 64-column blocks of a 16-bit tile
  constexpr int TILE = kRowsTile * D * 2;           // bytes of a Q, K or V tile in 16 bits
  constexpr int RAW = kRowsTile * D;                // of a page of codes
  constexpr uint32_t FMT = FP8 ? 0u : (1u << 7) | (1u << 10);   // f16 or bf16 operands
  constexpr uint32_t IDESC_QK = (1u << 4) | FMT | ((128u >> 3) << 17) | ((128u >> 4) << 24);
  constexpr uint32_t IDESC_PV = (1u << 4) | FMT | (1u << 16) | ((static_cast<uint32_t>(D) >> 3) << 17) |
                                ((128u >> 4) << 24);
  constexpr uint32_t TM_O = 256;                    // O of group s at 256 + 128 s, S / P at 128 s
  const RowsGeom& g = p.g;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int NST = p.nst, NRAW = p.nraw;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.off_bar);  // [NST] page ready for the UMMAs
  uint64_t* empty = full + NST;                                    // [NST] UMMAs done with it
  uint64_t* raw = empty + NST;      // bf16: [NST] V page landed (its relay then fills `full`); E4M3: [NRAW] codes landed
  uint64_t* rawfree = raw + (FP8 ? NRAW : NST);                    // E4M3: [NRAW] codes converted
  uint64_t* sfull = rawfree + (FP8 ? NRAW : 0);                    // [2] S of group s written
  uint64_t* pfull = sfull + 2;                                     // [2] P of group s written
  uint64_t* odone = pfull + 2;                                     // [2] last PV of the piece retired
  uint64_t* qfull = odone + 2;                                     // [2] Q tile landed
  uint64_t* qempty = qfull + 2;                                    // [2] last QK that reads it retired
  uint64_t* qconv = qempty + 2;                                    // [2] E4M3: Q tile converted to f16
  uint64_t* mdone = qconv + 2;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(mdone + 1);
  int* abortf = reinterpret_cast<int*>(mdone + 2);
  const Waits wt{g.err, abortf, p.wait_ns};
  int64_t* scan = reinterpret_cast<int64_t*>(smem + p.off_scan);
  float* ml = reinterpret_cast<float*>(smem + p.off_ml);           // [2 groups][128 rows] {maximum, sum}
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool causal = p.tree_mask == nullptr;
  const int toks = TWO ? 2 * p.tile_toks : p.tile_toks;

  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full[i], FP8 ? 4 : 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < (FP8 ? NRAW : NST); ++i) mbar_init(&raw[i], 1);
    if constexpr (FP8)
      for (int i = 0; i < NRAW; ++i) mbar_init(&rawfree[i], 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], 4);
      mbar_init(&odone[i], 1);
      mbar_init(&qfull[i], 1);
      mbar_init(&qempty[i], 1);
      mbar_init(&qconv[i], TWO ? 4 : 8);
    }
    mbar_init(mdone, 1);
    *abortf = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  }
  pdl_wait();   // inputs may come from the previous kernel of the stream
  rows_scan(p, toks, causal, scan, scan + g.batch + 1);
  pdl_trigger();
  const int64_t W = scan[g.batch];
  const int64_t u0 = cta_unit_begin(blockIdx.x, W, p.num_ctas), u1 = cta_unit_begin(blockIdx.x + 1, W, p.num_ctas);
  for (int b = blockIdx.x; b < g.batch; b += gridDim.x) {  // requests with a bad length: zero rows
    if (scan[b + 1] != scan[b]) continue;
    const RowSpan s = row_span(g, b);
    const int64_t o0 = static_cast<int64_t>(s.row0) * g.num_q_heads * D, o1 = o0 + static_cast<int64_t>(s.n) * g.num_q_heads * D;
    for (int64_t e = o0 + tid; e < o1; e += blockDim.x) {
      if (p.out_f32) static_cast<float*>(p.out)[e] = 0.f;
      else static_cast<__nv_bfloat16*>(p.out)[e] = __float2bfloat16(0.f);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  uint8_t* qbase = smem + p.off_q;
  uint8_t* ring = smem + p.off_ring;
  uint8_t* rring = smem + p.off_raw;
  const RowsWalk walk{p, scan, toks, causal};

  // second tile present; pages [j0, e) that group s has of a piece [j0, j1)
  auto has_two = [&](const RowsItem& it) -> bool { return TWO && it.j * toks + p.tile_toks < it.n; };
  auto group_end = [&](const RowsItem& it, int s, int j0, int j1) -> int {
    if (!TWO) return j1;
    if (s == 1 && !has_two(it)) return j0;
    return min(j1, walk.pages(it, it.j * toks + (s + 1) * p.tile_toks));
  };

  if (u0 >= u1) {
    if (tid == 0) p.splits[blockIdx.x].b = -1;
  } else if (warp == 8) {
    // ------------------------------------------------------------ page loads
    if (lane == 0) prefetch_tensormap(&kv_map);
    const int64_t vbuf = kGroups;
    RowsItem it = walk.at(u0);
    int first_b = -1, first_ids = 0;   // pages 0 .. 31 of request first_b, one per lane
    auto ids_of = [&](int b, int j) -> int {
      int s = 0;
      if (j + lane < g.max_pages && (j + lane) * kPage < it.ctx + it.n) {
        s = g.page_table[static_cast<int64_t>(b) * g.max_pages + j + lane];
        if (s < 0 || s >= g.num_slots) {
          atomicOr(g.err, TRTV_DEVERR_PAGE_ID);
          s = 0;
        }
      }
      return s;
    };
    int i = 0;                          // ring index: K page, V page, K page, ...
    int npg = 0;
    bool ok = true, stop = false;
    for (; it.valid && it.u < u1 && ok && !stop; walk.next(it)) {
      int j0, j1;
      walk.piece(it, u0, u1, j0, j1);
      if (j0 >= j1) continue;
      if (first_b != it.b) {
        first_b = it.b;
        first_ids = ids_of(it.b, 0);
      }
      int base = j0 & ~31;
      int ids = base == 0 ? first_ids : ids_of(it.b, base);
      int ahead = base + 32 < j1 ? ids_of(it.b, base + 32) : 0;
      for (int j = j0; j < j1 && ok; ++j) {
        if (j >= base + 32) {
          base += 32;
          ids = ahead;
          ahead = base + 32 < j1 ? ids_of(it.b, base + 32) : 0;
        }
        const int64_t sub = static_cast<int64_t>(__shfl_sync(0xffffffffu, ids, j - base)) * g.slot_stride * kGroups;
        stop = p.withhold >= 0 && npg >= p.withhold;   // tests of the give-up path only
        if (stop) break;
        ++npg;
        for (int kv = 0; kv < 2 && ok; ++kv, ++i) {
          if constexpr (FP8) {
            const int st = i % NRAW;
            if (lane == 0) {
              if (i >= NRAW) ok = mbar_wait(&rawfree[st], static_cast<uint32_t>(i / NRAW - 1) & 1u, wt);
              if (ok) {
                mbar_arrive_expect_tx(&raw[st], RAW);
                tma_load_page(rring + st * RAW, &kv_map, &raw[st], 0, it.h, static_cast<int>(sub + kv * vbuf));
              }
            }
          } else {
            const int st = i % NST;
            if (lane == 0) {
              if (i >= NST) ok = mbar_wait(&empty[st], static_cast<uint32_t>(i / NST - 1) & 1u, wt);
              if (ok) {
                uint64_t* bar = kv ? &raw[st] : &full[st];
                mbar_arrive_expect_tx(bar, TILE);
#pragma unroll
                for (int hb = 0; hb < HB; ++hb)
                  tma_load_page(ring + st * TILE + hb * (TILE / HB), &kv_map, bar, hb * 64, it.h,
                                static_cast<int>(sub + kv * vbuf));
              }
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
        }
      }
    }
    // never leave copies in flight.  A stage's V barrier of the bf16 ring
    // completes once per V page held there, so its parity is counted apart.
    if (lane == 0) {
      const int depth = FP8 ? NRAW : NST;
      if (!ok) --i;   // the load that gave up was not issued
      for (int k = (i > depth ? i - depth : 0); k < i; ++k) {
        const int st = k % depth;
        if constexpr (FP8) {
          mbar_drain(&raw[st], static_cast<uint32_t>(k / depth) & 1u, wt);
        } else if (k & 1) {
          mbar_drain(&raw[st], static_cast<uint32_t>(depth % 2 ? k / (2 * depth) : k / depth) & 1u, wt);
        } else {
          mbar_drain(&full[st], static_cast<uint32_t>(k / depth) & 1u, wt);
        }
      }
    }
    __syncwarp();
  } else if (warp == 11) {
    // --------------------------------------------------------------- Q loads
    // TWO: tile s in slot s; else items take the two slots in turn
    if (lane == 0) {
      prefetch_tensormap(&q_map);
      const uint32_t bytes = static_cast<uint32_t>(p.tile_toks * g.group * D * 2);
      int used[2] = {0, 0};
      bool ok = true;
      int seq = 0;
      for (RowsItem it = walk.at(u0); it.valid && it.u < u1 && ok; walk.next(it)) {
        int j0, j1;
        walk.piece(it, u0, u1, j0, j1);
        if (j0 >= j1) continue;
        for (int s = 0; s < (TWO ? 2 : 1) && ok; ++s) {
          if (TWO && group_end(it, s, j0, j1) <= j0) continue;
          const int slot = TWO ? s : seq & 1;
          const int k = used[slot]++;
          if (k > 0) ok = mbar_wait(&qempty[slot], static_cast<uint32_t>(k - 1) & 1u, wt);
          if (!ok) {
            --used[slot];
            break;
          }
          mbar_arrive_expect_tx(&qfull[slot], bytes);
#pragma unroll
          for (int hb = 0; hb < HB; ++hb)
            tma_load_q(qbase + slot * TILE + hb * (TILE / HB), &q_map, &qfull[slot], hb * 64, it.h * g.group,
                       it.row0 + it.j * toks + s * p.tile_toks);
        }
        ++seq;
      }
      for (int s = 0; s < 2; ++s)
        if (used[s] > 0) mbar_drain(&qfull[s], static_cast<uint32_t>(used[s] - 1) & 1u, wt);
    }
    __syncwarp();
  } else if (warp == 10) {
    // ---------------------------------------- V relay (bf16): zero rows, hand on
    if constexpr (!FP8) {
      int i = 1;
      uint32_t seen = 0;   // parity bit per stage of `raw`
      bool ok = true;
      for (RowsItem it = walk.at(u0); it.valid && it.u < u1 && ok; walk.next(it)) {
        int j0, j1;
        walk.piece(it, u0, u1, j0, j1);
        for (int j = j0; j < j1 && ok; ++j, i += 2) {
          const int st = i % NST;
          ok = __all_sync(0xffffffffu, lane != 0 || mbar_wait(&raw[st], (seen >> st) & 1u, wt));
          if (!ok) break;
          seen ^= 1u << st;
          const int live = it.ctx + it.n - j * kPage;   // rows below kv_len
          if (live < kPage) {
            mbar_wait(&raw[st], ((seen >> st) & 1u) ^ 1u, wt);   // every lane has seen the copy land
            for (int c = lane; c < (kPage - live) * 8 * HB; c += 32) {
              const int hb = c / ((kPage - live) * 8), r = c % ((kPage - live) * 8);
              *reinterpret_cast<uint4*>(ring + st * TILE + hb * (TILE / HB) + live * 128 + r * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(&full[st]);
        }
      }
    }
  } else if (warp == 9) {
    // ----------------------------------------------------------- UMMA issue
    // the whole warp runs the loop, one elected lane issues (umma.cuh)
    const uint64_t kd0 = umma_desc_sw128(smem_u32(ring)), qd0 = umma_desc_sw128(smem_u32(qbase));
    const uint64_t vd0 = umma_desc_sw128_mn(smem_u32(ring), TILE / 2);
    bool alive = true;
    auto wait1 = [&](uint64_t* bar, uint32_t par) {
      if (alive) alive = __all_sync(0xffffffffu, lane != 0 || mbar_wait(bar, par, wt));
    };
    int kst = 0, vst = 1 % NST;          // ring stages of the next K and V page
    uint32_t kph = 0, vph = 0;           // their parities
    auto ring_step = [&](int& st, uint32_t& ph) {
      st += 2;
      if (st >= NST) {
        st -= NST;
        ph ^= 1u;
      }
    };
    uint32_t pph[2] = {0, 0};
    int qn[2] = {0, 0};                  // Q tiles taken from each slot
    int seq = 0;
    auto issue_qk = [&](int s, int slot, int st) {
      tc_fence_after();
      const uint64_t qd = desc_add(qd0, static_cast<uint32_t>(slot * TILE)), kd = desc_add(kd0, static_cast<uint32_t>(st * TILE));
#pragma unroll
      for (int hb = 0; hb < HB; ++hb) {
        uint64_t a[4], b[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          a[k] = desc_add(qd, hb * (TILE / HB) + k * 32);
          b[k] = desc_add(kd, hb * (TILE / HB) + k * 32);
        }
        umma4_elect<false>(tmem + static_cast<uint32_t>(s * 128), a, b, IDESC_QK, hb > 0 ? 1u : 0u);
      }
      umma_commit_elect(&sfull[s]);
    };
    auto issue_pv = [&](int s, int st, bool first) {
      wait1(&pfull[s], pph[s]);
      pph[s] ^= 1u;
      if (!alive) return;
      tc_fence_after();
      const uint64_t vd = desc_add(vd0, static_cast<uint32_t>(st * TILE));
#pragma unroll
      for (int h4 = 0; h4 < 2; ++h4) {
        uint32_t a[4];
        uint64_t b[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          a[k] = tmem + static_cast<uint32_t>(s * 128 + (4 * h4 + k) * 8);
          b[k] = desc_add(vd, (4 * h4 + k) * 2048);
        }
        umma4_tmem_a_elect<false>(tmem + TM_O + static_cast<uint32_t>(s * 128), a, b, IDESC_PV, (!first || h4 > 0) ? 1u : 0u);
      }
    };
    auto take_q = [&](int slot) {
      wait1(FP8 ? &qconv[slot] : &qfull[slot], static_cast<uint32_t>(qn[slot]) & 1u);
      ++qn[slot];
    };
    for (RowsItem it = walk.at(u0); it.valid && it.u < u1 && alive; walk.next(it)) {
      int j0, j1;
      walk.piece(it, u0, u1, j0, j1);
      if (j0 >= j1) continue;
      if constexpr (TWO) {
        const int e[2] = {group_end(it, 0, j0, j1), group_end(it, 1, j0, j1)};
        // QK of page j for both tiles, the page's stage freed behind the last
        auto qk_both = [&](int j, int only) {
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if ((only >= 0 && s != only) || j >= e[s] || !alive) continue;
            issue_qk(s, s, kst);
            if (j == e[s] - 1) umma_commit_elect(&qempty[s]);
          }
        };
        for (int s = 0; s < 2; ++s)
          if (e[s] > j0) take_q(s);
        wait1(&full[kst], kph);
        if (!alive) break;
        qk_both(j0, -1);
        umma_commit_elect(&empty[kst]);
        ring_step(kst, kph);
        for (int j = j0; j < j1 && alive; ++j) {
          wait1(&full[vst], vph);
          bool have_k = false;
          for (int s = 0; s < 2 && alive; ++s) {
            if (j < e[s]) {
              issue_pv(s, vst, j == j0);
              if (!alive) break;
              if (j == e[s] - 1) umma_commit_elect(&odone[s]);
            }
            if (s == 1) umma_commit_elect(&empty[vst]);
            if (j + 1 < j1) {
              if (!have_k) {
                wait1(&full[kst], kph);
                have_k = true;
                if (!alive) break;
              }
              qk_both(j + 1, s);
              if (s == 1) {
                umma_commit_elect(&empty[kst]);
                ring_step(kst, kph);
              }
            }
          }
          ring_step(vst, vph);
        }
      } else {
        const int slot = seq & 1;
        take_q(slot);
        auto qk = [&](int j) {
          wait1(&full[kst], kph);
          if (!alive) return;
          issue_qk((j - j0) & 1, slot, kst);
          umma_commit_elect(&empty[kst]);
          ring_step(kst, kph);
          if (j == j1 - 1) umma_commit_elect(&qempty[slot]);
        };
        if (alive) qk(j0);
        if (alive && j0 + 1 < j1) qk(j0 + 1);
        for (int j = j0; j < j1 && alive; ++j) {
          const int s = (j - j0) & 1;
          wait1(&full[vst], vph);
          if (!alive) break;
          issue_pv(s, vst, j - j0 < 2);
          if (!alive) break;
          umma_commit_elect(&empty[vst]);
          if (j + 2 >= j1) umma_commit_elect(&odone[s]);
          ring_step(vst, vph);
          if (j + 2 < j1) qk(j + 2);
        }
        ++seq;
      }
    }
    umma_commit_elect(mdone);
    if (lane == 0) mbar_drain(mdone, 0, wt);
    __syncwarp();
  } else if (FP8 && warp >= 12) {
    // -------------------------------------------------- E4M3 codes -> f16 tiles
    if constexpr (FP8) {
      const int ct = tid - 384, c = ct & 7, r0 = ct >> 3;   // 16-byte chunk of a row, first row
      bool ok = true;
      int i = 0;
      for (RowsItem it = walk.at(u0); it.valid && it.u < u1 && ok; walk.next(it)) {
        int j0, j1;
        walk.piece(it, u0, u1, j0, j1);
        for (int x = 2 * j0; x < 2 * j1 && ok; ++x, ++i) {
          const int rs = i % NRAW, st = i % NST;
          ok = __all_sync(0xffffffffu, mbar_wait(&raw[rs], static_cast<uint32_t>(i / NRAW) & 1u, wt) &&
                                           (i < NST || mbar_wait(&empty[st], static_cast<uint32_t>(i / NST - 1) & 1u, wt)));
          if (!ok) break;
          const int live = (x & 1) ? it.ctx + it.n - (x >> 1) * kPage : kPage;   // V rows past kv_len are zeroed
          const uint8_t* src = rring + rs * RAW;
          uint8_t* dst = ring + st * TILE + (c >> 2) * (TILE / 2);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int r = r0 + 16 * (4 * half + k);
              v[k] = *reinterpret_cast<const uint4*>(src + r * 128 + ((c ^ (r & 7)) << 4));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int r = r0 + 16 * (4 * half + k);
              if (r >= live) v[k] = make_uint4(0, 0, 0, 0);
              const uint32_t in[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
              uint32_t o[8];
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                o[2 * w] = e4m3x2_to_f16x2(static_cast<uint16_t>(in[w] & 0xFFFFu));
                o[2 * w + 1] = e4m3x2_to_f16x2(static_cast<uint16_t>(in[w] >> 16));
              }
              // lanes of the two column blocks write opposite chunks first, so
              // that a row's eight stores fall into eight different banks groups
              const int f = c >> 2, q0 = (c & 3) * 2;
              const uint4 a = make_uint4(o[0], o[1], o[2], o[3]), b = make_uint4(o[4], o[5], o[6], o[7]);
              *reinterpret_cast<uint4*>(dst + r * 128 + (((q0 + f) ^ (r & 7)) << 4)) = f ? b : a;
              *reinterpret_cast<uint4*>(dst + r * 128 + (((q0 + 1 - f) ^ (r & 7)) << 4)) = f ? a : b;
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&rawfree[rs]);
            mbar_arrive(&full[st]);
          }
        }
      }
    }
  } else {
    // ------------------------------------------------- softmax and epilogue
    const int s = warp >> 2;                        // group
    const int r = tid & 127;                        // row of the tile, TMEM lane
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const int t = r / g.group, gl = r % g.group;    // token of the tile, head of the group
    bool dead = false;
    auto wait_all = [&](uint64_t* bar, uint32_t par) {
      if (!dead) dead = __any_sync(0xffffffffu, !mbar_wait(bar, par, wt));
    };
    uint32_t sph = 0, oph[2] = {0, 0}, qph = 0;
    int seq = 0;
    bool split = false;                             // this CTA holds the first page of a cut item
    for (RowsItem it = walk.at(u0); it.valid && it.u < u1; walk.next(it)) {
      int j0, j1;
      walk.piece(it, u0, u1, j0, j1);
      if (j0 >= j1) continue;
      const int je = group_end(it, s, j0, j1);
      const int tok = it.j * toks + (TWO ? s * p.tile_toks : 0) + t;   // of the request
      const bool live = t < p.tile_toks && tok < it.n;
      float scale = p.scale_log2;
      if constexpr (FP8) {
        // Q row -> f16, scaled by a power of two that brings its largest
        // magnitude to [2^14, 2^15)
        const int slot = TWO ? s : seq & 1;
        const bool have = TWO ? je > j0 : true;
        if (have) {
          if (TWO) {
            wait_all(&qfull[slot], qph);
            qph ^= 1u;
          } else {
            wait_all(&qfull[slot], (qph >> slot) & 1u);
            qph ^= 1u << slot;
          }
          uint8_t* row = qbase + slot * TILE + r * 128;
          float amax = 0.f;
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const uint4 v = *reinterpret_cast<const uint4*>(row + (c >> 3) * (TILE / 2) + (((c & 7) ^ (r & 7)) << 4));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              amax = max3(amax, fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xFFFF0000u)));
          }
          const int e = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -100);
          const float mul = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
          scale *= __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23);
          if (!TWO) named_barrier(1, 256);   // both groups have read the rows; each converts one half
#pragma unroll
          for (int c0 = 0; c0 < (TWO ? 16 : 8); ++c0) {
            const int c = TWO ? c0 : s * 8 + c0;
            uint4* q4 = reinterpret_cast<uint4*>(row + (c >> 3) * (TILE / 2) + (((c & 7) ^ (r & 7)) << 4));
            const uint4 v = *q4;
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              o[k] = pack2<true>(__uint_as_float(w[k] << 16) * mul, __uint_as_float(w[k] & 0xFFFF0000u) * mul);
            *q4 = make_uint4(o[0], o[1], o[2], o[3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&qconv[slot]);
        }
      }
      const float lazy = kRowsLazy / scale;
      uint32_t mw[4] = {0, 0, 0, 0};                // tree: this row's mask
      int bound = live ? it.ctx + tok : -1;         // causal: its last position
      if (!causal && live) {
        const uint32_t* m = p.tree_mask + (static_cast<int64_t>(it.row0) + tok) * p.mask_words;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int bits = it.n - 32 * k;           // bits of this word that are nodes
          if (bits > 0) mw[k] = m[k] & (bits >= 32 ? 0xffffffffu : (1u << bits) - 1u);
        }
      }
      // first position that some row of the tile does not see
      const int open = causal ? it.ctx + it.j * toks + (TWO ? s * p.tile_toks : 0) + 1 : it.ctx;
      float m = -INFINITY, negm = 0.f, l = 0.f;     // reference maximum (raw), -m scale, sum
      const int js = TWO ? j0 : j0 + s, step = TWO ? 1 : 2;
      for (int j = js; j < je; j += step) {
        wait_all(&sfull[s], sph);
        sph ^= 1u;
        tc_fence_after();
        uint32_t x[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32_async(tl + s * 128 + 32 * c, x[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_wait_dep(x[c]);
        const int pos0 = j * kPage;
        if (pos0 + kPage > open) {                  // the page holds positions that a row does not see
          if (causal) {
            const int last = bound - pos0;
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (c > last) x[c >> 5][c & 31] = 0xff800000u;
          } else {
            uint32_t w[4];
            tree_window(mw, pos0 - it.ctx, w);
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (!((w[c >> 5] >> (c & 31)) & 1u)) x[c >> 5][c & 31] = 0xff800000u;
          }
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          mx[c] = __uint_as_float(x[c][0]);
#pragma unroll
          for (int k = 1; k < 31; k += 2) mx[c] = max3(mx[c], __uint_as_float(x[c][k]), __uint_as_float(x[c][k + 1]));
          mx[c] = fmaxf(mx[c], __uint_as_float(x[c][31]));
        }
        const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
        const bool grow = m != -INFINITY && top > m + lazy;
        float alpha = 1.f;
        if (grow || m == -INFINITY) {
          const float mn = fmaxf(m, top);
          const float nn = mn == -INFINITY ? 0.f : -mn * scale;
          if (grow) alpha = fast_exp2(nn - negm);   // 2^((m - mn) scale)
          m = mn;
          negm = nn;
        }
        if (__any_sync(0xffffffffu, grow)) {
          // S ready: the PV before it has retired, O is stable
          l *= alpha;
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += 16) {
            uint32_t w[16];
            tmem_ld_async(tl + TM_O + s * 128 + c0, w);
            tmem_ld_wait_dep(w);
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(__uint_as_float(w[k]) * alpha);
            tmem_st16(tl + TM_O + s * 128 + c0, w);
          }
        }
        const float2 sc2 = make_float2(scale, scale), ng2 = make_float2(negm, negm);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float2 v = __ffma2_rn(make_float2(__uint_as_float(x[c][2 * k]), __uint_as_float(x[c][2 * k + 1])), sc2, ng2);
            v.x = fast_exp2(v.x);
            v.y = fast_exp2(v.y);
            sum[k & 1] = __fadd2_rn(sum[k & 1], v);
            w[k] = pack2<FP8>(v.x, v.y);
          }
          tmem_st16(tl + s * 128 + 16 * c, w);
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[s]);
      }
      // ------------------------------------------------------- end of the piece
      const int np = walk.item_pages(it);
      const bool whole = j0 == 0 && j1 == np;
      const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (j0 == 0 ? 1 : 0);
      constexpr int ROWS = TWO ? 256 : 128;
      if (j0 == 0 && j1 < np && tid == 0) {
        RowsSplit d;
        d.b = it.b; d.h = it.h; d.tok0 = it.j * toks; d.n = it.n; d.row0 = it.row0; d.pages = np; d.pad = 0;
        d.first = it.u + p.setup;
        d.W = W;
        d.c_last = static_cast<int>(cta_of_unit(d.first + static_cast<int64_t>(np - 1) * kPage, W, p.num_ctas));
        p.splits[blockIdx.x] = d;
        split = true;
      }
      const int64_t orow = (static_cast<int64_t>(it.row0 + tok) * g.num_q_heads + static_cast<int64_t>(it.h) * g.group + gl) * D;
      // D columns (TWO), or this group's half of them, scaled and written
      auto store = [&](int col, const float (&v)[32]) {
        if (!live) return;
        if (whole && !p.out_f32) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + orow + col);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            dst[k] = make_uint4(pack2<false>(v[8 * k], v[8 * k + 1]), pack2<false>(v[8 * k + 2], v[8 * k + 3]),
                                pack2<false>(v[8 * k + 4], v[8 * k + 5]), pack2<false>(v[8 * k + 6], v[8 * k + 7]));
        } else {
          float* base = whole ? static_cast<float*>(p.out) + orow
                              : p.ws_o + (slot * ROWS + (TWO ? s * 128 : 0) + r) * static_cast<int64_t>(D);
          float4* dst = reinterpret_cast<float4*>(base + col);
#pragma unroll
          for (int k = 0; k < 8; ++k) dst[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        }
      };
      if constexpr (TWO) {
        if (je > j0) {
          wait_all(&odone[s], oph[s]);
          oph[s] ^= 1u;
          tc_fence_after();
        }
        const float f = l == 0.f ? 0.f : (whole ? p.v_scale : 1.f) / l;  // a NaN stays one
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t o[32];
          float v[32];
          if (je > j0) {
            tmem_ld32_async(tl + TM_O + s * 128 + c0, o);
            tmem_ld_wait_dep(o);
          }
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = l == 0.f ? 0.f : __uint_as_float(o[k]) * f;
          store(c0, v);
        }
        if (!whole && live) p.ws_lse[slot * ROWS + s * 128 + r] = l == 0.f ? -INFINITY : __log2f(l) - negm;
      } else {
        // both groups' O of this row lie in this lane: exchange {maximum, sum},
        // then each group joins and writes half the columns
        float2* x2 = reinterpret_cast<float2*>(ml);
        x2[s * 128 + r] = make_float2(l == 0.f ? -INFINITY : -negm, l);
        named_barrier(1, 256);
        const int npieces = min(2, j1 - j0);
        for (int k = 0; k < npieces; ++k) {
          wait_all(&odone[k], oph[k]);
          oph[k] ^= 1u;
        }
        tc_fence_after();
        const float2 a = x2[r], b = x2[128 + r];
        const float top = fmaxf(a.x, b.x);
        const float wa = a.y == 0.f ? 0.f : fast_exp2(a.x - top), wb = b.y == 0.f ? 0.f : fast_exp2(b.x - top);
        const float lt = wa * a.y + wb * b.y;
        const float f = lt == 0.f ? 0.f : (whole ? p.v_scale : 1.f) / lt;
        const float fa = wa * f, fb = wb * f;   // zero where a group had no weight: its O may be anything
#pragma unroll
        for (int c0 = 0; c0 < D / 2; c0 += 32) {
          uint32_t o[32], q[32];
          float v[32];
          const int col = s * (D / 2) + c0;
          tmem_ld32_async(tl + TM_O + col, o);
          tmem_ld32_async(tl + TM_O + 128 + col, q);
          tmem_ld_wait_dep(o);
          tmem_ld_wait_dep(q);
#pragma unroll
          for (int k = 0; k < 32; ++k)
            v[k] = (fa == 0.f ? 0.f : __uint_as_float(o[k]) * fa) + (fb == 0.f ? 0.f : __uint_as_float(q[k]) * fb);
          store(col, v);
        }
        if (!whole && s == 0 && live) p.ws_lse[slot * ROWS + r] = lt == 0.f ? -INFINITY : top + __log2f(lt);
        tc_fence_before();
        named_barrier(1, 256);   // O may be overwritten, the exchange reused
      }
      tc_fence_before();
      ++seq;
    }
    if (tid == 0 && !split) p.splits[blockIdx.x].b = -1;
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool FP8, bool TWO>
cudaError_t launch_rows_attn_one(const CUtensorMap& kv_map, const CUtensorMap& q_map, const RowsAttnParams& p,
                                 size_t smem, cudaStream_t st) {
  const void* fn = reinterpret_cast<const void*>(&rows_attn_kernel<D, FP8, TWO>);
  const cudaError_t e = ensure_smem_attr(fn, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(rows_attn_kernel<D, FP8, TWO>, dim3(p.num_ctas), dim3(FP8 ? 512 : 384), smem, st, kv_map, q_map, p);
}

}  // namespace trtv
