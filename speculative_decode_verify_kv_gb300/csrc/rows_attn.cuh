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
// rows_join_kernel.  LANES: a tree of more than 256 rows has several items a KV
// head that read the same pages; the CTAs walk in as many lanes, abreast (see
// rows_scan; 16 trees of 512 rows over 16-32 k positions: 5 % faster, over E4M3
// 0.4 % slower).
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
// scale.  f16 has few exponents, so P is lifted by 2^7: the reference maximum's
// weight is 2^7, a row may outgrow it to 2^15, and down to 2^-21 of it a weight
// keeps its 11 bits.  Below, it is off by at most 2^-32 of it, less than the other
// weights' rounding in a piece of up to 2^21 positions (not lifted, weights under
// 2^-25 were lost: 0.4 % of the sum in a row of one large and 131072 small).  A
// reference that moves at 2^4, with a lift of 2^10, takes 2242 us where logits have a
// deviation of 6 (a prompt of 16384), 2206 so.
//
// What bounds a prompt's page is one group's chain: softmax, then PV and the
// next QK, which cannot start before P is written over S.  So a row's scores are
// read from TMEM twice (a read of 32 columns takes 35 cycles, spilt registers
// much more), and P is handed over in two halves, the first half's PV running
// under the second half's exponentials.
//
// Warps: 0-3 and 4-7 softmax groups, 8 page loads, 9 (TWO: and 10) UMMA issue
// (V rows at or past kv_len are zeroed first: P is zero there but 0 * NaN
// is not), 11 the CTA's schedule (its pieces, a few ahead, in shared memory; what
// the join needs) and Q loads, 12-15 (E4M3) conversion.
#pragma once

#include "rows.cuh"
#include "umma.cuh"

namespace trtv {

constexpr int kConvertWarps = 4;   // warps that convert a tile of E4M3 codes, all of them every tile
constexpr int kRowsLeast = 256;
constexpr float kRowsLazy = 8.0f;   // log2 of how far a row may outgrow its reference maximum
constexpr float kRowsLiftF16 = 7.0f;   // E4M3 caches: log2 of that maximum's weight

// ---- items ------------------------------------------------------------------

struct RowsItem {
  int b, h, j;        // request, KV head, item index within (b, h)
  int n, ctx, row0, nt;
  int64_t u;          // its first unit (setup, then positions)
  bool valid;
};

template <bool LANES>
struct RowsWalk {
  const RowsAttnParams& p;
  const int64_t* scan;   // [batch + 1] units before each request
  int toks;              // tokens per item
  bool causal;
  int lane_item;         // >= 0: this CTA takes item `lane_item` of every KV head, scan counts one item a head

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

  // the largest i in [0, n) with f(i) <= u, f rising, f(0) <= u: 32 candidates a
  // round, for the whole warp
  template <typename F>
  __device__ __forceinline__ int last_at_most(int n, int64_t u, int lane, F f) const {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, i = lo + lane * step;
      const unsigned m = __ballot_sync(0xffffffffu, i < hi && f(i) <= u);
      lo += (31 - __clz(m)) * step;
      hi = min(hi, lo + step);
    }
    return lo;
  }
  // the item that holds unit u (u < scan[batch]), for the whole warp
  __device__ __forceinline__ RowsItem at(int64_t u, int lane) const {
    RowsItem it{};
    request(it, last_at_most(p.g.batch, u, lane, [&](int i) { return scan[i]; }));
    const int64_t base = scan[it.b], head = before(it, LANES && lane_item >= 0 ? 1 : it.nt);
    it.h = last_at_most(p.g.num_kv_heads, u - base, lane, [&](int i) { return i * head; });
    it.u = base + it.h * head;
    if (LANES && lane_item >= 0) {
      it.j = lane_item;
    } else {
      it.j = last_at_most(it.nt, u - it.u, lane, [&](int i) { return before(it, i); });
      it.u += before(it, it.j);
    }
    it.valid = true;
    return it;
  }
  __device__ __forceinline__ void next(RowsItem& it) const {
    it.u += cost(it);
    if (!LANES || lane_item < 0) {
      if (++it.j < it.nt) return;
      it.j = 0;
    }
    if (++it.h < p.g.num_kv_heads) return;
    it.h = 0;
    int b = it.b + 1;
    while (b < p.g.batch && scan[b + 1] == scan[b]) ++b;
    it.valid = b < p.g.batch;
    if (it.valid) request(it, b);
  }
  // its pages [j0, j1) that lie in units [u0, u1)
  __device__ __forceinline__ void piece(const RowsItem& it, int64_t u0, int64_t u1, int& j0, int& j1) const {
    const int64_t f = it.u + p.setup, np = !LANES || it.j < it.nt ? item_pages(it) : 0;
    const int64_t a = u0 > f ? (u0 - f + kPage - 1) / kPage : 0, e = u1 > f ? (u1 - f + kPage - 1) / kPage : 0;
    j0 = static_cast<int>(a < np ? a : np);
    j1 = static_cast<int>(e < np ? e : np);
  }
};

// One piece of an item, as the scheduling warp hands it to the others: the
// item's place and the pages [j0, j1) of this CTA (e0, e1: where each softmax
// group's pages end); j1 = 0 ends the CTA's work.
struct __align__(16) RowsPiece {
  int row0, tok0, n, ctx;   // the request's first row, the item's first token, the request's tokens, positions before them
  int j0, j1, e0, e1;
  int np, h, b, pad;        // the item's pages, KV head, request
};
constexpr int kRowsPieces = 4;   // pieces scheduled ahead

// First unit of CTA c: floor(c W / P), W from the P-th on (c and P are at most
// 1024, so that little work needs no 64-bit division).
__device__ __forceinline__ int64_t rows_begin(int64_t c, int64_t W, int64_t P) {
  if (c >= P) return W;
  return W < (1 << 22) ? static_cast<uint32_t>(c * W) / static_cast<uint32_t>(P) : cta_unit_begin(c, W, P);
}

// Units of request b over all its items, 0 when it has none or is left out;
// `one`: of one item per KV head (trees: all items of a head cost the same).
__device__ __forceinline__ int64_t rows_units(const RowsAttnParams& p, int b, int toks, bool causal, bool flag, int64_t& one) {
  one = 0;
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
  one = (p.setup + static_cast<int64_t>(L)) * p.g.num_kv_heads;
  return causal ? (nt * (p.setup + static_cast<int64_t>(L - s.n)) + toks * (nt * (nt + 1) / 2)) * p.g.num_kv_heads : nt * one;
}

// Exclusive scan of the requests' units into scan[0 .. batch]; the whole block.
// LANES: true, and the scan is of one item per head, where the CTAs in
// `items` lanes, each with an item of every head, would be done at most a fifth
// later than with all items in one row: the lanes' CTAs read a head's pages at
// the same time, so that one read of HBM serves them.
template <bool LANES>
__device__ __forceinline__ bool rows_scan(const RowsAttnParams& p, int toks, bool causal, int items, int64_t* scan,
                                          int64_t* warp_tot, int& requests) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x, n = p.g.batch, warps = nthr / 32;
  const int seg = (n + nthr - 1) / nthr, lo = min(n, tid * seg), hi = min(n, lo + seg);
  int64_t all = 0, one = 0;
  for (int i = lo; i < hi; ++i) {
    int64_t o;
    const int64_t c = rows_units(p, i, toks, causal, blockIdx.x == 0, o);
    scan[i] = c;
    all += c;
    one += o;
  }
  int64_t incl = all, incl_one = one;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_tot[warp] = incl;
  if constexpr (LANES) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl_one, o);
      if (lane >= o) incl_one += v;
    }
    if (lane == 31) warp_tot[warps + warp] = incl_one;
  }
  requests = __syncthreads_count(all > 0);   // (batches beyond a thread each: fewer)
  bool lanes = false;
  if constexpr (LANES) {
    int64_t w_all = 0, w_one = 0;
    for (int w = 0; w < warps; ++w) {
      w_all += warp_tot[w];
      w_one += warp_tot[warps + w];
    }
    lanes = 5 * w_one * p.num_ctas <= 6 * w_all * (p.num_ctas / items);
  }
  int64_t run = lanes ? incl_one - one : incl - all;
  for (int w = 0; w < warp; ++w) run += warp_tot[lanes ? warps + w : w];
  for (int i = lo; i < hi; ++i) {
    int64_t c = scan[i];
    if (LANES && lanes) rows_units(p, i, toks, causal, false, c);
    scan[i] = run;
    run += c;
  }
  if (tid == nthr - 1) scan[n] = run;
  __syncthreads();
  return lanes;
}

// ---- small device helpers -----------------------------------------------------

// Named barrier; whether every thread brought true.
__device__ __forceinline__ bool barrier_all(int id, int threads, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbar.red.and.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(x))
      : "memory");
  return r != 0;
}

// four E4M3 codes -> four f16 (exact)
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// mbar_wait with the waiting loop out of line: a control warp's code runs once
// per page or item and is fetched each time, so it is kept short.
static __device__ __noinline__ bool rows_wait_slow(uint64_t* bar, uint32_t parity, int* err, volatile int* abort, uint64_t limit_ns) {
  return mbar_wait(bar, parity, Waits{err, abort, limit_ns});
}
__device__ __forceinline__ bool rows_wait(uint64_t* bar, uint32_t parity, const Waits& w) {
  return mbar_try_wait(bar, parity) || rows_wait_slow(bar, parity, w.err, w.abort, w.limit_ns);
}

// K or V page of one head: 128 positions x 64 columns (128 bytes each) per
// box.  ONCE: no other item reads the page, it need not stay in L2.
template <bool ONCE>
__device__ __forceinline__ void tma_load_page(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int h, int sub,
                                              uint64_t evict_first) {
  if constexpr (ONCE) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(0), "r"(h), "r"(sub), "r"(smem_u32(bar)), "l"(evict_first)
        : "memory");
  } else {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(0), "r"(h), "r"(sub), "r"(smem_u32(bar))
        : "memory");
  }
}

__device__ __forceinline__ void tma_load_q(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int head, int row) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(head), "r"(row), "r"(smem_u32(bar))
      : "memory");
}

// The products of one page and tile, issued by one elected lane (the whole warp
// executes the call): one asm block, only the low word of a descriptor moves.
//   S = Q K^T: HB x 4 steps of 16 head dims, 32 bytes apart in a 64-column
//   block, the blocks 16 KB apart
#define TRTV_QK_STEP(OFF, P)                                                                         \
  "add.u32 x, %1, " #OFF ";\n\tadd.u32 y, %2, " #OFF ";\n\tmov.b64 a, {x, %4};\n\tmov.b64 b, {y, %4};\n\t" \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, " #P ";\n\t"
template <int HB>
__device__ __forceinline__ void umma_qk(uint32_t d, uint32_t q, uint32_t k, uint32_t desc_hi, uint32_t idesc) {
  if constexpr (HB == 2) {
    asm volatile(
        "{\n\t.reg .pred e, f, t;\n\t.reg .b32 x, y;\n\t.reg .b64 a, b;\n\telect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 f, 0, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        TRTV_QK_STEP(0, f) TRTV_QK_STEP(2, t) TRTV_QK_STEP(4, t) TRTV_QK_STEP(6, t)
        TRTV_QK_STEP(1024, t) TRTV_QK_STEP(1026, t) TRTV_QK_STEP(1028, t) TRTV_QK_STEP(1030, t)
        "}\n" ::"r"(d), "r"(q), "r"(k), "r"(idesc), "r"(desc_hi)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred e, f, t;\n\t.reg .b32 x, y;\n\t.reg .b64 a, b;\n\telect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 f, 0, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        TRTV_QK_STEP(0, f) TRTV_QK_STEP(2, t) TRTV_QK_STEP(4, t) TRTV_QK_STEP(6, t)
        "}\n" ::"r"(d), "r"(q), "r"(k), "r"(idesc), "r"(desc_hi)
        : "memory");
  }
}
#undef TRTV_QK_STEP
//   O (+)= P V for half a page: 4 steps of 16 positions, 8 TMEM columns of P
//   and 2 KB of V apart
#define TRTV_PV_STEP(AO, BO, P)                                                          \
  "add.u32 x, %1, " #AO ";\n\tadd.u32 y, %2, " #BO ";\n\tmov.b64 b, {y, %5};\n\t"        \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, " #P ";\n\t"
__device__ __forceinline__ void umma_pv(uint32_t d, uint32_t pt, uint32_t v, uint32_t desc_hi, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, f, t;\n\t.reg .b32 x, y;\n\t.reg .b64 b;\n\telect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 f, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      TRTV_PV_STEP(0, 0, f) TRTV_PV_STEP(8, 128, t) TRTV_PV_STEP(16, 256, t) TRTV_PV_STEP(24, 384, t)
      "}\n" ::"r"(d), "r"(pt), "r"(v), "r"(idesc), "r"(accumulate), "r"(desc_hi)
      : "memory");
}
#undef TRTV_PV_STEP

// Allowed columns of a page for one row of a tree, as four words: positions
// before the tree all, node i by bit i of m (bits at n and above cleared).
// off = the first column's position minus the tree's first.
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

// The same for a causal bound: columns 0 .. last.
__device__ __forceinline__ void row_window(int last, uint32_t (&w)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int o = last - 32 * k;
    w[k] = o >= 31 ? 0xffffffffu : o < 0 ? 0u : (2u << o) - 1u;
  }
}

// Of 32 scores, those that the row does not see (bits of w not set) become
// minus infinity.
__device__ __forceinline__ void row_mask(uint32_t w, uint32_t (&x)[32]) {
#pragma unroll
  for (int k = 0; k < 32; ++k) x[k] = (w >> k) & 1u ? x[k] : 0xff800000u;
}

__device__ __forceinline__ float row_max(const uint32_t (&x)[32]) {
  float a = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1])), b = fmaxf(__uint_as_float(x[2]), __uint_as_float(x[3]));
#pragma unroll
  for (int k = 4; k < 32; k += 4) {
    a = max3(a, __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
    b = max3(b, __uint_as_float(x[k + 2]), __uint_as_float(x[k + 3]));
  }
  return fmaxf(a, b);
}

// A pair of weights as f16; past its range (the scores' own rounding can leave a
// row that far above its maximum where they pass 2^22) its largest value.
__device__ __forceinline__ uint32_t pack2_f16_sat(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Weights 2^(x scale + negm) of columns 32 c .. 32 c + 31, stored over the scores
// as 16-bit pairs (column ts + i of P holds positions 2i and 2i + 1); their sum
// is added to `sum`.
template <bool F16>
__device__ __forceinline__ void row_exp(uint32_t ts, int c, const uint32_t (&x)[32], float scale, float negm, float2& sum) {
  const float2 sc2 = make_float2(scale, scale), ng2 = make_float2(negm, negm);
  constexpr int N = F16 ? 8 : 16;   // pairs at a time (E4M3 kernels have fewer registers)
#pragma unroll
  for (int h = 0; h < 16; h += N) {
    uint32_t o[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float2 v = make_float2(__uint_as_float(x[2 * (h + k)]), __uint_as_float(x[2 * (h + k) + 1]));
      v = __ffma2_rn(v, sc2, ng2);
      v.x = fast_exp2(v.x);
      v.y = fast_exp2(v.y);
      sum = __fadd2_rn(sum, v);
      o[k] = F16 ? pack2_f16_sat(v.x, v.y) : pack2<false>(v.x, v.y);
    }
    if constexpr (F16) tmem_st8(ts + 16 * c + h, o);
    else tmem_st16(ts + 16 * c, o);
  }
}

// 32 bytes to 16-byte aligned memory; `wide`: it is 32-byte aligned
__device__ __forceinline__ void store_sector(uint8_t* dst, bool wide, const uint32_t (&w)[8]) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(dst + 16) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <int D, bool FP8, bool TWO, bool LANES>
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
  uint64_t* raw = empty + NST;                                     // E4M3: [NRAW] codes landed
  uint64_t* rawfree = raw + NRAW;                                  // E4M3: [NRAW] codes converted
  uint64_t* sfull = rawfree + NRAW;                                // [2] S of group s written
  uint64_t* pfull = sfull + 2;                                     // [2][2] P of group s, half h of the page, written
  uint64_t* odone = pfull + 4;                                     // [2] last PV of the piece retired
  uint64_t* qfull = odone + 2;                                     // [2] Q tile landed
  uint64_t* qempty = qfull + 2;                                    // [2] last QK that reads it retired
  uint64_t* qconv = qempty + 2;                                    // [2] E4M3: Q tile converted to f16
  uint64_t* ifull = qconv + 2;                                     // [kRowsPieces] piece scheduled
  uint64_t* iempty = ifull + kRowsPieces;                          // [kRowsPieces] every role has copied it
  uint64_t* turn = iempty + kRowsPieces;                           // [2] TWO: group s may issue
  uint64_t* mdone = turn + 2;                                      // [2] an issuer's last UMMA retired
  uint32_t* tslot = reinterpret_cast<uint32_t*>(mdone + 2);
  int* abortf = reinterpret_cast<int*>(mdone + 3);
  const Waits wt{g.err, abortf, p.wait_ns};
  int64_t* scan = reinterpret_cast<int64_t*>(smem + p.off_scan);
  float2* xml = reinterpret_cast<float2*>(smem + p.off_ml);        // [2 groups][128 rows] {reference maximum, sum}
  RowsPiece* pieces = reinterpret_cast<RowsPiece*>(smem + p.off_pieces);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool causal = p.tree_mask == nullptr;
  const int toks = TWO ? 2 * p.tile_toks : p.tile_toks;

  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full[i], FP8 ? kConvertWarps : 1);
      mbar_init(&empty[i], TWO ? 2 : 1);   // the groups' issuers that read the page
    }
    for (int i = 0; i < NRAW; ++i) {
      mbar_init(&raw[i], 1);
      mbar_init(&rawfree[i], kConvertWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[2 * i], 4);
      mbar_init(&pfull[2 * i + 1], 4);
      mbar_init(&odone[i], 1);
      mbar_init(&qfull[i], 1);
      mbar_init(&qempty[i], 1);
      mbar_init(&qconv[i], TWO ? 4 : 8);
    }
    for (int i = 0; i < kRowsPieces; ++i) {
      mbar_init(&ifull[i], 1);
      mbar_init(&iempty[i], 9 + (TWO ? 2 : 1) + (FP8 ? 4 : 0));   // softmax 8, page loads, UMMA issue, conversion 4
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&turn[i], 1);
      mbar_init(&mdone[i], 1);
    }
    *abortf = 0;
    fence_mbar_init();
  }
  pdl_wait();   // inputs may come from the previous kernel of the stream
  // (TMEM only now: a CTA that held it while it waits for the previous kernel could
  // keep it from a CTA of that kernel on the same SM)
  if (warp == 9) {
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  }
  int requests;
  const bool lanes = rows_scan<LANES>(p, toks, causal, LANES ? p.items : 1, scan, scan + g.batch + 1, requests);
  pdl_trigger();
  const int64_t W = scan[g.batch];
  // little work is spread over fewer CTAs: pieces of less than kRowsLeast
  // positions cost more to join than they save.  One-tile items of many pages (A
  // positions a head) are cut less than that: a page takes 0.35 us, four more pieces
  // 1.75 us of the join, so a piece is best some 10 sqrt(A) long (a tree of 8 over
  // 8000 positions 28.5 -> 21.2 us, over 30000 36.5 -> 32.0, two over 4-9 k 27.9 ->
  // 22.9; factors of 8, 12 and 16 21.2 / 21.3 / 23.2, 32.1 / 33.2 / 35.1), 64 off it
  // (0 / 32 / 64 / 96 / 128 off: one over 3000 17.7 / 17.6 / 17.0 / 16.9 / 17.5, three over
  // 700-1500 17.5 / 17.2 / 15.7 / 17.9 / 17.9, over 30000 34.5 / 34.3 / 34.1 / 34.3 / 34.1).
  const int stride = LANES && lanes ? p.items : 1, rank = static_cast<int>(blockIdx.x) / stride;
  int64_t P = max(int64_t{1}, min(static_cast<int64_t>(p.num_ctas / stride), W / kRowsLeast));
  if (!TWO && P > 16) {   // (16 pieces or fewer: not worth the arithmetic)
    const float per_head = static_cast<float>(W) / static_cast<float>(max(requests, 1) * g.num_kv_heads);
    P = min(P, W / max(kRowsLeast, static_cast<int>(10.f * sqrtf(per_head)) - 64));
  }
  // (a multiple of the KV heads: one request's heads are then all cut alike, no CTA
  // has the end of one and the start of the next; a tree of 8 over 900 positions
  // 14.0 us, 17.5 on 15 or 18 CTAs)
  if (P < p.num_ctas / stride && P > g.num_kv_heads) P -= static_cast<int>(P) % g.num_kv_heads;
  const int64_t u0 = rows_begin(rank, W, P), u1 = rows_begin(rank + 1, W, P);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  uint8_t* qbase = smem + p.off_q;
  uint8_t* ring = smem + p.off_ring;
  uint8_t* rring = smem + p.off_raw;
  // The next piece of this CTA, for the whole warp; false at the end, or when
  // the wait gave up.
  int piece_at = 0;
  uint32_t piece_ph = 0;
  auto next_piece = [&](RowsPiece& it) -> bool {
    if (!__all_sync(0xffffffffu, rows_wait(&ifull[piece_at], piece_ph, wt))) return false;
    it = pieces[piece_at];
    __syncwarp();
    if (lane == 0) mbar_arrive(&iempty[piece_at]);
    if (++piece_at == kRowsPieces) {
      piece_at = 0;
      piece_ph ^= 1u;
    }
    return it.j1 > 0;
  };

  if (u0 >= u1) {
    if (tid == 0) {
      p.splits[blockIdx.x].b = -1;
      p.cont[blockIdx.x] = 0;
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------ page loads
    if (lane == 0) prefetch_tensormap(&kv_map);
    const int64_t vbuf = kGroups;
    const uint64_t pol = policy_evict_first();
    RowsPiece it{};
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
    while (ok && !stop && next_piece(it)) {
      const int j0 = it.j0, j1 = it.j1;
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
              if (i >= NRAW) ok = rows_wait(&rawfree[st], static_cast<uint32_t>(i / NRAW - 1) & 1u, wt);
              if (ok) {
                mbar_arrive_expect_tx(&raw[st], RAW);
                tma_load_page<!TWO>(rring + st * RAW, &kv_map, &raw[st], 0, it.h, static_cast<int>(sub + kv * vbuf), pol);
              }
            }
          } else {
            const int st = i % NST;
            if (lane == 0) {
              if (i >= NST) ok = rows_wait(&empty[st], static_cast<uint32_t>(i / NST - 1) & 1u, wt);
              if (ok) {
                mbar_arrive_expect_tx(&full[st], TILE);
#pragma unroll
                for (int hb = 0; hb < HB; ++hb)
                  tma_load_page<!TWO>(ring + st * TILE + hb * (TILE / HB), &kv_map, &full[st], hb * 64, it.h,
                                      static_cast<int>(sub + kv * vbuf), pol);
              }
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
        }
      }
    }
    // never leave copies in flight
    if (lane == 0) {
      const int depth = FP8 ? NRAW : NST;
      uint64_t* bars = FP8 ? raw : full;
      if (!ok) --i;   // the load that gave up was not issued
      for (int k = (i > depth ? i - depth : 0); k < i; ++k) mbar_drain(&bars[k % depth], static_cast<uint32_t>(k / depth) & 1u, wt);
    }
    __syncwarp();
  } else if (warp == 11) {
    // ------------------------------------------------- schedule and Q loads
    // Q tiles: TWO: tile s in slot s; else one slot
    const RowsWalk<LANES> walk{p, scan, toks, causal, LANES && lanes ? static_cast<int>(blockIdx.x) % stride : -1};
    RowsItem it = walk.at(u0, lane);
    if (lane == 0) {
      prefetch_tensormap(&q_map);
      const uint32_t bytes = static_cast<uint32_t>(p.tile_toks * g.group * D * 2);
      int used[2] = {0, 0};
      bool ok = true, split = false;   // split: this CTA holds the first page of a cut item
      int seq = 0;
      for (;;) {
        RowsPiece x{};
        for (; it.valid && it.u < u1; walk.next(it)) {
          walk.piece(it, u0, u1, x.j0, x.j1);
          if (x.j0 < x.j1) break;
          x.j1 = 0;
        }
        if (x.j1 > 0) {
          x.row0 = it.row0;
          x.tok0 = it.j * toks;
          x.n = it.n;
          x.ctx = it.ctx;
          x.np = walk.item_pages(it);
          x.h = it.h;
          x.b = it.b;
          x.e0 = x.e1 = x.j1;
          if (TWO) {   // the tiles' own ends: the second may be empty, the first see fewer pages
            x.e0 = min(x.j1, walk.pages(it, x.tok0 + p.tile_toks));
            x.e1 = x.tok0 + p.tile_toks < x.n ? x.j1 : x.j0;
          }
        }
        const int k = seq % kRowsPieces;
        if (seq >= kRowsPieces) ok = rows_wait(&iempty[k], static_cast<uint32_t>(seq / kRowsPieces - 1) & 1u, wt);
        if (!ok) break;
        pieces[k] = x;
        mbar_arrive(&ifull[k]);
        if (x.j1 == 0) break;
        for (int s = 0; s < (TWO ? 2 : 1) && ok; ++s) {
          if (TWO && (s ? x.e1 : x.e0) <= x.j0) continue;
          const int slot = TWO ? s : 0;
          if (used[slot] > 0) ok = rows_wait(&qempty[slot], static_cast<uint32_t>(used[slot] - 1) & 1u, wt);
          if (!ok) break;
          ++used[slot];
          mbar_arrive_expect_tx(&qfull[slot], bytes);
#pragma unroll
          for (int hb = 0; hb < HB; ++hb)
            tma_load_q(qbase + slot * TILE + hb * (TILE / HB), &q_map, &qfull[slot], hb * 64, x.h * g.group,
                       x.row0 + x.tok0 + s * p.tile_toks);
        }
        if (!ok) break;
        // what the join needs to know
        if (seq == 0) p.cont[blockIdx.x] = x.j0 > 0;
        if (x.j0 == 0 && x.j1 < x.np) {
          RowsSplit d{};
          d.b = x.b;
          d.h = x.h;
          d.tok0 = x.tok0;
          d.n = x.n;
          d.row0 = x.row0;
          d.c_last = static_cast<int>(cta_of_unit(it.u + p.setup + static_cast<int64_t>(x.np - 1) * kPage, W, P));
          if constexpr (LANES) d.c_last = d.c_last * stride + static_cast<int>(blockIdx.x) % stride;
          d.stride = stride;
          p.splits[blockIdx.x] = d;
          split = true;
        }
        ++seq;
        walk.next(it);
      }
      if (!split) p.splits[blockIdx.x].b = -1;
      if (seq == 0) p.cont[blockIdx.x] = 0;   // no page starts in its units
      for (int s = 0; s < 2; ++s)
        if (used[s] > 0) mbar_drain(&qfull[s], static_cast<uint32_t>(used[s] - 1) & 1u, wt);
    }
    __syncwarp();
  } else if (warp == 9 || (TWO && warp == 10)) {
    // ----------------------------------------------------------- UMMA issue
    // Steps: PV of a page, then QK of the same group's next page.  The whole
    // warp runs the loop, one elected lane issues.
    // TWO: one issuing warp per softmax group, taking strict turns.  One
    // warp's waits (100-200 cycles each even when nothing is to be waited
    // for; the tensor core's queue is only a few UMMAs deep) run under the
    // other's products, and the turns keep the groups half a period apart, so
    // that one's softmax runs under the other's products too (left alone they
    // fell into step: 4250 cycles a page).  Both see every use of every ring
    // stage, pages that only the other tile sees included.
    // Else one warp for both groups: a stage's uses would alternate between two
    // issuers, and a parity does not tell a phase from the one two before it.
    const uint32_t kd0 = static_cast<uint32_t>(umma_desc_sw128(smem_u32(ring)));
    const uint32_t qd0 = static_cast<uint32_t>(umma_desc_sw128(smem_u32(qbase)));
    const uint32_t vd0 = static_cast<uint32_t>(umma_desc_sw128_mn(smem_u32(ring), TILE / 2));
    const uint32_t hi = static_cast<uint32_t>(umma_desc_sw128(0) >> 32);   // the same for all of them
    bool alive = true;
    auto wait1 = [&](uint64_t* bar, uint32_t par) {
      if (alive) alive = __all_sync(0xffffffffu, rows_wait(bar, par, wt));
    };
    int kst = 0, vst = 1;                // ring stages of the next K and V page
    uint32_t kph = 0, vph = 0;           // their parities
    auto ring_step = [&](int& st, uint32_t& ph) {
      st += 2;
      if (st >= NST) {
        st -= NST;
        ph ^= 1u;
      }
    };
    uint32_t pph = 0, qph = 0;           // parities of pfull[s][], of the Q slots (bits)
    uint32_t tph = warp == 9 ? 1 : 0;    // of turn[s]: group 0 begins
    int seq = 0;
    RowsPiece it;
    while (alive && next_piece(it)) {
      const int j0 = it.j0, s0 = TWO ? warp - 9 : 0, e = s0 == 0 ? it.e0 : it.e1;
      const int slot = TWO ? s0 : 0, lead = TWO ? 1 : 2;   // QK runs `lead` pages ahead of PV
      if (j0 < e) {
        wait1(FP8 ? &qconv[slot] : &qfull[slot], (qph >> slot) & 1u);
        qph ^= 1u << slot;
      }
#pragma unroll 1
      for (int j = j0 - lead; j < it.j1 && alive; ++j) {
        const int s = TWO ? s0 : (j - j0) & 1;
        const uint32_t ts = tmem + static_cast<uint32_t>(s * 128);
        const bool page = j >= j0, pv = page && j < e, next = j + lead < it.j1, qk = j + lead < e;
        if (page) {
          wait1(&full[vst], vph);
          if constexpr (!FP8) {
            const int live = it.ctx + it.n - j * kPage;   // V rows past kv_len are zeroed (TWO: by both groups alike)
            if (live < kPage && alive) {
              for (int c = lane; c < (kPage - live) * 8; c += 32)
#pragma unroll
                for (int hb = 0; hb < HB; ++hb)
                  *reinterpret_cast<uint4*>(ring + vst * TILE + hb * (TILE / HB) + live * 128 + c * 16) = make_uint4(0, 0, 0, 0);
              fence_proxy_async_smem();
              __syncwarp();
            }
          }
        }
        if (pv) wait1(&pfull[2 * s], (pph >> s) & 1u);
        if constexpr (TWO) {
          if (next) wait1(&full[kst], kph);
          wait1(&turn[s], tph);
          tph ^= 1u;
        }
        if (!alive) break;
        tc_fence_after();
        if (pv) {
          const uint32_t vd = vd0 + static_cast<uint32_t>(vst * (TILE >> 4));
          umma_pv(ts + TM_O, ts, vd, hi, IDESC_PV, j >= j0 + lead ? 1u : 0u);
          wait1(&pfull[2 * s + 1], (pph >> s) & 1u);
          if (!alive) break;
          tc_fence_after();
          umma_pv(ts + TM_O, ts + 32, vd + 512, hi, IDESC_PV, 1u);
          pph ^= 1u << s;
        }
        const auto release_v = [&] {
          umma_commit_elect(&empty[vst]);
          ring_step(vst, vph);
        };
        if (!TWO && page) release_v();   // (with three stages the next K page takes its place)
        if (!TWO && qk) {   // (bound by the pages' arrival: not ahead of PV)
          wait1(&full[kst], kph);
          if (!alive) break;
          tc_fence_after();
        }
        if (qk) {
          umma_qk<HB>(ts, qd0 + static_cast<uint32_t>(slot * (TILE >> 4)), kd0 + static_cast<uint32_t>(kst * (TILE >> 4)), hi,
                      IDESC_QK);
          umma_commit_elect(&sfull[s]);
        }
        if (TWO && lane == 0) mbar_arrive(&turn[s ^ 1]);
        if (pv && !qk) umma_commit_elect(&odone[s]);
        if (TWO && page) release_v();
        if (next) {
          umma_commit_elect(&empty[kst]);
          if (j + lead == e - 1) umma_commit_elect(&qempty[slot]);
          ring_step(kst, kph);
        }
      }
      ++seq;
    }
    umma_commit_elect(&mdone[warp - 9]);
    if (lane == 0) mbar_drain(&mdone[warp - 9], 0, wt);
    __syncwarp();
  } else if (FP8 && warp >= 12) {
    // -------------------------------------------------- E4M3 codes -> f16 tiles
    // All four warps work on each tile (a tile each would put two waits per
    // stage use out of order).  Sixteen threads take rows r and r ^ 5 of an 8-row block:
    // with the tiles' swizzle (16-byte chunk c of row r at c ^ (r % 8)) every
    // eight lanes' loads and stores then fall into eight different bank groups.
    if constexpr (FP8) {
      constexpr int TT = 32 * kConvertWarps, PER = kRowsTile * 8 / TT;   // 16-byte chunks a thread takes of a tile
      const int ct = tid - 384;
      const int c = (ct & 3) + 4 * ((ct >> 3) & 1), odd = (ct >> 2) & 1 ? 5 : 0, g0 = ct >> 4;
      const int q0 = (c & 3) * 2;
      auto row_of = [&](int k) -> int {
        const int pair = k * (TT / 16) + g0;
        return ((pair >> 2) << 3) + ((pair & 3) ^ odd);
      };
      int rs = 0, st = 0;              // stages of the codes and of the tile
      uint32_t rph = 0, sph = 1;       // parities: codes landed, stage free (the first round is)
      bool ok = true;
      RowsPiece it;
      while (ok && next_piece(it)) {
        for (int x = 2 * it.j0; x < 2 * it.j1; ++x) {
          ok = __all_sync(0xffffffffu, rows_wait(&raw[rs], rph, wt));
          if (!ok) break;
          const uint8_t* src = rring + rs * RAW;
          uint8_t* dst = ring + st * TILE + (c >> 2) * (TILE / 2);
          uint4 v[PER];
#pragma unroll
          for (int k = 0; k < PER; ++k) {
            const int r = row_of(k);
            v[k] = *reinterpret_cast<const uint4*>(src + r * 128 + ((c ^ (r & 7)) << 4));
          }
          const int live = x & 1 ? it.ctx + it.n - (x >> 1) * kPage : kPage;   // V rows past kv_len are zeroed
          if (live < kPage) {
#pragma unroll
            for (int k = 0; k < PER; ++k)
              if (row_of(k) >= live) v[k] = make_uint4(0, 0, 0, 0);
          }
          ok = __all_sync(0xffffffffu, rows_wait(&empty[st], sph, wt));
          if (!ok) break;
#pragma unroll
          for (int k = 0; k < PER; ++k) {
            const int r = row_of(k);
            uint4 a, b;
            e4m3x4_to_f16x4(v[k].x, a.x, a.y);
            e4m3x4_to_f16x4(v[k].y, a.z, a.w);
            e4m3x4_to_f16x4(v[k].z, b.x, b.y);
            e4m3x4_to_f16x4(v[k].w, b.z, b.w);
            *reinterpret_cast<uint4*>(dst + r * 128 + ((q0 ^ (r & 7)) << 4)) = a;
            *reinterpret_cast<uint4*>(dst + r * 128 + (((q0 + 1) ^ (r & 7)) << 4)) = b;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&rawfree[rs]);
            mbar_arrive(&full[st]);
          }
          if (++rs == NRAW) {
            rs = 0;
            rph ^= 1u;
          }
          if (++st == NST) {
            st = 0;
            sph ^= 1u;
          }
        }
      }
    }
  } else if (warp < 8) {   // (one-tile items leave warp 10 idle)
    // ------------------------------------------------- softmax and epilogue
    const int s = warp >> 2;                        // group
    const int r = tid & 127;                        // row of the tile, TMEM lane
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const uint32_t ts = tl + s * 128;               // this row's scores, then its weights
    const int t = r / g.group;                      // token of the tile
    bool dead = false;
    auto wait_all = [&](uint64_t* bar, uint32_t par) {
      if (!dead) dead = __any_sync(0xffffffffu, !mbar_wait(bar, par, wt));
    };
    uint32_t sph = 0, oph = 0, qph = 0;             // parities of sfull[s]; odone[], qfull[] (bits)
    int seq = 0;
    // The piece stays in shared memory until its end (registers hold scores).
    for (;; ++seq) {
      const RowsPiece& it = pieces[seq % kRowsPieces];
      bool got = mbar_wait(&ifull[seq % kRowsPieces], static_cast<uint32_t>(seq / kRowsPieces) & 1u, wt);
      // one-tile items meet at barriers below: all go on, or (a wait of the CTA
      // gave up meanwhile) none
      got = TWO ? __all_sync(0xffffffffu, got) : barrier_all(1, 256, got);
      if (!got) break;
      if (it.j1 == 0) break;
      const int je = s == 0 ? it.e0 : it.e1, ctx = it.ctx;
      const int tok = it.tok0 + (TWO ? s * p.tile_toks : 0) + t;   // of the request
      const bool live = t < p.tile_toks && tok < it.n;
      float scale = p.scale_log2;
      if constexpr (FP8) {
        // Q row -> f16, scaled by a power of two that brings its largest
        // magnitude to [2^14, 2^15).  Where both groups read one tile, both
        // look at the whole row, then convert a half each.  (Loops kept short:
        // unrolled by four, 4 chunks of 1600 tokens take 688 us against 595.)
        const int slot = TWO ? s : 0;
        if (!TWO || je > it.j0) {
          wait_all(&qfull[slot], (qph >> slot) & 1u);
          qph ^= 1u << slot;
          uint8_t* row = qbase + slot * TILE + r * 128;
          float amax = 0.f;
#pragma unroll 2
          for (int c = 0; c < 16; ++c) {
            const uint4 v = *reinterpret_cast<const uint4*>(row + (c >> 3) * (TILE / 2) + (((c & 7) ^ (r & 7)) << 4));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              amax = max3(amax, fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xFFFF0000u)));
          }
          // (rows below 2^-40 are taken as 2^-40: the scale stays a normal number)
          const int e = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -40);
          const float mul = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
          scale *= __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23);
          if (!TWO) named_barrier(1, 256);
#pragma unroll 1
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
      constexpr float LIFT = FP8 ? kRowsLiftF16 : 0.f;
      const float lazy = kRowsLazy / scale;
      const int bound = live ? ctx + tok : -1;      // causal: its last position
      // first position that some row of the tile does not see
      const int open = causal ? ctx + it.tok0 + (TWO ? s * p.tile_toks : 0) + 1 : ctx;
      float m = -INFINITY, negm = LIFT, l = 0.f;    // reference maximum (raw), -m scale + LIFT, sum
      for (int j = TWO ? it.j0 : it.j0 + s; j < je; j += TWO ? 1 : 2) {
        wait_all(&sfull[s], sph);
        sph ^= 1u;
        tc_fence_after();
        const bool masked = j * kPage + kPage > open;   // the page holds positions that some row does not see
        uint32_t w[4] = {0, 0, 0, 0};
        if (masked) {
          if (causal) {
            row_window(bound - j * kPage, w);
          } else {
            uint32_t mw[4];                         // this row's mask: bits below n, none for a dead row
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int bits = live ? it.n - 32 * k : 0;
              mw[k] = bits <= 0 ? 0u
                                : p.tree_mask[(static_cast<int64_t>(it.row0) + tok) * p.mask_words + k] &
                                      (bits >= 32 ? 0xffffffffu : (1u << bits) - 1u);
            }
            tree_window(mw, j * kPage - ctx, w);
          }
        }
        // Chunks of 32 columns; the last two are read first and read again for
        // their exponentials (128 scores in registers spill, and that costs more)
        uint32_t x[2][32];
        float top = -INFINITY;
#pragma unroll (FP8 && TWO ? 1 : 2)   // (rolled: 4 chunks of 1600 tokens over E4M3 583 against 595 us, over bf16 477 against 472)
        for (int half = 1; half >= 0; --half) {
          tmem_ld32_async(ts + 64 * half, x[0]);
          tmem_ld32_async(ts + 64 * half + 32, x[1]);
          tmem_ld_wait_dep(x[0]);
          tmem_ld_wait_dep(x[1]);
          if (masked) {
            row_mask(half ? w[2] : w[0], x[0]);
            row_mask(half ? w[3] : w[1], x[1]);
          }
          top = max3(top, row_max(x[0]), row_max(x[1]));
        }
        if (__any_sync(0xffffffffu, top > m + lazy)) {   // (a row without a maximum yet has m = -inf)
          const bool first = m == -INFINITY;
          const bool grow = top > m + lazy;
          if (grow) m = top;
          const float nn = (m == -INFINITY ? 0.f : -m * scale) + LIFT;
          if (__any_sync(0xffffffffu, grow && !first)) {
            // S ready: the PV before it has retired, O is stable
            const float alpha = grow && !first ? fast_exp2(nn - negm) : 1.f;   // 2^((old m - new m) scale)
            l *= alpha;
#pragma unroll
            for (int c0 = 0; c0 < D; c0 += 8) {
              uint32_t o[8];
              tmem_ld_async(tl + TM_O + s * 128 + c0, o);
              tmem_ld_wait_dep(o);
#pragma unroll
              for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
              tmem_st8(tl + TM_O + s * 128 + c0, o);
            }
          }
          negm = nn;
        }
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        auto hand_over = [&](int h) {
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&pfull[2 * s + h]);
        };
        row_exp<FP8>(ts, 0, x[0], scale, negm, sum[0]);
        row_exp<FP8>(ts, 1, x[1], scale, negm, sum[1]);
        tmem_ld32_async(ts + 64, x[0]);
        tmem_ld32_async(ts + 96, x[1]);
        hand_over(0);
        tmem_ld_wait_dep(x[0]);
        tmem_ld_wait_dep(x[1]);
        if (masked) {
          row_mask(w[2], x[0]);
          row_mask(w[3], x[1]);
        }
        row_exp<FP8>(ts, 2, x[0], scale, negm, sum[0]);
        row_exp<FP8>(ts, 3, x[1], scale, negm, sum[1]);
        hand_over(1);
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }
      // ------------------------------------------------------- end of the piece
      const int j0 = it.j0, j1 = it.j1, np = it.np;
      const bool whole = j0 == 0 && j1 == np;
      const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (j0 == 0 ? 1 : 0);
      constexpr int ROWS = TWO ? 256 : 128;
      // Each thread writes its own row, a sector (32 bytes) a store; 16 columns are
      // read while those before leave.  (This code runs once per piece: it is kept
      // short, its instructions come from far away.)
      const bool f32 = !whole || p.out_f32;
      const bool wide = !whole || (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
      uint8_t* const orow =
          whole ? static_cast<uint8_t*>(p.out) +
                      (static_cast<int64_t>(it.row0 + tok) * g.num_q_heads + it.h * g.group + (r - t * g.group)) * (D * (f32 ? 4 : 2))
                : reinterpret_cast<uint8_t*>(p.ws_o + (slot * ROWS + (TWO ? s * 128 : 0) + r) * D);
      __syncwarp();
      if (lane == 0) mbar_arrive(&iempty[seq % kRowsPieces]);
      // columns [c0, c1) of this row: fetch(c) starts reading 16 columns, take(v) gives them
      auto store = [&](int c0, int c1, const auto& fetch, const auto& take) {
        fetch(c0);
#pragma unroll 1
        for (int c = c0; c < c1; c += 16) {
          float v[16];
          take(v);
          if (c + 16 < c1) fetch(c + 16);
          if (!live) continue;
          if (f32) {
#pragma unroll
            for (int h = 0; h < 16; h += 8) {
              uint32_t w[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(v[h + k]);
              store_sector(orow + c * 4 + h * 4, wide, w);
            }
          } else {
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = pack2<false>(v[2 * k], v[2 * k + 1]);
            store_sector(orow + c * 2, wide, w);
          }
        }
      };
      uint32_t o[16];
      if constexpr (TWO) {
        if (je > j0) {
          wait_all(&odone[s], (oph >> s) & 1u);
          oph ^= 1u << s;
          tc_fence_after();
        }
        const float f = l == 0.f ? 0.f : (whole ? p.v_scale : 1.f) / l;  // a NaN stays one
        const bool none = l == 0.f;   // O may be anything
        store(
            0, D,
            [&](int c) { tmem_ld_async(tl + TM_O + s * 128 + c, o); },
            [&](float (&v)[16]) {
              tmem_ld_wait_dep(o);
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] = none ? 0.f : __uint_as_float(o[k]) * f;
            });
        if (!whole && live) p.ws_lse[slot * ROWS + s * 128 + r] = l == 0.f ? -INFINITY : __log2f(l) - negm;
      } else {
        // both groups' O of this row lie in this lane: exchange maxima and
        // sums, then each group joins and writes half the columns
        xml[s * 128 + r] = make_float2(l == 0.f ? -INFINITY : -negm, l);
        named_barrier(1, 256);
        for (int k = 0; k < min(2, j1 - j0); ++k) {
          wait_all(&odone[k], (oph >> k) & 1u);
          oph ^= 1u << k;
        }
        tc_fence_after();
        const float2 a = xml[r], b = xml[128 + r];
        const float top = fmaxf(a.x, b.x);
        const float wa = a.y == 0.f ? 0.f : fast_exp2(a.x - top), wb = b.y == 0.f ? 0.f : fast_exp2(b.x - top);
        const float lt = wa * a.y + wb * b.y;
        const float f = lt == 0.f ? 0.f : (whole ? p.v_scale : 1.f) / lt;
        const float fa = wa * f, fb = wb * f;   // zero where a group had no weight: its O may be anything
        uint32_t q[16];
        store(
            s * (D / 2), (s + 1) * (D / 2),
            [&](int c) {
              tmem_ld_async(tl + TM_O + c, o);
              tmem_ld_async(tl + TM_O + 128 + c, q);
            },
            [&](float (&v)[16]) {
              tmem_ld_wait_dep(o);
              tmem_ld_wait_dep(q);
#pragma unroll
              for (int k = 0; k < 16; ++k)
                v[k] = (fa == 0.f ? 0.f : __uint_as_float(o[k]) * fa) + (fb == 0.f ? 0.f : __uint_as_float(q[k]) * fb);
            });
        if (!whole && s == 0 && live) p.ws_lse[slot * ROWS + r] = lt == 0.f ? -INFINITY : top + __log2f(lt);
        tc_fence_before();
        named_barrier(1, 256);   // O may be overwritten, the exchange reused
      }
      tc_fence_before();
    }
  }

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
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool FP8, bool TWO, bool LANES>
cudaError_t launch_rows_attn_one(const CUtensorMap& kv_map, const CUtensorMap& q_map, const RowsAttnParams& p,
                                 size_t smem, cudaStream_t st) {
  const void* fn = reinterpret_cast<const void*>(&rows_attn_kernel<D, FP8, TWO, LANES>);
  const cudaError_t e = ensure_smem_attr(fn, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(rows_attn_kernel<D, FP8, TWO, LANES>, dim3(p.num_ctas), dim3(FP8 ? 512 : 384), smem, st, kv_map, q_map, p);
}

// two: 256-row items, in `items` lanes where a tree has more than one a head
template <int D, bool FP8>
cudaError_t launch_rows_attn_kind(bool two, const CUtensorMap& kv_map, const CUtensorMap& q_map, const RowsAttnParams& p,
                                  size_t smem, cudaStream_t st) {
  if (!two) return launch_rows_attn_one<D, FP8, false, false>(kv_map, q_map, p, smem, st);
  return p.items > 1 ? launch_rows_attn_one<D, FP8, true, true>(kv_map, q_map, p, smem, st)
                     : launch_rows_attn_one<D, FP8, true, false>(kv_map, q_map, p, smem, st);
}

}  // namespace trtv
