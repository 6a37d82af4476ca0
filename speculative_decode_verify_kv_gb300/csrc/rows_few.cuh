// rows_few.cuh -- attention of few rows over E2M1 caches: decoding, verify steps
// and small trees, at most 16 MT rows (tokens x query heads of one KV head).
//
// A page's K and V are 18 KB of codes and scales against 64 KB in 16 bits, so
// what matters is that nothing else passes through shared memory: a warp turns
// the codes of 16 positions into the registers of its matrix fragments
// (mma.sync m16n8k16, f16 operands, fp32 sums) and keeps scores, weights and
// the output in registers.  Written out to shared memory for tcgen05, a page's
// tiles cost 512 cycles of stores and as many of reads, above the 800 that its
// bytes take to arrive at the SM's share of the copy rate; an E2M1 conversion,
// a permute and a product of f16 pairs take 2 cycles each per warp, 5 of them
// per 4 elements.
//
// Fragments.  The order of the head dims inside QK^T, of the positions inside a
// slice and of the columns of O is free as long as both operands agree, so each
// lane reads what lies together: of a key a quarter of its dims (lane % 4), of a
// value an eighth (lane / 4), whole scale blocks in both.  S = Q K^T leaves the
// weights where P V wants its A operand.  Of 16 positions, column n of half i is
// row 8 i + n / 2 + 4 (n % 2): lanes of one load then read neighbouring rows.
// The code's scale is a factor of its f16 value, exact (see rows_attn.cuh).
//
// Each consumer warp has a running maximum, sum and O of its own over the slices
// that it takes of each page (every SETS-th page of the CTA is its).  At the end of
// a piece it leaves them in shared memory and goes on with the next; two merging
// warps join them in the warps' order and write the rows, under the next piece's
// pages.  Another warp prepares the next piece's Q: f16 in the order of the
// fragments.  So a piece costs the consumers little more than its pages (joined
// by all warps at a barrier, with Q loaded by each: 5.4 us a piece against 0.6 a
// page, 64 requests' decoding 68 us).
// Work split, pieces, the join between CTAs and the refusals are rows_attn.cuh's,
// with one item per (request, KV head).
#pragma once

#include "rows_attn.cuh"

namespace trtv {

constexpr int kFewLeast = 256;       // positions that a CTA takes at least

constexpr int kFewMergers = 2;       // merging warps

// Consumer warps, in whole warpgroups, tiles of 8 positions that one takes at a
// time, and whether Q's fragments stay in its registers.
constexpr int few_warps(int D, int MT) { return MT == 1 || D == 64 ? 12 : 8; }
constexpr int few_tiles(int D, int MT) { return 4; }
constexpr bool few_q_regs(int D, int MT) { return MT == 1; }
constexpr int few_threads(int D, int MT) { return 32 * few_warps(D, MT) + 128; }
constexpr int few_q_bytes(int D, int MT) { return MT * (D / 16) * 512 + MT * 64; }   // fragments and scales of a piece

// (not volatile: the compiler may move it among what it does not depend on)
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) { return pack2<true>(lo, hi); }

template <int REGS, bool INC>
__device__ __forceinline__ void set_registers() {
  if constexpr (INC) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

template <int D, int MT>
__global__ void __launch_bounds__(few_threads(D, MT), 1)
    rows_few_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ RowsAttnParams p) {
  constexpr int CW = few_warps(D, MT);
  constexpr int BLOCK = kFp4Row * D;           // bytes of 32 rows of a head
  constexpr int HALF = kGroups * BLOCK;        // a page's K (or V)
  constexpr int KW = D / 32;                   // words of codes that a lane takes of a key
  constexpr int VW = D / 64;                   // and of a value
  constexpr int NT = D / 8;                    // n-tiles of O
  constexpr int HT = few_tiles(D, MT);         // tiles of 8 positions that a warp takes at a time
  constexpr int UPP = kPage / (8 * HT);        // of which a page has
  constexpr int SETS = CW / UPP;               // pages at a time
  constexpr bool QREG = few_q_regs(D, MT);
  static_assert(CW % UPP == 0 && HT % 2 == 0, "whole pages");
  const RowsGeom& g = p.g;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int NST = p.nst;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.off_bar);   // [NST] page landed
  uint64_t* empty = full + NST;                                     // [NST] its slices done
  uint64_t* ifull = empty + NST;                                    // [kRowsPieces] piece scheduled
  uint64_t* iempty = ifull + kRowsPieces;                           // [kRowsPieces] every role has read it
  uint64_t* qfull = iempty + kRowsPieces;                           // [2] Q ready
  uint64_t* qempty = qfull + 2;                                     // [2] and done with
  uint64_t* mfull = qempty + 2;                                     // every consumer's share of a piece is there
  uint64_t* mempty = mfull + 1;                                     // and joined
  int* abortf = reinterpret_cast<int*>(mempty + 1);
  const Waits wt{g.err, abortf, p.wait_ns};
  int64_t* scan = reinterpret_cast<int64_t*>(smem + p.off_scan);
  RowsPiece* pieces = reinterpret_cast<RowsPiece*>(smem + p.off_pieces);
  uint8_t* ring = smem + p.off_ring;
  uint8_t* qbuf = smem + p.off_q;                                   // [2] fragments, then scales
  float2* xml = reinterpret_cast<float2*>(smem + p.off_ml);         // [CW][16 MT] {reference maximum, sum}
  float4* share = reinterpret_cast<float4*>(smem + p.off_raw);      // [CW][16 MT][D / 4] O of each consumer
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool causal = p.tree_mask == nullptr;
  // (chunk c of row r of O lies at c ^ swz: a warp's stores and loads fall into different banks)
  auto swz = [](int r, int c) { return c ^ ((c >> (D == 128 ? 3 : 2)) | (r & 1) << 2); };

  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], UPP);
    }
    for (int i = 0; i < kRowsPieces; ++i) {
      mbar_init(&ifull[i], 1);
      mbar_init(&iempty[i], CW + 1 + kFewMergers);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&qfull[i], 1);
      mbar_init(&qempty[i], CW);
    }
    mbar_init(mfull, CW);
    mbar_init(mempty, kFewMergers);
    *abortf = 0;
    fence_mbar_init();
  }
  pdl_wait();   // inputs may come from the previous kernel of the stream
  int requests;
  rows_scan<false>(p, p.tile_toks, causal, 1, scan, scan + g.batch + 1, requests);
  pdl_trigger();
  const int64_t W = scan[g.batch];
  int64_t P = max(int64_t{1}, min(static_cast<int64_t>(p.num_ctas), W / kFewLeast));
  if (P < p.num_ctas && P > g.num_kv_heads) P -= static_cast<int>(P) % g.num_kv_heads;   // (see rows_attn.cuh)
  const int64_t u0 = rows_begin(blockIdx.x, W, P), u1 = rows_begin(static_cast<int64_t>(blockIdx.x) + 1, W, P);
  __syncthreads();

  if (u0 >= u1) {
    if (tid == 0) {
      p.splits[blockIdx.x].b = -1;
      p.cont[blockIdx.x] = 0;
    }
  } else if (warp >= CW) {
    // ------------------------------------------------------------ producers
    set_registers<56, false>();
    if (warp == CW) {
      // page loads
      const uint64_t pol = policy_evict_first();
      if (lane == 0) prefetch_tensormap(&kv_map);
      int at = 0;
      uint32_t ph = 0;
      RowsPiece it{};
      auto ids_of = [&](int j) -> int {
        int s = 0;
        if (j + lane < it.j1) {
          s = g.page_table[static_cast<int64_t>(it.b) * g.max_pages + j + lane];
          if (s < 0 || s >= g.num_slots) {
            atomicOr(g.err, TRTV_DEVERR_PAGE_ID);
            s = 0;
          }
        }
        return s;
      };
      int i = 0, st = 0;   // pages so far, ring stage
      uint32_t eph = 1;    // parity of empty[st] (the first round is free)
      bool ok = true, stop = false;
      while (ok && !stop) {
        if (!__all_sync(0xffffffffu, mbar_wait(&ifull[at], ph, wt))) break;
        it = pieces[at];
        __syncwarp();
        if (lane == 0) mbar_arrive(&iempty[at]);
        if (++at == kRowsPieces) {
          at = 0;
          ph ^= 1u;
        }
        if (it.j1 == 0) break;
        int base = it.j0, ids = ids_of(base), ahead = base + 32 < it.j1 ? ids_of(base + 32) : 0;
        for (int j = it.j0; j < it.j1 && ok; ++j) {
          if (j >= base + 32) {
            base += 32;
            ids = ahead;
            ahead = base + 32 < it.j1 ? ids_of(base + 32) : 0;
          }
          const int64_t sub = static_cast<int64_t>(__shfl_sync(0xffffffffu, ids, j - base)) * g.slot_stride * kGroups;
          stop = p.withhold >= 0 && i >= p.withhold;   // tests of the give-up path only
          if (stop) break;
          ok = __all_sync(0xffffffffu, mbar_wait(&empty[st], eph, wt));
          if (!ok) break;
          if (lane == 0) {   // (V's buffer follows K's: one box has both)
            mbar_arrive_expect_tx(&full[st], 2 * HALF);
            tma_load_blocks<true>(ring + st * 2 * HALF, &kv_map, &full[st], it.h, static_cast<int>(sub), pol);
          }
          ++i;
          if (++st == NST) {
            st = 0;
            eph ^= 1u;
          }
        }
      }
      // never leave copies in flight
      if (lane == 0)
        for (int k = max(0, i - NST); k < i; ++k) mbar_drain(&full[k % NST], static_cast<uint32_t>(k / NST) & 1u, wt);
      __syncwarp();
    } else if (warp == CW + 1) {
      // schedule, and Q
      const RowsWalk<false> walk{p, scan, p.tile_toks, causal, -1};
      RowsItem it = walk.at(u0, lane);
      bool split = false;   // this CTA holds the first page of a cut item
      int seq = 0;
      for (;; ++seq) {
        RowsPiece x{};
        if (lane == 0) {
          for (; it.valid && it.u < u1; walk.next(it)) {
            walk.piece(it, u0, u1, x.j0, x.j1);
            if (x.j0 < x.j1) break;
            x.j1 = 0;
          }
          if (x.j1 > 0) {
            x.row0 = it.row0;
            x.n = it.n;
            x.ctx = it.ctx;
            x.np = walk.item_pages(it);
            x.h = it.h;
            x.b = it.b;
          }
        }
        const int k = seq % kRowsPieces;
        bool ok = true;
        if (seq >= kRowsPieces) ok = __all_sync(0xffffffffu, mbar_wait(&iempty[k], static_cast<uint32_t>(seq / kRowsPieces - 1) & 1u, wt));
        if (!ok) break;
        if (lane == 0) {
          pieces[k] = x;
          mbar_arrive(&ifull[k]);
          if (x.j1 > 0) {
            // what the join needs to know
            if (seq == 0) p.cont[blockIdx.x] = x.j0 > 0;
            if (x.j0 == 0 && x.j1 < x.np) {
              RowsSplit d{};
              d.b = x.b;
              d.h = x.h;
              d.n = x.n;
              d.row0 = x.row0;
              d.c_last = static_cast<int>(cta_of_unit(it.u + p.setup + static_cast<int64_t>(x.np - 1) * kPage, W, P));
              d.stride = 1;
              p.splits[blockIdx.x] = d;
              split = true;
            }
            walk.next(it);
          }
        }
        if (__shfl_sync(0xffffffffu, x.j1, 0) == 0) break;
        const int n = __shfl_sync(0xffffffffu, x.n, 0), row0 = __shfl_sync(0xffffffffu, x.row0, 0), h = __shfl_sync(0xffffffffu, x.h, 0);
        const int sl = seq & 1;
        if (seq >= 2) ok = __all_sync(0xffffffffu, mbar_wait(&qempty[sl], static_cast<uint32_t>(seq / 2 - 1) & 1u, wt));
        if (!ok) break;
        const int gi = lane >> 2, t = lane & 3;
        uint4* frag = reinterpret_cast<uint4*>(qbuf + sl * few_q_bytes(D, MT));
        float* qscale = reinterpret_cast<float*>(qbuf + sl * few_q_bytes(D, MT) + MT * (D / 16) * 512);
#pragma unroll 1
        for (int a = 0; a < MT; ++a) {
          uint32_t v[2][D / 8];   // rows gi and gi + 8 of the tile, this lane's quarter
#pragma unroll
          for (int k2 = 0; k2 < 2; ++k2) {
            const int r = gi + 8 * k2 + 16 * a, tk = r / g.group;
            const uint4* src = reinterpret_cast<const uint4*>(
                p.q + ((static_cast<int64_t>(row0) + tk) * g.num_q_heads + h * g.group + (r - tk * g.group)) * D + t * (D / 4));
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
              const uint4 w = tk < n ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
              v[k2][4 * i] = w.x; v[k2][4 * i + 1] = w.y; v[k2][4 * i + 2] = w.z; v[k2][4 * i + 3] = w.w;
            }
          }
#pragma unroll
          for (int k2 = 0; k2 < 2; ++k2) {
            // a power of two that brings the row's largest magnitude to [2^14, 2^15)
            // (rows below 2^-40 are taken as 2^-40: the scale stays a normal number)
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
              amax = max3(amax, fabsf(__uint_as_float(v[k2][i] << 16)), fabsf(__uint_as_float(v[k2][i] & 0xFFFF0000u)));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            const int e = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -40);
            const float mul = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
            if (t == 0) qscale[gi + 8 * k2 + 16 * a] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23);
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
              v[k2][i] = pack_f16(__uint_as_float(v[k2][i] << 16) * mul, __uint_as_float(v[k2][i] & 0xFFFF0000u) * mul);
          }
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            frag[(a * (D / 16) + ks) * 32 + lane] = make_uint4(v[0][2 * ks], v[1][2 * ks], v[0][2 * ks + 1], v[1][2 * ks + 1]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&qfull[sl]);
      }
      if (lane == 0) {
        if (!split) p.splits[blockIdx.x].b = -1;
        if (seq == 0) p.cont[blockIdx.x] = 0;   // no page starts in its units
      }
    } else {
      // joining the consumers' shares: a row at a time, its columns over the lanes
      const int mw = warp - CW - 2;
      constexpr int C4 = D / 4;   // 16-byte chunks of a row
      constexpr int RPW = 32 / C4;   // rows at a time (head_dim 64: two)
      const int c = lane % C4, rr = lane / C4;
      for (int seq = 0;; ++seq) {
        const int k = seq % kRowsPieces;
        if (!__all_sync(0xffffffffu, mbar_wait(&ifull[k], static_cast<uint32_t>(seq / kRowsPieces) & 1u, wt))) break;
        const int n = pieces[k].n, row0 = pieces[k].row0, h = pieces[k].h, j0 = pieces[k].j0, j1 = pieces[k].j1;
        const bool whole = j0 == 0 && j1 == pieces[k].np;
        __syncwarp();
        if (lane == 0) mbar_arrive(&iempty[k]);
        if (j1 == 0) break;
        if (!__all_sync(0xffffffffu, mbar_wait(mfull, static_cast<uint32_t>(seq) & 1u, wt))) break;
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (j0 == 0 ? 1 : 0);
        const int rows = n * g.group;
        // a consumer's factor for a row, in place of its maximum: a row per lane
        for (int r = mw * RPW + lane % RPW + lane / RPW * kFewMergers * RPW; r < rows; r += kFewMergers * 32) {
          float top = -INFINITY, lt = 0.f;
          float2 x[CW];
#pragma unroll
          for (int w = 0; w < CW; ++w) x[w] = xml[w * 16 * MT + r];
#pragma unroll
          for (int w = 0; w < CW; ++w) top = fmaxf(top, x[w].y == 0.f ? -INFINITY : x[w].x);
#pragma unroll
          for (int w = 0; w < CW; ++w) {
            x[w].x = x[w].y == 0.f ? 0.f : fast_exp2(x[w].x - top);
            lt += x[w].x * x[w].y;
          }
          const float f = lt == 0.f ? 0.f : (whole ? p.v_scale : 1.f) / lt;   // a NaN stays one
#pragma unroll
          for (int w = 0; w < CW; ++w) xml[w * 16 * MT + r].x = x[w].x * f;
          if (!whole) p.ws_lse[slot * 16 * MT + r] = lt == 0.f ? -INFINITY : top + __log2f(lt);
        }
        __syncwarp();
        for (int r0 = mw * RPW; r0 < rows; r0 += kFewMergers * RPW) {
          const int r = min(r0 + rr, 16 * MT - 1), tk = r / g.group;   // (beyond the rows: read, not written)
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w0 = 0; w0 < CW; w0 += 4) {
            float f[4];
            float4 v[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              f[w] = xml[(w0 + w) * 16 * MT + r].x;
              v[w] = share[((w0 + w) * 16 * MT + r) * C4 + swz(r, c)];
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              if (f[w] == 0.f) v[w] = make_float4(0.f, 0.f, 0.f, 0.f);   // no weight: its O may be anything
              a.x += f[w] * v[w].x; a.y += f[w] * v[w].y; a.z += f[w] * v[w].z; a.w += f[w] * v[w].w;
            }
          }
          if (r0 + rr >= rows) continue;
          if (!whole) {
            *reinterpret_cast<float4*>(p.ws_o + (slot * 16 * MT + r) * D + 4 * c) = a;
          } else {
            const int64_t at = (static_cast<int64_t>(row0 + tk) * g.num_q_heads + h * g.group + (r - tk * g.group)) * D + 4 * c;
            if (p.out_f32) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = a;
            else
              *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at) = make_uint2(pack2<false>(a.x, a.y), pack2<false>(a.z, a.w));
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(mempty);
      }
    }
  } else {
    // ------------------------------------------------------------ consumers
    set_registers<CW == 12 ? 152 : 224, true>();
    const int gi = lane >> 2, t = lane & 3;       // fragment row (or column), and place in it
    constexpr float LIFT = kRowsLiftF16;
    const int kpos = (gi >> 1) + 4 * (gi & 1);    // this lane's key of a half slice
    const int slice = warp % UPP, set = warp / UPP;   // its positions of a page, its pages
    int seq = 0, page0 = 0;                       // pieces and pages before this one
    int st = 0, at0 = 0;                          // ring stage of the CTA's page at0
    uint32_t ph = 0;                              // and its parity
    bool dead = false;
    for (; !dead; ++seq) {
      const int pk = seq % kRowsPieces;
      if (!__all_sync(0xffffffffu, mbar_wait(&ifull[pk], static_cast<uint32_t>(seq / kRowsPieces) & 1u, wt))) break;
      const int ctx = pieces[pk].ctx, n = pieces[pk].n, row0 = pieces[pk].row0, len = ctx + n, j0 = pieces[pk].j0, j1 = pieces[pk].j1;
      __syncwarp();
      if (lane == 0) mbar_arrive(&iempty[pk]);
      if (j1 == 0) break;
      const int qs = seq & 1;
      const uint4* frag = reinterpret_cast<const uint4*>(qbuf + qs * few_q_bytes(D, MT)) + lane;
      const float* qscale = reinterpret_cast<const float*>(qbuf + qs * few_q_bytes(D, MT) + MT * (D / 16) * 512);
      if (!__all_sync(0xffffffffu, mbar_wait(&qfull[qs], static_cast<uint32_t>(seq / 2) & 1u, wt))) break;
      uint4 q[QREG ? MT : 1][QREG ? D / 16 : 1];
      if constexpr (QREG) {
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) q[a][ks] = frag[(a * (D / 16) + ks) * 32];
      }
      // rows of this lane: gi + 8 k, k < 2 MT
      float scale[2 * MT], negm[2 * MT], lim[2 * MT], l[2 * MT];   // negm: LIFT - maximum scale; lim: when the maximum moves
#pragma unroll
      for (int k = 0; k < 2 * MT; ++k) {
        scale[k] = qscale[gi + 8 * k];
        lim[k] = -INFINITY;
        negm[k] = LIFT;
        l[k] = 0.f;
      }
      if constexpr (QREG) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&qempty[qs]);
      }
      float o[MT][NT][4];
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int b = 0; b < NT; ++b)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[a][b][c] = 0.f;
      const int open = causal ? ctx + 1 : ctx;   // first position that some row does not see

      // (this warp's pages: every SETS-th of the CTA's, so that short pieces spread evenly)
      int j = j0 + (set - page0 % SETS + SETS) % SETS;
      st += j - j0 - (at0 - page0);   // from the page that it stood at
      while (st >= NST) {
        st -= NST;
        ph ^= 1u;
      }
#pragma unroll 1
      for (; j < j1; j += SETS) {
        const int pos0 = j * kPage + slice * (8 * HT);
        dead = __any_sync(0xffffffffu, !mbar_wait(&full[st], ph, wt));
        if (dead) break;
        if (pos0 < len) {
          const uint8_t* kb = ring + st * 2 * HALF + slice * (8 * HT) / kSub * BLOCK;
          const uint8_t* vb = kb + HALF;
          constexpr int IN = kSub / (8 * HT);       // units of a 32-row block
          const int r0 = IN == 1 ? 0 : slice % IN * (8 * HT);
          const bool masked = pos0 + 8 * HT > open;
          // ---- S = Q K^T
          float s[MT][HT][4];
          uint32_t kw[HT][KW], ks[HT][2];
#pragma unroll
          for (int i = 0; i < HT; ++i) {
            const int r = r0 + 8 * i + kpos;
            if constexpr (KW == 4) {
              const uint4 v = *reinterpret_cast<const uint4*>(kb + r * (D / 2) + t * 16);
              kw[i][0] = v.x; kw[i][1] = v.y; kw[i][2] = v.z; kw[i][3] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(kb + r * (D / 2) + t * 8);
              kw[i][0] = v.x; kw[i][1] = v.y;
            }
            const uint32_t two = e4m3x2_to_f16x2_reg(
                D == 128 ? *reinterpret_cast<const uint16_t*>(kb + kSub * (D / 2) + r * (D / 16) + t * 2)
                         : kb[kSub * (D / 2) + r * (D / 16) + t]);
            ks[i][0] = __byte_perm(two, 0, 0x1010);
            ks[i][1] = __byte_perm(two, 0, 0x3232);
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
              for (int c = 0; c < 4; ++c) s[a][i][c] = 0.f;
          }
#pragma unroll
          for (int x = 0; x < KW; ++x) {
            uint32_t b[HT][4];
#pragma unroll
            for (int i = 0; i < HT; ++i) {
              e2m1x8_to_f16x8(kw[i][x], b[i]);
#pragma unroll
              for (int e = 0; e < 4; ++e) b[i][e] = mul_f16x2(b[i][e], ks[i][D == 128 ? x >> 1 : 0]);
            }
            // (sums of different tiles in turn: each waits for its last product)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int a = 0; a < MT; ++a) {
                uint4 f;
                if constexpr (QREG) f = q[a][2 * x + e];
                else f = frag[(a * (D / 16) + 2 * x + e) * 32];
                const uint32_t fa[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                for (int i = 0; i < HT; ++i) mma_f16(s[a][i], fa, b[i][2 * e], b[i][2 * e + 1]);
              }
          }
          if (masked) {
#pragma unroll
            for (int k = 0; k < 2 * MT; ++k) {
              const int tok = (gi + 8 * k) / g.group;
              const uint32_t* mask = causal ? nullptr : p.tree_mask + (static_cast<int64_t>(row0) + tok) * p.mask_words;
#pragma unroll
              for (int i = 0; i < HT; ++i)
#pragma unroll
                for (int c = 0; c < 2; ++c) {   // column 2 t + c of tile i
                  const int rel = pos0 + 8 * i + t + 4 * c - ctx;
                  bool see = tok < n;
                  if (see && rel >= 0) see = causal ? rel <= tok : rel < n && (mask[rel >> 5] >> (rel & 31) & 1u);
                  if (!see) s[k >> 1][i][2 * (k & 1) + c] = -INFINITY;
                }
            }
          }
          // ---- weights
          bool grow = false;
          float top[2 * MT];
#pragma unroll
          for (int k = 0; k < 2 * MT; ++k) {
            const int c = 2 * (k & 1);
            top[k] = fmaxf(s[k >> 1][0][c], s[k >> 1][0][c + 1]);
#pragma unroll
            for (int i = 1; i < HT; ++i) top[k] = max3(top[k], s[k >> 1][i][c], s[k >> 1][i][c + 1]);
            grow |= top[k] > lim[k];
          }
          if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int k = 0; k < 2 * MT; ++k) {
              float x = top[k];
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
              if (x > lim[k]) {   // (the same for the row's four lanes)
                const float to = LIFT - x * scale[k];
                const float alpha = lim[k] == -INFINITY ? 1.f : fast_exp2(to - negm[k]);
                lim[k] = x + kRowsLazy / scale[k];
                negm[k] = to;
                l[k] *= alpha;
#pragma unroll
                for (int b = 0; b < NT; ++b) {
                  o[k >> 1][b][2 * (k & 1)] *= alpha;
                  o[k >> 1][b][2 * (k & 1) + 1] *= alpha;
                }
              }
            }
          }
          uint32_t pw[MT][HT / 2][4];
#pragma unroll
          for (int k = 0; k < 2 * MT; ++k)
#pragma unroll
            for (int i = 0; i < HT; ++i) {
              const float a = fast_exp2(fmaf(s[k >> 1][i][2 * (k & 1)], scale[k], negm[k]));
              const float b = fast_exp2(fmaf(s[k >> 1][i][2 * (k & 1) + 1], scale[k], negm[k]));
              l[k] += a + b;
              pw[k >> 1][i >> 1][(k & 1) + 2 * (i & 1)] = pack2_f16_sat(a, b);
            }
          // ---- O += P V, 16 positions at a time
#pragma unroll
          for (int hh = 0; hh < HT / 2; ++hh) {
            uint32_t w[4][VW], sc[4];
#pragma unroll
            for (int a = 0; a < 4; ++a) {
              const int r = r0 + 16 * hh + 4 * a + t;
              if constexpr (VW == 2) {
                const uint2 v = *reinterpret_cast<const uint2*>(vb + r * (D / 2) + gi * 8);
                w[a][0] = v.x; w[a][1] = v.y;
                sc[a] = vb[kSub * (D / 2) + r * (D / 16) + gi];
              } else {
                w[a][0] = *reinterpret_cast<const uint32_t*>(vb + r * (D / 2) + gi * 4);
                sc[a] = vb[kSub * (D / 2) + r * (D / 16) + (gi >> 1)];
              }
              if (masked && pos0 + 16 * hh + 4 * a + t >= len) {   // (zero weights times what lies there)
#pragma unroll
                for (int x = 0; x < VW; ++x) w[a][x] = 0;
                sc[a] = 0;
              }
            }
            const uint32_t s01 = e4m3x2_to_f16x2_reg(sc[0] | sc[1] << 8), s23 = e4m3x2_to_f16x2_reg(sc[2] | sc[3] << 8);
#pragma unroll
            for (int x = 0; x < VW; ++x) {
              uint32_t v[4][4];
#pragma unroll
              for (int a = 0; a < 4; ++a) e2m1x8_to_f16x8(w[a][x], v[a]);
#pragma unroll
              for (int e = 0; e < 4; ++e) {   // dims 8 x + 2 e and the next of this lane's
                const uint32_t b00 = mul_f16x2(__byte_perm(v[0][e], v[1][e], 0x5410), s01);
                const uint32_t b01 = mul_f16x2(__byte_perm(v[2][e], v[3][e], 0x5410), s23);
                const uint32_t b10 = mul_f16x2(__byte_perm(v[0][e], v[1][e], 0x7632), s01);
                const uint32_t b11 = mul_f16x2(__byte_perm(v[2][e], v[3][e], 0x7632), s23);
#pragma unroll
                for (int a = 0; a < MT; ++a) {
                  mma_f16(o[a][8 * x + 2 * e], pw[a][hh], b00, b01);
                  mma_f16(o[a][8 * x + 2 * e + 1], pw[a][hh], b10, b11);
                }
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        st += SETS;
        if (st >= NST) {
          st -= NST;
          ph ^= 1u;
        }
      }
      if (dead) break;
      at0 = page0 + (j - j0);   // the page that st stands at
      page0 += j1 - j0;
      if constexpr (!QREG) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&qempty[qs]);
      }
      // ------------------------------------------------------- end of the piece
      if (seq > 0 && !__all_sync(0xffffffffu, mbar_wait(mempty, static_cast<uint32_t>(seq - 1) & 1u, wt))) break;
#pragma unroll
      for (int k = 0; k < 2 * MT; ++k) {
        const int r = gi + 8 * k;
        l[k] += __shfl_xor_sync(0xffffffffu, l[k], 1);
        l[k] += __shfl_xor_sync(0xffffffffu, l[k], 2);
        if (t == 0) xml[warp * 16 * MT + r] = make_float2(-negm[k], l[k]);
        // column 2 t + c of n-tile b is dim (D / 8) (2 t + c) + b
        float4* row = share + (warp * 16 * MT + r) * (D / 4);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int b = 0; b < NT; b += 4) {
            const int e = 2 * (k & 1) + c;
            row[swz(r, (2 * t + c) * (D / 32) + b / 4)] =
                make_float4(o[k >> 1][b][e], o[k >> 1][b + 1][e], o[k >> 1][b + 2][e], o[k >> 1][b + 3][e]);
          }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(mfull);
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
}

}  // namespace trtv
