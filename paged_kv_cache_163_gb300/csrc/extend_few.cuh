// Attention of few new tokens of each sequence over its paged cache: single
// tokens and drafted ones, a few query rows of a KV head.
//
// Same mathematics, items, shares, partials and merge as the kernel for many
// tokens; what differs is the product unit.  With 8 to 32 rows a 128-row tile
// is mostly padding, and its chain of copy, conversion, product, softmax and
// product through barriers sets the time (99 us for one token of 16 sequences
// with a 4096-token window over an E4M3 cache, 34 here; the bytes alone are
// 20).  Here a warp does all of a 16-token block by itself:
//   S^T[16 tokens x 8 rows] = K[16 x D] . Q^T[D x 8],  O^T[D x 8] += V^T P^T
// with mma.sync m16n8k16, the block's codes turned into f16 fragments in
// registers, so nothing but the copies goes through shared memory.  What bounds
// it: over long contexts the cache's bytes (16-bit: 6.1 TB/s beside a fixed 15 us)
// or the instructions on codes (E4M3: 5.2 TB/s, two warps a scheduler at one
// instruction in 2.5 cycles; 12 or 16 warps with fewer registers were no
// faster), over short ones the chain plan, table, copies, join (11 us).
//
// Eight warps share a 128-token step, a block each (two at once over coded
// caches, to overlap two chains: 78 -> 74 us for 16 x 8192 tokens), and
// every warp keeps its own ring of copies in flight (cp.async, chunks permuted
// so that fragment loads meet no bank twice; the head_dim order inside the
// products is whatever those loads give, the same for K and Q).  At a piece's
// end the warps' partial rows are joined through shared memory.  Rows beyond
// 8 NR of an item repeat its blocks.  A batch with no more items than CTAs is
// not cut when that costs more (kCut: 74 -> 68 us there, 27 -> 19 us for 1024 tokens).
#pragma once

#include "extend.cuh"
#include "decode_mma.cuh"
#include "extend_few.h"

namespace pkv {

template <int D, int CDT, int QDT, int NR>
struct FewCfg {
  static constexpr int KT = k_part(CDT), VT = v_part(CDT);
  static constexpr bool kCoded = is_coded(KT);
  static constexpr bool kInt4V = VT == kInt4;
  static constexpr bool kBf16 = !kCoded && QDT == PKV_BF16;  // operand type of the products, else f16
  static constexpr bool kCvtQ = kCoded && QDT == PKV_BF16;   // queries become f16, times a power of two a row
  static constexpr int PT = kBf16 ? PKV_BF16 : PKV_F16;
  static constexpr int kWarps = 8, kThreads = 256;
  static constexpr int kRows = 8 * NR;
  static constexpr int kKRow = D * (kCoded ? 1 : 2);        // bytes of a token's K, and of its V
  static constexpr int kVRow = kInt4V ? D / 2 : kKRow;
  static constexpr int kOffV = kBS * kKRow;
  static constexpr int kOffS = kOffV + kBS * kVRow;         // K scales, V scales
  static constexpr int kStage = kOffS + (kCoded ? 128 : 0);
  static constexpr int kJoinRows = NR == 1 ? 8 : 16;        // rows joined at a time
  static constexpr int kJoinRow = D + 4;                    // floats; padded against bank conflicts
  static constexpr int kOffQ = 0;                           // fragments [D / 16][NR][32 lanes] of 8 bytes
  static constexpr int kOffBack = kOffQ + kRows * D * 2;    // [rows] inverse of the query's power of two
  static constexpr int kOffMl = kOffBack + kRows * 4;       // [warps][rows] (m, l)
  static constexpr int kOffMisc = kOffMl + kWarps * kRows * 8;  // start of the share, merge flag
  static constexpr int kOffJoin = round_up_c(kOffMisc + 128, 128);
  static constexpr int kOffRing = round_up_c(kOffJoin + kWarps * kJoinRows * kJoinRow * 4, 128);
  static constexpr int kFit = (232448 - kOffRing) / (kWarps * kStage);
  static constexpr int kStages = kFit < 6 ? kFit : 6;
  // Blocks a warp computes at once: two with one group of rows, where one block's
  // chain of dependent steps leaves the warp idle.
  static constexpr int kBlocks = NR == 1 && kStages >= 4 ? 2 : 1;
  // What cutting an item costs, in 128-token steps: the second piece's start,
  // the count and the merge, some 17000 cycles together, in which the SM's share
  // of the memory bandwidth brings about 360 KB.
  static constexpr int kCut = 360 * 1024 / (128 * (kKRow + kVRow));
  static constexpr int kSmem = kOffRing + kWarps * kStages * kStage;
  // A reference may lag the largest score by 2^7; over coded caches P carries
  // the V scales relative to a power of two at or above them, times 2^8: at most 2^15.
  static constexpr float kLag = 7.f;
  static constexpr float kPTop = 256.f;
  static_assert(kStages >= 2, "a block in flight while another is computed");
  static_assert(kWarps * kStages * kStage >= (PKV_MAX_SEQS_PER_CALL + 1) * 8, "the plan's sums fit the ring");
  static_assert(sizeof(ExtStart) <= 96, "start of the share");
};

// Byte of 16-byte chunk c of row r in a block's shared-memory image with CH
// chunks a row: chunks are permuted within 128-byte lines so that the eight
// (or sixteen, of 8 bytes) lanes of a fragment load meet different banks.
template <int CH>
__device__ __forceinline__ int few_at(int r, int c) {
  const int l = r * CH + c;
  const int x = CH >= 8 ? r & 7 : CH == 4 ? (2 * (r >> 1)) & 7 : 2 * ((r >> 2) & 1);
  return ((l & ~7) | ((l & 7) ^ x)) * 16;
}

// 16 bytes to shared memory without a register; zeros when !there.
__device__ __forceinline__ void few_copy(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0)
               : "memory");
}

// A warp's blocks of a piece: from, from + 8 .. before `to`, `passes` times.
struct FewPiece {
  const int32_t *table;
  int kvh, near, gap, from, to, passes, more;
};
// The walk's piece (with `next`, the following one) or the first after it that has blocks for this warp.
template <int ROWS>
__device__ __noinline__ FewPiece few_piece(ExtWalk *w, int warp, bool next) {
  FewPiece a = {};
  for (;; next = true) {
    if (next) w->next();
    if (!w->more()) return a;
    a.from = 8 * w->j0 + warp;
    a.to = min(8 * w->j1, w->it.blocks);
    if (a.from < a.to) break;
  }
  a.table = w->p.block_tables + static_cast<int64_t>(w->b) * w->p.max_blocks_per_seq;
  a.kvh = w->kvh;
  a.near = w->it.near;
  a.gap = w->it.gap;
  a.passes = (w->rows() + ROWS - 1) / ROWS;
  a.more = 1;
  return a;
}

template <int D, int CDT, int QDT, int NR>
__global__ void __launch_bounds__(256, 1) paged_extend_few_kernel(const __grid_constant__ ExtendParams p) {
  using C = FewCfg<D, CDT, QDT, NR>;
  constexpr int S = C::kStages;
  constexpr int NB = C::kBlocks;
  constexpr int KS = D / 16;        // k-steps of the scores
  constexpr int MT = D / 16;        // 16-row tiles of the output
  constexpr int CHK = C::kKRow / 16, CHV = C::kVRow / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  uint2 *qf = reinterpret_cast<uint2 *>(smem + C::kOffQ);
  float *back = reinterpret_cast<float *>(smem + C::kOffBack);
  float2 *ml = reinterpret_cast<float2 *>(smem + C::kOffMl);
  volatile int32_t *last_flag = reinterpret_cast<volatile int32_t *>(smem + C::kOffMisc + 96);
  float *join = reinterpret_cast<float *>(smem + C::kOffJoin);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, q4 = lane & 3;
  uint8_t *ring = smem + C::kOffRing + warp * S * C::kStage;

  ExtStart st0;
  if (p.num_seqs <= 32) {
    st0 = ext_plan_warp<C::kCut>(p);
  } else {
    ExtStart *start = reinterpret_cast<ExtStart *>(smem + C::kOffMisc);
    ext_plan_cta<C::kThreads>(p, reinterpret_cast<long long *>(smem + C::kOffRing), start);
    st0 = *start;
  }

  // Queries of a pass, a warp a row.  The first are asked for before the copies:
  // behind them they came 9000 cycles later.
  uint2 q_rows[NR];
  auto load_queries = [&](const ExtWalk &w, int r0) {
#pragma unroll
    for (int e = 0; e < NR; ++e) {
      const int r = r0 + warp + 8 * e;
      q_rows[e] = make_uint2(0u, 0u);
      if (r < w.rows() && 4 * lane < D)
        q_rows[e] = __ldg(
            reinterpret_cast<const uint2 *>(p.q + (ext_row<D>(p, w, w.qb * kExtRows + r) + 4 * lane) * 2));
    }
  };
  ExtWalk w(p, st0);
  if (w.more()) load_queries(w, 0);
  bool loaded = true;

  // ---- copies: this warp's blocks, piece by piece, a group of copies each ----
  // The walk ahead stays in local memory, and what changes with a block only in
  // registers: opening a piece is long code that runs once in many blocks.
  ExtWalk ahead(p, st0);
  FewPiece a = few_piece<C::kRows>(&ahead, warp, false);
  const int two = p.tiles_per_block - 1;  // tokens' blocks of 32: two 16-token ones each
  int a_i = a.from, a_n = 0;  // the block to be copied next, its number in the pass
  int a_tab = 0;              // lane k: the table entry of block 32 (a_n / 32) + k of the pass
  auto table = [&]() {
    const int i = a_i + 8 * lane;
    if (a.more && i < a.to) a_tab = __ldg(a.table + ((i < a.near ? i : i + a.gap) >> two));
  };
  table();
  const uint32_t ring_addr = smem_addr(ring);
  uint32_t to_stage = ring_addr;  // where the next block goes
  auto issue = [&]() {
    if (a.more) {
      const int a_blk = __shfl_sync(kFull, a_tab, a_n & 31);
      const uint32_t dst = to_stage;
      to_stage = to_stage == ring_addr + (S - 1) * C::kStage ? ring_addr : to_stage + C::kStage;
      const bool good = a_blk >= 0 && a_blk < p.num_blocks;
      if (!good && lane == 0) report(p.d_error, PKV_DEVERR_BAD_BLOCK);
      const int lb = a_i < a.near ? a_i : a_i + a.gap;
      const int64_t tile =
          good ? static_cast<int64_t>(((a_blk * p.num_kv_heads + a.kvh) << two) + (lb & two)) : 0;  // (a row number is 31 bits)
      const uint8_t *k = p.k_cache + tile * (kBS * C::kKRow), *v = p.v_cache + tile * (kBS * C::kVRow);
#pragma unroll
      for (int u = lane; u < kBS * CHK; u += 32) few_copy(dst + few_at<CHK>(u / CHK, u % CHK), k + u * 16, good);
#pragma unroll
      for (int u = lane; u < kBS * CHV; u += 32)
        few_copy(dst + C::kOffV + few_at<CHV>(u / CHV, u % CHV), v + u * 16, good);
      if constexpr (C::kCoded) {
        if (lane < 8) {
          const int64_t si = scale_index(tile, p.tiles_per_block) + (lane & 3) * 4;
          few_copy(dst + C::kOffS + lane * 16, (lane < 4 ? p.k_scale : p.v_scale) + si, good);
        }
      }
      a_i += 8;
      if (a_i >= a.to) {
        if (--a.passes == 0) a = few_piece<C::kRows>(&ahead, warp, true);
        a_i = a.from;
        a_n = -1;
      }
      if ((++a_n & 31) == 0) table();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int i = 0; i < S - NB; ++i) issue();

  int used = 0;  // stage of the block computed next
  const float sl2 = p.negate ? -p.scale_log2 : p.scale_log2;
#pragma unroll 1
  for (; w.more(); w.next(), loaded = false) {
    const int rows = w.rows(), item_row = w.qb * kExtRows;
    if (w.it.steps == 0) {  // the rows see nothing: zeros
#pragma unroll 1
      for (int u = tid; u < rows * (D / 4); u += C::kThreads) {
        const int64_t at = ext_row<D>(p, w, item_row + u / (D / 4)) + 4 * (u % (D / 4));
        if (p.out_f32) *reinterpret_cast<float4 *>(p.out + at * 4) = make_float4(0.f, 0.f, 0.f, 0.f);
        else *reinterpret_cast<uint2 *>(p.out + at * 2) = make_uint2(0u, 0u);
      }
      continue;
    }
    const bool whole = w.whole();
    const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (w.j0 == 0 ? 1 : 0);
    const int i0 = 8 * w.j0 + warp, i1 = min(8 * w.j1, w.it.blocks);
    const int first_pos = w.s.len - w.s.n;
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += C::kRows) {
      // ---- queries to fragments: a warp a row (the last join's barrier is behind us) ----
      if (!loaded) load_queries(w, r0);
      loaded = false;
#pragma unroll
      for (int e = 0; e < NR; ++e) {
        const int r = warp + 8 * e;
        uint2 x = q_rows[e];
        if constexpr (C::kCvtQ) {
          // bf16 -> f16, times the power of two that takes the row's largest finite
          // element to [2^14, 2^15): elements 2^-29 of it and larger keep all bits
          const uint32_t q2[2] = {x.x, x.y};
          uint32_t top = 0;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t lo = q2[k] & 0x7FFFu, hi = (q2[k] >> 16) & 0x7FFFu;
            top = max(top, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
          }
          const uint32_t ex = max(__reduce_max_sync(kFull, top) >> 7, 15u);
          const float up = __uint_as_float((268u - ex) << 23);
          const float2 a = unpack2<PKV_BF16>(x.x), b = unpack2<PKV_BF16>(x.y);
          x = make_uint2(pack2<PKV_F16>(a.x * up, a.y * up), pack2<PKV_F16>(b.x * up, b.y * up));
          if (lane == 0) back[r] = __uint_as_float((ex - 14u) << 23);
        }
        // elements 4 lane .. 4 lane + 3 belong to k-step s of lane (row, quarter)
        int s, quarter;
        if constexpr (C::kCoded) {
          s = lane % KS;
          quarter = lane / KS;
        } else {
          s = (lane >> 4) * 4 + (lane & 3);
          quarter = (lane >> 2) & 3;
        }
        if (4 * lane < D) qf[(s * NR + (r >> 3)) * 32 + (r & 7) * 4 + quarter] = x;
      }
      __syncthreads();
      uint2 qreg[NR == 1 ? KS : 1];
      float qback[C::kCvtQ ? 2 * NR : 1];
      if constexpr (NR == 1) {
#pragma unroll
        for (int s = 0; s < KS; ++s) qreg[s] = qf[s * 32 + lane];
      }
      if constexpr (C::kCvtQ) {
#pragma unroll
        for (int e = 0; e < 2 * NR; ++e) qback[e] = back[8 * (e >> 1) + 2 * q4 + (e & 1)];
      }
      float o[NR][MT][4];  // O^T: rows of head_dim g, g + 8 of tile i, columns 2 q4, 2 q4 + 1
      float m[NR][2], l[NR][2];
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int i = 0; i < MT; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
      }
      float unit = 0.f, inv_unit = 0.f;  // of the V scales: a power of two, and kPTop / it
      const int top_row = min(r0 + C::kRows, rows) - 1;
      const int pos_min = first_pos + ((item_row + r0) >> p.group_shift);
      const int pos_max = first_pos + ((item_row + top_row) >> p.group_shift);

#pragma unroll 1
      for (int i = i0; i < i1; i += 8 * NB) {
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 2 * NB) : "memory");
        __syncwarp();  // the blocks are there for every lane, and all have read the last ones
        const int n_there = min((i1 - i + 7) / 8, NB);
        const uint8_t *kt[NB];
        int tok0[NB];  // (one that is not there: beyond every row and the context's end)
#pragma unroll
        for (int t = 0; t < NB; ++t) {
          if (t < n_there) issue();
          kt[t] = ring + (used + t < S ? used + t : used + t - S) * C::kStage;
          tok0[t] = t < n_there ? w.logical(i + 8 * t) * kBS : INT_MAX - 64;
        }
        used = used + n_there < S ? used + n_there : used + n_there - S;

        // ---- S^T = K Q^T ----
        float s4[NB][NR][4] = {};
#pragma unroll
        for (int t = 0; t < NB; ++t) {
          constexpr bool kTwo = NR == 1;  // two chains of products when there is one group of rows
          float alt[4] = {};
          auto product = [&](int s, const uint32_t (&x)[4]) {
#pragma unroll
            for (int n = 0; n < NR; ++n) {
              uint2 b;
              if constexpr (NR == 1) b = qreg[s];
              else b = qf[(s * NR + n) * 32 + lane];
              mma_16816(kTwo && (s & 1) ? alt : s4[t][n], x, b.x, b.y, C::kBf16);
            }
          };
          if constexpr (C::kCoded) {
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
              const int c = (D / 64) * q4 + j;
              const uint4 lo = *reinterpret_cast<const uint4 *>(kt[t] + few_at<CHK>(g, c));
              const uint4 hi = *reinterpret_cast<const uint4 *>(kt[t] + few_at<CHK>(g + 8, c));
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t x[4];
                code4_to_f16x2<C::KT>(word(lo, e), x[0], x[2]);
                code4_to_f16x2<C::KT>(word(hi, e), x[1], x[3]);
                product(4 * j + e, x);
              }
            }
          } else {
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
              const int c = 8 * (e >> 1) + 2 * q4 + (e & 1);
              const uint4 lo = *reinterpret_cast<const uint4 *>(kt[t] + few_at<CHK>(g, c));
              const uint4 hi = *reinterpret_cast<const uint4 *>(kt[t] + few_at<CHK>(g + 8, c));
              const uint32_t x0[4] = {lo.x, hi.x, lo.y, hi.y}, x1[4] = {lo.z, hi.z, lo.w, hi.w};
              product(2 * e, x0);
              product(2 * e + 1, x1);
            }
          }
          if constexpr (kTwo) {
#pragma unroll
            for (int c = 0; c < 4; ++c) s4[t][0][c] += alt[c];
          }
        }
        // ---- scores, masked where a row does not see a token ----
        uint32_t hide[NB];
        bool lags = false;
#pragma unroll
        for (int t = 0; t < NB; ++t) {
          const float *sc = reinterpret_cast<const float *>(kt[t] + C::kOffS);
          float sc0 = sl2, sc1 = sl2;
          if constexpr (C::kCoded) {
            sc0 *= sc[g];
            sc1 *= sc[g + 8];
          }
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            float b0 = 1.f, b1 = 1.f;
            if constexpr (C::kCvtQ) {
              b0 = qback[2 * n];
              b1 = qback[2 * n + 1];
            }
            s4[t][n][0] *= sc0 * b0;
            s4[t][n][1] *= sc0 * b1;
            s4[t][n][2] *= sc1 * b0;
            s4[t][n][3] *= sc1 * b1;
          }
          const bool inner = tok0[t] + kBS - 1 <= pos_min &&
                             (!p.window || tok0[t] > pos_max - p.window || tok0[t] + kBS <= p.sinks);
          hide[t] = 0;
          if (!inner) {
#pragma unroll
            for (int n = 0; n < NR; ++n) {
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const int row = min(r0 + 8 * n + 2 * q4 + (c & 1), rows - 1);
                const int pos = first_pos + ((item_row + row) >> p.group_shift);
                const int tok = tok0[t] + g + 8 * (c >> 1);
                const bool sees = tok <= pos && (!p.window || tok > pos - p.window || tok < p.sinks);
                if (!sees) {
                  hide[t] |= 1u << (4 * n + c);
                  s4[t][n][c] = -INFINITY;
                }
              }
            }
          }
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            lags |= fmaxf(s4[t][n][0], s4[t][n][2]) > m[n][0] + C::kLag;
            lags |= fmaxf(s4[t][n][1], s4[t][n][3]) > m[n][1] + C::kLag;
          }
        }
        // ---- a reference that lags too far (or is not set) is renewed: l and O change units ----
        if (__any_sync(kFull, lags)) {
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            float al[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float mx = -INFINITY;
#pragma unroll
              for (int t = 0; t < NB; ++t) mx = fmaxf(mx, fmaxf(s4[t][n][c], s4[t][n][c + 2]));
              mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
              mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
              mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
              const float mn = fmaxf(m[n][c], mx);
              al[c] = mn == -INFINITY ? 1.f : fast_exp2(m[n][c] - mn);
              m[n][c] = mn;
              l[n][c] *= al[c];
            }
#pragma unroll
            for (int i2 = 0; i2 < MT; ++i2) {
              o[n][i2][0] *= al[0];
              o[n][i2][1] *= al[1];
              o[n][i2][2] *= al[0];
              o[n][i2][3] *= al[1];
            }
          }
        }
        // ---- V scales relative to the unit, which grows with them ----
        float w0[NB], w1[NB];
        if constexpr (C::kCoded) {
          float top = 0.f;
#pragma unroll
          for (int t = 0; t < NB; ++t) {
            const float *sc = reinterpret_cast<const float *>(kt[t] + C::kOffS);
            w0[t] = tok0[t] + g < w.s.len ? sc[16 + g] : 0.f;
            w1[t] = tok0[t] + g + 8 < w.s.len ? sc[24 + g] : 0.f;
            top = fmaxf(top, fmaxf(w0[t] < INFINITY ? w0[t] : 0.f, w1[t] < INFINITY ? w1[t] : 0.f));
          }
          if (__any_sync(kFull, top > unit)) {
            top = fmaxf(top, __shfl_xor_sync(kFull, top, 4));
            top = fmaxf(top, __shfl_xor_sync(kFull, top, 8));
            top = fmaxf(top, __shfl_xor_sync(kFull, top, 16));
            const uint32_t e = min(max((__float_as_uint(top) + 0x7FFFFFu) >> 23, 1u), 253u);
            const float inv = __uint_as_float((254u - e) << 23);
            const float by = unit * inv;  // powers of two
            unit = __uint_as_float(e << 23);
            inv_unit = inv * C::kPTop;
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
              for (int i2 = 0; i2 < MT; ++i2)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[n][i2][c] *= by;
          }
        }
        // ---- P^T, transposed to the second product's operand ----
        uint32_t pb[NB][NR][2];
#pragma unroll
        for (int t = 0; t < NB; ++t) {
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            const float n0 = m[n][0] == -INFINITY ? 0.f : m[n][0], n1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
            float p0 = fast_exp2(s4[t][n][0] - n0), p1 = fast_exp2(s4[t][n][1] - n1);
            float p2 = fast_exp2(s4[t][n][2] - n0), p3 = fast_exp2(s4[t][n][3] - n1);
            l[n][0] += p0 + p2;
            l[n][1] += p1 + p3;
            if constexpr (C::kCoded) {
              const float v0 = w0[t] * inv_unit, v1 = w1[t] * inv_unit;
              p0 *= v0;
              p1 *= v0;
              p2 *= v1;
              p3 *= v1;
              if (hide[t]) {  // whatever the scale of a token that the row does not see
                const uint32_t h = hide[t] >> (4 * n);
                p0 = h & 1 ? 0.f : p0;
                p1 = h & 2 ? 0.f : p1;
                p2 = h & 4 ? 0.f : p2;
                p3 = h & 8 ? 0.f : p3;
              }
            }
            pb[t][n][0] = movmatrix_t(pack2<C::PT>(p0, p1));
            pb[t][n][1] = movmatrix_t(pack2<C::PT>(p2, p3));
          }
        }
        // ---- O^T += V^T P^T; tokens past the context's end count as zeros ----
        const int tk[4] = {2 * q4, 2 * q4 + 1, 2 * q4 + 8, 2 * q4 + 9};
#pragma unroll
        for (int t = 0; t < NB; ++t) {
          const uint8_t *vt = kt[t] + C::kOffV;
          const bool tail = tok0[t] + kBS > w.s.len;
          auto add = [&](int i2, const uint32_t (&x)[4]) {
#pragma unroll
            for (int n = 0; n < NR; ++n) mma_16816(o[n][i2], x, pb[t][n][0], pb[t][n][1], C::kBf16);
          };
          if constexpr (!C::kCoded) {
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
              uint4 v[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                v[k] = *reinterpret_cast<const uint4 *>(vt + few_at<CHV>(tk[k], 8 * h + g));
                if (tail && tok0[t] + tk[k] >= w.s.len) v[k] = make_uint4(0u, 0u, 0u, 0u);
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t x0 = word(v[0], e), y0 = word(v[1], e), x1 = word(v[2], e), y1 = word(v[3], e);
                const uint32_t x[4] = {prmt(x0, y0, 0x5410), prmt(x0, y0, 0x7632), prmt(x1, y1, 0x5410),
                                       prmt(x1, y1, 0x7632)};
                add(4 * h + e, x);
              }
            }
          } else {
            constexpr int W = C::kInt4V ? D / 64 : D / 32;  // 32-bit words of a token that a lane reads
            uint32_t v[4][W];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint8_t *src = vt + few_at<CHV>(tk[k], (g * W) >> 2) + ((g * W) & 3) * 4;
              if constexpr (W == 4) {
                const uint4 x = *reinterpret_cast<const uint4 *>(src);
                v[k][0] = x.x;
                v[k][1] = x.y;
                v[k][2] = x.z;
                v[k][3] = x.w;
              } else if constexpr (W == 2) {
                const uint2 x = *reinterpret_cast<const uint2 *>(src);
                v[k][0] = x.x;
                v[k][1] = x.y;
              } else {
                v[k][0] = *reinterpret_cast<const uint32_t *>(src);
              }
              if (tail && tok0[t] + tk[k] >= w.s.len) {
#pragma unroll
                for (int e = 0; e < W; ++e) v[k][e] = 0u;
              }
            }
#pragma unroll
            for (int e = 0; e < W; ++e) {
              if constexpr (C::kInt4V) {
                // byte b: element 2b (low nibble) and 2b + 1 of the lane's slice
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                  const uint32_t sel = 0x4400u + 0x1111u * b;
                  uint32_t x[4];
                  int4_pair_to_f16x2(prmt(v[0][e], v[1][e], sel), x[0], x[1]);
                  int4_pair_to_f16x2(prmt(v[2][e], v[3][e], sel), x[2], x[3]);
                  add(4 * e + b, x);
                }
              } else {
                uint32_t x[4], y[4];
                code4_to_f16x2<C::VT>(prmt(v[0][e], v[1][e], 0x5140), x[0], x[1]);
                code4_to_f16x2<C::VT>(prmt(v[2][e], v[3][e], 0x5140), x[2], x[3]);
                code4_to_f16x2<C::VT>(prmt(v[0][e], v[1][e], 0x7362), y[0], y[1]);
                code4_to_f16x2<C::VT>(prmt(v[2][e], v[3][e], 0x7362), y[2], y[3]);
                add(2 * e, x);
                add(2 * e + 1, y);
              }
            }
          }
        }
      }

      // ---- join the warps' rows ----
      const float put = C::kCoded ? unit * (1.f / C::kPTop) : 1.f;
#pragma unroll
      for (int n = 0; n < NR; ++n) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float t = l[n][c];
          t += __shfl_xor_sync(kFull, t, 4);
          t += __shfl_xor_sync(kFull, t, 8);
          t += __shfl_xor_sync(kFull, t, 16);
          l[n][c] = t;
          if (g == 0) ml[warp * C::kRows + 8 * n + 2 * q4 + c] = make_float2(m[n][c], t);
        }
      }
#pragma unroll 1
      for (int b = 0; b < C::kRows && r0 + b < rows; b += C::kJoinRows) {
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          if (8 * n < b || 8 * n >= b + C::kJoinRows) continue;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float *to = join + (warp * C::kJoinRows + 8 * n + 2 * q4 + c - b) * C::kJoinRow;
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
              const int d = C::kCoded ? (D / 8) * g + 8 * h : 64 * h + 8 * g;
              float x[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] = o[n][4 * h + (e >> 1)][2 * (e & 1) + c] * put;
              reinterpret_cast<float4 *>(to + d)[0] = make_float4(x[0], x[1], x[2], x[3]);
              reinterpret_cast<float4 *>(to + d)[1] = make_float4(x[4], x[5], x[6], x[7]);
            }
          }
        }
        __syncthreads();
#pragma unroll 1
        for (int u = tid; u < C::kJoinRows * (D / 4); u += C::kThreads) {
          const int row = b + u / (D / 4), d4 = u % (D / 4), at_row = r0 + row;
          if (at_row >= rows) break;
          float2 a[C::kWarps];
          float mj = -INFINITY, lj = 0.f;
#pragma unroll
          for (int k = 0; k < C::kWarps; ++k) {
            a[k] = ml[k * C::kRows + row];
            mj = fmaxf(mj, a[k].x);
          }
          float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < C::kWarps; ++k) {
            const float f = a[k].x > -INFINITY ? fast_exp2(a[k].x - mj) : 0.f;
            lj += a[k].x > -INFINITY ? a[k].y * f : a[k].y;  // (without a reference: 0, or not a number)
            const float4 x = *reinterpret_cast<const float4 *>(join + (k * C::kJoinRows + row - b) * C::kJoinRow + 4 * d4);
            if (f != 0.f) {
              r.x = fmaf(f, x.x, r.x);
              r.y = fmaf(f, x.y, r.y);
              r.z = fmaf(f, x.z, r.z);
              r.w = fmaf(f, x.w, r.w);
            }
          }
          if (__builtin_expect(!(fabsf(r.x + r.y + r.z + r.w) < INFINITY) && lj == lj, 0)) {
            float y[4];  // the piece's blocks against the row's reference, once more
            ext_exact<D, CDT, QDT>(p, ext_exact_row<D>(p, w, item_row + at_row), 8 * w.j0, i1, 8, 8, 4 * d4, mj, y);
            r = make_float4(y[0], y[1], y[2], y[3]);
          }
          if (whole) {
            const float inv = lj > 0.f ? 1.f / lj : (lj == 0.f ? 0.f : lj);
            const int64_t at = ext_row<D>(p, w, item_row + at_row) + 4 * d4;
            if (p.out_f32)
              *reinterpret_cast<float4 *>(p.out + at * 4) = make_float4(r.x * inv, r.y * inv, r.z * inv, r.w * inv);
            else
              *reinterpret_cast<uint2 *>(p.out + at * 2) =
                  make_uint2(pack2<QDT>(r.x * inv, r.y * inv), pack2<QDT>(r.z * inv, r.w * inv));
          } else {
            reinterpret_cast<float4 *>(p.ws_o)[(slot * (D / 4) + d4) * kExtRows + at_row] = r;
            if (d4 == 0) reinterpret_cast<float2 *>(p.ws_ml)[slot * kExtRows + at_row] = make_float2(mj, lj);
          }
        }
        __syncthreads();
      }
    }
    if (!whole) {  // count the piece in at the CTA that begins the item; whoever counts last merges
      const int64_t item0 = w.pos - w.u;
      const int64_t shares = st0.shares, total = st0.total;
      const int c0 = static_cast<int>(((item0 + kExtItemCost + 1) * shares - 1) / total);
      const int c1 = static_cast<int>(((item0 + ext_weight(w.it)) * shares - 1) / total);
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        __threadfence();
        const bool last = atomicAdd(p.ws_ctr + c0, 1u) == static_cast<uint32_t>(c1 - c0);
        if (last) p.ws_ctr[c0] = 0;
        __threadfence();
        *last_flag = last ? 1 : 0;
      }
      __syncthreads();
      if (*last_flag) ext_merge<D, QDT>(p, w, c0, c1);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int D, int CDT, int QDT, int NR>
cudaError_t launch_extend_few(const ExtendParams &p, int grid) {
  using C = FewCfg<D, CDT, QDT, NR>;
  cudaError_t e = cudaFuncSetAttribute(paged_extend_few_kernel<D, CDT, QDT, NR>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  paged_extend_few_kernel<D, CDT, QDT, NR><<<grid, C::kThreads, C::kSmem, p.stream>>>(p);
  return cudaGetLastError();
}

template <int CDT, int QDT>
cudaError_t extend_few_family(const ExtendParams &p, int head_dim, int rows, int grid) {
  if (head_dim == 128)
    return rows <= 8 ? launch_extend_few<128, CDT, QDT, 1>(p, grid) : launch_extend_few<128, CDT, QDT, 4>(p, grid);
  return rows <= 8 ? launch_extend_few<64, CDT, QDT, 1>(p, grid) : launch_extend_few<64, CDT, QDT, 4>(p, grid);
}

}  // namespace pkv
