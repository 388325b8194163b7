// Attention of several new tokens of each sequence over its paged cache:
// prompts, prompt chunks, drafted tokens and single tokens, causal, with an
// optional sliding window and first tokens that stay visible (sinks).
//
// Mathematics.  Query i of a sequence of L cached tokens, n of them new,
// stands at position p = L - n + i and sees tokens j <= p that lie in its
// window (j > p - window) or among the sinks (j < sinks).  One pass over the
// visible tokens keeps, per query row, a reference maximum m, the sum l of
// 2^(s - m) and the accumulator o of 2^(s - m) V, s = scale log2(e) <q, K_j>;
// the result is o / l.
//
// Work split.  A row is one (token, query head of the KV head's group); 256
// consecutive rows of one (sequence, KV head) are an item: two 128-row MMA
// tiles that share one stream of keys and values.  An item walks its visible
// 16-token blocks only (the sink blocks, then the window's), eight to a
// 128-token step.  All items' steps, in order, are cut into equal shares, one
// per CTA, so that ragged batches and the causal triangle balance to one step;
// an item cut by a share boundary leaves fp32 partials in the workspace, and
// the CTA that stores its last one merges them (nothing waits).
//
// One CTA per SM, warp-specialised:
//  * a copy warp moves Q (tensor TMA, boxes of group x tokens rows), and K
//    and V blocks through a ring of 128-token stages;
//  * a warp for each tile issues the tcgen05 MMAs of half steps, 64 tokens:
//    O_t += P_t V of one step's half with P_t read from tensor memory, then
//    S_t = Q_t K^T of the next step's, which overwrites it, then one commit;
//  * two groups of four softmax warps, one per tile, own one row per thread.
//    P is formed against a reference that may lag the row's maximum (kLag), and
//    no maximum is looked for while the sums stay small, so the accumulator is
//    rescaled rarely;
//  * items of 64 rows or less: both tiles take the same rows and every other
//    step, and the second tile's result is joined to the first's;
//  * coded caches: the copy warp brings the raw codes and four more warps turn
//    them into f16 operands (exact: every code is a binary16 number).  K scales
//    multiply the scores; V scales, relative to a running power of two, the V
//    operand.
//
// What bounds it, measured: a prompt of 8192 tokens, 32/8 heads of 128, BF16,
// takes 445 us, 1230 TFLOP/s of the causal half.  The two products of a step
// need some 2100 cycles of the tensor core, the softmax of a tile's half 800
// cycles of its warps alone and about 1600 beside the other tile's: the
// softmax sets the pace.  Over codes the shared memory does (operands written
// once and read by both products' tiles, and the conversions): windowed chunks
// over E4M3 reach 580 TFLOP/s.
//
// Waits are bounded as in the other kernels: a wait that runs out reports
// PKV_DEVERR_WAIT_TIMEOUT and the CTA winds down.
#pragma once

#include <cuda.h>

#include <climits>
#include <type_traits>

#include "extend.h"
#include "umma.cuh"

namespace pkv {

template <int D, int CDT, int QDT>
struct ExtendCfg {
  static constexpr int KT = k_part(CDT), VT = v_part(CDT);
  static constexpr bool kCoded = is_coded(KT);
  static constexpr bool kQkBf16 = !kCoded && QDT == PKV_BF16;
  // bf16 queries over coded caches become f16 too (times a power of two that is
  // common to the item), so that a code costs one conversion instruction and
  // not four: bf16 has no conversion from codes.
  static constexpr bool kCvtQ = kCoded && QDT == PKV_BF16;
  static constexpr bool kPvBf16 = !kCoded && QDT == PKV_BF16;  // V codes become f16
  static constexpr int PT = kPvBf16 ? PKV_BF16 : PKV_F16;      // type of P (and of V's operand)
  static constexpr int kHalves = D / 64;
  static constexpr int kHalf = 128 * 128;             // 64 head_dim elements of 128 rows
  static constexpr int kTile = kHalves * kHalf;       // 128 rows of 16-bit elements: a Q tile, a K or V stage
  static constexpr int kStages = kCoded ? (D == 128 ? 3 : 4) : (D == 128 ? 5 : 8);
  static constexpr int kRawCodes = 128 * D;           // codes of a step's K or V (4-bit V: half of it)
  static constexpr int kRaw = kRawCodes + 512;        // ... and the scales of its 128 tokens
  static constexpr int kRawStages = kCoded ? (D == 128 ? 3 : 6) : 0;
  static constexpr int kOffStage = 2 * kTile;
  static constexpr int kOffRaw = kOffStage + kStages * kTile;
  static constexpr int kOffScale = kOffRaw + kRawStages * kRaw;  // [4 steps] K scales of 128 tokens
  static constexpr int kOffUnit = kOffScale + (kCoded ? 4 * 128 * 4 : 0);  // [4 steps] V unit
  static constexpr int kOffBars = kOffUnit + 16;
  static constexpr int kBars = 2 * kStages + 2 * kRawStages + 20;
  static constexpr int kOffMisc = kOffBars + kBars * 8;  // tensor-memory address, abort flag, merge flag, start
  static constexpr int kSmem = 1024 + kOffMisc + 112 + 512;  // ... and (m, l) of 64 joined rows
  static constexpr int kMmaWarp = 8, kCopyWarp = 9, kCvtWarp = 12;
  static constexpr int kThreads = kCoded ? 512 : 384;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColO = 256;              // S / P of the tiles: columns 0, 128
  // A row's reference is renewed when the P of 64 tokens sum to more than
  // kSumTop, which an f16 P then stays below (bf16 and the fp32 sums have
  // room for far more); a sum beyond it has an exponent beyond kLag.
  static constexpr float kSumTop = kPvBf16 ? 1.152921504606847e18f : 16384.f;  // 2^60, 2^14
  static constexpr float kLag = kPvBf16 ? 53.f : 7.f;
  // V operand of a coded cache: code x scale / unit x kVTop, the unit being a
  // power of two at or above every scale so far; the largest code x kVTop is an
  // f16 number, and a token's scale may be 2^-20 of the largest and keep 11 bits.
  static constexpr float kVTop = VT == PKV_FP8_E5M2 ? 1.f : (VT == kInt4 ? 4096.f : 128.f);
  static_assert(kSmem <= 232448, "shared memory budget");
  static_assert(kStages <= 7 || !kCoded, "scale ring of four steps");
  static_assert(kOffMisc % 8 == 0, "alignment");
};

// Tensor-map load of a 2D box with an L2 policy.
__device__ __forceinline__ void ext_tma_2d(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar,
                                           uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void ext_tma_3d(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ uint64_t policy_evict_normal() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ uint64_t ext_desc(uint32_t lo, uint32_t hi) {
  return static_cast<uint64_t>(hi) << 32 | lo;
}
// Pairs of floats in one 64-bit register, and the packed fp32 instructions on them.
__device__ __forceinline__ uint64_t f2_pack(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// A in tensor memory (K-major, two 16-bit elements a column).
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                            bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}

// ---- sequences, items, shares --------------------------------------------------------

// A sequence's cached tokens, new tokens and first query row.  Lengths or
// query ranges that cannot be are reported (by one thread of the grid) and
// leave the sequence without tokens (its rows become zeros) or without queries.
struct ExtSeq {
  int len, n, q0;
};
__device__ __forceinline__ ExtSeq ext_seq(const ExtendParams &p, int b, bool tell) {
  ExtSeq s;
  s.len = __ldg(p.context_lens + b);
  s.q0 = __ldg(p.query_starts + b);
  const int q1 = __ldg(p.query_starts + b + 1);
  s.n = q1 - s.q0;
  const bool bad_len = s.len < 0 || s.len > static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size;
  const bool bad_rows = s.q0 < 0 || q1 < s.q0 || q1 > p.num_queries;
  if (tell && (bad_len || bad_rows)) report(p.d_error, PKV_DEVERR_BAD_CONTEXT_LEN);
  if (bad_len) s.len = 0;
  if (bad_rows) s.n = s.q0 = 0;
  return s;
}

// The blocks that 256 rows of a sequence see: visible block i is logical
// 16-token block i (i < near: the sinks) or i + gap.
struct ExtItem {
  int blocks, near, gap, steps;
};
__device__ __forceinline__ ExtItem ext_item(const ExtendParams &p, const ExtSeq &s, int qb) {
  const int r0 = qb * kExtRows;
  const int r1 = min(r0 + kExtRows, s.n << p.group_shift);
  const int p0 = max(s.len - s.n + (r0 >> p.group_shift), 0);
  const int p1 = s.len - s.n + ((r1 - 1) >> p.group_shift);
  ExtItem it = {0, 0, 0, 0};
  if (p1 < 0) return it;
  const int end = (p1 + kBS) / kBS;
  it.blocks = end;
  if (p.window) {
    const int first = max(p0 - p.window + 1, 0) / kBS;
    const int near = min((min(p.sinks, p1 + 1) + kBS - 1) / kBS, end);
    if (near < first) {
      it.near = near;
      it.gap = first - near;
      it.blocks = end - it.gap;
    }
  }
  it.steps = (it.blocks + 7) / 8;
  return it;
}
// An item's share of the work, in steps: its own, at least one, and kExtItemCost
// for loading Q, filling the pipeline and writing the result (measured at two
// steps; without it a CTA with many short items ended 10% after the others).
constexpr int kExtItemCost = 2;
__device__ __forceinline__ int ext_weight(const ExtItem &it) { return max(it.steps, 1) + kExtItemCost; }
__device__ __forceinline__ int ext_qblocks(const ExtendParams &p, int n) {
  return ((n << p.group_shift) + kExtRows - 1) / kExtRows;
}

struct ExtStart {
  long long pos, end, total;  // this CTA's share of the work, and all of it
  int b, kvh, qb, u, shares;  // where it starts (unit u of an item), and how many CTAs have one
  ExtSeq s;                   // that sequence
};

// Walks the pieces of a share: (item, steps j0 .. j1).  A share that begins or
// ends within an item's cost units has no step of it there and no piece.
struct ExtWalk {
  const ExtendParams &p;
  int64_t pos, end;
  int b, kvh, qb, nqb;
  int u, j0, j1;
  ExtSeq s;
  ExtItem it;
  __device__ ExtWalk(const ExtendParams &pp, const ExtStart &st) : p(pp), pos(st.pos), end(st.end), b(st.b), kvh(st.kvh), qb(st.qb) {
    if (pos < end) {
      s = st.s;
      nqb = ext_qblocks(p, s.n);
      open(st.u);
      if (j0 == j1) next();
    }
  }
  __device__ __forceinline__ bool more() const { return pos < end; }
  __device__ __forceinline__ void open(int unit) {
    it = ext_item(p, s, qb);
    u = unit;
    j0 = max(unit - kExtItemCost, 0);
    j1 = static_cast<int>(max(min(static_cast<int64_t>(ext_weight(it)), unit + (end - pos)) - kExtItemCost, static_cast<int64_t>(0)));
  }
  __device__ __forceinline__ void next() {
    do {
      pos += j1 + kExtItemCost - u;
      if (j1 == 0 || pos >= end) {  // the share ends in this item
        pos = end;
        return;
      }
      if (++qb == nqb) {
        qb = 0;
        if (++kvh == p.num_kv_heads) {
          kvh = 0;
          do {
            ++b;
            s = ext_seq(p, b, false);
            nqb = ext_qblocks(p, s.n);
          } while (nqb == 0);
        }
      }
      open(0);
    } while (j0 == j1);
  }
  __device__ __forceinline__ int rows() const { return min((s.n << p.group_shift) - qb * kExtRows, kExtRows); }
  __device__ __forceinline__ bool two() const { return rows() > 128; }
  // Few rows (a decode step, drafted tokens): both tiles take the same rows and
  // every other step, and the second's result is joined to the first's, so that
  // two chains of products and exponentials run instead of one.
  __device__ __forceinline__ bool split() const { return rows() <= 64 && j1 - j0 >= 2; }
  __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == max(it.steps, 1); }
  __device__ __forceinline__ int logical(int i) const { return i < it.near ? i : i + it.gap; }
};

__device__ __forceinline__ long long ext_div(long long a, long long b) {  // of numbers that are not negative
  return (a | b) >> 32 ? a / b : static_cast<long long>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}

// One lane a sequence: its work (all KV heads).  Whole warps take part: long
// prompts' items are added up by the warp together.
__device__ __forceinline__ long long ext_seq_work(const ExtendParams &p, const ExtSeq &s) {
  const int lane = threadIdx.x & 31;
  const int nqb = ext_qblocks(p, s.n);
  long long sum = 0;
  if (nqb <= 4) {
#pragma unroll 1
    for (int qb = 0; qb < nqb; ++qb) sum += ext_weight(ext_item(p, s, qb));
  }
  for (unsigned todo = __ballot_sync(kFull, nqb > 4); todo; todo &= todo - 1) {
    const int from = __ffs(todo) - 1;
    const ExtSeq o = {__shfl_sync(kFull, s.len, from), __shfl_sync(kFull, s.n, from), 0};
    const int onqb = __shfl_sync(kFull, nqb, from);
    long long part = 0;
#pragma unroll 1
    for (int qb = lane; qb < onqb; qb += 32) part += ext_weight(ext_item(p, o, qb));
#pragma unroll
    for (int off = 16; off; off >>= 1) part += __shfl_xor_sync(kFull, part, off);
    if (lane == from) sum = part;
  }
  return sum * p.num_kv_heads;
}

// This CTA's share of `total`.
__device__ __forceinline__ ExtStart ext_share(long long total) {
  // shares of at least kExtMinShare units (an item of two steps): a cut costs a merge
  constexpr int kExtMinShare = kExtItemCost + 2;
  const long long shares =
      max(1ll, min(static_cast<long long>(gridDim.x), ext_div(total + kExtMinShare - 1, kExtMinShare)));
  ExtStart st = {0, 0, total, 0, 0, 0, 0, static_cast<int>(shares), {0, 0, 0}};
  if (blockIdx.x < shares) {
    st.pos = ext_div(blockIdx.x * total, shares);
    st.end = ext_div((blockIdx.x + 1) * total, shares);
  }
  return st;
}

// The whole warp: where in sequence st.b, whose work is `work`, unit `rem` lies.
__device__ __forceinline__ void ext_locate(const ExtendParams &p, ExtStart &st, long long work, long long rem) {
  const int lane = threadIdx.x & 31;
  const long long per_head = p.num_kv_heads == 1 ? work : ext_div(work, p.num_kv_heads);
  st.kvh = p.num_kv_heads == 1 ? 0 : static_cast<int>(ext_div(rem, per_head));
  rem -= st.kvh * per_head;
  const int nqb = ext_qblocks(p, st.s.n);
  st.qb = 0;
  st.u = static_cast<int>(rem);
#pragma unroll 1
  for (int q0 = 0; nqb > 1 && q0 < nqb; q0 += 32) {
    const int own = q0 + lane < nqb ? ext_weight(ext_item(p, st.s, q0 + lane)) : 0;
    int v = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(kFull, v, off);
      if (lane >= off) v += u;
    }
    const int sum = __shfl_sync(kFull, v, 31);
    if (rem < sum) {
      const int at = __ffs(__ballot_sync(kFull, rem < v)) - 1;
      st.qb = q0 + at;
      st.u = static_cast<int>(rem) - (__shfl_sync(kFull, v, at) - __shfl_sync(kFull, own, at));
      break;
    }
    rem -= sum;
  }
}

__device__ __forceinline__ long long ext_scan(long long v) {  // inclusive, over the warp
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long u = __shfl_up_sync(kFull, v, off);
    if (lane >= off) v += u;
  }
  return v;
}

// Batches of up to 32 sequences: each warp plans for itself, without shared
// memory or barriers (the plan is on the path of the smallest calls).
// CUT > 0: what a cut item costs in steps.  When there are no more items than
// CTAs and the longest is shorter than an equal share with a cut, each CTA
// takes one whole item.
template <int CUT = 0>
__device__ __forceinline__ ExtStart ext_plan_warp(const ExtendParams &p) {
  const int lane = threadIdx.x & 31;
  ExtSeq s = {0, 0, 0};
  if (lane < p.num_seqs) s = ext_seq(p, lane, blockIdx.x == 0 && threadIdx.x < 32);
  const long long work = ext_seq_work(p, s);
  const long long upto = ext_scan(work);
  const long long total = __shfl_sync(kFull, upto, 31);
  if constexpr (CUT > 0) {
    // items: a row block for each KV head; the last row block of a sequence is (nearly) its longest
    const int nqb = ext_qblocks(p, s.n);
    const int own = min(static_cast<int>(gridDim.x) + 1, min(nqb, 4096)) * min(p.num_kv_heads, 4096);
    int items = min(own, 1 << 24);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(kFull, items, off);
      if (lane >= off) items += v;
    }
    const int count = __shfl_sync(kFull, items, 31);
    int longest = 0;
    if (nqb > 0) longest = ext_weight(ext_item(p, s, nqb - 1));
    longest = __reduce_max_sync(kFull, longest);
    if (count <= static_cast<int>(gridDim.x) && longest <= ext_div(total, gridDim.x) + CUT) {
      ExtStart st = {0, 0, total, 0, 0, 0, 0, count, {0, 0, 0}};
      const int c = static_cast<int>(blockIdx.x);
      if (c < count) {
        st.b = __ffs(__ballot_sync(kFull, items > c)) - 1;
        st.s = {__shfl_sync(kFull, s.len, st.b), __shfl_sync(kFull, s.n, st.b), __shfl_sync(kFull, s.q0, st.b)};
        const int r = c - (__shfl_sync(kFull, items, st.b) - __shfl_sync(kFull, own, st.b));
        const int blocks = __shfl_sync(kFull, nqb, st.b);
        st.kvh = r / blocks;
        st.qb = r - st.kvh * blocks;
        st.end = ext_weight(ext_item(p, st.s, st.qb));
      }
      return st;
    }
  }
  ExtStart st = ext_share(total);
  if (st.pos < st.end) {
    st.b = __ffs(__ballot_sync(kFull, upto > st.pos)) - 1;
    st.s = {__shfl_sync(kFull, s.len, st.b), __shfl_sync(kFull, s.n, st.b), __shfl_sync(kFull, s.q0, st.b)};
    const long long own = __shfl_sync(kFull, work, st.b);
    ext_locate(p, st, own, st.pos - (__shfl_sync(kFull, upto, st.b) - own));
  }
  return st;
}

// Larger batches: all threads of the CTA, `cum` being shared memory for
// num_seqs + 1 prefix sums of work per sequence.
template <int THREADS>
__device__ __noinline__ void ext_plan_cta(const ExtendParams &p, long long *cum, ExtStart *start) {
  const int tid = threadIdx.x, lane = tid & 31;
#pragma unroll 1
  for (int b0 = 0; b0 < p.num_seqs; b0 += THREADS) {
    const int b = b0 + tid;
    ExtSeq s = {0, 0, 0};
    if (b < p.num_seqs) s = ext_seq(p, b, blockIdx.x == 0);
    const long long work = ext_seq_work(p, s);
    if (b < p.num_seqs) cum[b] = work;
  }
  __syncthreads();
  if (tid < 32) {
    long long total = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < p.num_seqs; b0 += 32) {
      const long long own = b0 + lane < p.num_seqs ? cum[b0 + lane] : 0;
      const long long v = ext_scan(own);
      if (b0 + lane < p.num_seqs) cum[b0 + lane] = total + v - own;
      total += __shfl_sync(kFull, v, 31);
    }
    if (lane == 0) cum[p.num_seqs] = total;
    __syncwarp();
    ExtStart st = ext_share(total);
    if (st.pos < st.end) {
      int lo = 0, hi = p.num_seqs - 1;
      while (lo < hi) {  // the last sequence that starts at or before pos
        const int mid = (lo + hi + 1) >> 1;
        if (cum[mid] <= st.pos) lo = mid; else hi = mid - 1;
      }
      st.b = lo;
      st.s = ext_seq(p, lo, false);
      ext_locate(p, st, cum[lo + 1] - cum[lo], st.pos - cum[lo]);
    }
    if (lane == 0) *start = st;
  }
  fence_proxy_async_smem();  // `cum` lies where the copies will land
  __syncthreads();
}

// Sixteen codes (one 16-byte vector, or 8 bytes of 4-bit codes) -> eight words
// of two binary16 numbers, exact.
template <int DT>
__device__ __forceinline__ void ext_codes(const uint4 &v, uint32_t (&o)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (DT == kInt4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // byte i: elements 2i (low nibble), 2i + 1
      const uint32_t t = w[i >> 2] >> (8 * (i & 3));
      const uint32_t n = (t & 0xFu) | ((t & 0xF0u) << 12) | 0x64006400u;
      asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(o[i]) : "r"(n), "r"(0x64086408u));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) code4_to_f16x2<DT>(w[i], o[2 * i], o[2 * i + 1]);
  }
}

// Element offset in out (and q) of row `row` of a sequence's KV head.
template <int D>
__device__ __forceinline__ int64_t ext_row(const ExtendParams &p, const ExtWalk &w, int row) {
  return (static_cast<int64_t>(w.s.q0 + (row >> p.group_shift)) * p.num_q_heads + (w.kvh << p.group_shift) +
          (row & ((1 << p.group_shift) - 1))) * D;
}

// The whole warp: 32 columns, from column d on, of 32 consecutive rows of out,
// each lane holding its own row's.  Lanes of four exchange 16-byte units, so
// that a store writes 64 contiguous bytes of eight rows and not 16 of 32
// (measured on a 256-row item: a thread storing its own row took 7000 cycles).
template <int D, int QDT>
__device__ __forceinline__ void ext_store32(const ExtendParams &p, const ExtWalk &w, int row, int d, const float (&v)[32]) {
  const int lane = threadIdx.x & 31, rows = w.s.n << p.group_shift;
  auto exchange = [&](uint4 (&u)[4]) {
#pragma unroll
    for (int s = 1; s <= 2; s <<= 1) {
      const bool up = lane & s;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k & s) continue;
        const uint4 send = up ? u[k] : u[k | s];
        const uint4 got = make_uint4(__shfl_xor_sync(kFull, send.x, s), __shfl_xor_sync(kFull, send.y, s),
                                     __shfl_xor_sync(kFull, send.z, s), __shfl_xor_sync(kFull, send.w, s));
        if (up) u[k] = got; else u[k | s] = got;
      }
    }
  };
  const int row0 = row & ~3;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if (half && !p.out_f32) break;
    uint4 u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (p.out_f32) {
        const int e = 16 * half + 4 * k;
        u[k] = make_uint4(__float_as_uint(v[e]), __float_as_uint(v[e + 1]), __float_as_uint(v[e + 2]), __float_as_uint(v[e + 3]));
      } else {
        u[k] = make_uint4(pack2<QDT>(v[8 * k], v[8 * k + 1]), pack2<QDT>(v[8 * k + 2], v[8 * k + 3]),
                          pack2<QDT>(v[8 * k + 4], v[8 * k + 5]), pack2<QDT>(v[8 * k + 6], v[8 * k + 7]));
      }
    }
    exchange(u);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (row0 + k >= rows) continue;
      const int64_t at = ext_row<D>(p, w, row0 + k) + d;
      uint8_t *to = p.out_f32 ? p.out + (at + 16 * half + 4 * (lane & 3)) * 4 : p.out + (at + 8 * (lane & 3)) * 2;
      *reinterpret_cast<uint4 *>(to) = u[k];
    }
  }
}

// Element d of row `row` (token of the pool) of a cache half, without its scale.
template <int D, int DT>
__device__ __forceinline__ float ext_element(const uint8_t *cache, int64_t row, int d) {
  if constexpr (DT == kInt4) {
    const uint32_t b = cache[row * (D / 2) + d / 2];
    return static_cast<float>(d & 1 ? b >> 4 : b & 15u) - 8.f;
  } else if constexpr (is_code8(DT)) {
    float f[4];
    unpack_code4<DT>(cache[row * D + d], f);
    return f[0];
  } else {
    const float2 f = unpack2<DT>(reinterpret_cast<const uint16_t *>(cache)[row * D + d]);
    return f.x;
  }
}

// N columns, from d on, of a row's accumulator from the definition: over the
// visible tokens of the item's blocks i0, i0 + 1 .. (run of them), i0 + stride
// .. before i1, with the row's reference m.  For rows whose accumulator is not
// finite: the products also multiply the V of tokens that a row does not see,
// by zero, which an infinity or a NaN there turns into NaN.  What the row does
// see decides here.
struct ExtRow {
  int pos, b, kvh, near, gap;
  int64_t q;  // element offset of the query
};
template <int D>
__device__ __forceinline__ ExtRow ext_exact_row(const ExtendParams &p, const ExtWalk &w, int row) {
  return {w.s.len - w.s.n + (row >> p.group_shift), w.b, w.kvh, w.it.near, w.it.gap, ext_row<D>(p, w, row)};
}
template <int D, int CDT, int QDT, int N>
__device__ __noinline__ void ext_exact(const ExtendParams &p, ExtRow w, int i0, int i1, int run, int stride, int d,
                                       float m, float (&v)[N]) {
  constexpr int KT = k_part(CDT), VT = v_part(CDT);
  const int pos = w.pos;
  const int lo = p.window ? max(pos - p.window + 1, 0) : 0;
  const uint16_t *q = reinterpret_cast<const uint16_t *>(p.q) + w.q;
  const float scale = p.negate ? -p.scale_log2 : p.scale_log2;
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] = 0.f;
#pragma unroll 1
  for (int i = i0; i < i1; i += (i - i0) % stride == run - 1 ? stride - run + 1 : 1) {
    const int lb = i < w.near ? i : i + w.gap;
    const int32_t blk = __ldg(p.block_tables + static_cast<int64_t>(w.b) * p.max_blocks_per_seq + lb / p.tiles_per_block);
    if (blk < 0 || blk >= p.num_blocks) continue;
    const int64_t bh = static_cast<int64_t>(blk) * p.num_kv_heads + w.kvh;
#pragma unroll 1
    for (int u = 0; u < kBS; ++u) {
      const int tok = lb * kBS + u;
      if (tok > pos || (tok < lo && tok >= p.sinks)) continue;
      const int off = tok % p.block_size;
      const int64_t at = bh * p.block_size + off, sat = bh * 2 * p.block_size + off;
      float dot = 0.f;
#pragma unroll 1
      for (int e = 0; e < D; ++e) dot = fmaf(unpack2<QDT>(q[e]).x, ext_element<D, KT>(p.k_cache, at, e), dot);
      if constexpr (is_coded(KT)) dot *= p.k_scale[sat];
      float f = fast_exp2(fmaf(dot, scale, m == -INFINITY ? 0.f : -m));
      if constexpr (is_coded(VT)) f *= p.v_scale[sat];
      bool known = true;
#pragma unroll 1
      for (int e = 0; e < N; ++e) {
        v[e] = fmaf(f, ext_element<D, VT>(p.v_cache, at, d + e), v[e]);
        known &= v[e] != v[e];
      }
      if (known) return;  // all NaN: nothing can change that
    }
  }
}

// v += f x a row's 32 elements of the joined result ([D / 4][64 rows] in shared memory)
__device__ __forceinline__ void ext_join(float (&v)[32], const float4 *o, float f) {
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    const float4 a = o[(e / 4) * 64];
    v[e] = fmaf(a.x, f, v[e]);
    v[e + 1] = fmaf(a.y, f, v[e + 1]);
    v[e + 2] = fmaf(a.z, f, v[e + 2]);
    v[e + 3] = fmaf(a.w, f, v[e + 3]);
  }
}

// The 256 softmax threads: partials of an item, left by CTAs c0 .. c1, to its
// output rows.  With more than 128 rows a thread takes a row; else several
// threads share one, each with every tper-th group of four elements.
template <int D, int QDT>
__device__ __forceinline__ void ext_merge(const ExtendParams &p, const ExtWalk &w, int c0, int c1) {
  const int rows = w.rows();
  const int tper = min(kExtRows / rows, D / 4);  // threads a row
  const int rr = static_cast<int>(threadIdx.x) % (tper == 1 ? kExtRows : rows);
  const int sub = tper == 1 ? 0 : static_cast<int>(threadIdx.x) / rows;
  const bool mine = sub < tper && rr < rows;
  if (!__any_sync(kFull, mine)) return;
  const float2 *ml = reinterpret_cast<const float2 *>(p.ws_ml) + rr;
  const float4 *wo = reinterpret_cast<const float4 *>(p.ws_o) + rr;
  auto slot = [&](int c) { return static_cast<int64_t>(2 * c + (c == c0 ? 1 : 0)); };
  float m = -INFINITY, l = 0.f;
  if (mine) {
#pragma unroll 4
    for (int c = c0; c <= c1; ++c) {
      const float2 a = __ldcg(ml + slot(c) * kExtRows);
      const float m_new = fmaxf(m, a.x);
      if (m_new > -INFINITY) {
        l = l * fast_exp2(m - m_new) + a.y * fast_exp2(a.x - m_new);
        m = m_new;
      } else {
        l += a.y;  // 0, or not a number
      }
    }
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  const int row = w.qb * kExtRows + rr;
  constexpr int kBatch = 8;
#pragma unroll 1
  for (int d0 = sub; d0 < D / 4; d0 += kBatch * tper) {
    float4 o[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (mine) {
#pragma unroll 2
      for (int c = c0; c <= c1; ++c) {
        const float a = __ldcg(ml + slot(c) * kExtRows).x;
        const float f = a > -INFINITY ? fast_exp2(a - m) : 0.f;
        float4 v[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int d4 = d0 + u * tper;
          v[u] = d4 < D / 4 && f != 0.f ? __ldcg(wo + (slot(c) * (D / 4) + d4) * kExtRows) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          o[u].x += v[u].x * f;
          o[u].y += v[u].y * f;
          o[u].z += v[u].z * f;
          o[u].w += v[u].w * f;
        }
      }
    }
    if (tper == 1) {
      float v[32];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        v[4 * u] = o[u].x * inv;
        v[4 * u + 1] = o[u].y * inv;
        v[4 * u + 2] = o[u].z * inv;
        v[4 * u + 3] = o[u].w * inv;
      }
      ext_store32<D, QDT>(p, w, row, 4 * d0, v);
    } else if (mine) {
      const int64_t out_row = ext_row<D>(p, w, row);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int d4 = d0 + u * tper;
        if (d4 >= D / 4) break;
        const int64_t at = out_row + 4 * d4;
        if (p.out_f32)
          *reinterpret_cast<float4 *>(p.out + at * 4) =
              make_float4(o[u].x * inv, o[u].y * inv, o[u].z * inv, o[u].w * inv);
        else
          *reinterpret_cast<uint2 *>(p.out + at * 2) =
              make_uint2(pack2<QDT>(o[u].x * inv, o[u].y * inv), pack2<QDT>(o[u].z * inv, o[u].w * inv));
      }
    }
  }
}

// ---- the kernel ------------------------------------------------------------------------

template <int D, int CDT, int QDT>
__global__ void __launch_bounds__(ExtendCfg<D, CDT, QDT>::kThreads, 1)
    paged_extend_kernel(const __grid_constant__ ExtendParams p, const __grid_constant__ CUtensorMap tmq,
                        const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
  using C = ExtendCfg<D, CDT, QDT>;
  constexpr int S = C::kStages;
  constexpr int RS = C::kRawStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kOffBars);
  uint64_t *full = bars;              // [S] a stage's 16-bit operand is ready
  uint64_t *empty = full + S;         // [S] the MMAs that read it are done (once a tile)
  uint64_t *rfull = empty + S;        // [RS] a raw stage's copies landed
  uint64_t *rempty = rfull + RS;      // [RS] converted
  uint64_t *sfull = rempty + RS;      // [2 tiles][2 halves] P V of the last step's half and S of this one done (commit)
  uint64_t *pfull = sfull + 4;        // [2][2] P of a half written, O rescaled if needed (a warp each)
  uint64_t *pvhalf = pfull + 4;       // [2] split items: P V of a first half done (commit)
  uint64_t *joined = pvhalf + 2;      // [2] split items: rows 0-31, 32-63 of the second tile's result are in shared memory
  uint64_t *qfull = joined + 2;       // Q landed
  uint64_t *qmax = qfull + 1;         // kCvtQ: largest query known, Q converted (a converting warp each)
  uint64_t *qready = C::kCvtQ ? qfull + 2 : qfull;  // Q in the type of the products
  uint64_t *qempty = qfull + 3;       // last S of the piece done (commit)
  uint64_t *stored = qempty + 1;      // a piece's partials are in the workspace (a softmax warp each)
  uint64_t *counted = stored + 1;     // ... and counted in
  uint64_t *done = counted + 1;       // [2] every MMA of the tile's warp is done (commit)
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffMisc);
  volatile int32_t *abort_flag = reinterpret_cast<volatile int32_t *>(tmem_slot + 1);
  volatile int32_t *last_flag = abort_flag + 1;
  float *scales = reinterpret_cast<float *>(smem + C::kOffScale);
  uint32_t *qtop = reinterpret_cast<uint32_t *>(smem + C::kOffMisc + 96);  // [2] by piece: bits of the largest finite |query|
  volatile float *units = reinterpret_cast<volatile float *>(smem + C::kOffUnit);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full + s, C::kCoded ? 4 : 1);
      mbar_init(empty + s, 2);
    }
    for (int s = 0; s < RS; ++s) {
      mbar_init(rfull + s, 1);
      mbar_init(rempty + s, 4);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(pvhalf + t, 1);
      mbar_init(joined + t, 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(sfull + 2 * t + h, 1);
        mbar_init(pfull + 2 * t + h, 4);
      }
    }
    mbar_init(qfull, 1);
    mbar_init(qfull + 1, 4);
    mbar_init(qfull + 2, 4);
    qtop[0] = qtop[1] = 0;
    mbar_init(qempty, 2);
    mbar_init(stored, 8);
    mbar_init(counted, 1);
    mbar_init(done, 1);
    mbar_init(done + 1, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == C::kMmaWarp) tmem_alloc(tmem_slot, C::kTmemCols);
  tmem_fence_before();
  ExtStart st0;
  if (p.num_seqs <= 32) {
    st0 = ext_plan_warp(p);
    __syncthreads();
  } else {
    ExtStart *start = reinterpret_cast<ExtStart *>(smem + C::kOffMisc + 16);
    ext_plan_cta<C::kThreads>(p, reinterpret_cast<long long *>(smem + C::kOffStage), start);
    st0 = *start;
  }
  tmem_fence_after();
  const uint32_t tmem = *tmem_slot;

  // A bounded wait.  Once any thread of the CTA gave up, the others stop waiting too.
  auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
    if (mbar_try_wait(bar, parity)) return true;
#pragma unroll 1
    for (uint32_t i = 0; i < kWaitLimit; ++i) {
      if (mbar_try_wait(bar, parity)) return true;
      if (*abort_flag) return false;
    }
    *abort_flag = 1;
    report(p.d_error, PKV_DEVERR_WAIT_TIMEOUT);
    return false;
  };
  auto uwait = [&](uint64_t *bar, uint32_t parity) -> bool { return __all_sync(kFull, wait(bar, parity)); };

  // The softmax groups take registers from the others; the sums are what the
  // launch holds (2 x 184 + 136 = 3 x 168, 2 x 176 + 80 + 80 = 4 x 128).
  if (warp >= 8 && warp < 12) {
   if constexpr (C::kCoded) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
   else asm volatile("setmaxnreg.dec.sync.aligned.u32 136;");
   if (warp == C::kCopyWarp) {
    // ---- copies: Q of a piece, then its K and V blocks step by step ----
    uint32_t cnt = 0, qn = 0;
    bool ok = true;
    for (ExtWalk w(p, st0); ok && w.more(); w.next()) {
      if (w.it.steps == 0) continue;
      // several items read the same keys and values unless a sequence has one item per KV head
      const uint64_t pol = w.nqb > 1 ? policy_evict_normal() : policy_evict_first();
      if (qn) ok = uwait(qempty, (qn - 1) & 1);
      if (!ok) break;
      if (lane == 0) {
        const int tiles = w.two() ? 2 : 1;
        mbar_arrive_expect_tx(qfull, tiles * C::kTile);
        const int tok = 128 >> p.group_shift;  // tokens of a 128-row tile
        const int t0 = w.s.q0 + ((w.qb * kExtRows) >> p.group_shift);
        for (int t = 0; t < tiles; ++t)
          for (int h = 0; h < C::kHalves; ++h)
            ext_tma_3d(smem + t * C::kTile + h * C::kHalf, &tmq, 64 * h, w.kvh << p.group_shift, t0 + t * tok, qfull);
      }
      ++qn;
      const int32_t *table = p.block_tables + static_cast<int64_t>(w.b) * p.max_blocks_per_seq;
      const int tpb = p.tiles_per_block;
      auto block_of = [&](int j) -> int32_t {
        const int i = 8 * j + lane;
        return lane < 8 && i < w.it.blocks ? __ldg(table + w.logical(i) / tpb) : -1;
      };
      int32_t blk = block_of(w.j0);
      for (int j = w.j0; ok && j < w.j1; ++j) {
        const int i = 8 * j + lane;
        const bool there = lane < 8 && i < w.it.blocks;
        const int lb = w.logical(i);
        const bool good = there && blk >= 0 && blk < p.num_blocks;
        if (there && !good) report(p.d_error, PKV_DEVERR_BAD_BLOCK);
        const int64_t tile = good ? (static_cast<int64_t>(blk) * p.num_kv_heads + w.kvh) * tpb + lb % tpb : 0;
        const bool cut = good && (lb + 1) * kBS > w.s.len;  // tokens past the context: V must read as zeros
        const unsigned bads = __ballot_sync(kFull, there && !good);
        const unsigned cuts = __ballot_sync(kFull, cut);
        const unsigned goods = __ballot_sync(kFull, good);
        blk = j + 1 < w.j1 ? block_of(j + 1) : -1;
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
          if constexpr (C::kCoded) {
            const int st = cnt % RS;
            if (cnt >= RS && !(ok = uwait(rempty + st, (cnt / RS - 1) & 1))) break;
            uint8_t *dst = smem + C::kOffRaw + st * C::kRaw;
            const int rb = row_bytes(kind ? C::VT : C::KT, D);
            for (unsigned m = bads; m; m &= m - 1) {  // a bad block reads as zeros
              const int u = __ffs(m) - 1;
              for (int e = lane; e < kBS * rb / 16; e += 32)
                *reinterpret_cast<uint4 *>(dst + u * kBS * rb + e * 16) = make_uint4(0u, 0u, 0u, 0u);
              if (lane < kBS) *reinterpret_cast<float *>(dst + C::kRawCodes + (u * kBS + lane) * 4) = 0.f;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(rfull + st, __popc(goods) * (kBS * rb + kBS * 4));
            __syncwarp();
            if (good) {
              const uint8_t *cache = kind ? p.v_cache : p.k_cache;
              const float *sc = (kind ? p.v_scale : p.k_scale) + scale_index(tile, tpb);
              bulk_g2s(dst + lane * kBS * rb, cache + tile * kBS * rb, kBS * rb, rfull + st, pol);
              bulk_g2s(dst + C::kRawCodes + lane * kBS * 4, sc, kBS * 4, rfull + st, pol);
            }
          } else {
            const int st = cnt % S;
            if (cnt >= S && !(ok = uwait(empty + st, (cnt / S - 1) & 1))) break;
            uint8_t *dst = smem + C::kOffStage + st * C::kTile;
            const unsigned by_hand = bads | (kind ? cuts : 0u);
            const unsigned by_tma = goods & ~by_hand;
            if ((by_tma >> lane) & 1) {
              const int row = static_cast<int>(tile * kBS);
#pragma unroll
              for (int h = 0; h < C::kHalves; ++h)
                ext_tma_2d(dst + h * C::kHalf + lane * kBS * 128, kind ? &tmv : &tmk, 64 * h, row, full + st, pol);
            }
            for (unsigned m = by_hand; m; m &= m - 1) {
              const int u = __ffs(m) - 1;
              const int64_t utile = __shfl_sync(kFull, tile, u);
              const bool ugood = (goods >> u) & 1;
              const int left = w.s.len - w.logical(8 * j + u) * kBS;  // valid tokens of the block
              const uint4 *src = reinterpret_cast<const uint4 *>((kind ? p.v_cache : p.k_cache) + utile * kBS * D * 2);
#pragma unroll
              for (int e = lane; e < kBS * D / 8; e += 32) {
                const int r = e / (D / 8), ch = e % (D / 8);
                const uint4 v = ugood && r < left ? src[e] : make_uint4(0u, 0u, 0u, 0u);
                *reinterpret_cast<uint4 *>(dst + (ch >> 3) * C::kHalf + (u * kBS + r) * 128 +
                                           (((ch & 7) ^ (r & 7)) << 4)) = v;
              }
            }
            if (by_hand) fence_proxy_async_smem();
            __syncwarp();
            // the one arrival of the phase: the copies' bytes and what was written above
            if (lane == 0) mbar_arrive_expect_tx(full + st, __popc(by_tma) * kBS * D * 2);
          }
          __syncwarp();
          ++cnt;
        }
      }
    }
    // copies in flight land before the CTA can retire (bounded)
    if constexpr (C::kCoded) {
      for (uint32_t c = cnt > RS ? cnt - RS : 0; c < cnt; ++c) mbar_wait(rfull + c % RS, (c / RS) & 1);
    } else {
      for (uint32_t c = cnt > S ? cnt - S : 0; c < cnt; ++c) mbar_wait(full + c % S, (c / S) & 1);
    }
    if (qn) mbar_wait(qfull, (qn - 1) & 1);
    __syncwarp();
   } else if (warp == C::kMmaWarp || warp == C::kMmaWarp + 2) {
    // ---- MMA issue, a warp for each tile.  A commit holds the issuing thread until
    // the MMAs before it have nearly run, and with one warp for both tiles the
    // tensor core then idled between groups (3000 cycles a step for 2100 of work).
    // The warp stays together and elects a lane for each group: operands then
    // reach their uniform registers directly (20 cycles an instruction; 54 when
    // the whole role ran in one divergent lane). ----
    const int t = warp == C::kMmaWarp ? 0 : 1;
    constexpr uint32_t kIdescPV = umma_idesc_f16(128, D, C::kPvBf16, true);
    // Shared-memory descriptors by words: the high one is the same for all (8-row
    // atoms of 1024 bytes), the low one holds the address and, for V, whose
    // rows are the product's K, the step from 64 columns to the next.
    constexpr uint32_t kHi = static_cast<uint32_t>(umma_sdesc(0, 0, 1024) >> 32);
    constexpr uint32_t kStep = C::kTile >> 4;
    const uint32_t dk0 = (smem_addr(smem) + C::kOffStage) >> 4;
    int st = 0;        // stage of the next K or V
    uint32_t ph = 0;   // ... and its parity
    uint32_t qn = 0, pn = 0;
    bool ok = true;
    auto uniform = [](int x) { return __shfl_sync(kFull, x, 0); };
    auto step = [&]() {
      if (++st == S) {
        st = 0;
        ph ^= 1;
      }
    };
    // One lane: S of half h, 64 tokens of the K in stage k; O += P V of half h, V in stage v.
    uint32_t dq = 0;
    auto scores = [&](int h, int k, int blocks) {
      const uint32_t kd = dk0 + k * kStep + h * (64 * 128 >> 4), d = tmem + 128 * t + 64 * h;
      const uint32_t idesc = umma_idesc_f16(128, 16 * min(blocks - 4 * h, 4), C::kQkBf16, false);
      if (blocks > 4 * h) {
#pragma unroll
        for (int e = 0; e < D / 16; ++e) {
          const uint32_t off = ((e >> 2) * C::kHalf + (e & 3) * 32) >> 4;
          umma_f16(d, ext_desc(dq + off, kHi), ext_desc(kd + off, kHi), idesc, e > 0);
        }
      }
    };
    auto values = [&](int h, int v, int blocks, bool accumulate) {
      const uint32_t vd = ((dk0 + v * kStep) | (C::kHalf >> 4) << 16) + h * (64 * 128 >> 4);
      const uint32_t d = tmem + C::kColO + D * t, a = tmem + 128 * t + 64 * h;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < blocks - 4 * h)
          umma_f16_ts(d, a + 8 * e, ext_desc(vd + e * (2048 >> 4), kHi), kIdescPV, accumulate || e > 0);
    };
    for (ExtWalk w(p, st0); ok && w.more(); w.next()) {
      if (w.it.steps == 0) continue;
      const int all = uniform(w.it.blocks), j0 = uniform(w.j0), j1 = uniform(w.j1);
      auto blocks = [&](int j) { return min(8, all - 8 * j); };
      dq = (smem_addr(smem) >> 4) + (w.two() ? t * kStep : 0);
      if (w.split()) {  // every other step, the stages of the others freed as they fill
        if (!(ok = uwait(qready, qn & 1))) break;
        ++qn;
        bool begun = false;
        for (int j = j0; ok && j < j1; ++j) {
          if (((j - j0) & 1) != t) {
#pragma unroll 1
            for (int q = 0; ok && q < 2; ++q) {
              ok = uwait(full + st, ph);
              if (ok && lane == 0) mbar_arrive(empty + st);
              __syncwarp();
              step();
            }
            continue;
          }
          if (!(ok = uwait(full + st, ph))) break;
          tmem_fence_after();
          if (elect_one()) {
            scores(0, st, blocks(j));
            umma_commit(sfull + 2 * t);
            scores(1, st, blocks(j));
            umma_commit(sfull + 2 * t + 1);
            umma_commit(empty + st);
          }
          __syncwarp();
          step();
          if (!(ok = uwait(full + st, ph) && uwait(pfull + 2 * t, pn & 1))) break;
          tmem_fence_after();
          if (elect_one()) {
            values(0, st, blocks(j), begun);
            umma_commit(pvhalf + t);
          }
          __syncwarp();
          if (!(ok = uwait(pfull + 2 * t + 1, pn & 1))) break;
          ++pn;
          tmem_fence_after();
          if (elect_one()) {
            values(1, st, blocks(j), true);
            umma_commit(empty + st);
          }
          __syncwarp();
          step();
          begun = true;
        }
        if (ok && elect_one()) {
          umma_commit(sfull + 2 * t);
          umma_commit(sfull + 2 * t + 1);
        }
        __syncwarp();
        continue;  // the softmax warps free Q, whose second tile holds the joined rows
      }
      if (t && !w.two()) {  // the item has no second tile: free the stages as they fill
        for (int j = 2 * j0; ok && j < 2 * j1; ++j) {
          ok = uwait(full + st, ph);
          if (ok && lane == 0) mbar_arrive(empty + st);
          __syncwarp();
          step();
        }
        if (!(ok = ok && uwait(qready, qn & 1))) break;
        ++qn;
        if (lane == 0) mbar_arrive(qempty);
        __syncwarp();
        continue;
      }
      ok = uwait(qready, qn & 1) && uwait(full + st, ph);
      ++qn;
      if (!ok) break;
      tmem_fence_after();
      if (elect_one()) {
        scores(0, st, blocks(j0));
        umma_commit(sfull + 2 * t);
        scores(1, st, blocks(j0));
        umma_commit(sfull + 2 * t + 1);
        if (j1 - j0 == 1) umma_commit(qempty);
      }
      __syncwarp();
      step();
      for (int j = j0; ok && j < j1; ++j) {
        const bool next = j + 1 < j1;
        const int vst = st;  // V of this step, then K of the next
        if (!(ok = uwait(full + st, ph))) break;
        step();
        if (next) {
          if (!(ok = uwait(full + st, ph))) break;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!(ok = uwait(pfull + 2 * t + h, pn & 1))) break;
          tmem_fence_after();
          if (elect_one()) {
            values(h, vst, blocks(j), j > j0 || h);
            if (next) scores(h, st, blocks(j + 1));
            // the only commit of a group, as each costs the tensor core some 100 cycles:
            // the softmax warps, who wait for it, free the stages
            umma_commit(sfull + 2 * t + h);
            if (h && j + 2 == j1) umma_commit(qempty);
          }
          __syncwarp();
        }
        ++pn;
        if (next) step();
      }
    }
    // nothing may still write tensor memory or read shared memory when the CTA ends (bounded)
    if (elect_one()) umma_commit(done + t);
    __syncwarp();
    mbar_wait(done + t, 0);
    __syncwarp();
   }
  } else if (warp < 8) {
    if constexpr (C::kCoded) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    // ---- softmax: thread = row of tile t ----
    const int t = warp >> 2;
    const int r = tid & 127;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_row = tmem + lane_base + 128 * t;
    const uint32_t o_row = tmem + lane_base + C::kColO + D * t;
    const float sl2 = p.negate ? -p.scale_log2 : p.scale_log2;
    uint32_t sn = 0, hn = 0, jn = 0, merges = 0;  // phases of sfull, pvhalf, joined, stored used
    uint32_t steps_done = 0;              // steps of this CTA before the piece
    bool ok = true;
    for (ExtWalk w(p, st0); ok && w.more(); w.next()) {
      const bool split = w.it.steps != 0 && w.split();
      const int row = w.qb * kExtRows + (split ? 0 : t * 128) + r;
      const bool real = (split ? 0 : t * 128) + r < w.rows();
      const int pos = w.s.len - w.s.n + (row >> p.group_shift);
      float m_run = -INFINITY, l_run = 0.f, unit = 0.f;
      const bool mine_t = t == 0 || split || w.two();  // this tile has rows
      const bool some = __any_sync(kFull, real);
      if (w.it.steps != 0 && mine_t) {
        const int lo = p.window ? max(pos - p.window + 1, 0) : 0;
        const int sinks = p.sinks, blocks = w.it.blocks, near = w.it.near, gap = w.it.gap, j0 = w.j0, j1 = w.j1;
        auto logical = [&](int i) { return i < near ? i : i + gap; };
        // Steps whose 128 tokens every row of the warp sees: j < j_sinks (among
        // the sinks) and j_from <= j < j_to (in every row's window, none ahead).
        const int pos_min = __reduce_min_sync(kFull, real ? pos : INT_MAX);
        const int lo_max = __reduce_max_sync(kFull, real ? lo : 0);
        const int j_sinks = p.window ? max(min(min(sinks, pos_min + 1) / kBS, gap ? near : blocks), 0) / 8 : 0;
        const int j_from = (max(near, (lo_max + kBS - 1) / kBS - gap) + 7) / 8;
        const int j_to = min(blocks, max((min(pos_min, INT_MAX - 1) + 1) / kBS - gap, 0)) / 8;
        const int first = split ? j0 + t : j0;
        bool set = false;  // every row of the warp has a reference
        for (int j = first; ok && j < j1; j += split ? 2 : 1) {
          const uint32_t step = steps_done + (j - j0);
          const bool masked = !(j < j_sinks || (j >= j_from && j < j_to));
          const ulonglong2 *ks4 = reinterpret_cast<const ulonglong2 *>(scales + (step & 3) * 128);
          // x = s - m of 64 tokens against the reference so far (minus infinity where this row sees nothing)
          auto scores = [&](auto hide, int h, float neg, float (&x)[64]) {
            const uint64_t scale2 = f2_pack(sl2, sl2), neg2 = f2_pack(neg, neg);
#pragma unroll
            for (int e = 0; e < 64; e += 4) {
              uint64_t k0 = scale2, k1 = scale2;
              if constexpr (C::kCoded) {
                const ulonglong2 k4 = ks4[16 * h + e / 4];
                k0 = k4.x;
                k1 = k4.y;
              }
              f2_unpack(f2_fma(f2_pack(x[e], x[e + 1]), k0, neg2), x[e], x[e + 1]);
              f2_unpack(f2_fma(f2_pack(x[e + 2], x[e + 3]), k1, neg2), x[e + 2], x[e + 3]);
            }
            if constexpr (decltype(hide)::value) {
              uint32_t see[2] = {0u, 0u};  // the tokens this row sees, one bit each
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const int i = 8 * j + 4 * h + u;
                const int base = logical(i) * kBS;
                uint32_t m = 0;
                if (real && i < blocks && base <= pos) {
                  m = pos - base >= 15 ? 0xFFFFu : (2u << (pos - base)) - 1;
                  if (lo > base) {
                    uint32_t in = lo - base >= 16 ? 0u : 0xFFFFu << (lo - base);
                    if (sinks > base) in |= sinks - base >= 16 ? 0xFFFFu : (1u << (sinks - base)) - 1;
                    m &= in;
                  }
                }
                see[u >> 1] |= u & 1 ? m << 16 : m;
              }
#pragma unroll
              for (int e = 0; e < 64; ++e) x[e] = (see[e >> 5] >> (e & 31)) & 1 ? x[e] : -INFINITY;
            }
          };
          auto maximum = [&](const float (&x)[64]) {
            float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 64; e += 8) {
#pragma unroll
              for (int i = 0; i < 4; ++i) mx4[i] = fmaxf(mx4[i], fmaxf(x[e + i], x[e + i + 4]));
            }
            return fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
          };
          // A row whose reference lags its maximum too far (or is not set) takes
          // a new one: x, l and O change units, the latter by the factor returned.
          auto renew = [&](float mx, float (&x)[64]) {
            float factor = 1.f;
            const bool lags = mx > (m_run == -INFINITY ? -INFINITY : C::kLag);
            {
              if (lags) {
                const float m_new = mx + (m_run == -INFINITY ? 0.f : m_run);
                factor = fast_exp2(m_run - m_new);
                m_run = m_new;
                l_run *= factor;
              }
              const float by = lags ? mx : 0.f;
#pragma unroll
              for (int e = 0; e < 64; ++e) x[e] -= by;
            }
            return factor;
          };
          // O by a factor; the MMAs must be done with it
          auto rescale = [&](float factor) {
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              float o[16];
              tmem_ld16(o_row + 16 * c, o);
              tmem_ld_wait();
              uint32_t w16[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) w16[e] = __float_as_uint(o[e] * factor);
              tmem_st16(o_row + 16 * c, w16);
            }
          };
          // P = 2^x of 32 tokens, packed, and their sum
          auto weights = [&](const float *x, uint32_t (&pk)[16]) {
            uint64_t s2[2] = {0ull, 0ull};
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              float y[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) y[i] = fast_exp2(x[e + i]);
              s2[0] = f2_add(s2[0], f2_pack(y[0], y[1]));
              s2[1] = f2_add(s2[1], f2_pack(y[2], y[3]));
              pk[e / 2] = pack2<C::PT>(y[0], y[1]);
              pk[e / 2 + 1] = pack2<C::PT>(y[2], y[3]);
            }
            float a, b;
            f2_unpack(f2_add(s2[0], s2[1]), a, b);
            return a + b;
          };
          // The step's two halves of 64 tokens, each handed to the MMAs when its P is
          // written (in the columns of S that have been read already).  A loop, not
          // unrolled: the body has to stay in the instruction cache.
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            if (!(ok = uwait(sfull + 2 * t + h, sn & 1))) break;
            tmem_fence_after();
            if constexpr (C::kCoded) {
              // V's unit of this step (never smaller than the last one's).  Waited for
              // after S: by then the stage's phase before this one has passed, which a
              // wait by parity needs.
              const uint32_t vc = 2 * step + 1;
              if (!h && !(ok = uwait(full + vc % S, (vc / S) & 1))) break;
            }
            if (h && !split && (warp & 3) == 0 && lane == 0) {  // done with this K and the last step's V
              mbar_arrive(empty + 2 * step % S);
              if (j > j0) mbar_arrive(empty + (2 * step - 1) % S);
            }
            if (some && 8 * j + 4 * h < blocks) {
              // P = 2^(s - m) and its sum against the reference so far.  No maximum is
              // looked for: a sum within kSumTop shows that no P is beyond it.  Only
              // otherwise, where a row has no reference yet, or where tokens are
              // hidden, does the second form run (S is there until P is stored).
              uint32_t pk[2][16];
              float sum;
              bool usual = !masked && set;
              if (__builtin_expect(usual, 1)) {
                float x[64];
                tmem_ld64(s_row + 64 * h, x);
                tmem_ld_wait();
                scores(std::false_type(), h, -m_run, x);
                sum = weights(x, pk[0]) + weights(x + 32, pk[1]);
                usual = !__any_sync(kFull, real && !(sum <= C::kSumTop));
                if constexpr (C::kCoded) usual &= units[step & 3] == unit;  // the same for the whole warp
              }
              if (__builtin_expect(!usual, 0)) {
                float x[64];
                tmem_ld64(s_row + 64 * h, x);
                tmem_ld_wait();
                scores(std::true_type(), h, m_run == -INFINITY ? 0.f : -m_run, x);
                float factor = renew(maximum(x), x);
                sum = weights(x, pk[0]) + weights(x + 32, pk[1]);
                set = !__any_sync(kFull, real && m_run == -INFINITY);
                if constexpr (C::kCoded) {
                  const float u = units[step & 3];
                  if (u != unit) {
                    factor *= unit * __uint_as_float((254u << 23) - __float_as_uint(u));  // unit / u, powers of two
                    unit = u;
                  }
                }
                if ((j > first || h) && __any_sync(kFull, factor != 1.f)) {
                  // O must not be in the MMAs' hands: wait for P V of the half before
                  ok = split && h ? uwait(pvhalf + t, hn & 1) : uwait(sfull + 2 * t + (h ^ 1), (sn + h) & 1);
                  if (!ok) break;
                  tmem_fence_after();
                  rescale(factor);
                }
              }
              l_run += sum;
              tmem_st16(s_row + 64 * h, pk[0]);
              tmem_st16(s_row + 64 * h + 16, pk[1]);
              tmem_st_wait();
              tmem_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(pfull + 2 * t + h);
          }
          if (!ok) break;
          ++sn;
          if (split) ++hn;
        }
        if (ok) ok = uwait(sfull + 2 * t, sn & 1) && uwait(sfull + 2 * t + 1, sn & 1);  // O is complete
        if (ok && !split && (warp & 3) == 0 && lane == 0) mbar_arrive(empty + (2 * (steps_done + j1 - j0) - 1) % S);
        ++sn;
        if (!ok) break;
        tmem_fence_after();
      }
      float put = C::kCoded ? unit * (1.f / C::kVTop) : 1.f;
      // 32 columns of the accumulator, finite or what the definition gives.
      const int i_from = 8 * (split ? w.j0 + t : w.j0), i_to = min(8 * w.j1, w.it.blocks), stride = split ? 16 : 8;
      const float m_own = m_run, unit_own = put;
      auto columns = [&](int c, float (&v)[32]) {
        tmem_ld32(o_row + 32 * c, v);
        tmem_ld_wait();
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 32; ++e) sum = fmaf(v[e], 0.f, sum);
        const bool wrong = real && sum != 0.f && l_run == l_run;
        if (__builtin_expect(__any_sync(kFull, wrong), 0)) {
          if (wrong) {
            float x[32];
            ext_exact<D, CDT, QDT>(p, ext_exact_row<D>(p, w, row), i_from, i_to, 8, stride, 32 * c, m_own, x);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = C::kCoded ? x[e] / unit_own : x[e];
          }
          __syncwarp();
        }
      };
      // A split item: the second tile's rows go through shared memory (Q's second
      // tile, free here) to the first tile's threads, which join them to theirs.
      float join = 0.f;
      const float4 *joined_o = reinterpret_cast<const float4 *>(smem + C::kTile) + r;
      if (split && (warp & 3) < 2) {
        float2 *ml = reinterpret_cast<float2 *>(smem + C::kOffMisc + 112) + r;
        if (t) {
          float4 *so = reinterpret_cast<float4 *>(smem + C::kTile) + r;
          if (some) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              float v[32];
              columns(c, v);
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                so[(8 * c + e / 4) * 64] = make_float4(v[e] * put, v[e + 1] * put, v[e + 2] * put, v[e + 3] * put);
            }
            *ml = make_float2(m_run, l_run);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(joined + warp - 4);
        } else {
          if (!(ok = uwait(joined + warp, jn & 1))) break;
          ++jn;
          const float2 o = *ml;
          const float m = fmaxf(m_run, o.x);
          const float f0 = m > -INFINITY ? fast_exp2(m_run - m) : 0.f;
          join = m > -INFINITY ? fast_exp2(o.x - m) : 0.f;
          l_run = l_run * f0 + o.y * join;
          put *= f0;
          m_run = m;
        }
      }
      const bool writes = some && !(split && t);  // this warp has rows to write
      if (w.whole()) {
        // the whole item: O / l (zeros for rows that see nothing)
        if (writes) {
          const float inv = l_run > 0.f ? 1.f / l_run : (l_run == 0.f ? 0.f : l_run);
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float v[32];
            if (w.it.steps != 0) columns(c, v);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = l_run == 0.f ? 0.f : v[e] * put;
            if (split && l_run != 0.f) ext_join(v, joined_o + 8 * c * 64, join);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] *= inv;
            ext_store32<D, QDT>(p, w, row, 32 * c, v);
          }
        }
      } else {
        // A piece: fp32 partial in this CTA's slot (0: an item begun by an
        // earlier CTA, 1: one that this CTA begins), counted in at the CTA
        // that begins the item; whoever counts last merges.
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (w.j0 == 0 ? 1 : 0);
        if (writes) {
          float4 *po = reinterpret_cast<float4 *>(p.ws_o) + slot * (D / 4) * kExtRows + t * 128 + r;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float v[32];
            columns(c, v);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] *= put;
            if (split) ext_join(v, joined_o + 8 * c * 64, join);
            if (real) {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                po[(8 * c + e / 4) * kExtRows] = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
            }
          }
          if (real) reinterpret_cast<float2 *>(p.ws_ml)[slot * kExtRows + t * 128 + r] = make_float2(m_run, l_run);
        }
        // CTAs that hold the item's first and last step
        const int64_t item0 = w.pos - w.u;
        const int64_t shares = st0.shares, total = st0.total;
        const int c0 = static_cast<int>(((item0 + kExtItemCost + 1) * shares - 1) / total);
        const int c1 = static_cast<int>(((item0 + ext_weight(w.it)) * shares - 1) / total);
        __threadfence();
        __syncwarp();
        if (lane == 0) mbar_arrive(stored);
        if (tid == 0 && (ok = wait(stored, merges & 1))) {
          __threadfence();
          const bool last = atomicAdd(p.ws_ctr + c0, 1u) == static_cast<uint32_t>(c1 - c0);
          if (last) p.ws_ctr[c0] = 0;
          __threadfence();
          *last_flag = last ? 1 : 0;
          mbar_arrive(counted);
        }
        if (!(ok = uwait(counted, merges & 1))) break;
        ++merges;
        if (*last_flag) ext_merge<D, QDT>(p, w, c0, c1);
      }
      if (split && warp < 2) {  // the joined rows have been read: Q may be loaded again
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(qempty);
      }
      if (w.it.steps != 0) steps_done += w.j1 - w.j0;
      tmem_fence_before();
    }
  } else {
    // ---- coded caches: raw codes -> 16-bit operands in the MMA's layout ----
    if constexpr (C::kCoded) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
      const int ct = tid - C::kCvtWarp * 32;
      const float ksign = p.negate ? -p.scale_log2 : p.scale_log2;
      uint32_t cnt = 0, qn = 0;
      bool ok = true;
      for (ExtWalk w(p, st0); ok && w.more(); w.next()) {
        if (w.it.steps == 0) continue;
        float k_norm = ksign;
        if constexpr (C::kCvtQ) {
          // Queries: bf16 -> f16 in place, times the power of two that takes the
          // item's largest finite one to [2^14, 2^15): values 2^-29 of it and
          // larger keep all their bits.  The K scales undo the power.
          const int vecs = w.rows() * (D / 8);
          auto at = [&](int u) {
            const int row = u / (D / 8), ch = u % (D / 8);
            return reinterpret_cast<uint4 *>(smem + (row >> 7) * C::kTile + (ch >> 3) * C::kHalf + (row & 127) * 128 +
                                             (((ch & 7) ^ (row & 7)) << 4));
          };
          if (!(ok = uwait(qfull, qn & 1))) break;
          uint32_t top = 0;
          for (int u = ct; u < vecs; u += 128) {
            const uint4 v = *at(u);
            const uint32_t q4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t lo = q4[e] & 0x7FFFu, hi = (q4[e] >> 16) & 0x7FFFu;
              top = max(top, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
            }
          }
          top = __reduce_max_sync(kFull, top);
          if (lane == 0) {
            atomicMax(qtop + (qn & 1), top);
            mbar_arrive(qmax);
          }
          if (!(ok = uwait(qmax, qn & 1))) break;
          const uint32_t e = max(*reinterpret_cast<volatile uint32_t *>(qtop + (qn & 1)) >> 7, 15u);
          const float up = __uint_as_float((268u - e) << 23);
          k_norm = ksign * __uint_as_float((e - 14u) << 23);
          for (int u = ct; u < vecs; u += 128) {
            const uint4 v = *at(u);
            uint32_t q4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 f = unpack2<PKV_BF16>(q4[i]);
              q4[i] = pack2<PKV_F16>(f.x * up, f.y * up);
            }
            *at(u) = make_uint4(q4[0], q4[1], q4[2], q4[3]);
          }
          if (ct == 0) qtop[(qn & 1) ^ 1] = 0;  // for the next piece: nobody reads it before
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(qready);
          ++qn;
        }
        uint32_t unit_e = 1;  // biased exponent of V's unit, a power of two; it only grows within a piece
        for (int j = w.j0; ok && j < w.j1; ++j) {
#pragma unroll
          for (int kind = 0; kind < 2; ++kind) {
            const int rst = cnt % RS, st = cnt % S;
            if (!(ok = uwait(rfull + rst, (cnt / RS) & 1))) break;
            if (cnt >= S && !(ok = uwait(empty + st, (cnt / S - 1) & 1))) break;
            const uint8_t *raw = smem + C::kOffRaw + rst * C::kRaw;
            const float *rsc = reinterpret_cast<const float *>(raw + C::kRawCodes);
            uint8_t *dst = smem + C::kOffStage + st * C::kTile;
            const uint32_t step = cnt >> 1;
            float *ring = scales + (step & 3) * 128;
            // tokens of the step that are there: those of its blocks, up to the context's end
            const int there = min(16 * (w.it.blocks - 8 * j), 128);
            const int last = w.logical(8 * j + (there - 1) / kBS);  // the last block may end past the context
            const int valid = there - max((last + 1) * kBS - w.s.len, 0);
            float v_norm = 0.f;  // kVTop / unit
            if (kind == 0) {
              ring[ct] = rsc[ct] * k_norm;  // K scales with the softmax scale in them
            } else {
              float top = 0.f;
#pragma unroll
              for (int h = 0; h < 4; ++h)
                if (lane + 32 * h < valid && rsc[lane + 32 * h] < INFINITY) top = fmaxf(top, rsc[lane + 32 * h]);
#pragma unroll
              for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
              // the power of two at or above the largest scale
              const uint32_t e = min(max((__float_as_uint(top) + 0x7FFFFFu) >> 23, 1u), 253u);
              unit_e = max(unit_e, e);
              v_norm = __uint_as_float((254u - unit_e) << 23) * C::kVTop;
              if (ct == 0) units[step & 3] = __uint_as_float(unit_e << 23);
            }
            // Sixteen codes a unit; four units are loaded before the first is stored, to
            // keep the chain of load, conversion and store of one from setting the pace.
            constexpr int kCh = D / 16;  // units of a row
            constexpr int kBatch = 4;
#pragma unroll 1
            for (int u0 = ct; u0 < 128 * kCh; u0 += 128 * kBatch) {
              uint4 v[kBatch];
              float f[kBatch];
#pragma unroll
              for (int q = 0; q < kBatch; ++q) {
                const int row = (u0 + 128 * q) / kCh, ch = (u0 + 128 * q) % kCh;
                if (kind == 1 && C::VT == kInt4) {
                  const uint2 half = *reinterpret_cast<const uint2 *>(raw + row * (D / 2) + ch * 8);
                  v[q] = make_uint4(half.x, half.y, 0u, 0u);
                } else {
                  v[q] = *reinterpret_cast<const uint4 *>(raw + row * D + ch * 16);
                }
                if (kind == 1) f[q] = rsc[row];
              }
#pragma unroll
              for (int q = 0; q < kBatch; ++q) {
                const int row = (u0 + 128 * q) / kCh, ch = (u0 + 128 * q) % kCh;
                uint32_t o[8];
                if (kind == 0) {
                  ext_codes<C::KT>(v[q], o);
                } else {
                  ext_codes<C::VT>(v[q], o);
                  // V = code x scale / unit, the scale rounded to f16 first; zeros for
                  // tokens that are not there, whatever their bytes hold
                  const __half2 s2 = __float2half2_rn(f[q] * v_norm);
#pragma unroll
                  for (int e = 0; e < 8; ++e) {
                    const __half2 x = __hmul2(*reinterpret_cast<__half2 *>(&o[e]), s2);
                    o[e] = row < valid ? *reinterpret_cast<const uint32_t *>(&x) : 0u;
                  }
                }
                // two 16-byte chunks of the row's half; the order alternates between
                // the halves so that a quarter warp's stores hit different banks
                uint8_t *to = dst + (ch >> 2) * C::kHalf + row * 128;
                const int c0 = (2 * ch) & 7, flip = (ch >> 2) & 1;
                const uint4 a = make_uint4(o[0], o[1], o[2], o[3]), b = make_uint4(o[4], o[5], o[6], o[7]);
                *reinterpret_cast<uint4 *>(to + (((c0 + flip) ^ (row & 7)) << 4)) = flip ? b : a;
                *reinterpret_cast<uint4 *>(to + (((c0 + 1 - flip) ^ (row & 7)) << 4)) = flip ? a : b;
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(full + st);
              mbar_arrive(rempty + rst);
            }
            ++cnt;
          }
        }
      }
    }
  }

  tmem_fence_before();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tmem_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int D, int CDT, int QDT>
cudaError_t launch_extend(const ExtendParams &p, const CUtensorMap &tmq, const CUtensorMap &tmk,
                          const CUtensorMap &tmv, int grid) {
  using C = ExtendCfg<D, CDT, QDT>;
  cudaError_t e = cudaFuncSetAttribute(paged_extend_kernel<D, CDT, QDT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::kSmem);
  if (e != cudaSuccess) return e;
  paged_extend_kernel<D, CDT, QDT><<<grid, C::kThreads, C::kSmem, p.stream>>>(p, tmq, tmk, tmv);
  return cudaGetLastError();
}

}  // namespace pkv
