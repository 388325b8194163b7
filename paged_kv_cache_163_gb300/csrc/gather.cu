// Reading the cache back: cached rows of K and V as contiguous rows, coded
// ones as code x scale (one fp32 product, rounded once to the output type).
//
// Bound by memory: every cached row is read once and every output row written
// once.  A CTA takes 8 to 32 consecutive output rows (of one of K and V), finds
// their slots once (a thread a row, from the tables), and then moves rows x
// heads pieces of one row of one head: D / 8 lanes a piece, 8 elements a
// lane, so the 16-bit side moves in 16-byte vectors and all sectors are whole
// (a piece is 64 to 256 contiguous bytes on each side).  kUnroll pieces per
// lane are in flight before the first is stored.  16 sequences of 16k-32k tokens
// of 8 heads of 128, E4M3 to BF16: 368 us, 6.6 TB/s, 98% of a plain copy.
#include "common.cuh"
#include "gather.h"

namespace pkv {

namespace {

constexpr int kMaxRows = 32;  // output rows of a CTA
constexpr int kUnroll = 4;

// Eight elements of storage type DT (16, 8 or 4 bytes), as loaded.
template <int DT>
struct Raw8 {
  static constexpr int kBytes = row_bytes(DT, 8);
  uint32_t w[kBytes / 4];
};

template <int DT>
__device__ __forceinline__ void load8(const uint8_t *from, Raw8<DT> &r) {
  if constexpr (Raw8<DT>::kBytes == 16) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(from));
    r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
  } else if constexpr (Raw8<DT>::kBytes == 8) {
    const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(from));
    r.w[0] = v.x; r.w[1] = v.y;
  } else {
    r.w[0] = __ldcs(reinterpret_cast<const uint32_t *>(from));
  }
}

template <int DT>
__device__ __forceinline__ void values8(const Raw8<DT> &r, float (&x)[8]) {
  if constexpr (is_code8(DT)) {
    unpack_code4<DT>(r.w[0], x);
    unpack_code4<DT>(r.w[1], x + 4);
  } else if constexpr (DT == kInt4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // bytes 2i, 2i + 1: elements 4i .. 4i + 3
      uint32_t pair, lo, hi;
      asm("prmt.b32 %0, %1, 0, %2;" : "=r"(pair) : "r"(r.w[0]), "r"(i ? 0x4342 : 0x4140));
      int4_pair_to_f16x2(pair, lo, hi);
      const float2 l = __half22float2(*reinterpret_cast<__half2 *>(&lo));
      const float2 h = __half22float2(*reinterpret_cast<__half2 *>(&hi));
      x[4 * i] = l.x;
      x[4 * i + 1] = h.x;
      x[4 * i + 2] = l.y;
      x[4 * i + 3] = h.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<DT>(r.w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

// Eight values to the output row (element e0 on), in the output type.
template <int ODT>
__device__ __forceinline__ void store8(uint8_t *to, const float (&x)[8]) {
  if constexpr (ODT == PKV_F32) {
    __stcs(reinterpret_cast<float4 *>(to), make_float4(x[0], x[1], x[2], x[3]));
    __stcs(reinterpret_cast<float4 *>(to) + 1, make_float4(x[4], x[5], x[6], x[7]));
  } else {
    __stcs(reinterpret_cast<uint4 *>(to), make_uint4(pack2<ODT>(x[0], x[1]), pack2<ODT>(x[2], x[3]),
                                                     pack2<ODT>(x[4], x[5]), pack2<ODT>(x[6], x[7])));
  }
}

// One of K and V (storage type DT) of this CTA's rows.
template <int D, int DT, int ODT>
__device__ __forceinline__ void gather_part(const GatherArgs &a, const uint8_t *cache, const float *scales,
                                            uint8_t *out, const int2 *slot, int rows, int64_t row0) {
  constexpr int LANES = D / 8;
  constexpr int GROUPS = 256 / LANES;
  constexpr int ESZ = ODT == PKV_F32 ? 4 : 2;
  const int l = threadIdx.x & (LANES - 1);
  const int hkv = a.num_kv_heads;
  const int pieces = rows * hkv;
  for (int p0 = threadIdx.x / LANES; p0 < pieces; p0 += kUnroll * GROUPS) {
    Raw8<DT> raw[kUnroll];
    float sc[kUnroll];
    bool ok[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int piece = p0 + u * GROUPS;
      ok[u] = false;
      if (piece < pieces) {
        const int r = piece / hkv, h = piece - r * hkv;
        const int2 sl = slot[r];
        if (sl.x >= 0) {
          ok[u] = true;
          const int64_t row = sl.x + h * a.block_size;
          load8<DT>(cache + row * row_bytes(DT, D) + l * Raw8<DT>::kBytes, raw[u]);
          if constexpr (is_coded(DT)) sc[u] = scales[2 * row - sl.y];  // [block x head][2][block_size]
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (!ok[u]) continue;
      const int piece = p0 + u * GROUPS;
      float x[8];
      values8<DT>(raw[u], x);
      if constexpr (is_coded(DT)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= sc[u];
      }
      // piece = row x heads + head is also the order of the output
      store8<ODT>(out + ((row0 * hkv + piece) * D + l * 8) * ESZ, x);
    }
  }
}

template <int D, int CDT, int ODT>
__global__ void __launch_bounds__(256) gather_kernel(const GatherArgs a, const int rows) {
  __shared__ int2 slot[kMaxRows];  // cache row of head 0 (-1: none), and its place in the block
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows;
  // The sequence of the first row: how many sequences end at or before it
  // (starts ascend), counted by the whole CTA in one pass of loads.
  int seq = 0;
  for (int b0 = 0; b0 < a.num_seqs; b0 += 256) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    seq += __syncthreads_count(b < a.num_seqs && a.out_starts[b + 1] <= row0);
  }
  if (threadIdx.x < rows) {
    const int64_t row = row0 + threadIdx.x;
    int2 sl = make_int2(-1, 0);
    int b = seq;
    while (b < a.num_seqs && a.out_starts[b + 1] <= row) ++b;
    if (b < a.num_seqs && row < a.num_rows && row >= a.out_starts[b]) {
      const int64_t token = (a.token_starts ? a.token_starts[b] : 0) + (row - a.out_starts[b]);
      const int32_t len = a.context_lens[b];
      if (token < 0 || token >= len || token >= static_cast<int64_t>(a.max_blocks_per_seq) * a.block_size) {
        report(a.d_error, PKV_DEVERR_BAD_CONTEXT_LEN);
      } else {
        const int32_t blk = a.block_tables[static_cast<int64_t>(b) * a.max_blocks_per_seq + token / a.block_size];
        if (blk < 0 || blk >= a.num_blocks) report(a.d_error, PKV_DEVERR_BAD_BLOCK);
        else {
          sl.y = static_cast<int32_t>(token % a.block_size);
          sl.x = blk * a.num_kv_heads * a.block_size + sl.y;  // (a pool's rows are numbered in 31 bits)
        }
      }
    }
    slot[threadIdx.x] = sl;
  }
  __syncthreads();
  if (blockIdx.y == 0)
    gather_part<D, k_part(CDT), ODT>(a, a.k_cache, a.k_scale, a.k_out, slot, rows, row0);
  else
    gather_part<D, v_part(CDT), ODT>(a, a.v_cache, a.v_scale, a.v_out, slot, rows, row0);
}

template <int D, int CDT, int ODT>
cudaError_t launch_gather(const GatherArgs &a) {
  // Few rows: enough CTAs for the SMs; many: longer runs of a CTA on neighbouring
  // addresses.  Measured with 8, 16 and 32 rows a CTA, us: 1500 rows of 8 heads,
  // BF16, 6.7, 8.5, 10.6; 393000, E4M3 to BF16, 454, 424, 410.
  const int rows = a.num_rows <= 2400 ? 8 : a.num_rows <= 40000 ? 16 : kMaxRows;
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.num_rows) + rows - 1) / rows), 2);
  gather_kernel<D, CDT, ODT><<<grid, 256, 0, a.stream>>>(a, rows);
  return cudaGetLastError();
}

template <int D, int CDT>
cudaError_t by_output(const GatherArgs &a) {
  switch (a.out_dtype) {
    case PKV_F32: return launch_gather<D, CDT, PKV_F32>(a);
    case PKV_BF16: return launch_gather<D, CDT, PKV_BF16>(a);
    default: return launch_gather<D, CDT, PKV_F16>(a);
  }
}

template <int D>
cudaError_t by_cache(const GatherArgs &a) {
  switch (a.cache_dtype) {
    case PKV_FP8_E4M3: return by_output<D, PKV_FP8_E4M3>(a);
    case PKV_FP8_E5M2: return by_output<D, PKV_FP8_E5M2>(a);
    case PKV_INT8: return by_output<D, PKV_INT8>(a);
    case PKV_FP8_E4M3_INT4: return by_output<D, PKV_FP8_E4M3_INT4>(a);
    case PKV_BF16: return a.out_dtype == PKV_F32 ? launch_gather<D, PKV_BF16, PKV_F32>(a)
                                                 : launch_gather<D, PKV_BF16, PKV_BF16>(a);
    default: return a.out_dtype == PKV_F32 ? launch_gather<D, PKV_F16, PKV_F32>(a)
                                           : launch_gather<D, PKV_F16, PKV_F16>(a);
  }
}

}  // namespace

cudaError_t run_gather(const GatherArgs &a) {
  if (a.num_rows == 0 || a.num_seqs == 0) return cudaSuccess;
  return a.head_dim == 128 ? by_cache<128>(a) : by_cache<64>(a);
}

}  // namespace pkv
