// Rotary positions: the table of cosines and sines, and the append that
// rotates queries and keys on the way.
//
// A pair (a, b) of a row's first rot_dim elements at position n and pair
// index i becomes (a c - b s, b c + a s) with c, s = cos, sin(n f_i) from the
// table; every product and the sum or difference is one fp32 operation (no
// fused multiply-add), so the result does not depend on how it is compiled
// and the codes of a coded cache can be compared bit for bit.  The rotated
// key goes to the cache straight from fp32: rounded once to a 16-bit type, or
// quantised with its own scale exactly as paged_kv_append does (common.cuh).
//
// Both are bound by memory: the append reads each row once and writes it once.
// A row is held by D / 8 lanes with 16 bytes each, so every load and store is
// a whole 32-byte sector, and a half-split pair's other element arrives by a
// shuffle.  A thread keeps one table slice for all of the rows it turns
// (they belong to one token), so the table costs one read per token and CTA.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "rope.h"

namespace pkv {

// One thread per (position, pair): angles in 64 bits, because a far
// position's angle (10^6 radians and more) has no fractional precision left
// in 32.
__global__ void __launch_bounds__(256) rope_table_kernel(float *__restrict__ table, int64_t entries, int32_t half,
                                                         const RopeTable t) {
  const int64_t nth = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; e < entries; e += nth) {
    const int64_t pos = e / half;
    const int i = static_cast<int>(e - pos * half);
    double f = pow(t.base, -static_cast<double>(i) / half);
    if (t.scaling == PKV_ROPE_LINEAR) {
      f /= t.factor;
    } else if (t.scaling == PKV_ROPE_BY_PARTS) {
      // turns of this pair over the original context: many turns keep their
      // frequency, few are interpolated, and a ramp joins the two
      const double turns = t.original_max * f / 6.283185307179586476925286766559;
      const double g = fmin(fmax((turns - t.slow_turns) / (t.fast_turns - t.slow_turns), 0.0), 1.0);
      f = f / t.factor * (1.0 - g) + f * g;
    }
    double s, c;
    sincos(static_cast<double>(pos) * f, &s, &c);
    table[pos * 2 * half + i] = static_cast<float>(c * t.magnitude);
    table[pos * 2 * half + half + i] = static_cast<float>(s * t.magnitude);
  }
}

cudaError_t run_rope_table(float *table, int64_t max_positions, int32_t rot_dim, const RopeTable &t,
                           cudaStream_t stream) {
  const int64_t entries = max_positions * (rot_dim / 2);
  if (entries == 0) return cudaSuccess;
  const int64_t blocks = std::min<int64_t>((entries + 255) / 256, 1 << 16);
  rope_table_kernel<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(table, entries, rot_dim / 2, t);
  return cudaGetLastError();
}

namespace {

// The lanes of one row (a power of two of them, aligned within the warp).
template <int LANES>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = LANES / 2; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

// Eight fp32 values of a row, 8 l .. 8 l + 7, into cache row `row` of storage
// type CDT.  All lanes of the warp take part in the row's maximum; `write`
// says whether this row is stored.
template <int D, int IDT, int CDT>
__device__ __forceinline__ void store_cache8(const float (&x)[8], uint8_t *cache, float *scales, int64_t row,
                                             int64_t srow, int l, bool write) {
  constexpr int LANES = D / 8;
  if constexpr (!is_coded(CDT)) {
    if (write) {
      const uint4 v = make_uint4(pack2<CDT>(x[0], x[1]), pack2<CDT>(x[2], x[3]), pack2<CDT>(x[4], x[5]),
                                 pack2<CDT>(x[6], x[7]));
      *reinterpret_cast<uint4 *>(cache + row * (2 * D) + l * 16) = v;
    }
  } else {
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));
    amax = row_max<LANES>(amax);
    const float s = (amax == 0.f) ? 1.f : __fdiv_rn(amax, code_range<CDT>());
    constexpr int kBits = CDT == kInt4 ? 4 : 8;
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const uint32_t c2 = encode2<CDT>(__fdiv_rn(x[e], s), __fdiv_rn(x[e + 1], s));
      w[(e * kBits) >> 5] |= c2 << ((e * kBits) & 31);
    }
    if (write) {
      if constexpr (CDT == kInt4)
        *reinterpret_cast<uint32_t *>(cache + row * (D / 2) + l * 4) = w[0];
      else
        *reinterpret_cast<uint2 *>(cache + row * D + l * 8) = make_uint2(w[0], w[1]);
      if (l == 0) scales[srow] = s;
    }
  }
}

// Block (token, part): D / 8 lanes a row, each group of lanes every
// (groups x parts)-th row of the token's Hq + 2 Hkv rows.
template <int D, int IDT, int CDT>
__global__ void __launch_bounds__(256) append_rope_kernel(const AppendRopeArgs a) {
  constexpr int LANES = D / 8;
  constexpr int GROUPS = 256 / LANES;
  const int l = threadIdx.x & (LANES - 1);
  const int group = threadIdx.x / LANES;
  const int64_t t = blockIdx.x;
  const int32_t pos = a.positions[t];
  if (pos < 0 || pos >= a.max_positions) {
    if (threadIdx.x == 0 && blockIdx.y == 0) report(a.d_error, PKV_DEVERR_BAD_POSITION);
    return;
  }
  const int32_t slot = a.slot_mapping[t];
  const bool in_pool = slot < static_cast<int64_t>(a.num_blocks) * a.block_size;
  if (!in_pool && threadIdx.x == 0 && blockIdx.y == 0) report(a.d_error, PKV_DEVERR_BAD_SLOT);
  const bool keep = slot >= 0 && in_pool;
  const int64_t blk = keep ? slot / a.block_size : 0;
  const int off = keep ? slot % a.block_size : 0;

  // This lane's cosines and sines: elements e0 .. e0 + 7 of every row.  Half
  // layout: pair of element e is e (first half) or e - half; interleaved:
  // e / 2.  The partner of a half-layout lane is `half / 8` lanes away.
  const int half = a.rot_dim >> 1;
  const int e0 = l * 8;
  const bool turned = e0 < a.rot_dim;
  const bool second = !a.interleaved && e0 >= half;
  const int src = turned && !a.interleaved ? (second ? l - half / 8 : l + half / 8) : l;
  float c[8], s[8];
  if (turned) {
    const float *row = a.cos_sin + static_cast<int64_t>(pos) * a.rot_dim;
    if (a.interleaved) {
      const float4 c4 = __ldg(reinterpret_cast<const float4 *>(row + e0 / 2));
      const float4 s4 = __ldg(reinterpret_cast<const float4 *>(row + half + e0 / 2));
      c[0] = c[1] = c4.x; c[2] = c[3] = c4.y; c[4] = c[5] = c4.z; c[6] = c[7] = c4.w;
      s[0] = s[1] = s4.x; s[2] = s[3] = s4.y; s[4] = s[5] = s4.z; s[6] = s[7] = s4.w;
    } else {
      const int i0 = second ? e0 - half : e0;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float4 c4 = __ldg(reinterpret_cast<const float4 *>(row + i0) + q);
        const float4 s4 = __ldg(reinterpret_cast<const float4 *>(row + half + i0) + q);
        c[4 * q] = c4.x; c[4 * q + 1] = c4.y; c[4 * q + 2] = c4.z; c[4 * q + 3] = c4.w;
        s[4 * q] = s4.x; s[4 * q + 1] = s4.y; s[4 * q + 2] = s4.z; s[4 * q + 3] = s4.w;
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) { c[e] = 1.f; s[e] = 0.f; }
  }

  const int hq = a.num_q_heads, hkv = a.num_kv_heads;
  const int rows = hq + 2 * hkv;
  constexpr int U = 4;  // rows in flight per group of lanes
  const int step = GROUPS * gridDim.y;
  // whole warps run together (shuffles): groups past the last row idle along
  for (int r0 = blockIdx.y * GROUPS + group; r0 - group < rows; r0 += U * step) {
    uint4 in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * step;
      const uint8_t *from = nullptr;
      if (r < hq) from = a.q + (t * a.q_stride + static_cast<int64_t>(r) * D) * 2;
      else if (r < hq + hkv) from = a.k + (t * a.k_stride + static_cast<int64_t>(r - hq) * D) * 2;
      else if (r < rows) from = a.v + (t * a.v_stride + static_cast<int64_t>(r - hq - hkv) * D) * 2;
      const bool skip = r >= hq && !keep;  // a key or value that goes nowhere
      in[u] = from && !skip ? *reinterpret_cast<const uint4 *>(from + l * 16) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * step;
      if (r - group >= rows) break;  // the same for the whole block
      float x[8];
      const uint32_t w[4] = {in[u].x, in[u].y, in[u].z, in[u].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<IDT>(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
      float y[8];
      if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          y[e] = __fsub_rn(__fmul_rn(x[e], c[e]), __fmul_rn(x[e + 1], s[e]));
          y[e + 1] = __fadd_rn(__fmul_rn(x[e + 1], c[e]), __fmul_rn(x[e], s[e]));
        }
      } else {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = __shfl_sync(kFull, w[i], src, LANES);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = unpack2<IDT>(o[i]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int e = 2 * i + h;
            const float other = h ? f.y : f.x;
            const float mine = __fmul_rn(x[e], c[e]), theirs = __fmul_rn(other, s[e]);
            y[e] = second ? __fadd_rn(mine, theirs) : __fsub_rn(mine, theirs);
          }
        }
      }
      if (!turned) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[e];
      }
      if (r < hq) {
        const uint4 v = make_uint4(pack2<IDT>(y[0], y[1]), pack2<IDT>(y[2], y[3]), pack2<IDT>(y[4], y[5]),
                                   pack2<IDT>(y[6], y[7]));
        *reinterpret_cast<uint4 *>(a.q_out + (t * hq + r) * (D * 2) + l * 16) = v;
      }
      // Rows of keys and values: a warp may hold rows of several kinds, so
      // the row maximum is taken by every lane and the stores are guarded.
      const bool is_k = r >= hq && r < hq + hkv, is_v = r >= hq + hkv && r < rows;
      if (__any_sync(kFull, is_k)) {
        const int h = is_k ? r - hq : 0;
        const int64_t bh = blk * hkv + h;
        store_cache8<D, IDT, k_part(CDT)>(y, a.k_cache, a.k_scale, bh * a.block_size + off,
                                          bh * 2 * a.block_size + off, l, is_k && keep);
      }
      if (__any_sync(kFull, is_v)) {
        const int h = is_v ? r - hq - hkv : 0;
        const int64_t bh = blk * hkv + h;
        store_cache8<D, IDT, v_part(CDT)>(x, a.v_cache, a.v_scale, bh * a.block_size + off,
                                          bh * 2 * a.block_size + off, l, is_v && keep);
      }
    }
  }
}

template <int D, int IDT, int CDT>
cudaError_t launch_append_rope(const AppendRopeArgs &a) {
  constexpr int GROUPS = 256 * 8 / D;
  const int rows = a.num_q_heads + 2 * a.num_kv_heads;
  // One CTA per token keeps its table slice for all of the token's rows; with
  // fewer tokens than would fill the SMs the rows are spread over more CTAs
  // (one row per group of lanes).
  const int parts = a.num_tokens >= kRopeFullTokens ? 1 : (rows + GROUPS - 1) / GROUPS;
  append_rope_kernel<D, IDT, CDT><<<dim3(static_cast<unsigned>(a.num_tokens), static_cast<unsigned>(parts)), 256, 0,
                                    a.stream>>>(a);
  return cudaGetLastError();
}

template <int D, int CDT>
cudaError_t by_input(const AppendRopeArgs &a) {
  return a.in_dtype == PKV_BF16 ? launch_append_rope<D, PKV_BF16, CDT>(a) : launch_append_rope<D, PKV_F16, CDT>(a);
}

template <int D>
cudaError_t by_cache(const AppendRopeArgs &a) {
  switch (a.cache_dtype) {
    case PKV_FP8_E4M3: return by_input<D, PKV_FP8_E4M3>(a);
    case PKV_FP8_E5M2: return by_input<D, PKV_FP8_E5M2>(a);
    case PKV_INT8: return by_input<D, PKV_INT8>(a);
    case PKV_FP8_E4M3_INT4: return by_input<D, PKV_FP8_E4M3_INT4>(a);
    case PKV_BF16: return launch_append_rope<D, PKV_BF16, PKV_BF16>(a);
    default: return launch_append_rope<D, PKV_F16, PKV_F16>(a);
  }
}

}  // namespace

cudaError_t run_append_rope(const AppendRopeArgs &a) {
  if (a.num_tokens == 0) return cudaSuccess;
  return a.head_dim == 128 ? by_cache<128>(a) : by_cache<64>(a);
}

}  // namespace pkv
