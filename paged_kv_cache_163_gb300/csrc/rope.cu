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
// A row is held by D / 8 lanes with 16 bytes each, two 8-byte vectors that hold
// both elements of four pairs, so loads and stores fill whole sectors and no
// element crosses lanes.  A thread keeps one table slice for all of the rows it
// turns (they belong to one token), so the table costs one read per token and
// CTA.
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

// Eight fp32 values of a row, four from element e0 and four from e1, into
// cache row `row` of storage type CDT (a pool's rows are numbered in 31 bits),
// place `off` of its block.  The D / 8 lanes of the row (`lanes`)
// call it together.
template <int D, int CDT>
__device__ __forceinline__ void store_cache8(const float (&x)[8], uint8_t *cache, float *scales, int32_t row,
                                             int32_t off, int e0, int e1, unsigned lanes) {
  if constexpr (!is_coded(CDT)) {
    uint8_t *to = cache + static_cast<int64_t>(row) * (2 * D);
    *reinterpret_cast<uint2 *>(to + 2 * e0) = make_uint2(pack2<CDT>(x[0], x[1]), pack2<CDT>(x[2], x[3]));
    *reinterpret_cast<uint2 *>(to + 2 * e1) = make_uint2(pack2<CDT>(x[4], x[5]), pack2<CDT>(x[6], x[7]));
  } else {
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));
#pragma unroll
    for (int o = D / 16; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(lanes, amax, o));
    const float s = (amax == 0.f) ? 1.f : __fdiv_rn(amax, code_range<CDT>());
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 8; e += 2) c[e / 2] = encode2<CDT>(__fdiv_rn(x[e], s), __fdiv_rn(x[e + 1], s));
    if constexpr (CDT == kInt4) {
      uint8_t *to = cache + static_cast<int64_t>(row) * (D / 2);
      *reinterpret_cast<uint16_t *>(to + e0 / 2) = static_cast<uint16_t>(c[0] | c[1] << 8);
      *reinterpret_cast<uint16_t *>(to + e1 / 2) = static_cast<uint16_t>(c[2] | c[3] << 8);
    } else {
      uint8_t *to = cache + static_cast<int64_t>(row) * D;
      *reinterpret_cast<uint32_t *>(to + e0) = c[0] | c[1] << 16;
      *reinterpret_cast<uint32_t *>(to + e1) = c[2] | c[3] << 16;
    }
    if (e0 == 0) scales[2 * static_cast<int64_t>(row) - off] = s;  // [block x head][2][block_size]
  }
}

// Block (tokens, part): D / 8 lanes a row, each group of lanes every
// (groups of the token x parts)-th row of a token's Hq + 2 Hkv rows.  A lane holds both
// elements of four pairs, in 8-byte vectors: elements 4l .. and rot_dim / 2 +
// 4l .. (half layout), 8l .. 8l + 7 (interleaved); the lanes past the rotated
// part, and all lanes of a value row, hold eight elements that pass through.
// Measured: 16384 tokens of 48 rows of 128, BF16, 70 us (5.9 TB/s; 89 with three rows
// in flight, streaming loads and six CTAs an SM); 4097 tokens of 12 rows of 64, F16
// to E5M2, 6 us, 13.6 with a CTA a token; 16 tokens 2.6 us.
constexpr int kRopeRows = 6;  // rows in flight per group of lanes
template <int D, int IDT, int CDT, bool IL>
__global__ void __launch_bounds__(256, 4) append_rope_kernel(const AppendRopeArgs a, const int per_token) {
  constexpr int LANES = D / 8;
  constexpr int GROUPS = 256 / LANES;
  const int l = threadIdx.x & (LANES - 1);
  const int group = threadIdx.x / LANES;
  const unsigned lanes = (LANES == 32 ? 0u : 1u << LANES) - 1u << (threadIdx.x & 31 & ~(LANES - 1));
  // `per_token` groups of lanes take a token's rows, so a CTA has GROUPS / per_token tokens
  const int own = group / per_token, share = group - own * per_token;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (GROUPS / per_token) + own;
  if (own >= GROUPS / per_token || t >= a.num_tokens) return;
  const bool speaks = l == 0 && share == 0 && blockIdx.y == 0;  // reports for the token
  const int hq = a.num_q_heads, hkv = a.num_kv_heads;
  const int rows = hq + 2 * hkv;
  const int half = a.rot_dim >> 1;
  const bool turned = 8 * l < a.rot_dim;
  const int e0 = IL || !turned ? 8 * l : 4 * l;
  const int e1 = IL || !turned ? e0 + 4 : half + e0;
  constexpr int U = kRopeRows;
  const int step = per_token * gridDim.y;
  const int first = blockIdx.y * per_token + share;
  // Addresses are formed once a token, and 32-bit steps from there: with 64-bit
  // products for every row the kernel was bound by its instructions (570 a warp).
  const uint8_t *q_from = a.q + t * a.q_stride * 2;
  const uint8_t *k_from = a.k + t * a.k_stride * 2 - hq * (2 * D);
  const uint8_t *v_from = a.v + t * a.v_stride * 2 - (hq + hkv) * (2 * D);
  uint8_t *q_to = a.q_out + t * hq * (2 * D);
  auto load = [&](int r, uint2 (&in)[2]) {
    if (r >= rows) return;
    const bool v = r >= hq + hkv;
    const uint8_t *from = (r < hq ? q_from : v ? v_from : k_from) + r * (2 * D);
    in[0] = *reinterpret_cast<const uint2 *>(from + 2 * (v ? 8 * l : e0));
    in[1] = *reinterpret_cast<const uint2 *>(from + 2 * (v ? 8 * l + 4 : e1));
  };
  // The first rows need nothing but the token's number, so they are under way
  // while the position, and then its table row, arrive.
  uint2 in[U][2];
#pragma unroll
  for (int u = 0; u < U; ++u) load(first + u * step, in[u]);
  const int32_t pos = a.positions[t];
  const int32_t slot = a.slot_mapping[t];
  if (pos < 0 || pos >= a.max_positions) {
    if (speaks) report(a.d_error, PKV_DEVERR_BAD_POSITION);
    return;
  }
  const bool in_pool = slot < static_cast<int64_t>(a.num_blocks) * a.block_size;
  if (!in_pool && speaks) report(a.d_error, PKV_DEVERR_BAD_SLOT);
  const bool keep = slot >= 0 && in_pool;
  const int sh = a.block_size == 32 ? 5 : 4;
  const int off = slot & (a.block_size - 1);
  const int row0 = keep ? ((slot >> sh) * hkv << sh) + off : 0;  // of KV head 0; a head's rows are block_size apart
  float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
  if (turned) {
    const float *row = a.cos_sin + static_cast<int64_t>(pos) * a.rot_dim + 4 * l;
    const float4 c4 = __ldg(reinterpret_cast<const float4 *>(row));
    const float4 s4 = __ldg(reinterpret_cast<const float4 *>(row + half));
    c[0] = c4.x; c[1] = c4.y; c[2] = c4.z; c[3] = c4.w;
    s[0] = s4.x; s[1] = s4.y; s[2] = s4.z; s[3] = s4.w;
  }
  for (int r0 = first; r0 < rows; r0 += U * step) {
    if (r0 != first) {
#pragma unroll
      for (int u = 0; u < U; ++u) load(r0 + u * step, in[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * step;
      if (r >= rows || (r >= hq && !keep)) break;  // the rest are keys and values, too
      float x[8];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 f = unpack2<IDT>(in[u][i].x), g = unpack2<IDT>(in[u][i].y);
        x[4 * i] = f.x; x[4 * i + 1] = f.y; x[4 * i + 2] = g.x; x[4 * i + 3] = g.y;
      }
      if (r >= hq + hkv) {
        store_cache8<D, v_part(CDT)>(x, a.v_cache, a.v_scale, row0 + (r - hq - hkv << sh), off, 8 * l, 8 * l + 4,
                                     lanes);
        continue;
      }
      if (turned) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int p = IL ? 2 * i : i, q = IL ? 2 * i + 1 : i + 4;
          const float u0 = x[p], u1 = x[q];
          x[p] = __fsub_rn(__fmul_rn(u0, c[i]), __fmul_rn(u1, s[i]));
          x[q] = __fadd_rn(__fmul_rn(u1, c[i]), __fmul_rn(u0, s[i]));
        }
      }
      if (r < hq) {
        uint8_t *to = q_to + r * (2 * D);
        *reinterpret_cast<uint2 *>(to + 2 * e0) = make_uint2(pack2<IDT>(x[0], x[1]), pack2<IDT>(x[2], x[3]));
        *reinterpret_cast<uint2 *>(to + 2 * e1) = make_uint2(pack2<IDT>(x[4], x[5]), pack2<IDT>(x[6], x[7]));
      } else {
        store_cache8<D, k_part(CDT)>(x, a.k_cache, a.k_scale, row0 + (r - hq << sh), off, e0, e1, lanes);
      }
    }
  }
}

template <int D, int IDT, int CDT>
cudaError_t launch_append_rope(const AppendRopeArgs &a) {
  constexpr int GROUPS = 256 * 8 / D;
  const int rows = a.num_q_heads + 2 * a.num_kv_heads;
  // A token's groups keep its table slice for kRopeRows rows each, all in flight
  // at once, and a CTA takes as many tokens as that leaves room for; with fewer
  // tokens than would fill the SMs the rows are spread over more CTAs (one row
  // per group of lanes).
  const int parts = a.num_tokens >= kRopeFullTokens ? 1 : (rows + GROUPS - 1) / GROUPS;
  const int per_token = parts > 1 ? GROUPS : std::max(1, std::min(GROUPS, (rows + kRopeRows - 1) / kRopeRows));
  const int tokens = GROUPS / per_token;  // of a CTA
  const dim3 grid(static_cast<unsigned>((a.num_tokens + tokens - 1) / tokens), static_cast<unsigned>(parts));
  if (a.interleaved) append_rope_kernel<D, IDT, CDT, true><<<grid, 256, 0, a.stream>>>(a, per_token);
  else append_rope_kernel<D, IDT, CDT, false><<<grid, 256, 0, a.stream>>>(a, per_token);
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
