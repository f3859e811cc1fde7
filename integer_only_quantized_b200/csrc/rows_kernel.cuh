// Row operators between the projections and the KV caches: the norm and
// position rotation of query and key heads, quantising rows with fixed
// scales as they are written into a cache, and reading cache rows back.
//
// A row is one head of one token: d = 64 or 128 channels.  D / 8 lanes hold a
// row, eight channels (one 16-byte load) each, and everything between the
// load and the store stays in fp32 registers:
//   norm      y = x / sqrt(mean x^2 + eps) * w, the sum over the row's lanes
//             by shuffles
//   rotation  pairs (a, b) of the first rot channels -> (a c - b s, a s + b c)
//             with (c, s) from the caller's table at the token's position;
//             half-split pairs (f, f + rot/2) sit rot/16 lanes apart (one
//             shuffle per channel), interleaved pairs (2f, 2f + 1) in one lane
//   codes     clamp(rint(RN32(y inv)) + z), or one rounding to fp16 / bf16
// All of it is bound by memory (2 bytes in, 2, 1 or 1/2 byte out per channel
// for a handful of instructions), or, for the few rows of a decode step, by
// the launch and one round trip.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "params_kernel.cuh"
#include "quantize_kernel.cuh"
#include "sm100.cuh"

namespace intattn {

// One tensor of rows: element (b, h, t, c) at b sb + h sh + t sl + c.
struct RowTensor {
  const void* in;         // fp16 / bf16
  void* out;              // fp16 / bf16, or codes
  int64_t isb, ish, isl;  // input strides, elements
  int64_t osb, osh, osl;  // output strides, elements (4-bit codes: also in elements, two to a byte)
  const float* w;         // [d] norm weight, or null: no norm
  int32_t heads;
  int32_t rope;           // rotate
  int32_t cache;          // output row = start[b] + t, checked against Lmax; else t
  int32_t bits;           // codes: 8 or 4; unused for fp output
  int32_t asym;           // codes: unsigned with zero-points
  int32_t sc;             // codes: first entry of the call's scale arrays
};

struct RowArgs {
  RowTensor t[3];              // heads of tensor 0, then 1, then 2
  int32_t n_tensors, heads;    // heads: over all tensors
  int32_t B, L, Lmax, bf16, per_head;
  int32_t heads_per_item;      // heads of one token that a warp handles
  int32_t items_per_token;
  int64_t items;               // B * L * items_per_token
  const int32_t* start;        // [B] first cache row, or null
  const int32_t* lengths;      // [B] rows of each sequence, or null: all L
  const int32_t* positions;    // [B, L], or null: no rotation
  const float2* table;         // [n_positions, rot / 2] (cos, sin)
  int32_t n_positions, rot, interleaved;
  float eps;
  float inv[3 * INTATTN_MAX_HEADS];    // codes: RN32(1 / scale)
  uint8_t zero[3 * INTATTN_MAX_HEADS];
};

struct ReadArgs {
  const uint8_t* in[2];   // caches [B, H, Lmax, d] (4 bits: d / 2 bytes a row)
  void* out[2];           // [B, H, L, d] fp16 / bf16
  int32_t n_tensors, B, H, L, Lmax, bf16, per_head, bits, asym_k, asym_v;
  int64_t rows;           // per tensor: B * H * L
  const int32_t* start;
  const int32_t* lengths;
  float scale[2 * INTATTN_MAX_HEADS];
  uint8_t zero[2 * INTATTN_MAX_HEADS];
};

namespace rows {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

// rint(RN32(y inv)) as an integer in [-2^21, 2^21]: infinities and values
// beyond the range saturate there (every code range lies inside), NaN gives 0.
__device__ __forceinline__ int32_t code_of(float y, float inv) {
  const float p = __fmul_rn(y, inv);
  const float q = fminf(fmaxf(p, -2097152.0f), 2097152.0f);  // NaN: -2097152
  return p == p ? __float2int_rn(q) : 0;
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b, bool bf16) {
  if (bf16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// kCodes: the output is codes; else fp16 / bf16.
template <int D, bool kCodes>
__global__ void __launch_bounds__(kThreads) rows_kernel(const __grid_constant__ RowArgs a) {
  constexpr int kLpr = D / 8;           // lanes per row
  constexpr int kRpw = 32 / kLpr;       // rows (heads) per warp and step
  constexpr int kUnroll = 4;            // steps whose loads are in flight together
  const int lane = threadIdx.x & 31;
  const int piece = lane % kLpr;        // channels 8 piece .. 8 piece + 7
  const int sub = lane / kLpr;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (item >= a.items) return;
  const int64_t token = item / a.items_per_token;
  const int h0 = static_cast<int>(item - token * a.items_per_token) * a.heads_per_item;
  const int h1 = min(a.heads, h0 + a.heads_per_item);
  const int b = static_cast<int>(token / a.L);
  const int t = static_cast<int>(token - static_cast<int64_t>(b) * a.L);

  if (a.lengths != nullptr && t >= a.lengths[b]) return;  // a padded row
  int slot = t;
  if (a.start != nullptr) {
    const int64_t row = static_cast<int64_t>(a.start[b]) + t;
    if (row < 0 || row >= a.Lmax) {
      if (lane == 0) atomicOr(&g_device_error, kErrParamRange);
      return;
    }
    slot = static_cast<int>(row);
  }

  // cos and sin of this lane's channels (kept for every head of the token)
  float cs[8], sn[8];
  bool turn = false;
  if (a.positions != nullptr) {
    const int pos = a.positions[token];
    if (pos < 0) return;  // a padded row
    if (pos >= a.n_positions) {
      if (lane == 0) atomicOr(&g_device_error, kErrParamRange);
      return;
    }
    turn = 8 * piece < a.rot;
    if (turn) {
      const int half = a.rot / 2;
      const float2* row = a.table + static_cast<int64_t>(pos) * half;
      if (a.interleaved) {
        const float4* p = reinterpret_cast<const float4*>(row + 4 * piece);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 v = __ldg(p + i);
          cs[4 * i] = cs[4 * i + 1] = v.x;
          sn[4 * i] = -v.y;  // the pair's first: a c - b s
          sn[4 * i + 1] = v.y;
          cs[4 * i + 2] = cs[4 * i + 3] = v.z;
          sn[4 * i + 2] = -v.w;
          sn[4 * i + 3] = v.w;
        }
      } else {
        const bool first = 8 * piece < half;
        const float4* p = reinterpret_cast<const float4*>(row + (first ? 8 * piece : 8 * piece - half));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 v = __ldg(p + i);
          cs[2 * i] = v.x;
          sn[2 * i] = first ? -v.y : v.y;
          cs[2 * i + 1] = v.z;
          sn[2 * i + 1] = first ? -v.w : v.w;
        }
      }
    }
  }
  // the lane that holds the other half of this lane's pairs (half-split)
  const int hop = a.rot / 16;
  const int partner = !turn ? lane : (8 * piece < a.rot / 2 ? lane + hop : lane - hop);

  // tensor of head g of the token, and the head within it
  auto locate = [&](int g, int& x, int& h) {
    x = 0;
    h = g;
    if (h >= a.t[0].heads) {
      h -= a.t[0].heads;
      x = 1;
      if (a.n_tensors > 2 && h >= a.t[1].heads) {
        h -= a.t[1].heads;
        x = 2;
      }
    }
  };

  for (int base = h0; base < h1; base += kRpw * kUnroll) {
    uint4 raw[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int g = base + u * kRpw + sub;
      raw[u] = make_uint4(0, 0, 0, 0);
      if (g < h1) {
        int x, h;
        locate(g, x, h);
        const RowTensor& rt = a.t[x];
        raw[u] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(rt.in) + b * rt.isb + h * rt.ish +
                                                 t * rt.isl + 8 * piece);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int g = base + u * kRpw + sub;
      if (base + u * kRpw >= h1) break;  // uniform over the warp
      const bool mine = g < h1;
      int x, h;
      locate(mine ? g : h1 - 1, x, h);
      const RowTensor& rt = a.t[x];
      float y[8];
      quant::to_float8(raw[u], a.bf16, y);
      // norm (the shuffles run on every lane: rows of a warp may differ in kind)
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
      for (int o = kLpr / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (rt.w != nullptr) {
        const float r = __fdiv_rn(1.0f, __fsqrt_rn(ss * (1.0f / D) + a.eps));
        const float4* wp = reinterpret_cast<const float4*>(rt.w + 8 * piece);
        const float4 w0 = __ldg(wp), w1 = __ldg(wp + 1);
        const float wv[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = y[i] * r * wv[i];
      }
      if (a.positions != nullptr) {  // uniform over the warp
        const bool rot = turn && rt.rope;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          float o0, o1;
          if (a.interleaved) {
            o0 = y[i + 1];
            o1 = y[i];
          } else {
            o0 = __shfl_sync(0xffffffffu, y[i], partner);
            o1 = __shfl_sync(0xffffffffu, y[i + 1], partner);
          }
          if (rot) {
            y[i] = fmaf(y[i], cs[i], o0 * sn[i]);
            y[i + 1] = fmaf(y[i + 1], cs[i + 1], o1 * sn[i + 1]);
          }
        }
      }
      if (!mine) continue;
      const int64_t at = b * rt.osb + h * rt.osh + static_cast<int64_t>(rt.cache ? slot : t) * rt.osl + 8 * piece;
      if constexpr (!kCodes) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(rt.out) + at) =
            make_uint4(pack_half2(y[0], y[1], a.bf16), pack_half2(y[2], y[3], a.bf16), pack_half2(y[4], y[5], a.bf16),
                       pack_half2(y[6], y[7], a.bf16));
      } else {
        const int e = rt.sc + (a.per_head ? h : 0);
        const float inv = a.inv[e];
        const int32_t z = rt.asym ? a.zero[e] : 0;
        const int32_t hi = rt.asym ? (1 << rt.bits) - 1 : (1 << (rt.bits - 1)) - 1;
        const int32_t lo = rt.asym ? 0 : -hi;
        uint32_t c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = static_cast<uint32_t>(min(max(code_of(y[i], inv) + z, lo), hi));
        if (rt.bits == 8) {
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(rt.out) + at) =
              make_uint2(__byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410),
                         __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410));
        } else {
          uint32_t w = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) w |= (c[i] & 15u) << (4 * i);  // channel 2t in the low nibble of byte t
          *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(rt.out) + at / 2) = w;
        }
      }
    }
  }
}

// Values s (c - z) of cache rows.  Sixteen channels per thread: one 16-byte
// load of int8 codes (8 bytes of int4 codes) and two 16-byte stores.
template <int D>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ ReadArgs a) {
  constexpr int kLpr = D / 16;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int piece = static_cast<int>(i % kLpr);
  int64_t row = i / kLpr;  // over the tensors' rows
  if (row >= a.rows * a.n_tensors) return;
  const int x = row >= a.rows ? 1 : 0;
  row -= x * a.rows;
  const int64_t bh = row / a.L;
  const int t = static_cast<int>(row - bh * a.L);
  const int b = static_cast<int>(bh / a.H);
  const int h = static_cast<int>(bh - static_cast<int64_t>(b) * a.H);
  if (a.lengths != nullptr && t >= a.lengths[b]) return;
  const int64_t slot = static_cast<int64_t>(a.start[b]) + t;
  if (slot < 0 || slot >= a.Lmax) {
    if (piece == 0) atomicOr(&g_device_error, kErrParamRange);
    return;
  }
  const int e = x * INTATTN_MAX_HEADS + (a.per_head ? h : 0);
  const float s = a.scale[e];
  const bool asym = x ? a.asym_v : a.asym_k;
  const int32_t z = asym ? a.zero[e] : 0;
  const int64_t src = (bh * a.Lmax + slot) * D + 16 * piece;  // channels
  int32_t c[16];
  if (a.bits == 8) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(a.in[x] + src));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const uint32_t u = (w[k / 4] >> (8 * (k % 4))) & 255u;
      c[k] = asym ? static_cast<int32_t>(u) - z : static_cast<int32_t>(static_cast<int8_t>(u));
    }
  } else {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(a.in[x] + src / 2));
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const uint32_t u = (w[k / 8] >> (4 * (k % 8))) & 15u;
      c[k] = asym ? static_cast<int32_t>(u) - z : static_cast<int32_t>(u ^ 8u) - 8;
    }
  }
  uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out[x]) + row * D + 16 * piece);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      o[k] = pack_half2(__fmul_rn(s, static_cast<float>(c[8 * q + 2 * k])),
                        __fmul_rn(s, static_cast<float>(c[8 * q + 2 * k + 1])), a.bf16);
    dst[q] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

}  // namespace rows
}  // namespace intattn
