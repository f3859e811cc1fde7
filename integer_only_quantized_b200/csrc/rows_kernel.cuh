// Row operators between the projections and the KV caches: the norm and
// position rotation of query and key heads, quantising rows with fixed
// scales as they are written into a cache, and reading cache rows back.
//
// A row is one head of one token: d = 64 or 128 channels.  D / 8 lanes hold a
// row, two groups of four channels each, and everything between the load
// and the store stays in fp32 registers:
//   norm      y = x / sqrt(mean x^2 + eps) * w, the sum over the row's lanes
//             by shuffles
//   rotation  pairs (a, b) of the first rot channels -> (a c - b s, a s + b c)
//             with (c, s) from the caller's table at the token's position.  A
//             lane's two groups are those that pair with each other (f and
//             f + rot/2, or neighbours where pairs are interleaved), so the rotation
//             needs no other lane: with eight consecutive channels per lane
//             and a shuffle per channel the rows of a LLaMA-7B prefill (B1
//             H32/32 L8192 d128 bf16) took 82 us instead of
//             64, both before the paired arithmetic
//   codes     clamp(rint(RN32(y inv)) + z), or one rounding to fp16 / bf16
// All of it is bound by memory (2 bytes in, 2, 1 or 1/2 byte out per channel),
// closely followed by the instructions in between; for the few rows of a
// decode step by the launch and one round trip.  Measured, per call in a CUDA graph:
// those LLaMA-7B rows, norm and rotation, 51.2 us (5.3 TB/s; a copy of the bytes
// takes 41.7); one token of 12 heads 1.8 us.  B4 L4096 H32 d128 K and V rows, beside the
// copy of each direction's own bytes:
//   write  int8 93.4 us (61.5), u8 91.2, with the keys' norm and rotation 108.5, and
//          with the queries too 167.8 (92.3); int4 99.1 (51.3), with zero-points the same
//   read   int8 or u8 62.0 us (61.5), int4 56.5 (51.3)
// The write is bound by its instructions (76 % of the issue slots), the read by memory.  In fp32
// pairs (mul2, fma2) norm and rotation went from 64 to 57 us, with four loads
// per lane and a tensor per grid row to 52.7; two, six or eight loads per
// lane, and 64 or 256 threads, were slower.
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
  float lo, hi;           // codes: their range
  int32_t sc;             // codes: first entry of the call's scale arrays
  int32_t warps;          // per token: ceil(heads / batch)
};

struct RowArgs {
  RowTensor t[3];              // heads of tensor 0, then 1, then 2
  int32_t n_tensors;
  int32_t B, L, Lmax, bf16, per_head;
  int32_t batch;               // heads of one token that a warp handles
  uint32_t tokens;             // B * L
  const int32_t* start;        // [B] first cache row, or null
  const int32_t* lengths;      // [B] rows of each sequence, or null: all L
  const int32_t* positions;    // [B, L], or null: no rotation
  const float2* table;         // [n_positions, rot / 2] (cos, sin)
  int32_t n_positions, rot, interleaved;
  int32_t zero_left_out;       // rows left out (padding, out of range) of outputs other than a cache become 0
  float eps;
};
// with codes: 3 KB more, which a call without them need not hand over
struct RowCodeArgs : RowArgs {
  float inv[3 * INTATTN_MAX_HEADS];    // RN32(1 / scale)
  float zero[3 * INTATTN_MAX_HEADS];   // zero-points (0: symmetric)
};
template <bool kCodes> struct RowCallOf { using type = RowArgs; };
template <> struct RowCallOf<true> { using type = RowCodeArgs; };
template <bool kCodes> using RowCall = typename RowCallOf<kCodes>::type;

struct ReadArgs {
  const uint8_t* in[2];   // caches [B, H, Lmax, d] (4 bits: d / 2 bytes a row)
  void* out[2];           // [B, H, L, d] fp16 / bf16
  int32_t n_tensors, B, H, L, Lmax, bf16, per_head, bits, asym_k, asym_v;
  int32_t chunks;         // CTAs per (b, h): each takes kRows rows
  int32_t zero_left_out;  // as in RowArgs
  const int32_t* start;
  const int32_t* lengths;
  float scale[2 * INTATTN_MAX_HEADS];
  float zero[2 * INTATTN_MAX_HEADS];
};

namespace rows {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

template <bool kBf16>
__device__ __forceinline__ void to_float4(uint2 v, float (&f)[4]) {
  const uint32_t w[2] = {v.x, v.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (kBf16) {
      f[2 * i] = __uint_as_float(w[i] << 16);  // bf16 = high half of an fp32
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = h.x;
      f[2 * i + 1] = h.y;
    }
  }
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b, bool bf16) {
  if (bf16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Two fp32 operations in one instruction: (a0, a1) * (b0, b1), and + (c0, c1).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 z, x, y;\n\t"
      "mov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\t"
      "mov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 z, x, y;\n\t"
      "mov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// clamp(rint(RN32(y inv)), lo, hi) + z of four values, in the low byte of
// each word.  Adding 1.5 * 2^23 rounds to an integer with ties to even and leaves it in
// the sum's low bits; z is a whole number, so adding it is exact.  Infinities
// end at lo or hi; a NaN gives z (`careful`: there may be one).
__device__ __forceinline__ void codes4(const float2 (&y)[2], float inv, float lo, float hi, float z, bool careful,
                                       uint32_t (&c)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 p = mul2(y[i], both(inv));
    float2 q = make_float2(fminf(fmaxf(p.x, lo), hi), fminf(fmaxf(p.y, lo), hi));
    if (careful) q = make_float2(p.x == p.x ? q.x : 0.f, p.y == p.y ? q.y : 0.f);
    q = add2(add2(q, both(12582912.0f)), both(z));
    c[2 * i] = __float_as_uint(q.x);
    c[2 * i + 1] = __float_as_uint(q.y);
  }
}

// 0 into the warp's output rows, which the call leaves out (not those of a
// cache).  A function of its own, finding everything again: inlined beside the kernel's
// loop it made the write of a LLaMA-7B prompt 99.6 us instead of 93.3, which leaves nothing out.
template <int D, bool kCodes>
__device__ __noinline__ void zero_rows(const RowCall<kCodes>& a) {
  constexpr int kLpr = D / 8;
  const RowTensor& rt = a.t[blockIdx.y];
  if (rt.cache) return;
  const uint32_t id = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const uint32_t token = id / static_cast<uint32_t>(rt.warps);
  const int h0 = static_cast<int>(id - token * rt.warps) * a.batch;
  const int h1 = min(rt.heads, h0 + a.batch);
  const int b = static_cast<int>(token / static_cast<uint32_t>(a.L));
  const int t = static_cast<int>(token) - b * a.L;
  for (int i = threadIdx.x & 31; i < (h1 - h0) * kLpr; i += 32) {  // eight channels each
    const int64_t at = b * rt.osb + t * rt.osl + (h0 + i / kLpr) * rt.osh + 8 * (i % kLpr);
    if constexpr (kCodes) *reinterpret_cast<uint2*>(static_cast<uint8_t*>(rt.out) + at) = make_uint2(0, 0);
    else *reinterpret_cast<uint4*>(static_cast<uint16_t*>(rt.out) + at) = make_uint4(0, 0, 0, 0);
  }
}

// kCodes: the output is codes; else fp16 / bf16.
template <int D, bool kCodes, bool kBf16>
__global__ void __launch_bounds__(kThreads) rows_kernel(const __grid_constant__ RowCall<kCodes> a) {
  constexpr int kLpr = D / 8;           // lanes per row
  constexpr int kRpw = 32 / kLpr;       // rows (heads) per warp and load
  constexpr int kUnroll = 4;            // loads in flight per lane
  const int lane = threadIdx.x & 31;
  const int piece = lane % kLpr;
  const int sub = lane / kLpr;
  const RowTensor& rt = a.t[blockIdx.y];
  const uint32_t id = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const uint32_t token = id / static_cast<uint32_t>(rt.warps);
  if (token >= a.tokens) return;
  const int h0 = static_cast<int>(id - token * rt.warps) * a.batch;
  const int h1 = min(rt.heads, h0 + a.batch);
  const int b = static_cast<int>(token / static_cast<uint32_t>(a.L));
  const int t = static_cast<int>(token) - b * a.L;

  // The lane's groups: channels g0 .. g0 + 3 and g1 .. g1 + 3.
  const bool rope = a.positions != nullptr && rt.rope;  // uniform over the warp
  const bool split = rope && !a.interleaved;
  const bool turn = rope && 8 * piece < a.rot;
  const int g0 = split && turn ? 4 * piece : 8 * piece;
  const int g1 = split && turn ? 4 * piece + a.rot / 2 : 8 * piece + 4;

  // the rows first: nothing below is needed for them
  const uint16_t* in = static_cast<const uint16_t*>(rt.in) + b * rt.isb + t * rt.isl + (h0 + sub) * rt.ish + g0;
  const int64_t in_step = kRpw * rt.ish;
  uint2 raw[kUnroll][2];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u, in += in_step) {
    raw[u][0] = raw[u][1] = make_uint2(0, 0);
    if (h0 + u * kRpw + sub < h1) {
      raw[u][0] = *reinterpret_cast<const uint2*>(in);
      raw[u][1] = *reinterpret_cast<const uint2*>(in + (g1 - g0));
    }
  }

  if (a.lengths != nullptr && t >= a.lengths[b]) {  // a padded row
    if (a.zero_left_out) zero_rows<D, kCodes>(a);
    return;
  }
  int row = t;
  if (a.start != nullptr) {
    const int64_t slot = static_cast<int64_t>(a.start[b]) + t;
    if (slot < 0 || slot >= a.Lmax) {
      if (lane == 0) atomicOr(&g_device_error, kErrParamRange);
      if (a.zero_left_out) zero_rows<D, kCodes>(a);
      return;
    }
    if (rt.cache) row = static_cast<int>(slot);
  }
  // cos and sin of the lane's four pairs: split, pair i is channels g0 + i and
  // g1 + i; interleaved, pairs 0 and 1 lie in the first group, 2 and 3 in the second
  float2 cs[2], sn[2], ns[2];  // ns: -sin
  if (a.positions != nullptr) {
    const int pos = a.positions[token];
    if (pos < 0 || pos >= a.n_positions) {  // negative: a padded row
      if (pos >= 0 && lane == 0) atomicOr(&g_device_error, kErrParamRange);
      if (a.zero_left_out) zero_rows<D, kCodes>(a);
      return;
    }
    if (turn) {
      const float4* p = reinterpret_cast<const float4*>(a.table + static_cast<int64_t>(pos) * (a.rot / 2) + 4 * piece);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 v = __ldg(p + i);
        cs[i] = make_float2(v.x, v.z);
        sn[i] = make_float2(v.y, v.w);
        ns[i] = make_float2(-v.y, -v.w);
      }
    }
  }
  float2 w[2][2];
  if (rt.w != nullptr) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(rt.w + (g ? g1 : g0)));
      w[g][0] = make_float2(v.x, v.y);
      w[g][1] = make_float2(v.z, v.w);
    }
  }
  int64_t at = b * rt.osb + static_cast<int64_t>(row) * rt.osl + (h0 + sub) * rt.osh + g0;
  const int64_t out_step = kRpw * rt.osh;
#pragma unroll
  for (int u = 0; u < kUnroll; ++u, at += out_step) {
    if (h0 + u * kRpw >= h1) break;  // uniform over the warp
    const int h = h0 + u * kRpw + sub;
    float f[2][4];
    to_float4<kBf16>(raw[u][0], f[0]);
    to_float4<kBf16>(raw[u][1], f[1]);
    float2 y[2][2] = {{make_float2(f[0][0], f[0][1]), make_float2(f[0][2], f[0][3])},
                      {make_float2(f[1][0], f[1][1]), make_float2(f[1][2], f[1][3])}};
    if (rt.w != nullptr) {
      float2 sq = mul2(y[0][0], y[0][0]);
      sq = fma2(y[0][1], y[0][1], sq);
      sq = fma2(y[1][0], y[1][0], sq);
      sq = fma2(y[1][1], y[1][1], sq);
      float ss = sq.x + sq.y;
#pragma unroll
      for (int o = kLpr / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float r = rsqrtf(fmaf(ss, 1.0f / D, a.eps));  // within 2 units in the last place
      const float2 rr = make_float2(r, r);
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int i = 0; i < 2; ++i) y[g][i] = mul2(mul2(y[g][i], rr), w[g][i]);
    }
    if (turn) {
      if (split) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 p = y[0][i], q = y[1][i];
          y[0][i] = fma2(q, ns[i], mul2(p, cs[i]));
          y[1][i] = fma2(p, sn[i], mul2(q, cs[i]));
        }
      } else {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const float2 p = y[g][0], q = y[g][1], c = cs[g], s = sn[g];
          y[g][0] = make_float2(fmaf(p.x, c.x, -(p.y * s.x)), fmaf(p.y, c.x, p.x * s.x));
          y[g][1] = make_float2(fmaf(q.x, c.y, -(q.y * s.y)), fmaf(q.y, c.y, q.x * s.y));
        }
      }
    }
    if (h >= h1) continue;
    if constexpr (!kCodes) {
      uint16_t* dst = static_cast<uint16_t*>(rt.out) + at;
#pragma unroll
      for (int g = 0; g < 2; ++g)
        *reinterpret_cast<uint2*>(dst + (g ? g1 - g0 : 0)) =
            make_uint2(pack_half2(y[g][0].x, y[g][0].y, kBf16), pack_half2(y[g][1].x, y[g][1].y, kBf16));
    } else {
      const int e = rt.sc + (a.per_head ? h : 0);
      const float inv = a.inv[e], z = a.zero[e];
      const float lo = rt.lo - z, hi = rt.hi - z;
      // no NaN among the eight values (an infinity may say so too)
      const float2 sum = add2(add2(y[0][0], y[0][1]), add2(y[1][0], y[1][1]));
      const bool careful = !(fabsf(sum.x + sum.y) < 3.402823466e38f);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        uint32_t c[4];
        codes4(y[g], inv, lo, hi, z, careful, c);
        const int64_t to = at + (g ? g1 - g0 : 0);
        if (rt.bits == 8) {
          *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(rt.out) + to) =
              __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
        } else {  // channel 2t in the low nibble of byte t
          *reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(rt.out) + to / 2) = static_cast<uint16_t>(
              (c[0] & 15u) | ((c[1] & 15u) << 4) | ((c[2] & 15u) << 8) | ((c[3] & 15u) << 12));
        }
      }
    }
  }
}

// Values s (c - z) of cache rows.  A lane takes eight channels of a row (an 8-byte
// load of int8 codes, 4 bytes of int4 codes; one 16-byte store, so that a warp's store is one
// contiguous run), of kUnroll rows.
constexpr int kReadThreads = 128;
constexpr int kReadUnroll = 4;
template <int D, bool kBf16>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ ReadArgs a) {
  constexpr int kLpr = D / 8;
  constexpr int kStep = kReadThreads / kLpr;      // rows per load
  constexpr int kRows = kStep * kReadUnroll;      // rows per CTA
  const int piece = threadIdx.x % kLpr;
  const uint32_t bhx = blockIdx.x / static_cast<uint32_t>(a.chunks);  // (tensor, b, h)
  const int t0 = static_cast<int>(blockIdx.x - bhx * a.chunks) * kRows + threadIdx.x / kLpr;
  const uint32_t planes = static_cast<uint32_t>(a.B) * a.H;
  const int x = bhx >= planes ? 1 : 0;
  const uint32_t bh = bhx - x * planes;
  const int b = static_cast<int>(bh / static_cast<uint32_t>(a.H));
  const int h = static_cast<int>(bh) - b * a.H;
  const int start = a.start[b];
  const int n = a.lengths != nullptr ? min(a.L, a.lengths[b]) : a.L;
  const int e = x * INTATTN_MAX_HEADS + (a.per_head ? h : 0);
  const float s = a.scale[e];
  const bool asym = x ? a.asym_v : a.asym_k;
  // A code as an unsigned byte u (two's complement: its sign bit flipped) is
  // the float 2^23 + u with u in the low byte; `off` takes 2^23, the flip and z from it.
  const uint32_t flip = asym ? 0u : a.bits == 8 ? 0x80808080u : 0x08080808u;
  const float off = -(8388608.0f + (asym ? a.zero[e] : a.bits == 8 ? 128.0f : 8.0f));
  const uint8_t* in = a.in[x];
  uint2 raw[kReadUnroll];
  bool ok[kReadUnroll];
#pragma unroll
  for (int u = 0; u < kReadUnroll; ++u) {
    const int t = t0 + u * kStep;
    const int64_t slot = static_cast<int64_t>(start) + t;
    ok[u] = t < n && slot >= 0 && slot < a.Lmax;
    if (t < n && !ok[u] && piece == 0) atomicOr(&g_device_error, kErrParamRange);
    raw[u] = make_uint2(0, 0);
    if (ok[u]) {
      const int64_t at = (static_cast<int64_t>(bh) * a.Lmax + slot) * D + 8 * piece;  // channels
      if (a.bits == 8) raw[u] = __ldg(reinterpret_cast<const uint2*>(in + at));
      else raw[u].x = __ldg(reinterpret_cast<const uint32_t*>(in + at / 2));
    }
  }
#pragma unroll
  for (int u = 0; u < kReadUnroll; ++u) {
    if (!ok[u] && !(a.zero_left_out && t0 + u * kStep < a.L)) continue;
    // u words: bytes in the order of the channels (8 bits), or even and odd channels (4 bits)
    uint32_t u0 = raw[u].x ^ flip, u1 = raw[u].y ^ flip;
    if (a.bits == 4) {
      u1 = (raw[u].x >> 4 & 0x0F0F0F0Fu) ^ flip;
      u0 = (raw[u].x & 0x0F0F0F0Fu) ^ flip;
    }
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // channels 2k and 2k + 1
      uint32_t x0, x1;
      if (a.bits == 8) {
        const uint32_t v = k < 2 ? u0 : u1;
        x0 = __byte_perm(v, 0x4B000000u, 0x7650 + 2 * (k & 1));
        x1 = __byte_perm(v, 0x4B000000u, 0x7651 + 2 * (k & 1));
      } else {
        x0 = __byte_perm(u0, 0x4B000000u, 0x7650 + k);
        x1 = __byte_perm(u1, 0x4B000000u, 0x7650 + k);
      }
      // the sum is a whole number and exact; a product of it and then one rounding to 16 bits
      const float2 f = mul2(add2(make_float2(__uint_as_float(x0), __uint_as_float(x1)), both(off)), both(s));
      o[k] = ok[u] ? pack_half2(f.x, f.y, kBf16) : 0u;
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out[x]) + (static_cast<int64_t>(bh) * a.L + t0 + u * kStep) * D +
                              8 * piece) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

}  // namespace rows
}  // namespace intattn
