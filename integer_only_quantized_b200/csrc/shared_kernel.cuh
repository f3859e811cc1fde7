// Decode for a batch whose sequences share a prefix: one query per (b, h)
// against the prefix rows of its K / V head followed by the rows of its own
// cache, by the definition of intattn.h over the joined keys.
//
// One CTA per (b, h), three sweeps over its keys with the scores recomputed:
// row max, sum of pseudo-exponentials, P.V.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <climits>
#include <cstdint>

#include "common.cuh"
#include "decode_kernel.cuh"
#include "params_kernel.cuh"
#include "sm100.cuh"

namespace intattn {

struct SharedArgs {
  const int8_t* q;            // [B, H, d]
  const int8_t* kp;           // [Hkv, Lp_max, d] prefix rows, Lp of them valid
  const int8_t* vp;
  const int8_t* kc;           // [B, Hkv, Lmax, d] each sequence's own rows
  const int8_t* vc;
  const int32_t* lengths;     // [B], or null: Lmax
  void* out;                  // [B, H, d] int8 codes, or fp16 / bf16 values
  int32_t B, H, Hkv, G, Lp, Lp_max, Lmax, per_head, out_kind, k_u8, v_u8;
  float s_o[INTATTN_MAX_HEADS];
  uint32_t lut[INTATTN_MAX_CLIPS][32];
  HeadParamsDev hp[INTATTN_MAX_HEADS];
};

namespace shared {

constexpr int kThreads = 256;

template <int D>
__global__ void __launch_bounds__(kThreads) shared_simple_kernel(const __grid_constant__ SharedArgs a) {
  const int b = blockIdx.x / a.H, h = blockIdx.x % a.H, hk = h / a.G;
  const int tid = threadIdx.x;
  const HeadParamsDev hp = a.hp[a.per_head ? h : 0];
  const int n_own = a.lengths ? a.lengths[b] : a.Lmax;
  if (n_own < 0 || n_own > a.Lmax) {
    if (tid == 0) atomicOr(&g_device_error, kErrParamRange);
    return;
  }
  const int n = a.Lp + n_own;
  __shared__ uint32_t qs[D / 4];
  __shared__ uint32_t lut[32];
  __shared__ uint8_t ps[kThreads];
  __shared__ int32_t red;
  __shared__ int32_t total;
  if (tid < D / 4) qs[tid] = reinterpret_cast<const uint32_t*>(a.q + static_cast<size_t>(blockIdx.x) * D)[tid];
  if (tid < 32) lut[tid] = a.lut[hp.lut][tid];
  if (tid == 0) {
    red = INT_MIN;
    total = 0;
  }
  __syncthreads();
  auto row = [&](const int8_t* prefix, const int8_t* cache, int j) {
    return j < a.Lp ? prefix + (static_cast<size_t>(hk) * a.Lp_max + j) * D
                    : cache + ((static_cast<size_t>(b) * a.Hkv + hk) * a.Lmax + (j - a.Lp)) * D;
  };
  auto score = [&](int j) {
    const uint32_t* k = reinterpret_cast<const uint32_t*>(row(a.kp, a.kc, j));
    int32_t s = 0;
    for (int i = 0; i < D / 4; ++i) s = a.k_u8 ? decode::dp4a_su(qs[i], k[i], s) : decode::dp4a_ss(qs[i], k[i], s);
    return s;
  };
  int32_t m = INT_MIN;
  for (int j = tid; j < n; j += kThreads) m = max(m, score(j));
  atomicMax(&red, m);
  __syncthreads();
  m = red;
  auto index = [&](int32_t s) {
    const long long gap = min(static_cast<long long>(m) - s, static_cast<long long>(hp.D));
    return static_cast<int>((gap * hp.M + (1ll << (hp.s - 1))) >> hp.s);
  };
  int32_t z = 0;
  for (int j = tid; j < n; j += kThreads) z += static_cast<int32_t>(lut[index(score(j))]);
  atomicAdd(&total, z);
  __syncthreads();
  const unsigned long long Z = static_cast<uint32_t>(total);
  const unsigned long long R = n ? ((255ull << 32) + (Z >> 1)) / Z : 0;
  int32_t acc = 0;
  for (int base = 0; base < n; base += kThreads) {
    const int j = base + tid;
    __syncthreads();
    ps[tid] = j < n ? static_cast<uint8_t>((lut[index(score(j))] * R + (1ull << 31)) >> 32) : 0;
    __syncthreads();
    if (tid < D)
      for (int i = 0; i < min(kThreads, n - base); ++i) {
        const int8_t v = row(a.vp, a.vc, base + i)[tid];
        acc += ps[i] * ((a.v_u8 ? static_cast<int32_t>(static_cast<uint8_t>(v)) : v) - hp.zv);
      }
  }
  if (tid < D) {
    const long long t = (static_cast<long long>(acc) * hp.Mo + (1ll << (hp.so - 1))) >> hp.so;
    const int y = static_cast<int>(min(max(t, -127ll), 127ll));
    const size_t at = static_cast<size_t>(blockIdx.x) * D + tid;
    const float val = __fmul_rn(a.s_o[a.per_head ? h : 0], static_cast<float>(y));
    if (a.out_kind == INTATTN_DTYPE_INT8) static_cast<int8_t*>(a.out)[at] = static_cast<int8_t>(y);
    else if (a.out_kind == INTATTN_DTYPE_BF16) static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(val);
    else static_cast<__half*>(a.out)[at] = __float2half_rn(val);
  }
}

}  // namespace shared
}  // namespace intattn
