// Host side of the shared-prefix decode (see intattn.h).  Included by
// intattn.cu, whose helpers it uses.
#pragma once

namespace {

using intattn::SharedArgs;

// Head parameters of H query heads from scales whose K and V entries belong
// to Hkv heads.
int shared_params(const intattn_scales_t* sc, int H, int Hkv, int d, float clip_c, SharedArgs* a) {
  if (!sc->s_q || !sc->s_k || !sc->s_v || !sc->s_o) return INTATTN_ERR_INVALID_ARG;
  const int n = sc->per_head ? H : 1;
  if (n > INTATTN_MAX_HEADS) return INTATTN_ERR_UNSUPPORTED;
  float s_k[INTATTN_MAX_HEADS], s_v[INTATTN_MAX_HEADS];
  int32_t z_k[INTATTN_MAX_HEADS], z_v[INTATTN_MAX_HEADS];
  const int G = H / Hkv;
  for (int i = 0; i < n; ++i) {
    const int e = sc->per_head ? i / G : 0;
    s_k[i] = sc->s_k[e];
    s_v[i] = sc->s_v[e];
    z_k[i] = sc->z_k ? sc->z_k[e] : 0;
    z_v[i] = sc->z_v ? sc->z_v[e] : 0;
    a->s_o[i] = sc->s_o[i];
  }
  intattn_scales_t x = *sc;
  x.s_k = s_k;
  x.s_v = s_v;
  x.z_k = sc->z_k ? z_k : nullptr;
  x.z_v = sc->z_v ? z_v : nullptr;
  return derive(&x, H, d, clip_c, a->lut, a->hp, INTATTN_MAX_HEADS);
}

}  // namespace

extern "C" {

size_t intattn_decode_shared_workspace_size(int B, int H, int Hkv, int Lmax, int d) {
  if (B < 0 || H <= 0 || Hkv <= 0 || H % Hkv || Lmax < 0 || (d != 64 && d != 128)) return 0;
  return 256;
}

int intattn_decode_shared(const int8_t* q, const int8_t* k_prefix, const int8_t* v_prefix, int Lp, int Lp_max,
                          const int8_t* k_cache, const int8_t* v_cache, const int32_t* lengths,
                          const intattn_scales_t* scales, int B, int H, int Hkv, int Lmax, int d, float clip_c,
                          int out_dtype, void* out, void* workspace, size_t workspace_bytes, intattn_stream_t stream) {
  if (B < 0 || H <= 0 || Hkv <= 0 || H % Hkv || Lp < 0 || Lp_max < Lp || Lmax < 0 || Lp > 65535 || Lmax > 65535 ||
      Lp + Lmax < 1 || Lp + Lmax > 65535)
    return INTATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return INTATTN_ERR_UNSUPPORTED;
  if (out_dtype != INTATTN_DTYPE_INT8 && out_dtype != INTATTN_DTYPE_FP16 && out_dtype != INTATTN_DTYPE_BF16)
    return INTATTN_ERR_UNSUPPORTED;
  if (!scales) return INTATTN_ERR_INVALID_ARG;
  static_assert(sizeof(SharedArgs) <= 8192, "kernel argument block too large");
  SharedArgs a;
  std::memset(&a, 0, sizeof(a));
  const int rc = shared_params(scales, H, Hkv, d, clip_c, &a);
  if (rc) return rc;
  const long long BH = static_cast<long long>(B) * H;
  if (BH == 0) return INTATTN_OK;
  if (BH > 65535) return INTATTN_ERR_UNSUPPORTED;
  if (!q || !out || (Lp && (!k_prefix || !v_prefix)) || (Lmax && (!k_cache || !v_cache))) return INTATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(k_prefix) || !aligned16(v_prefix) || !aligned16(k_cache) ||
      !aligned16(v_cache) || !aligned4(lengths))
    return INTATTN_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < intattn_decode_shared_workspace_size(B, H, Hkv, Lmax, d) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return INTATTN_ERR_WORKSPACE;
  a.q = q;
  a.kp = k_prefix;
  a.vp = v_prefix;
  a.kc = k_cache;
  a.vc = v_cache;
  a.lengths = lengths;
  a.out = out;
  a.B = B;
  a.H = H;
  a.Hkv = Hkv;
  a.G = H / Hkv;
  a.Lp = Lp;
  a.Lp_max = Lp_max;
  a.Lmax = Lmax;
  a.per_head = scales->per_head ? 1 : 0;
  a.out_kind = out_dtype;
  a.k_u8 = scales->z_k ? 1 : 0;
  a.v_u8 = scales->z_v ? 1 : 0;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (d == 64)
    intattn::shared::shared_simple_kernel<64><<<static_cast<unsigned>(BH), intattn::shared::kThreads, 0, st>>>(a);
  else
    intattn::shared::shared_simple_kernel<128><<<static_cast<unsigned>(BH), intattn::shared::kThreads, 0, st>>>(a);
  return note_launch(cudaGetLastError());
}

}  // extern "C"
