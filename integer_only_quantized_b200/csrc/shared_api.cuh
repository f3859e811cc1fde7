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
  return derive(&x, H, d, clip_c, a->lut, a->hp, INTATTN_MAX_HEADS, &a->n_luts);
}

struct SharedLayout {
  int ld_s;
  size_t zeroed;  // words the zero kernel clears: counters and row maxima
  size_t off_z, off_p, off_acc, off_s, off_i, total;
};

SharedLayout shared_layout(long long BH, int Lmax, int d) {
  SharedLayout L{};
  const size_t rows = static_cast<size_t>(BH);
  L.zeroed = 8 + rows;
  L.off_z = round256(4 * L.zeroed);
  // row_z, row_p and acc are consecutive (cleared together by the kernel);
  // acc starts on 16 bytes
  L.off_acc = (L.off_z + 8 * rows + 15) & ~size_t(15);
  L.off_z = L.off_acc - 8 * rows;
  L.off_p = L.off_z + 4 * rows;
  L.ld_s = (Lmax + 63) & ~63;  // whole blocks
  L.off_s = round256(L.off_acc + 4 * rows * d);
  L.off_i = L.off_s + round256(4 * rows * static_cast<size_t>(L.ld_s));
  L.total = L.off_i + round256(rows * static_cast<size_t>(L.ld_s));
  return L;
}

template <int D, bool ZP>
int shared_launch(const SharedArgs& a, int grid, const SharedLayout& L, cudaStream_t st) {
  using C = intattn::shared::Cfg<D>;
  static bool attr_set[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return INTATTN_ERR_CUDA;
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(intattn::shared::shared_kernel<D, ZP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(C::kSmemBytes)) != cudaSuccess)
      return note_launch(cudaGetLastError());
    attr_set[dev] = true;
  }
  const int n = static_cast<int>(L.zeroed);
  intattn::shared::shared_zero_kernel<<<std::min(32, (n + 255) / 256), 256, 0, st>>>(a.ctr, n);
  const int rc = note_launch(cudaGetLastError());
  if (rc) return rc;
  // cooperative: all CTAs resident (the grid barriers); programmatic
  // serialisation: set-up and the first loads overlap the zero kernel
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeCooperative;
  attrs[0].val.cooperative = 1;
  attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(intattn::shared::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = st;
  cfg.attrs = attrs;
  cfg.numAttrs = 2;
  return note_launch(cudaLaunchKernelEx(&cfg, intattn::shared::shared_kernel<D, ZP>, a));
}

// [planes, rows of capacity, d] bytes with the first `rows` rows of a plane
// visible (rows past them read as 0), box {d, box_rows, 1}, swizzle = d bytes.
bool encode_rows(CUtensorMap* m, const void* base, int d, int rows, int capacity, long long planes, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(planes)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(capacity) * d};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(d), static_cast<cuuint32_t>(box_rows), 1u};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

extern "C" {

size_t intattn_decode_shared_workspace_size(int B, int H, int Hkv, int Lmax, int d) {
  if (B < 0 || H <= 0 || Hkv <= 0 || H % Hkv || Lmax < 0 || (d != 64 && d != 128)) return 0;
  return shared_layout(static_cast<long long>(B) * H, Lmax, d).total;
}

int intattn_decode_shared(const int8_t* q, const int8_t* k_prefix, const int8_t* v_prefix, int Lp, int Lp_max,
                          const int8_t* k_cache, const int8_t* v_cache, const int32_t* lengths,
                          const intattn_scales_t* scales, int B, int H, int Hkv, int Lmax, int d, float clip_c,
                          int out_dtype, void* out, void* workspace, size_t workspace_bytes, intattn_stream_t stream) {
  if (B < 0 || H <= 0 || Hkv <= 0 || H % Hkv || Lp < 0 || Lp_max < Lp || Lmax < 0 || Lp > 65535 || Lmax > 65535 ||
      Lp + Lmax < 1 || Lp + Lmax > 65535)
    return INTATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return INTATTN_ERR_UNSUPPORTED;
  const bool zero_left_out = out_dtype >= 0 && (out_dtype & INTATTN_ZERO_LEFT_OUT);
  if (zero_left_out) out_dtype &= ~INTATTN_ZERO_LEFT_OUT;
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
  const SharedLayout L = shared_layout(BH, Lmax, d);
  char* ws = static_cast<char*>(workspace);
  a.q = q;
  a.lengths = lengths;
  a.out = out;
  a.ctr = reinterpret_cast<uint32_t*>(ws);
  a.row_max = a.ctr + 8;
  a.row_z = reinterpret_cast<int32_t*>(ws + L.off_z);
  a.row_p = reinterpret_cast<int32_t*>(ws + L.off_p);
  a.acc = reinterpret_cast<float*>(ws + L.off_acc);
  a.scores = reinterpret_cast<int32_t*>(ws + L.off_s);
  a.index = reinterpret_cast<uint32_t*>(ws + L.off_i);
  a.ld_s = L.ld_s;
  a.B = B;
  a.H = H;
  a.Hkv = Hkv;
  a.G = H / Hkv;
  a.R = B * a.G;
  a.Lp = Lp;
  a.Lmax = Lmax;
  a.key_tiles = (Lp + intattn::shared::kBN - 1) / intattn::shared::kBN;
  a.row_tiles = (a.R + intattn::shared::kBM - 1) / intattn::shared::kBM;
  a.per_head = scales->per_head ? 1 : 0;
  a.out_kind = out_dtype;
  a.zero_left_out = zero_left_out ? 1 : 0;
  a.k_u8 = scales->z_k ? 1 : 0;
  a.v_u8 = scales->z_v ? 1 : 0;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int sms = 0;
  if (sm_count(&sms) != INTATTN_OK) return INTATTN_ERR_CUDA;
  // Few queries fold F key tiles into a tile, as long as every SM still gets
  // one: B9 H32/8 d128 over 50000 shared keys 48.0 us a call, without folding 61.3;
  // B2 H32/8 over 30000 35.1, without 43.7; B8 H12 d64 over 9000 25.3, without 31.3.  Too
  // few tiles: B4 H12 d64 over 500 18.0 us, folded all the same 18.5; B16 H32/8 over 2000
  // 29.1 and 30.6; one shape the other way, B16 H16 d64 over 1500 20.7 and 19.8.
  a.fold = 1;
  for (int f = 2; f <= 4; f *= 2)
    if (a.R <= intattn::shared::kBM / f && static_cast<long long>(Hkv) * ((a.key_tiles + f - 1) / f) >= sms) a.fold = f;
  a.seg_tiles = (a.key_tiles + a.fold - 1) / a.fold;
  const long long tiles = static_cast<long long>(Hkv) * a.row_tiles * a.seg_tiles;
  if (tiles > 0x7fffffffll) return INTATTN_ERR_UNSUPPORTED;
  a.tiles = static_cast<int32_t>(tiles);
  if (Lp > 0 && (!encode_rows(&a.tm_k, k_prefix, d, Lp, Lp_max, Hkv, intattn::shared::kBN) ||
                 !encode_rows(&a.tm_v, v_prefix, d, Lp, Lp_max, Hkv, intattn::shared::kBN)))
    return INTATTN_ERR_CUDA;
  const long long planes = static_cast<long long>(B) * Hkv;
  if (Lmax > 0 && (!encode_rows(&a.tm_kc, k_cache, d, Lmax, Lmax, planes, intattn::shared::kOwnBytes / d) ||
                   !encode_rows(&a.tm_vc, v_cache, d, Lmax, Lmax, planes, intattn::shared::kOwnBytes / d)))
    return INTATTN_ERR_CUDA;
  // The K / V ring and the own warps' rings share their memory (kRingBytes):
  // one block per own warp instead of two where the prefix is the longer stream
  // (B9 H32/8 over 50000 shared and up to 333 own keys: 48.0 us against 48.9 with
  // two; one everywhere: B64 H32, 4001 shared and up to 777 own keys 84.0 us against 68.4, B64
  // H32/8 over up to 8192 own keys 173 against 142).  The rule knows the caches' capacity, not
  // the lengths on the device; caches of 8192 rows that hold 100 (B64 H32/8, 8192 shared): two
  // blocks 35.9 us, one 36.5.
  const long long own_keys = static_cast<long long>(B) * Hkv * Lmax, prefix_keys = static_cast<long long>(Hkv) * Lp;
  a.own_slots = Lmax == 0 ? 0 : 2 * own_keys <= prefix_keys ? 1 : 2;
  a.stages = (intattn::shared::kRingBytes - a.own_slots * intattn::shared::kOwnWarps * intattn::shared::kOwnBytes) /
             (intattn::shared::kBN * d);
  // as many CTAs as there are prefix tiles or 128-key pieces of own rows
  const long long own = static_cast<long long>(B) * Hkv * ((Lmax + 127) / 128);
  const int grid = static_cast<int>(std::min<long long>(sms, std::max<long long>(std::max(tiles, own), 1)));
  // A CTA whose tiles belong to two heads pays for the second segment (tables, O read out
  // twice): four tiles' worth.  B64 H32/8 over 8192 + 1024 keys 42.5 us a call instead
  // of 46.0 without it (two tiles' worth 43.8, eight 42.8), B9 L50000 48.0 instead of 51.0, B128 H8 d64 over
  // 16000 35.1 instead of 38.1, B30 H32 over 2400 29.2 instead of 32.4 (two 28.6, eight 33.1).  Not where a CTA has
  // one tile at most: B4 H12 L500 18.0 us, with it 19.4 (two tiles here, none there).
  a.seg_cost = tiles > grid ? 4 : 0;
  const long long cost = static_cast<long long>(Hkv) * a.row_tiles * (a.seg_tiles + a.seg_cost);
  if (cost > 0x7fffffffll) return INTATTN_ERR_UNSUPPORTED;
  a.cta_cost = static_cast<int32_t>(cost / grid);
  a.cta_more = static_cast<int32_t>(cost % grid);
  if (a.k_u8 || a.v_u8) return d == 64 ? shared_launch<64, true>(a, grid, L, st) : shared_launch<128, true>(a, grid, L, st);
  return d == 64 ? shared_launch<64, false>(a, grid, L, st) : shared_launch<128, false>(a, grid, L, st);
}

}  // extern "C"
