// Host side of the row operators (see intattn.h): argument checks and
// launches.  Included by intattn.cu, whose helpers it uses.
#pragma once

namespace {

using intattn::ReadArgs;
using intattn::RowArgs;
using intattn::RowCodeArgs;
using intattn::RowTensor;

// The element type of a call's floating tensors; whether rows left out become 0.
bool row_dtype(int dtype, int32_t* bf16, int32_t* zero) {
  *zero = dtype >= 0 && (dtype & INTATTN_ZERO_LEFT_OUT) ? 1 : 0;
  if (*zero) dtype &= ~INTATTN_ZERO_LEFT_OUT;
  *bf16 = dtype == INTATTN_DTYPE_BF16 ? 1 : 0;
  return dtype == INTATTN_DTYPE_FP16 || dtype == INTATTN_DTYPE_BF16;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A strided [B, heads, L, d] tensor of 16-bit elements whose rows start on
// 16-byte boundaries.  An output may not repeat rows.
int check_rows(const intattn_rows_t* r, int B, int heads, int L, bool output) {
  if (!r || !r->ptr) return INTATTN_ERR_INVALID_ARG;
  if (!aligned16(r->ptr) || r->stride_b % 8 || r->stride_h % 8 || r->stride_l % 8) return INTATTN_ERR_UNSUPPORTED;
  if (output && ((B > 1 && r->stride_b == 0) || (heads > 1 && r->stride_h == 0) || (L > 1 && r->stride_l == 0)))
    return INTATTN_ERR_INVALID_ARG;
  return INTATTN_OK;
}

// Whether n bytes at a and m bytes at b share any.
bool overlap(const void* a, unsigned long long n, const void* b, unsigned long long m) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y ? y - x < n : x - y < m;
}

// Whether the rows of x are those of y, one by one.
bool same_rows(const intattn_rows_t* x, const intattn_rows_t* y, int B, int heads, int L) {
  return x->ptr == y->ptr && (B <= 1 || x->stride_b == y->stride_b) && (heads <= 1 || x->stride_h == y->stride_h) &&
         (L <= 1 || x->stride_l == y->stride_l);
}

int check_rope_norm(const intattn_rope_norm_t* rn, int d, RowArgs* a) {
  if (rn->positions && !rn->table) return INTATTN_ERR_INVALID_ARG;
  if (rn->table) {
    if (!rn->positions || rn->n_positions < 1 || rn->rot < 0 || rn->rot > d) return INTATTN_ERR_INVALID_ARG;
    if (rn->rot % 16 || !aligned16(rn->table) || !aligned4(rn->positions)) return INTATTN_ERR_UNSUPPORTED;
    a->table = reinterpret_cast<const float2*>(rn->table);
    a->positions = rn->positions;
    a->n_positions = rn->n_positions;
    a->rot = rn->rot;
    a->interleaved = rn->interleaved ? 1 : 0;
  }
  if ((rn->w_q && !aligned16(rn->w_q)) || (rn->w_k && !aligned16(rn->w_k))) return INTATTN_ERR_UNSUPPORTED;
  if (rn->w_q || rn->w_k) {
    if (!std::isfinite(rn->eps) || !(rn->eps > 0.0f)) return INTATTN_ERR_PARAM_RANGE;
    a->eps = rn->eps;
  }
  return INTATTN_OK;
}

void set_input(RowTensor* t, const intattn_rows_t* r, int heads) {
  t->in = r->ptr;
  t->isb = r->stride_b;
  t->ish = r->stride_h;
  t->isl = r->stride_l;
  t->heads = heads;
}

// A warp takes a batch of one tensor's heads of a token: as many as it holds in
// flight (D / 8 lanes and four loads per lane) when that still gives every SM
// several warps, else one load's worth, so that few tokens spread over more SMs.
// Always four loads: one token 2.9 us instead of 2.4, the cache write of 64 tokens with
// eight K / V heads 3.7 instead of 2.8; always one: the rows of a LLaMA-7B
// prefill 101 us instead of 51, their cache write 177 instead of 91.
template <bool kCodes>
int rows_launch(intattn::RowCall<kCodes>& a, int d, cudaStream_t st) {
  int sms = 0;
  if (sm_count(&sms) != INTATTN_OK) return INTATTN_ERR_CUDA;
  const int per_load = 256 / d;
  const long long tokens = static_cast<long long>(a.B) * a.L;
  if (tokens > 0x7fffffffll) return INTATTN_ERR_UNSUPPORTED;
  a.tokens = static_cast<uint32_t>(tokens);
  long long most = 0;
  for (a.batch = 4 * per_load;; a.batch = per_load) {
    long long warps = 0;
    most = 0;
    for (int i = 0; i < a.n_tensors; ++i) {
      a.t[i].warps = (a.t[i].heads + a.batch - 1) / a.batch;
      warps += tokens * a.t[i].warps;
      most = std::max(most, tokens * a.t[i].warps);
    }
    if (a.batch == per_load || warps >= 8ll * sms) break;
  }
  if (most > 0x7fffffffll) return INTATTN_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>((most + intattn::rows::kWarps - 1) / intattn::rows::kWarps),
                  static_cast<unsigned>(a.n_tensors));
  auto* kernel = d == 64 ? (a.bf16 ? intattn::rows::rows_kernel<64, kCodes, true> : intattn::rows::rows_kernel<64, kCodes, false>)
                         : (a.bf16 ? intattn::rows::rows_kernel<128, kCodes, true> : intattn::rows::rows_kernel<128, kCodes, false>);
  kernel<<<grid, intattn::rows::kThreads, 0, st>>>(a);
  return note_launch(cudaGetLastError());
}

// Scales and zero-points of one tensor's heads: RN32(1 / s), or s itself.
int code_params(const float* s, const int32_t* z, int n, int bits, bool reciprocal, float* out, float* zero) {
  if (!s) return INTATTN_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    if (!std::isfinite(s[i]) || !(s[i] > 0.0f)) return INTATTN_ERR_PARAM_RANGE;
    out[i] = reciprocal ? std::min(1.0f / s[i], 3.402823466e38f) : s[i];
    if (z) {
      if (z[i] < 0 || z[i] >= (1 << bits)) return INTATTN_ERR_INVALID_ARG;
      zero[i] = static_cast<float>(z[i]);
    }
  }
  return INTATTN_OK;
}

}  // namespace

extern "C" {

int intattn_qk_norm_rope(const intattn_rows_t* q, const intattn_rows_t* k, const intattn_rope_norm_t* rn, int dtype,
                         int B, int H, int Hkv, int L, int d, const intattn_rows_t* q_out, const intattn_rows_t* k_out,
                         intattn_stream_t stream) {
  if (B < 0 || H <= 0 || Hkv < 0 || L < 0 || !rn || !q || !q_out || (Hkv > 0) != (k != nullptr) ||
      (k != nullptr) != (k_out != nullptr))
    return INTATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return INTATTN_ERR_UNSUPPORTED;
  int32_t bf16, zero;
  if (!row_dtype(dtype, &bf16, &zero)) return INTATTN_ERR_UNSUPPORTED;
  if (H > 65535 || Hkv > 65535) return INTATTN_ERR_UNSUPPORTED;
  RowArgs a;
  std::memset(&a, 0, sizeof(a));
  int rc = check_rope_norm(rn, d, &a);
  if (rc) return rc;
  if (static_cast<long long>(B) * L == 0) return INTATTN_OK;
  const intattn_rows_t* in[2] = {q, k};
  const intattn_rows_t* out[2] = {q_out, k_out};
  const int heads[2] = {H, Hkv};
  a.n_tensors = k ? 2 : 1;
  for (int i = 0; i < a.n_tensors; ++i) {
    if ((rc = check_rows(in[i], B, heads[i], L, false)) || (rc = check_rows(out[i], B, heads[i], L, true))) return rc;
    set_input(&a.t[i], in[i], heads[i]);
    a.t[i].out = const_cast<void*>(out[i]->ptr);
    a.t[i].osb = out[i]->stride_b;
    a.t[i].osh = out[i]->stride_h;
    a.t[i].osl = out[i]->stride_l;
    a.t[i].w = i ? rn->w_k : rn->w_q;
    a.t[i].rope = 1;
  }
  // An output that starts where another tensor does: only in place.  (Views of
  // one packed buffer interleave, so their extents say nothing.)
  for (int i = 0; i < a.n_tensors; ++i)
    for (int j = 0; j < a.n_tensors; ++j) {
      if (i == j ? out[i]->ptr == in[i]->ptr && !same_rows(out[i], in[i], B, heads[i], L)
                 : out[i]->ptr == in[j]->ptr || out[i]->ptr == out[j]->ptr)
        return INTATTN_ERR_INVALID_ARG;
    }
  a.B = B;
  a.L = L;
  a.bf16 = bf16;
  a.zero_left_out = zero;
  return rows_launch<false>(a, d, reinterpret_cast<cudaStream_t>(stream));
}

int intattn_cache_write(const intattn_rows_t* k, const intattn_rows_t* v, const intattn_rows_t* q, int dtype,
                        const intattn_scales_t* scales, int bits, const intattn_rope_norm_t* rn, int B, int H, int Hkv,
                        int L, int Lmax, int d, const int32_t* start, const int32_t* lengths, void* k_cache,
                        void* v_cache, int8_t* q_out, intattn_stream_t stream) {
  if (B < 0 || Hkv <= 0 || L < 0 || Lmax < 0 || !scales || (q != nullptr) != (q_out != nullptr) || (q && H <= 0))
    return INTATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return INTATTN_ERR_UNSUPPORTED;
  int32_t bf16, zero;
  if (!row_dtype(dtype, &bf16, &zero)) return INTATTN_ERR_UNSUPPORTED;
  if (bits != 8 && bits != 4) return INTATTN_ERR_UNSUPPORTED;
  if (Hkv > 65535 || (q && H > 65535)) return INTATTN_ERR_UNSUPPORTED;
  if (scales->per_head && (Hkv > INTATTN_MAX_HEADS || (q && H > INTATTN_MAX_HEADS))) return INTATTN_ERR_UNSUPPORTED;
  static_assert(sizeof(RowCodeArgs) <= 8192, "kernel argument block too large");
  RowCodeArgs a;
  std::memset(&a, 0, sizeof(a));
  int rc;
  if (rn && (rc = check_rope_norm(rn, d, &a))) return rc;
  const int n_kv = scales->per_head ? Hkv : 1, n_q = scales->per_head ? H : 1;
  constexpr int S = INTATTN_MAX_HEADS;
  if ((rc = code_params(scales->s_k, scales->z_k, n_kv, bits, true, a.inv, a.zero)) ||
      (rc = code_params(scales->s_v, scales->z_v, n_kv, bits, true, a.inv + S, a.zero + S)) ||
      (q && (rc = code_params(scales->s_q, nullptr, n_q, 8, true, a.inv + 2 * S, a.zero + 2 * S))))
    return rc;
  if (static_cast<long long>(B) * L == 0) return INTATTN_OK;
  if (!start || !k_cache || !v_cache) return INTATTN_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(q_out) || !aligned4(start) || !aligned4(lengths))
    return INTATTN_ERR_UNSUPPORTED;
  const intattn_rows_t* in[3] = {k, v, q};
  void* out[3] = {k_cache, v_cache, q_out};
  a.n_tensors = q ? 3 : 2;
  for (int i = 0; i < a.n_tensors; ++i) {
    const int heads = i < 2 ? Hkv : H;
    if ((rc = check_rows(in[i], B, heads, L, false))) return rc;
    RowTensor& t = a.t[i];
    set_input(&t, in[i], heads);
    const long long rows = i < 2 ? Lmax : L;
    t.out = out[i];
    t.osb = rows * heads * d;
    t.osh = rows * d;
    t.osl = d;
    t.w = rn ? (i == 0 ? rn->w_k : i == 2 ? rn->w_q : nullptr) : nullptr;
    t.rope = i != 1;
    t.cache = i < 2;
    t.bits = i < 2 ? bits : 8;
    const bool asym = (i == 0 && scales->z_k) || (i == 1 && scales->z_v);
    t.hi = static_cast<float>(asym ? (1 << t.bits) - 1 : (1 << (t.bits - 1)) - 1);
    t.lo = asym ? 0.0f : -t.hi;
    t.sc = i * S;
  }
  const unsigned long long cache = static_cast<unsigned long long>(B) * Hkv * Lmax * (d * bits / 8);
  const unsigned long long queries = static_cast<unsigned long long>(B) * H * L * d;
  if (overlap(k_cache, cache, v_cache, cache) ||
      (q && (overlap(q_out, queries, k_cache, cache) || overlap(q_out, queries, v_cache, cache))))
    return INTATTN_ERR_INVALID_ARG;
  a.B = B;
  a.L = L;
  a.Lmax = Lmax;
  a.bf16 = bf16;
  a.zero_left_out = zero;
  a.per_head = scales->per_head ? 1 : 0;
  a.start = start;
  a.lengths = lengths;
  return rows_launch<true>(a, d, reinterpret_cast<cudaStream_t>(stream));
}

int intattn_cache_read(const void* k_cache, const void* v_cache, const intattn_scales_t* scales, int bits, int B,
                       int Hkv, int L, int Lmax, int d, const int32_t* start, const int32_t* lengths, int dtype,
                       void* k_out, void* v_out, intattn_stream_t stream) {
  if (B < 0 || Hkv <= 0 || L < 0 || Lmax < 0 || !scales || (v_cache != nullptr) != (v_out != nullptr))
    return INTATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return INTATTN_ERR_UNSUPPORTED;
  int32_t bf16, zero;
  if (!row_dtype(dtype, &bf16, &zero)) return INTATTN_ERR_UNSUPPORTED;
  if (bits != 8 && bits != 4) return INTATTN_ERR_UNSUPPORTED;
  if (scales->per_head && Hkv > INTATTN_MAX_HEADS) return INTATTN_ERR_UNSUPPORTED;
  ReadArgs a;
  std::memset(&a, 0, sizeof(a));
  const int n = scales->per_head ? Hkv : 1;
  constexpr int S = INTATTN_MAX_HEADS;
  int rc;
  if ((rc = code_params(scales->s_k, scales->z_k, n, bits, false, a.scale, a.zero)) ||
      (v_out && (rc = code_params(scales->s_v, scales->z_v, n, bits, false, a.scale + S, a.zero + S))))
    return rc;
  if (static_cast<long long>(B) * L == 0) return INTATTN_OK;
  if (!k_cache || !k_out || !start) return INTATTN_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_out) || !aligned16(v_out) || !aligned4(start) ||
      !aligned4(lengths))
    return INTATTN_ERR_UNSUPPORTED;
  const unsigned long long values = 2ull * B * Hkv * L * d;
  if (v_out && overlap(k_out, values, v_out, values)) return INTATTN_ERR_INVALID_ARG;
  a.in[0] = static_cast<const uint8_t*>(k_cache);
  a.in[1] = static_cast<const uint8_t*>(v_cache);
  a.out[0] = k_out;
  a.out[1] = v_out;
  a.n_tensors = v_out ? 2 : 1;
  a.B = B;
  a.H = Hkv;
  a.L = L;
  a.Lmax = Lmax;
  a.bf16 = bf16;
  a.zero_left_out = zero;
  a.per_head = scales->per_head ? 1 : 0;
  a.bits = bits;
  a.asym_k = scales->z_k ? 1 : 0;
  a.asym_v = scales->z_v ? 1 : 0;
  a.start = start;
  a.lengths = lengths;
  const int per_cta = intattn::rows::kReadThreads / (d / 8) * intattn::rows::kReadUnroll;
  a.chunks = (L - 1) / per_cta + 1;
  const long long grid = static_cast<long long>(a.chunks) * B * Hkv * a.n_tensors;
  if (grid > 0x7fffffffll) return INTATTN_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto* kernel = d == 64 ? (a.bf16 ? intattn::rows::read_kernel<64, true> : intattn::rows::read_kernel<64, false>)
                         : (a.bf16 ? intattn::rows::read_kernel<128, true> : intattn::rows::read_kernel<128, false>);
  kernel<<<static_cast<unsigned>(grid), intattn::rows::kReadThreads, 0, st>>>(a);
  return note_launch(cudaGetLastError());
}

}  // extern "C"
