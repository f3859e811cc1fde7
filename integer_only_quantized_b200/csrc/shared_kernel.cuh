// Decode for a batch whose sequences share a prefix: one query per (b, h)
// against the prefix rows of its K / V head followed by the rows of its own
// cache, by the definition of intattn.h over the joined keys.
//
// The definition needs the row max before any table index and the row sum
// before any probability, over the joined keys, so the work is three phases
// with a grid-wide barrier between them, in one cooperative launch of at
// most one CTA per SM:
//   A  scores -> row max            (global atomic max)
//   B  scores -> Z = sum of LUT     (global atomic add)
//   C  scores -> u8 P, P.V          (global adds), then a barrier and requantisation
// Integer sums do not depend on their order, so the bytes do not depend on
// the split.  acc is added up in fp32: every partial sum is a whole number
// below 2^24 (sum of P <= 510 times 255), so those sums are exact too, and one
// instruction adds four channels.
//
// Prefix.  The R = B G queries that share a K / V head are the rows of a
// 128-row tile, so the prefix streams once per 128 queries and the products
// run on the tensor cores: tcgen05.mma kind::i8 for S = Q.K^T and O += P.V as
// in the prefill kernel (whose warp roles, barriers and index arithmetic this
// follows), scores recomputed in each phase (K comes from L2 after phase A;
// keeping 4 bytes per score would move more than re-reading D bytes per key
// does for every row of the tile at once).  The (head, row tile, 128-key
// tile) triples are cut into equal consecutive ranges, one per CTA; the part of
// a range within one (head, row tile) is a segment.
//
// Own rows.  They are read by one sequence only: an HBM stream with up to
// eight query rows per K / V row.  Each softmax warp takes an equal
// consecutive share of all blocks of own rows and streams it through a ring
// of its own (two 2 KB TMA tiles, in the memory of the tables, which those
// parts of the phases do not use): 64 KB in flight per SM without registers
// or barriers shared by warps.  The products are m16n8k32 integer MMAs, keys or
// channels on the 16 side and the grouped heads on the 8 side; the contraction order
// is free, so a thread's 16 consecutive bytes of K serve as its fragments.
// Scores (4 bytes per key and head), and from phase B on their table indices
// (one byte), wait in the workspace.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <climits>
#include <cstdint>

#include "common.cuh"
#include "decode_kernel.cuh"
#include "params_kernel.cuh"
#include "prefill_kernel.cuh"
#include "quantize_kernel.cuh"
#include "rows_kernel.cuh"
#include "sm100.cuh"

namespace intattn {

struct SharedArgs {
  CUtensorMap tm_k, tm_v;     // prefix [Hkv, Lp, d], box {d, 128, 1}
  CUtensorMap tm_kc, tm_vc;   // own rows [B Hkv, Lmax, d], boxes {d, 2048 / d, 1} and {64, 32, 1}
  const int8_t* q;            // [B, H, d]
  const int32_t* lengths;     // [B], or null: Lmax
  void* out;                  // [B, H, d] int8 codes, or fp16 / bf16 values
  // workspace; row r of K / V head hk (r = b G + g) is row hk R + r
  uint32_t* ctr;              // [8] barrier counters (zeroed before the kernel, with row_max)
  uint32_t* row_max;          // [Hkv R] score + 2^31
  int32_t* row_z;             // [Hkv R] Z (zeroed in phase A, as the next two)
  int32_t* row_p;             // [Hkv R] sum of P (V zero-points)
  float* acc;                 // [Hkv R, d] sum of P.V
  int32_t* scores;            // [B H, ld_s] scores of the own rows
  uint32_t* index;            // [B H, ld_s / 4] their table indices, a byte each
  int32_t B, H, Hkv, G, R, Lp, Lmax, ld_s, per_head, out_kind, k_u8, v_u8, n_luts;
  int32_t key_tiles, row_tiles;  // 128-key tiles of the prefix, 128-row tiles of R
  int32_t tiles;                 // Hkv * row_tiles * key_tiles
  float s_o[INTATTN_MAX_HEADS];
  uint32_t lut[INTATTN_MAX_CLIPS][32];
  HeadParamsDev hp[INTATTN_MAX_HEADS];
};

namespace shared {

using prefill::exact_R;
using prefill::fma2_rz;
using prefill::fma_rz_sat;
using prefill::imax;
using prefill::pack2;

constexpr int kBM = 128;                   // query rows per tile
constexpr int kBN = 128;                   // keys per tile
constexpr int kTeams = 2;                  // teams taking alternate S tiles
constexpr int kSoftWarps = 16;
constexpr int kTeamWarps = kSoftWarps / kTeams;
constexpr int kCols = 64;                  // S columns per thread and tile (two halves)
constexpr int kProducerWarp = 16;
constexpr int kMmaWarp = 17;
constexpr int kQWarp = 18;                 // warps 18-19: Q rows into shared memory
constexpr int kEpiWarp0 = 20;              // warps 20-23: O of a finished segment
constexpr int kEpiWarps = 4;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;              // two S buffers
constexpr uint32_t kColO = 256;
constexpr uint32_t kColP = 384;            // four P buffers of 32 columns
constexpr int kPBufs = 4;
constexpr uint32_t kNbSoft = 1;            // named barrier of the softmax warps
constexpr uint32_t kNbBoth = 2;            // softmax and epilogue warps

enum Role : unsigned { kRoleSoftmax = 5, kRoleProducer = 6, kRoleMma = 7, kRoleEpilogue = 8, kRoleQ = 9 };

enum Bar : int {
  kBarQFull = 0,    // [2]
  kBarQEmpty = 2,   // [2]
  kBarSFull = 4,    // [2]
  kBarSEmpty = 6,   // [2]
  kBarPFull = 8,    // [4]
  kBarPEmpty = 12,  // [4]
  kBarOFull = 16,
  kBarOEmpty = 17,
  kBarDrain = 18,
  kBarOwn = 19,     // [16][2] tiles of the softmax warps' own rings
  kBarKvFull = 51,  // [stages], then kv_empty[stages]
};

template <int D>
struct Cfg {
  static constexpr int kStages = (D == 64) ? 8 : 6;
  static constexpr uint32_t kTileBytes = kBN * D;
  static constexpr uint32_t kQBytes = kBM * D;
  static constexpr uint32_t kSwizzle = (D == 128) ? 2u : 4u;  // 128B / 64B swizzle
  static constexpr uint32_t kSBO = 8 * D;
  static constexpr int kNumBars = kBarKvFull + 2 * kStages;
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffKV = kOffQ + 2 * kQBytes;
  // per-row tables [33][kBM] u32, row k for index code k (see idx_bits): in
  // phase B the first holds LUT, in phase C table b holds P << 8b
  static constexpr uint32_t kTabBytes = 33 * kBM * 4;
  static constexpr uint32_t kOffTab = kOffKV + kStages * kTileBytes;
  static constexpr uint32_t kOffLut = kOffTab + 4 * kTabBytes;
  static constexpr uint32_t kOffHp = kOffLut + INTATTN_MAX_CLIPS * 32 * 4;
  static constexpr uint32_t kOffBars = kOffHp + INTATTN_MAX_HEADS * sizeof(HeadParamsDev);
  static constexpr uint32_t kOffMisc = kOffBars + kNumBars * 8;  // TMEM address, barrier verdict
  static constexpr uint32_t kUsed = kOffMisc + 16;
  static_assert(4 * kTabBytes >= kSoftWarps * 4096 && kOffTab % 1024 == 0, "own rings in the tables' memory");
  // one CTA per SM: every CTA takes all 512 TMEM columns
  static constexpr uint32_t kSmemBytes = (kUsed + 1024 > 120 * 1024) ? kUsed + 1024 : 120 * 1024;
};

// Consecutive tiles of one (head, row tile).
struct Segment {
  int hk, rt, j0, n;
};
__device__ __forceinline__ Segment segment_at(const SharedArgs& a, int t, int t1) {
  Segment s;
  const int u = t / a.key_tiles;
  s.j0 = t - u * a.key_tiles;
  s.n = min(t1 - t, a.key_tiles - s.j0);
  s.hk = u / a.row_tiles;
  s.rt = u - s.hk * a.row_tiles;
  return s;
}

__device__ __forceinline__ uint32_t bias(int32_t s) { return static_cast<uint32_t>(s) ^ 0x80000000u; }
__device__ __forceinline__ int32_t unbias(uint32_t u) { return static_cast<int32_t>(u ^ 0x80000000u); }

// Four fp32 adds to consecutive addresses (16-byte aligned).
__device__ __forceinline__ void red_add4(float* p, float a, float b, float c, float d) {
  asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}

// D[16 x 8] += A[16 x 32] B[32 x 8], bytes, row x column fragments.
template <bool kASigned, bool kBSigned>
__device__ __forceinline__ void mma16832(int32_t (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (kASigned && kBSigned)
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else if constexpr (kBSigned)
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else if constexpr (kASigned)
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.u8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.u8.u8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Own rows of a sequence; 0 for a length out of range (its output is skipped).
__device__ __forceinline__ int own_rows(const SharedArgs& a, int b) {
  if (a.lengths == nullptr) return a.Lmax;
  const int n = __ldg(a.lengths + b);
  return n < 0 || n > a.Lmax ? 0 : n;
}

// Blocks of `keys` keys over the own rows of every sequence and `units`
// units per sequence, in the order (b, unit, block): their number, and the
// block at position p.  Warp-collective.
__device__ __forceinline__ long long own_blocks(const SharedArgs& a, int keys, int units) {
  const int lane = threadIdx.x & 31;
  long long n = 0;
  for (int b = lane; b < a.B; b += 32) n += (own_rows(a, b) + keys - 1) / keys;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n * units;
}

struct Walk {
  int b, u, blk, nb;  // nb: blocks of sequence b
  __device__ __forceinline__ void seek(const SharedArgs& a, int keys, int units, long long p) {
    const int lane = threadIdx.x & 31;
    b = u = blk = nb = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int mine = b0 + lane < a.B ? (own_rows(a, b0 + lane) + keys - 1) / keys : 0;
      long long incl = static_cast<long long>(mine) * units;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, incl > p);
      if (past) {
        const int l = __ffs(past) - 1;
        nb = __shfl_sync(0xffffffffu, mine, l);
        p -= __shfl_sync(0xffffffffu, incl, l) - static_cast<long long>(nb) * units;
        b = b0 + l;
        u = static_cast<int>(p / nb);
        blk = static_cast<int>(p - static_cast<long long>(u) * nb);
        return;
      }
      p -= __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  // to the next block (there is one); true if the unit changed
  __device__ __forceinline__ bool next(const SharedArgs& a, int keys, int units) {
    if (++blk < nb) return false;
    blk = 0;
    if (++u == units) {
      u = 0;
      do {
        ++b;
        nb = (own_rows(a, b) + keys - 1) / keys;
      } while (nb == 0);
    }
    return true;
  }
};

// A warp's private ring of two 2 KB slots for the own rows' tiles: lane 0
// issues the loads, every lane waits.
struct OwnRing {
  uint32_t base, bar;  // shared addresses: slot i at base + 2048 i, barrier i at bar + 8 i
  uint32_t issued, used;
  __device__ __forceinline__ void issue(const CUtensorMap* tm, int x, int y, int z) {
    if ((threadIdx.x & 31) == 0) {
      const uint32_t i = issued & 1;
      mbar_arrive_expect_tx(bar + 8 * i, 2048);
      tma_load_3d(base + 2048 * i, tm, bar + 8 * i, x, y, z);
    }
    ++issued;
  }
  // the oldest tile not yet used (its address), or 0 when the wait ran out
  __device__ __forceinline__ uint32_t wait(unsigned role) {
    const uint32_t i = used & 1, par = (used >> 1) & 1;
    ++used;
    if (mbar_wait_warp(bar + 8 * i, par, role)) return base + 2048 * i;
    if (used < issued) {  // give up, but leave no copy in flight
      mbar_wait_warp(bar + 8 * (used & 1), (used >> 1) & 1, role);
      ++used;
    }
    return 0u;
  }
};

__device__ __forceinline__ uint4 lds_u128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds_u64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// Where the score of key kk of a 32-key block is kept: thread t of phase C
// reads the four scores of a word with one load (position 16 g + 4 t + i) and
// the V bytes of their keys from rows whose 16-byte pieces lie in other
// banks than those of the other threads' rows (see own_pv).
__device__ __forceinline__ int score_at(int kk) {
  return (kk & 16) | ((kk & 4) << 1) | ((kk & 1) << 2) | ((kk & 8) >> 2) | ((kk & 2) >> 1);
}
__device__ __forceinline__ int key_of(int t, int i) {  // word 4 g + .. of thread t: i = 0 .. 7
  return (t & 1) + 4 * (t >> 1) + 2 * (i & 1) + 8 * ((i >> 1) & 1) + 16 * (i >> 2);
}

// ---- phase A of the own rows: scores and row max ----
// Units (hk, group of eight query heads).  A key past the sequence's last
// (in its last 32-key block) gets the lowest score, whose table entry is 0.
template <int D, bool kKSigned>
__device__ __forceinline__ bool own_scores(const SharedArgs& a, OwnRing& ring, int warp, int warps) {
  constexpr int kKeys = 2048 / D;      // 16 or 32
  constexpr int kSub = kKeys / 16;     // 16-key products per block
  constexpr int kCh = D / 64;          // 16-byte pieces of a row per thread: piece t (and t + 4)
  const int lane = threadIdx.x & 31, n8 = lane >> 2, t = lane & 3;
  const int groups = (a.G + 7) / 8, units = a.Hkv * groups;
  const long long total = own_blocks(a, kKeys, units);
  const long long lo = total * warp / warps, hi = total * (warp + 1) / warps;
  const int n = static_cast<int>(hi - lo);
  if (n == 0) return true;
  Walk ld, w;
  w.seek(a, kKeys, units, lo);
  ld = w;
  auto issue = [&]() { ring.issue(&a.tm_kc, 0, ld.blk * kKeys, ld.b * a.Hkv + ld.u / groups); };
  issue();
  if (n > 1) {
    ld.next(a, kKeys, units);
    issue();
  }
  uint4 q[kCh];
  int hk = 0, rows = 0, len = 0;
  size_t at = 0;       // first query row of the unit, in the row arrays
  int32_t* sp = nullptr;
  int32_t m[2];
  auto enter = [&]() {
    hk = w.u / groups;
    const int g0 = 8 * (w.u - hk * groups);
    rows = min(8, a.G - g0);
    len = own_rows(a, w.b);
    at = static_cast<size_t>(hk) * a.R + w.b * a.G + g0;
    const size_t head = static_cast<size_t>(w.b) * a.H + hk * a.G + g0;
    sp = a.scores + (head + 2 * t) * a.ld_s;
#pragma unroll
    for (int c = 0; c < kCh; ++c)
      q[c] = n8 < rows ? __ldg(reinterpret_cast<const uint4*>(a.q + (head + n8) * D + 16 * t + 64 * c))
                       : make_uint4(0, 0, 0, 0);
    m[0] = m[1] = INT_MIN;
  };
  auto leave = [&]() {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      m[0] = imax(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
      m[1] = imax(m[1], __shfl_xor_sync(0xffffffffu, m[1], o));
    }
    if (n8 < 2 && 2 * t + n8 < rows) atomicMax(a.row_max + at + 2 * t + n8, bias(n8 ? m[1] : m[0]));
  };
  enter();
  for (int i = 0; i < n; ++i) {
    const uint32_t tile = ring.wait(kRoleSoftmax);
    if (tile == 0) return false;
    uint4 k[kSub][2][kCh];
#pragma unroll
    for (int s = 0; s < kSub; ++s)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int c = 0; c < kCh; ++c) {
          const int row = 16 * s + 8 * e + n8;  // the TMA's swizzle on the 16-byte piece
          const int piece = D == 128 ? ((t + 4 * c) ^ (row & 7)) : (t ^ ((row >> 1) & 3));
          k[s][e][c] = lds_u128(tile + row * D + 16 * piece);
        }
    __syncwarp();  // every lane has read the tile
    if (i + 2 < n) {
      ld.next(a, kKeys, units);
      issue();
    }
#pragma unroll
    for (int s = 0; s < kSub; ++s) {
      int32_t d[4] = {0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < kCh; ++c) {
        mma16832<kKSigned, true>(d, k[s][0][c].x, k[s][1][c].x, k[s][0][c].y, k[s][1][c].y, q[c].x, q[c].y);
        mma16832<kKSigned, true>(d, k[s][0][c].z, k[s][1][c].z, k[s][0][c].w, k[s][1][c].w, q[c].z, q[c].w);
      }
      // d[0], d[1]: key n8, rows 2t and 2t + 1; d[2], d[3]: key n8 + 8
      const int j0 = w.blk * kKeys + 16 * s;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = j0 + 8 * e + n8;
        int32_t* dst = sp + (j & ~31) + score_at(j & 31);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int32_t v = j < len ? d[2 * e + r] : INT_MIN;
          if (2 * t + r < rows) {
            dst[static_cast<size_t>(r) * a.ld_s] = v;
            // the second half of a last 32-key block that no tile covers
            if (kKeys == 16 && (j0 & 16) == 0 && j0 + 16 >= len)
              (dst + 16)[static_cast<size_t>(r) * a.ld_s] = INT_MIN;
          }
          m[r] = imax(m[r], v);
        }
      }
    }
    if (i + 1 < n && w.blk + 1 == w.nb) {
      leave();
      w.next(a, kKeys, units);
      enter();
    } else if (i + 1 < n) {
      w.next(a, kKeys, units);
    }
  }
  leave();
  return true;
}

// Index arithmetic of one row on the integer pipe (as decode_kernel.cuh):
// idx = (Cm - max(S, lo) M) >> s in wrapping 32-bit arithmetic.  lo = m - D
// stays above the lowest int: D < 61 2^25 and |m| < 2^23.
struct RowIndex {
  int32_t lo;
  uint32_t M, s, Cm;
  __device__ __forceinline__ void set(const HeadParamsDev& hp, int32_t m) {
    lo = m - hp.D;
    M = static_cast<uint32_t>(hp.M);
    s = static_cast<uint32_t>(hp.s);
    Cm = static_cast<uint32_t>(m) * M + (1u << (s - 1));
  }
  __device__ __forceinline__ uint32_t operator()(int32_t sc) const {
    return (Cm - static_cast<uint32_t>(imax(sc, lo)) * M) >> s;
  }
};

// ---- phase B of the own rows: Z, 128 scores of one query row per block ----
__device__ __forceinline__ void own_sums(const SharedArgs& a, const HeadParamsDev* hp_s, const uint32_t* lut_s, int warp,
                                         int warps) {
  const int lane = threadIdx.x & 31;
  const long long total = own_blocks(a, 128, a.H);
  const long long lo = total * warp / warps, hi = total * (warp + 1) / warps;
  const int n = static_cast<int>(hi - lo);
  if (n == 0) return;
  Walk w;
  w.seek(a, 128, a.H, lo);
  size_t at = 0;
  int rounded = 0;
  const int32_t* sp = nullptr;
  uint32_t* ip = nullptr;
  const uint32_t* lut = nullptr;
  RowIndex index;
  uint32_t z = 0;
  auto enter = [&]() {
    const int hk = w.u / a.G;
    at = static_cast<size_t>(hk) * a.R + w.b * a.G + (w.u - hk * a.G);
    const HeadParamsDev hp = hp_s[a.per_head ? w.u : 0];
    index.set(hp, unbias(__ldcg(a.row_max + at)));
    lut = lut_s + 32 * hp.lut;
    const size_t row = (static_cast<size_t>(w.b) * a.H + w.u) * a.ld_s + 4 * lane;
    sp = a.scores + row;
    ip = a.index + row / 4;
    rounded = (own_rows(a, w.b) + 31) & ~31;  // every score of a started 32-key block is set
    z = 0;
  };
  auto leave = [&]() {
    z = __reduce_add_sync(0xffffffffu, z);
    if (lane == 0) atomicAdd(a.row_z + at, static_cast<int32_t>(z));
  };
  enter();
  for (int i = 0; i < n; ++i) {
    if (128 * w.blk + 4 * lane < rounded) {
      const int4 s = __ldcg(reinterpret_cast<const int4*>(sp + 128 * w.blk));
      const uint32_t i0 = index(s.x), i1 = index(s.y), i2 = index(s.z), i3 = index(s.w);
      z += (lut[i0] + lut[i1]) + (lut[i2] + lut[i3]);
      ip[32 * w.blk] = prefill::pack4(i0, i1, i2, i3);
    }
    if (i + 1 < n && w.blk + 1 == w.nb) {
      leave();
      w.next(a, 128, a.H);
      enter();
    } else if (i + 1 < n) {
      w.next(a, 128, a.H);
    }
  }
  leave();
}

// ---- phase C of the own rows: P.V, 32 keys and 64 channels per block ----
// Units (hk, group of eight query heads, half of the channels).  A = V^T: the
// thread (n8, t) reads eight channels (8 n8 ..) of the eight keys key_of(t, i);
// four keys of a channel make a fragment word.  B = P: query row n8, the
// same keys.
template <int D, bool kVSigned>
__device__ __forceinline__ bool own_pv(const SharedArgs& a, OwnRing& ring, const HeadParamsDev* hp_s,
                                       const uint32_t* lut_s, int warp, int warps) {
  constexpr int kHalves = D / 64;
  const int lane = threadIdx.x & 31, n8 = lane >> 2, t = lane & 3;
  const int groups = (a.G + 7) / 8, units = a.Hkv * groups * kHalves;
  const long long total = own_blocks(a, 32, units);
  const long long lo = total * warp / warps, hi = total * (warp + 1) / warps;
  const int n = static_cast<int>(hi - lo);
  if (n == 0) return true;
  Walk ld, w;
  w.seek(a, 32, units, lo);
  ld = w;
  auto issue = [&]() {
    ring.issue(&a.tm_vc, 64 * (ld.u % kHalves), 32 * ld.blk, ld.b * a.Hkv + ld.u / (groups * kHalves));
  };
  issue();
  if (n > 1) {
    ld.next(a, 32, units);
    issue();
  }
  size_t at = 0;
  int rows = 0, dh = 0;
  const uint32_t* ip = nullptr;
  const uint32_t* lut = nullptr;
  uint32_t R = 0;  // < 2^25: Z is at least 2^15
  int32_t psum = 0;
  int32_t o[4][4];
  uint32_t ix[2][2];  // indices of this block and the next
  auto enter = [&]() {
    dh = w.u % kHalves;
    const int u = w.u / kHalves, hk = u / groups, g0 = 8 * (u - hk * groups);
    rows = min(8, a.G - g0);
    at = static_cast<size_t>(hk) * a.R + w.b * a.G + g0;
    const int h = hk * a.G + g0 + min(n8, rows - 1);
    ip = a.index + (static_cast<size_t>(w.b) * a.H + h) * (a.ld_s / 4) + t;
    R = static_cast<uint32_t>(exact_R(__ldcg(a.row_z + at + min(n8, rows - 1))));
    lut = lut_s + 32 * hp_s[a.per_head ? h : 0].lut;
    psum = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[c][i] = 0;
  };
  auto load_index = [&](uint32_t (&x)[2], int blk) {
    x[0] = __ldcg(ip + 8 * blk);
    x[1] = __ldcg(ip + 8 * blk + 4);
  };
  auto leave = [&]() {
    if (a.v_u8 && dh == 0) {
      psum += __shfl_xor_sync(0xffffffffu, psum, 1);
      psum += __shfl_xor_sync(0xffffffffu, psum, 2);
      if (t == 0 && n8 < rows) atomicAdd(a.row_p + at + n8, psum);
    }
    // o[c][0..1]: channel 8 n8 + 2c, rows 2t, 2t + 1; o[c][2..3]: channel 8 n8 + 2c + 1
#pragma unroll
    for (int r = 0; r < 2; ++r)
      if (2 * t + r < rows) {
        float* dst = a.acc + (at + 2 * t + r) * D + 64 * dh + 8 * n8;
        red_add4(dst, static_cast<float>(o[0][r]), static_cast<float>(o[0][2 + r]), static_cast<float>(o[1][r]),
                 static_cast<float>(o[1][2 + r]));
        red_add4(dst + 4, static_cast<float>(o[2][r]), static_cast<float>(o[2][2 + r]), static_cast<float>(o[3][r]),
                 static_cast<float>(o[3][2 + r]));
      }
  };
  enter();
  load_index(ix[0], w.blk);
  for (int i = 0; i < n; ++i) {
    const bool last = i + 1 == n;
    const bool moves = !last && w.blk + 1 == w.nb;  // the next block is another unit's
    if (!last && !moves) load_index(ix[1], w.blk + 1);
    // P of this block (0 for rows the unit does not have)
    uint32_t p[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      uint32_t b[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        b[e] = static_cast<uint32_t>(
            (static_cast<unsigned long long>(lut[(ix[0][g] >> (8 * e)) & 255u]) * R + (1ull << 31)) >> 32);
      p[g] = n8 < rows ? prefill::pack4(b[0], b[1], b[2], b[3]) : 0u;
      psum = static_cast<int32_t>(__dp4a(p[g], 0x01010101u, static_cast<uint32_t>(psum)));
    }
    if (!last && !moves) w.next(a, 32, units);
    ix[0][0] = ix[1][0];
    ix[0][1] = ix[1][1];
    const uint32_t tile = ring.wait(kRoleSoftmax);
    if (tile == 0) return false;
    uint2 v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int row = key_of(t, e);  // the TMA's 64-byte swizzle on the 16-byte piece
      v[e] = lds_u64(tile + row * 64 + 16 * ((n8 >> 1) ^ ((row >> 1) & 3)) + 8 * (n8 & 1));
    }
    __syncwarp();
    if (i + 2 < n) {
      ld.next(a, 32, units);
      issue();
    }
    // bytes (key, channel c) -> word c holds four keys of channel c
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t x[2][4];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const uint32_t r0 = half ? v[4 * g].y : v[4 * g].x, r1 = half ? v[4 * g + 1].y : v[4 * g + 1].x;
        const uint32_t r2 = half ? v[4 * g + 2].y : v[4 * g + 2].x, r3 = half ? v[4 * g + 3].y : v[4 * g + 3].x;
        const uint32_t ab_lo = __byte_perm(r0, r1, 0x5140), ab_hi = __byte_perm(r0, r1, 0x7362);
        const uint32_t cd_lo = __byte_perm(r2, r3, 0x5140), cd_hi = __byte_perm(r2, r3, 0x7362);
        x[g][0] = __byte_perm(ab_lo, cd_lo, 0x5410);
        x[g][1] = __byte_perm(ab_lo, cd_lo, 0x7632);
        x[g][2] = __byte_perm(ab_hi, cd_hi, 0x5410);
        x[g][3] = __byte_perm(ab_hi, cd_hi, 0x7632);
      }
      mma16832<kVSigned, false>(o[2 * half], x[0][0], x[0][1], x[1][0], x[1][1], p[0], p[1]);
      mma16832<kVSigned, false>(o[2 * half + 1], x[0][2], x[0][3], x[1][2], x[1][3], p[0], p[1]);
    }
    if (moves) {
      leave();
      w.next(a, 32, units);
      enter();
      load_index(ix[0], w.blk);
    }
  }
  leave();
  return true;
}

// Requantised outputs of all rows, four channels per thread.
template <int D>
__device__ __forceinline__ void finish(const SharedArgs& a, const HeadParamsDev* hp_s, int thread, int threads) {
  const long long n = static_cast<long long>(a.Hkv) * a.R * (D / 4);
  for (long long i = thread; i < n; i += threads) {
    const int row = static_cast<int>(i / (D / 4)), c = 4 * static_cast<int>(i % (D / 4));
    const int hk = row / a.R, r = row - hk * a.R, b = r / a.G, h = hk * a.G + (r - b * a.G);
    if (a.lengths != nullptr) {
      const int len = __ldg(a.lengths + b);
      if (len < 0 || len > a.Lmax) continue;
    }
    const float4 v = __ldcg(reinterpret_cast<const float4*>(a.acc + static_cast<size_t>(row) * D + c));
    const HeadParamsDev hp = hp_s[a.per_head ? h : 0];
    const int32_t fix = hp.zv != 0 ? hp.zv * __ldcg(a.row_p + row) : 0;  // sum P (v - z_v)
    const float f[4] = {v.x, v.y, v.z, v.w};
    int32_t y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      y[k] = static_cast<int8_t>(prefill::requant_byte(static_cast<int32_t>(f[k]) - fix, hp.Mo, hp.so));
    const size_t at = (static_cast<size_t>(b) * a.H + h) * D + c;
    if (a.out_kind == INTATTN_DTYPE_INT8) {
      *reinterpret_cast<uint32_t*>(static_cast<int8_t*>(a.out) + at) = prefill::pack4(
          static_cast<uint32_t>(y[0]) & 255u, static_cast<uint32_t>(y[1]) & 255u, static_cast<uint32_t>(y[2]) & 255u,
          static_cast<uint32_t>(y[3]) & 255u);
    } else {
      const float s = a.s_o[a.per_head ? h : 0];
      const bool bf16 = a.out_kind == INTATTN_DTYPE_BF16;
      float o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = __fmul_rn(s, static_cast<float>(y[k]));
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
          make_uint2(rows::pack_half2(o[0], o[1], bf16), rows::pack_half2(o[2], o[3], bf16));
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) shared_kernel(const __grid_constant__ SharedArgs args) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t s_base = smem_u32(smem);
  const uint32_t sKV = s_base + C::kOffKV;
  uint32_t* tab = reinterpret_cast<uint32_t*>(smem + C::kOffTab);
  uint32_t* lut_s = reinterpret_cast<uint32_t*>(smem + C::kOffLut);
  HeadParamsDev* hp_s = reinterpret_cast<HeadParamsDev*>(smem + C::kOffHp);
  const uint32_t bars = s_base + C::kOffBars;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile uint32_t* verdict = reinterpret_cast<volatile uint32_t*>(smem + C::kOffMisc + 4);
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
  auto bar_kv_full = [&](int i) { return bar(kBarKvFull + i); };
  auto bar_kv_empty = [&](int i) { return bar(kBarKvFull + C::kStages + i); };
  auto sQ = [&](uint32_t i) { return s_base + C::kOffQ + i * C::kQBytes; };

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  // this CTA's tiles
  const int t0 = static_cast<int>(static_cast<long long>(args.tiles) * blockIdx.x / gridDim.x);
  const int t1 = static_cast<int>(static_cast<long long>(args.tiles) * (blockIdx.x + 1) / gridDim.x);

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarQFull + i), 2);
      mbar_init(bar(kBarQEmpty + i), 1);
      mbar_init(bar(kBarSFull + i), 1);
      mbar_init(bar(kBarSEmpty + i), kTeamWarps);
    }
    for (int i = 0; i < kPBufs; ++i) {
      mbar_init(bar(kBarPFull + i), kTeamWarps);
      mbar_init(bar(kBarPEmpty + i), 1);
    }
    mbar_init(bar(kBarOFull), 1);
    mbar_init(bar(kBarOEmpty), kEpiWarps);
    mbar_init(bar(kBarDrain), 1);
    for (int i = 0; i < 2 * kSoftWarps; ++i) mbar_init(bar(kBarOwn + i), 1);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(bar_kv_full(i), 1);
      mbar_init(bar_kv_empty(i), 1);
    }
    mbar_fence_init();
  }
  for (int i = tid; i < args.n_luts * 32; i += blockDim.x) lut_s[i] = args.lut[i >> 5][i & 31];
  for (int i = tid; i < (args.per_head ? args.H : 1); i += blockDim.x) hp_s[i] = args.hp[i];
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < kSoftWarps) {
    // ======================= softmax warps =======================
    const int sw = warp;
    const int quad = warp & 3;
    const int half = (sw >> 2) & 1;
    const int team = sw / kTeamWarps;
    const int grp = team * 2 + half;
    const int r = quad * 32 + lane;  // row of the tile == TMEM lane
    const uint32_t tlane = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t trow = tlane + half * kCols;
    const uint32_t prow = smem_u32(tab) + 4u * r;
    const int ow = sw * gridDim.x + blockIdx.x, ows = kSoftWarps * gridDim.x;  // share of the own rows
    OwnRing ring{s_base + C::kOffTab + 4096u * sw, bar(kBarOwn + 2 * sw), 0u, 0u};
    if (args.lengths != nullptr && blockIdx.x == 0 && sw == 0)
      for (int b = lane; b < args.B; b += 32) {
        const int n = __ldg(args.lengths + b);
        if (n < 0 || n > args.Lmax) atomicOr(&g_device_error, kErrParamRange);
      }
    bool ok = true;
    uint32_t sc = 0;  // S tiles so far
    uint32_t pc = 0;  // P tiles so far
    auto soft_sync = [&](bool mine) { return bar_red_and(kNbSoft, 32 * kSoftWarps, mine); };
    auto arrive_warp = [&](uint32_t b) {
      __syncwarp();
      if (lane == 0) mbar_arrive(b);
    };
    // grid-wide barrier k; `both`: the epilogue warps arrive at its first step too
    auto grid_sync = [&](int k, bool both) {
      __threadfence();
      const bool v = both ? bar_red_and(kNbBoth, 32 * (kSoftWarps + kEpiWarps), ok) : soft_sync(ok);
      if (tid == 0) {
        uint32_t good = 0;
        if (v) {
          __threadfence();
          atomicAdd(args.ctr + k, 1u);
          good = quant::wait_count(args.ctr + k, gridDim.x) ? 1u : 0u;
          __threadfence();
        }
        *verdict = good;
      }
      soft_sync(true);
      ok = *verdict != 0u;
      soft_sync(true);  // the verdict may now be written again
    };
    auto walk_s = [&](uint32_t idx, auto&& body) {
      const uint32_t buf = idx & 1;
      if (!mbar_wait_warp(bar(kBarSFull + buf), (idx >> 1) & 1, kRoleSoftmax)) return false;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < kCols / 32; ++c) {
        uint32_t v[32];
        tmem_ld32(trow + kColS + buf * kBN + 32 * c, v);
        tmem_wait_ld();
        if (c == kCols / 32 - 1) {
          tc_fence_before();
          arrive_warp(bar(kBarSEmpty + buf));
        }
        body(v, c);
      }
      return true;
    };
    auto first_j = [&](uint32_t s0) { return static_cast<int>((static_cast<uint32_t>(team) - s0) & 1u); };
    // keys of this thread's half of tile j that exist: a prefix
    auto nvalid = [&](int j) { return min(max(args.Lp - (j * kBN + half * kCols), 0), kCols); };

    quant::griddep_wait();  // the counters and row maxima are zeroed

    // ---- phase A ----
    if (args.Lmax > 0)
      ok = args.k_u8 ? own_scores<D, false>(args, ring, ow, ows) : own_scores<D, true>(args, ring, ow, ows);
    for (int t = t0; t < t1 && ok;) {
      const Segment sg = segment_at(args, t, t1);
      int32_t m = INT_MIN;
      for (int j = first_j(sc); j < sg.n; j += kTeams) {
        int32_t m4[4] = {INT_MIN, INT_MIN, INT_MIN, INT_MIN};
        const int nv = nvalid(sg.j0 + j);
        const bool got = walk_s(sc + j, [&](const uint32_t (&v)[32], int c) {
          if (nv == kCols) {
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
              m4[0] = __vimax3_s32(m4[0], static_cast<int32_t>(v[k + 0]), static_cast<int32_t>(v[k + 1]));
              m4[1] = __vimax3_s32(m4[1], static_cast<int32_t>(v[k + 2]), static_cast<int32_t>(v[k + 3]));
              m4[2] = __vimax3_s32(m4[2], static_cast<int32_t>(v[k + 4]), static_cast<int32_t>(v[k + 5]));
              m4[3] = __vimax3_s32(m4[3], static_cast<int32_t>(v[k + 6]), static_cast<int32_t>(v[k + 7]));
            }
          } else {
            const int nc = nv - 32 * c;
#pragma unroll
            for (int k = 0; k < 32; ++k) m4[k & 3] = imax(m4[k & 3], k < nc ? static_cast<int32_t>(v[k]) : INT_MIN);
          }
        });
        if (!got) { ok = false; break; }
        m = imax(m, imax(imax(m4[0], m4[1]), imax(m4[2], m4[3])));
      }
      sc += sg.n;
      const int row = sg.rt * kBM + r;
      if (row < args.R && m != INT_MIN) atomicMax(args.row_max + static_cast<size_t>(sg.hk) * args.R + row, bias(m));
      t += sg.n;
    }
    grid_sync(0, true);

    // index code of a score (see the prefill kernel): the bits of
    // 0x4B000000 + k, k = idx + 1 (idx <= 30) or 32 (clipped); 0 for a masked key
    uint32_t Cx = 0;
    float Ms32 = 0.f, c1 = 0.f;
    const uint32_t* lut_h = lut_s;
    auto row_index = [&](const Segment& sg) {
      const int row = min(sg.rt * kBM + r, args.R - 1);  // rows past R repeat the last one and are dropped
      const int h = sg.hk * args.G + row % args.G;
      const HeadParamsDev hp = hp_s[args.per_head ? h : 0];
      lut_h = lut_s + 32 * hp.lut;
      Cx = 0x4B000000u + static_cast<uint32_t>(unbias(__ldcg(args.row_max + static_cast<size_t>(sg.hk) * args.R + row)));
      const float Mf = __int2float_rn(hp.M);
      Ms32 = Mf * __uint_as_float(static_cast<uint32_t>(127 - 5 - hp.s) << 23);
      c1 = (1.5f - Mf * __uint_as_float(static_cast<uint32_t>(127 + 23 - hp.s) << 23)) * 0.03125f;
      return static_cast<size_t>(sg.hk) * args.R + row;
    };
    auto idx_bits = [&](uint32_t sv) {
      const float y = fma_rz_sat(__uint_as_float(Cx - sv), Ms32, c1);
      return __float_as_uint(__fmaf_rz(y, 32.0f, 8388608.0f));
    };
    auto idx_bits2 = [&](uint32_t s0, uint32_t s1, uint32_t& b0, uint32_t& b1) {
      const float y0 = fma_rz_sat(__uint_as_float(Cx - s0), Ms32, c1);
      const float y1 = fma_rz_sat(__uint_as_float(Cx - s1), Ms32, c1);
      float k0, k1;
      fma2_rz(y0, y1, pack2(32.0f), pack2(8388608.0f), k0, k1);
      b0 = __float_as_uint(k0);
      b1 = __float_as_uint(k1);
    };
    constexpr uint32_t kMaskedBits = 0x4B000000u;

    // ---- phase B ----
    if (ok) {
      if (sw < 4) tab[r] = 0u;  // row 0: masked keys
      if (args.Lmax > 0) own_sums(args, hp_s, lut_s, ow, ows);
      for (int t = t0; t < t1;) {
        const Segment sg = segment_at(args, t, t1);
        const size_t at = row_index(sg);
#pragma unroll
        for (int i = grp * 8; i < grp * 8 + 8; ++i) tab[(i + 1) * kBM + r] = lut_h[i];
        if (!soft_sync(ok)) { ok = false; break; }
        int32_t Z = 0;
        for (int j = first_j(sc); j < sg.n; j += kTeams) {
          const int nv = nvalid(sg.j0 + j);
          int32_t z4[4] = {0, 0, 0, 0};
          const bool got = walk_s(sc + j, [&](const uint32_t (&v)[32], int c) {
            if (nv == kCols) {
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                uint32_t b0, b1;
                idx_bits2(v[k], v[k + 1], b0, b1);
                z4[k & 3] += static_cast<int32_t>(lds_u32(b0 * 512u + prow));
                z4[(k + 1) & 3] += static_cast<int32_t>(lds_u32(b1 * 512u + prow));
              }
            } else {
              const int nc = nv - 32 * c;
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                const uint32_t ib = k < nc ? idx_bits(v[k]) : kMaskedBits;
                z4[k & 3] += static_cast<int32_t>(lds_u32(ib * 512u + prow));
              }
            }
          });
          if (!got) { ok = false; break; }
          Z += (z4[0] + z4[1]) + (z4[2] + z4[3]);
        }
        sc += sg.n;
        if (sg.rt * kBM + r < args.R && Z != 0) atomicAdd(args.row_z + at, Z);
        t += sg.n;
        if (!soft_sync(ok)) { ok = false; break; }  // the table may be written again
      }
      grid_sync(1, false);
    }

    // ---- phase C ----
    if (ok) {
      if (args.Lmax > 0) {
        fence_proxy_async_smem();  // the tables' last accesses, before the ring's tiles land there
        ok = args.v_u8 ? own_pv<D, false>(args, ring, hp_s, lut_s, ow, ows)
                       : own_pv<D, true>(args, ring, hp_s, lut_s, ow, ows);
        ok = soft_sync(ok);  // every ring is done with the tables' memory
      }
      if (sw < 4)
        for (int b = 0; b < 4; ++b) tab[b * (C::kTabBytes / 4) + r] = 0u;
      for (int t = t0; t < t1 && ok;) {
        const Segment sg = segment_at(args, t, t1);
        const size_t at = row_index(sg);
        const unsigned long long R = exact_R(__ldcg(args.row_z + at));
#pragma unroll
        for (int i = grp * 8; i < grp * 8 + 8; ++i) {
          const uint32_t P = static_cast<uint32_t>((static_cast<unsigned long long>(lut_h[i]) * R + (1ull << 31)) >> 32);
#pragma unroll
          for (int b = 0; b < 4; ++b) tab[b * (C::kTabBytes / 4) + (i + 1) * kBM + r] = P << (8 * b);
        }
        if (!soft_sync(ok)) { ok = false; break; }
        uint32_t psum = 0;
        for (int j = first_j(sc); j < sg.n; j += kTeams) {
          const uint32_t pi = pc + j;
          const uint32_t pb = pi & (kPBufs - 1);
          if (!mbar_wait_warp(bar(kBarPEmpty + pb), ((pi / kPBufs) & 1) ^ 1, kRoleSoftmax)) { ok = false; break; }
          const int nv = nvalid(sg.j0 + j);
          const bool got = walk_s(sc + j, [&](const uint32_t (&v)[32], int c) {
            uint32_t pw[8];
            if (nv == kCols) {
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                uint32_t kb[4], p[4];
                idx_bits2(v[q * 4], v[q * 4 + 1], kb[0], kb[1]);
                idx_bits2(v[q * 4 + 2], v[q * 4 + 3], kb[2], kb[3]);
#pragma unroll
                for (int b = 0; b < 4; ++b) p[b] = lds_u32(kb[b] * 512u + prow + b * C::kTabBytes);
                pw[q] = (p[0] + p[1]) + (p[2] + p[3]);
              }
            } else {
              const int nc = nv - 32 * c;
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                uint32_t p[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                  const int k = q * 4 + b;
                  const uint32_t ib = k < nc ? idx_bits(v[k]) : kMaskedBits;
                  p[b] = lds_u32(ib * 512u + prow + b * C::kTabBytes);
                }
                pw[q] = (p[0] + p[1]) + (p[2] + p[3]);
              }
            }
            if (args.v_u8) {
#pragma unroll
              for (int q = 0; q < 8; ++q) psum = __dp4a(pw[q], 0x01010101u, psum);
            }
            tmem_st8(tlane + kColP + pb * 32 + half * (kCols / 4) + c * 8, pw);
          });
          if (!got) { ok = false; break; }
          tmem_wait_st();
          tc_fence_before();
          arrive_warp(bar(kBarPFull + pb));
        }
        sc += sg.n;
        pc += sg.n;
        if (psum != 0 && sg.rt * kBM + r < args.R) atomicAdd(args.row_p + at, static_cast<int32_t>(psum));
        t += sg.n;
        if (!soft_sync(ok)) { ok = false; break; }
      }
    }
    grid_sync(2, true);
    if (ok)
      finish<D>(args, hp_s, blockIdx.x * 32 * kSoftWarps + tid, gridDim.x * 32 * kSoftWarps);
  } else if (warp >= kEpiWarp0) {
    // ============================ epilogue ============================
    // phase A: zero what the later phases add to
    {
      const size_t rows = static_cast<size_t>(args.Hkv) * args.R;
      const size_t n = 2 * rows + rows * D;  // row_z, row_p and acc are consecutive words
      for (size_t i = static_cast<size_t>(blockIdx.x) * (32 * kEpiWarps) + (tid - 32 * kEpiWarp0); i < n;
           i += static_cast<size_t>(gridDim.x) * (32 * kEpiWarps))
        args.row_z[i] = 0;
    }
    __threadfence();
    const bool go = bar_red_and(kNbBoth, 32 * (kSoftWarps + kEpiWarps), true);
    // phase C: O (int32, TMEM) of each segment -> acc
    const int quad = warp & 3;
    const int r = quad * 32 + lane;
    const uint32_t tlane = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    bool ok = go;
    int n = 0;
    for (int t = t0; t < t1 && ok; ++n) {
      const Segment sg = segment_at(args, t, t1);
      if (!mbar_wait_warp(bar(kBarOFull), n & 1, kRoleEpilogue)) { ok = false; break; }
      tc_fence_after();
      const int row = sg.rt * kBM + r;
      float* dst = args.acc + (static_cast<size_t>(sg.hk) * args.R + row) * D;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        uint32_t v[16];
        tmem_ld16(tlane + kColO + 16 * c, v);
        tmem_wait_ld();
        if (c == D / 16 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarOEmpty));
        }
        if (row < args.R) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            red_add4(dst + 16 * c + 4 * q, __int2float_rn(static_cast<int32_t>(v[4 * q])),
                     __int2float_rn(static_cast<int32_t>(v[4 * q + 1])), __int2float_rn(static_cast<int32_t>(v[4 * q + 2])),
                     __int2float_rn(static_cast<int32_t>(v[4 * q + 3])));
        }
      }
      t += sg.n;
    }
    __threadfence();
    bar_red_and(kNbBoth, 32 * (kSoftWarps + kEpiWarps), ok);
  } else if (warp == kProducerWarp) {
    // ============================ TMA producer ============================
    // lane s owns ring slot s (see the prefill kernel)
    if (lane == 0 && t0 < t1) {
      tma_prefetch_desc(&args.tm_k);
      tma_prefetch_desc(&args.tm_v);
    }
    __syncwarp();
    if (lane < C::kStages) {
      const uint32_t slot = static_cast<uint32_t>(lane);
      const uint32_t dst = sKV + slot * C::kTileBytes;
      uint32_t n = 0, mine = 0;
      bool ok = true;
      auto load = [&](const CUtensorMap* tm, int j, int hk) {
        if (ok && n % C::kStages == slot) {
          if (!mbar_wait(bar_kv_empty(slot), (mine & 1) ^ 1, kRoleProducer)) {
            ok = false;
          } else {
            mbar_arrive_expect_tx(bar_kv_full(slot), C::kTileBytes);
            tma_load_3d(dst, tm, bar_kv_full(slot), 0, j * kBN, hk);
            ++mine;
          }
        }
        ++n;
      };
      for (int phase = 0; phase < 2; ++phase)
        for (int t = t0; t < t1 && ok;) {
          const Segment sg = segment_at(args, t, t1);
          for (int j = 0; j < sg.n; ++j) load(&args.tm_k, sg.j0 + j, sg.hk);
          t += sg.n;
        }
      for (int t = t0; t < t1 && ok;) {
        const Segment sg = segment_at(args, t, t1);
        load(&args.tm_k, sg.j0, sg.hk);
        if (sg.n > 1) load(&args.tm_k, sg.j0 + 1, sg.hk);
        for (int j = 0; j < sg.n; ++j) {
          if (j + 2 < sg.n) load(&args.tm_k, sg.j0 + j + 2, sg.hk);
          load(&args.tm_v, sg.j0 + j, sg.hk);
        }
        t += sg.n;
      }
      if (mine > 0) mbar_wait(bar_kv_full(slot), (mine - 1) & 1, kRoleProducer);  // no copy left in flight
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ============================= MMA issuer =============================
    const uint32_t idesc_qk = idesc_i8(kBM, kBN, 1, args.k_u8 ? 0u : 1u, 0);
    const uint32_t idesc_pv = idesc_i8(kBM, D, 0, args.v_u8 ? 0u : 1u, 1);
    const uint64_t kv_desc0 = smem_desc(sKV, 16, C::kSBO, C::kSwizzle);
    constexpr uint32_t kSlotDesc = C::kTileBytes >> 4;
    bool ok = true;
    uint32_t slot = 0, kv_par = 0, sc = 0, pc = 0, nq = 0, no = 0;
    auto next_slot = [&]() {
      if (++slot == static_cast<uint32_t>(C::kStages)) {
        slot = 0;
        kv_par ^= 1;
      }
    };
    for (int phase = 0; phase < 3 && ok; ++phase) {
      for (int t = t0; t < t1 && ok; ++nq) {
        const Segment sg = segment_at(args, t, t1);
        const uint32_t qb = nq & 1;
        if (!mbar_wait_warp(bar(kBarQFull + qb), (nq >> 1) & 1, kRoleMma)) { ok = false; break; }
        const uint64_t q_desc = smem_desc(sQ(qb), 16, C::kSBO, C::kSwizzle);
        auto issue_qk = [&]() {
          if (!ok) return;
          const uint32_t buf = sc & 1;
          if (!mbar_wait2_warp(bar(kBarSEmpty + buf), ((sc >> 1) & 1) ^ 1, bar_kv_full(slot), kv_par, kRoleMma)) {
            ok = false;
            return;
          }
          tc_fence_after();
          const uint64_t k_desc = kv_desc0 + slot * kSlotDesc;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
              mma_i8_ss(tmem + kColS + buf * kBN, q_desc + 2 * kk, k_desc + 2 * kk, idesc_qk, kk > 0);
            mma_commit(bar_kv_empty(slot));
            mma_commit(bar(kBarSFull + buf));
          }
          __syncwarp();
          next_slot();
          ++sc;
        };
        if (phase < 2) {
          for (int j = 0; j < sg.n; ++j) issue_qk();
        } else {
          issue_qk();
          if (sg.n > 1) issue_qk();
          for (int j = 0; ok && j < sg.n; ++j, ++pc) {
            if (j + 2 < sg.n) issue_qk();
            if (!ok) break;
            if (j == 0 && !mbar_wait_warp(bar(kBarOEmpty), (no & 1) ^ 1, kRoleMma)) { ok = false; break; }
            const uint32_t pb = pc & (kPBufs - 1);
            if (!mbar_wait2_warp(bar(kBarPFull + pb), (pc / kPBufs) & 1, bar_kv_full(slot), kv_par, kRoleMma)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t v_desc = kv_desc0 + slot * kSlotDesc;
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kBN / 32; ++kk)
                mma_i8_ts(tmem + kColO, tmem + kColP + pb * 32 + kk * 8, v_desc + ((32u * D * kk) >> 4), idesc_pv,
                          (j > 0 || kk > 0) ? 1u : 0u);
              mma_commit(bar_kv_empty(slot));
              mma_commit(bar(kBarPEmpty + pb));
            }
            __syncwarp();
            next_slot();
          }
          if (!ok) break;
          mma_commit_elect(bar(kBarOFull));
          ++no;
        }
        if (!ok) break;
        mma_commit_elect(bar(kBarQEmpty + qb));
        t += sg.n;
      }
    }
    mma_commit_elect(bar(kBarDrain));
    mbar_wait_warp(bar(kBarDrain), 0, kRoleMma);
  } else {
    // ============================== Q rows ==============================
    // two warps, a half of the tile each, eight loads in flight per lane
    uint32_t nq = 0;
    bool ok = true;
    for (int phase = 0; phase < 3 && ok; ++phase)
      for (int t = t0; t < t1; ++nq) {
        const Segment sg = segment_at(args, t, t1);
        const uint32_t qb = nq & 1;
        if (!mbar_wait_warp(bar(kBarQEmpty + qb), ((nq >> 1) & 1) ^ 1, kRoleQ)) { ok = false; break; }
        constexpr int kPieces = D / 16;
        constexpr int kBatch = 8;
        for (int i0 = (warp - kQWarp) * kBM / 2 * kPieces; i0 < (warp - kQWarp + 1) * kBM / 2 * kPieces; i0 += 32 * kBatch) {
          uint4 v[kBatch];
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const int i = i0 + 32 * k + lane;
            const int row = sg.rt * kBM + i / kPieces;
            v[k] = make_uint4(0, 0, 0, 0);
            if (row < args.R) {
              const int b = row / args.G, g = row - b * args.G;
              v[k] = __ldg(reinterpret_cast<const uint4*>(
                  args.q + (static_cast<size_t>(b) * args.H + sg.hk * args.G + g) * D + 16 * (i % kPieces)));
            }
          }
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const int i = i0 + 32 * k + lane;
            const int rr = i / kPieces, c = i % kPieces;
            // the TMA's swizzle: 16-byte piece c of row rr
            const int piece = D == 128 ? (c ^ (rr & 7)) : (c ^ ((rr >> 1) & 3));
            *reinterpret_cast<uint4*>(smem + C::kOffQ + qb * C::kQBytes + rr * D + 16 * piece) = v[k];
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarQFull + qb));
        t += sg.n;
      }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Barrier counters and row maxima to 0 (below every score).
__global__ void shared_zero_kernel(uint32_t* p, int n) {
  quant::griddep_trigger();  // shared_kernel waits for completion before it uses them
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) p[i] = 0u;
}

}  // namespace shared
}  // namespace intattn
