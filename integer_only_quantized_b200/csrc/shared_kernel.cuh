// Decode for a batch whose sequences share a prefix: one query per (b, h)
// against the prefix rows of its K / V head followed by the rows of its own
// cache, by the definition of intattn.h over the joined keys.
//
// The definition needs the row max before any table index and the row sum
// before any probability, over the joined keys, so the work is three phases
// with a grid-wide barrier after each, in one cooperative launch of at most
// one CTA per SM:
//   A  scores -> row max            (global atomic max)
//   B  scores -> Z = sum of LUT     (global atomic add)
//   C  scores -> u8 P, P.V          (global adds); after the barrier, requantisation
// Integer sums do not depend on their order, so the bytes do not depend on
// the split.  acc is added up in fp32: every partial sum is a whole number
// below 2^24 (sum of P <= 510 times 255), so those sums are exact too, and one
// instruction adds four channels.
//
// In every phase two groups of warps work side by side, one on the prefix
// (bound by the tensor pipe and the index arithmetic), one on the own rows (bound
// by HBM), so that neither resource waits for the other's phase.
//
// Prefix.  The R = B G queries that share a K / V head are the rows of a
// 128-row tile, so the prefix streams once per 128 queries and the products
// run on the tensor cores: tcgen05.mma kind::i8 for S = Q.K^T and O += P.V as
// in the prefill kernel (whose warp roles, barriers and index arithmetic this
// follows), scores recomputed in each phase (K comes from L2 after phase A).
// Few queries fold: with R <= 64 (32) a tile holds F = 2 (4) key tiles, each
// against the same queries in its own 128 / F lanes.  Its S is the sum of F
// products whose Q operand is a window into zero-padded rows that puts the
// queries into lanes f 128 / F .. only; O adds up over F P buffers whose other
// lanes stay zero.  The tensor work per key tile is unchanged and the softmax
// work, which the padding lanes would double (quadruple), is not.
// The (head, row tile, key tile) triples are cut into equal consecutive
// ranges, one per CTA; the part of a range within one (head, row tile) is a
// segment.
//
// Own rows.  They are read by one sequence only: an HBM stream with up to
// eight query rows per K / V row.  Each of the own warps takes an equal
// consecutive share of all blocks of own rows (4 KB each) and streams it through
// a ring of its own TMA tiles: 64 KB in flight per SM, no registers held by loads, no
// barrier shared by warps.  The products are m16n8k32 integer MMAs, keys or channels on
// the 16 side and the grouped heads on the 8 side.  Scores
// (4 bytes per key and head), and from phase B on their table indices (one
// byte), wait in the workspace; a warp reads back what it wrote itself.
//
// Measured, per call in a CUDA graph over several sets of inputs (zero kernel and this
// one; own lengths uniform up to the number given), beside the time of a copy of the bytes:
//   B4 H12/12 d64, 500 shared, 64 own            17.8 us   (launches and three
//                                                phases of one tile each)
//   B64 H32/8 d128, 8192 shared, 1024 own        45.6 us   12.9 us
//   B64 H32/32 d128 u8, 4001 shared, 777 own     69.0 us   36.3 us (3.4 TB/s)
//   B9 H32/8 d128, 50000 shared, 333 own         50.2 us   16.1 us
//   B64 H32/8 d128, none shared, 8192 own        156.6 us  82.2 us
//   B64 H64/8 d64, 500 shared, 8192 own          140.1 us  41.2 us
//   B64 H32/32 d128, 500 shared, 8192 own        416 us    329 us
// (The comparisons beside the rules below and in shared_api.cuh repeat a call on
// the same inputs, so the smaller cases come partly from L2: 42.5, 68.4 and 48.0 us for
// the second, third and fourth.)
// Bound: the three dependent phases (scores of the prefix are made three
// times), in each the latency of the softmax warps' loops and of fetching them: the issue
// slots are a third used, the tensor pipe 9 to 21 %, DRAM 21 to 44 %.  Long own caches: the scores and index
// bytes of every query head, 10 G bytes per key beside 2 d of K and V.  Every
// change that made a loop's code smaller made it faster, and unrolling,
// reading ahead and prefetching V into L2 during phase B made it slower.
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
  CUtensorMap tm_kc, tm_vc;   // own rows [B Hkv, Lmax, d], box {d, 4096 / d, 1}
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
  int32_t fold;                  // F: key tiles per tile of 128 lanes
  int32_t stages, own_slots;     // of the K / V ring and of each own warp's ring (see kRingBytes)
  int32_t key_tiles;             // 128-key tiles of the prefix
  int32_t row_tiles, seg_tiles;  // 128-row tiles of R; tiles per (head, row tile): ceil(key_tiles / F)
  int32_t tiles;                 // Hkv * row_tiles * seg_tiles
  int32_t seg_cost;              // of a segment, in tiles, for equal shares (see first_tile)
  int32_t cta_cost, cta_more;    // a CTA's share of the cost, and one more for the first cta_more
  int32_t none;                  // 0 (see OwnRing)
  int32_t zero_left_out;         // outputs of a sequence whose length is out of range become 0
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

constexpr int kBM = 128;                   // lanes of a tile
constexpr int kBN = 128;                   // keys per key tile
constexpr int kTeams = 2;                  // softmax teams taking alternate tiles
constexpr int kSoftWarps = 16;
constexpr int kTeamWarps = kSoftWarps / kTeams;
constexpr int kCols = 64;                  // S columns per thread and tile (two halves)
constexpr int kChunk = 16;                 // of them read from TMEM at a time (tmem_ld16, tmem_st4)
constexpr int kProducerWarp = 16;
constexpr int kMmaWarp = 17;               // issues S = Q.K^T
constexpr int kPvWarp = 18;                // issues O += P.V
constexpr int kQWarp = 19;                 // Q rows into shared memory
constexpr int kOwnWarp0 = 20;              // warps 20-27: own rows
constexpr int kOwnWarps = 8;
constexpr int kOwnBytes = 4096;            // bytes of an own-row block
// K / V tiles of the prefix and the own warps' rings share these bytes: with S
// slots per own warp (0, 1 or 2) the prefix has (kRingBytes - 32 KB S) / tile stages
constexpr int kRingBytes = 144 * 1024;
constexpr int kMaxOwnSlots = 2;
constexpr int kThreads = 32 * (kOwnWarp0 + kOwnWarps);
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;              // two S buffers
constexpr uint32_t kColO = 256;
constexpr uint32_t kColP = 384;            // four P buffers of 32 columns
constexpr int kPBufs = 4;
constexpr uint32_t kNbSoft = 1;            // named barrier of the softmax warps
constexpr uint32_t kNbBoth = 2;            // softmax and own warps

enum Role : unsigned { kRoleSoftmax = 5, kRoleProducer = 6, kRoleMma = 7, kRoleOwn = 8, kRoleQ = 9 };

enum Bar : int {
  kBarQFull = 0,    // [2]
  kBarQEmpty = 2,   // [2]
  kBarSFull = 4,    // [2]
  kBarSEmpty = 6,   // [2]
  kBarPFull = 8,    // [4]
  kBarPEmpty = 12,  // [4]
  kBarOFull = 16,
  kBarOEmpty = 17,
  kBarDrain = 18,   // [2]
  kBarOwn = 20,     // [kOwnWarps][kMaxOwnSlots]
  kBarKvFull = kBarOwn + kOwnWarps * kMaxOwnSlots,  // K [kMaxStages], V [kMaxStages], then kv_empty[kMaxStages]
};

template <int D>
struct Cfg {
  static constexpr uint32_t kTileBytes = kBN * D;
  static constexpr int kMaxStages = kRingBytes / kTileBytes;
  static constexpr uint32_t kSwizzle = (D == 128) ? 2u : 4u;  // 128B / 64B swizzle
  static constexpr uint32_t kSBO = 8 * D;
  static constexpr int kNumBars = kBarKvFull + 3 * kMaxStages;
  // Q rows: buffer i at row 128 - 128 / F + 128 i, the other rows zero (F > 1)
  static constexpr int kQRows = 352;
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffKV = kOffQ + kQRows * D;
  // per-row tables [33][kBM] u32, row k for index code k (see idx_bits2; 1 .. 32): in
  // phase B the first holds LUT, in phase C table b holds P << 8b
  static constexpr uint32_t kTabBytes = 33 * kBM * 4;
  static constexpr uint32_t kOffTab = kOffKV + kRingBytes;
  static constexpr uint32_t kOffLut = kOffTab + 2 * kTabBytes;
  static constexpr uint32_t kOffHp = kOffLut + INTATTN_MAX_CLIPS * 32 * 4;
  static constexpr uint32_t kOffBars = kOffHp + INTATTN_MAX_HEADS * sizeof(HeadParamsDev);
  static constexpr uint32_t kOffMisc = kOffBars + kNumBars * 8;  // TMEM address, barrier verdict
  static constexpr uint32_t kUsed = kOffMisc + 16;
  static_assert(kOffKV % 1024 == 0, "swizzled tiles");
  // one CTA per SM: every CTA takes all 512 TMEM columns
  // (dynamic shared memory starts on 128 bytes: at most 896 go to the alignment)
  static constexpr uint32_t kSmemBytes = (kUsed + 896 > 120 * 1024) ? kUsed + 896 : 120 * 1024;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

// Consecutive tiles of one (head, row tile).
struct Segment {
  int hk, rt, j0, n;
};
__device__ __forceinline__ Segment segment_at(const SharedArgs& a, int t, int t1) {
  Segment s;
  const int u = t / a.seg_tiles;
  s.j0 = t - u * a.seg_tiles;
  s.n = min(t1 - t, a.seg_tiles - s.j0);
  s.hk = u / a.row_tiles;
  s.rt = u - s.hk * a.row_tiles;
  return s;
}
// Where CTA i's tiles start: equal shares of a cost that counts seg_cost tiles
// more for each (head, row tile).
__device__ __forceinline__ int first_tile(const SharedArgs& a, int i) {
  if (a.tiles == 0) return 0;
  const int each = a.seg_tiles + a.seg_cost;
  const int p = a.cta_cost * i + min(i, a.cta_more);
  const int u = p / each;
  return u * a.seg_tiles + min(p - u * each, a.seg_tiles);
}
// key tiles of tile j of a segment's (head, row tile)
__device__ __forceinline__ int folds_at(const SharedArgs& a, int j) { return min(a.fold, a.key_tiles - j * a.fold); }

__device__ __forceinline__ uint32_t bias(int32_t s) { return static_cast<uint32_t>(s) ^ 0x80000000u; }
__device__ __forceinline__ int32_t unbias(uint32_t u) { return static_cast<int32_t>(u ^ 0x80000000u); }

// Four fp32 adds to consecutive addresses (16-byte aligned).
__device__ __forceinline__ void red_add4(float* p, float a, float b, float c, float d) {
  asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}

// D[16 x 8] += A[16 x 32] B[32 x 8], row x column fragments: A s8 or u8 (K), B s8 (queries).
__device__ __forceinline__ void mma16832(int32_t (&c)[4], bool a_u8, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if (a_u8)
    asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with A s8 or u8 (V), B u8 (P).
__device__ __forceinline__ void mma16832_pv(int32_t (&c)[4], bool a_u8, uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  if (a_u8)
    asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.u8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.u8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Own rows of a sequence; 0 for a length out of range (its output is skipped).
__device__ __forceinline__ int own_rows(const SharedArgs& a, int b) {
  if (a.lengths == nullptr) return a.Lmax;
  const int n = __ldg(a.lengths + b);
  return n < 0 || n > a.Lmax ? 0 : n;
}

// The blocks of `keys` own rows of every sequence and unit (K / V head, group
// of eight query heads), in the order (b, unit, block), and a warp's
// place among them.  Warp-collective.
// Blocks' worth of work in changing the unit, for equal shares.  LLaMA-7B heads, B64,
// up to 777 own keys: 68.4 us a call, with 1 71.7, with 3 67.9; B64 H64/8 d64, up to 8192:
// 142.2, with 1 141.4, with 3 144.0; B32 H12 d64, up to 500: 21.5, 20.9, 21.8.  Twelve other shapes differ by 2 %
// or less.
constexpr int kUnitCost = 2;
struct Walk {
  int b, hk, g, blk, nb;  // sequence, K / V head, group of eight query heads; nb: blocks of the sequence
  // Goes to the start of the share of warp `w` of `warps`; its cost, 0 when there is nothing in it.
  // A unit costs its blocks and kUnitCost; a block belongs to the share in which it starts.
  __device__ __forceinline__ int share(const SharedArgs& a, int keys, int w, int warps) {
    const int lane = threadIdx.x & 31;
    const int groups = (a.G + 7) / 8, units = a.Hkv * groups;
    auto blocks = [&](int i) { return i < a.B ? (own_rows(a, i) + keys - 1) / keys : 0; };
    auto cost = [&](int n) { return n > 0 ? n + kUnitCost : 0; };
    int total = 0;
    for (int i = lane; i < a.B; i += 32) total += cost(blocks(i));
    total = __reduce_add_sync(0xffffffffu, total) * units;
    const int each = total / warps, more = total - each * warps;
    int left = each + (w < more ? 1 : 0);
    int p = each * w + min(w, more);  // from sequence b0 on
    b = hk = g = blk = nb = 0;
    if (left == 0) return 0;
#pragma unroll 1
    for (int b0 = 0;; b0 += 32) {
      const int mine = blocks(b0 + lane);
      int c = cost(mine);  // summed up to and with this lane's sequence
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) c += up;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, c * units > p);  // p < total: some lane's in the end
      if (past) {
        const int l = __ffs(past) - 1;
        nb = __shfl_sync(0xffffffffu, mine, l);
        b = b0 + l;
        p -= (__shfl_sync(0xffffffffu, c, l) - cost(nb)) * units;  // within sequence b
        break;
      }
      p -= __shfl_sync(0xffffffffu, c, 31) * units;
    }
    int u = p / cost(nb);
    blk = p - u * cost(nb);
    const bool between = blk >= nb;  // the first block is the next unit's, or the next sequence's
    if (between) {
      left -= cost(nb) - blk;
      blk = nb - 1;
    }
    hk = u / groups;
    g = u - hk * groups;
    if (left <= 0) return 0;
    if (between) next(a, keys);
    return left;
  }
  // Past `run` blocks of this unit: the cost left of `left`; at the next block while there is one.
  __device__ __forceinline__ int skip(const SharedArgs& a, int keys, int left, int run) {
    blk += run - 1;
    left -= blk + 1 == nb ? run + kUnitCost : run;
    if (left > 0) next(a, keys);
    return left;
  }
  // to the next block (there is one)
  __device__ __forceinline__ void next(const SharedArgs& a, int keys) {
    if (++blk < nb) return;
    blk = 0;
    if (8 * ++g < a.G) return;
    g = 0;
    if (++hk < a.Hkv) return;
    hk = 0;
    do {
      ++b;
      nb = (own_rows(a, b) + keys - 1) / keys;
    } while (nb == 0);
  }
};

// The query rows of a unit.
struct Unit {
  int head, rows, len;  // first query head; 1 .. 8 of them; own rows of the sequence
  int at, row;          // first row in the row arrays; in [B, H]
  __device__ __forceinline__ void set(const SharedArgs& a, const Walk& w) {
    const int g0 = 8 * w.g;
    rows = min(8, a.G - g0);
    head = w.hk * a.G + g0;
    len = own_rows(a, w.b);
    at = w.hk * a.R + w.b * a.G + g0;
    row = w.b * a.H + head;
  }
};

// A warp's private ring of blocks for the own rows' tiles.  The warp that reads a
// block also starts the copy that replaces it, so the copy (async proxy) has to come after every
// lane's reads (generic proxy): each lane's proxy fence, then the warp's barrier, then
// one lane's copy.  That lane's own reads moreover reach it as a value: `issue` takes
// one made of what was read, `read` & args.none, which is 0 when it arrives.  Without
// any of this a copy did overtake reads still on their way to registers, with
// other warps keeping shared memory busy.  Fence and barrier cost little beside that value:
// LLaMA-7B heads, B64, up to 777 own keys 68.1 us a call (68.0 without them), B64 H32/8 over
// 8192 + 1024 keys 42.5 (41.7), up to 8192 own keys of H32/8 alone 142.5 (142.7).
struct OwnRing {
  uint32_t base, bar;    // shared addresses: slot i at base + kOwnBytes i, barrier i at bar + 8 i
  uint32_t slots;
  uint32_t issued, used; // tiles, both counted over the slots as 2 slots states
  __device__ __forceinline__ uint32_t step(uint32_t n) const { return n + 1 == 2 * slots ? 0u : n + 1; }
  __device__ __forceinline__ uint32_t slot(uint32_t n) const { return n < slots ? n : n - slots; }
  __device__ __forceinline__ void issue(const CUtensorMap* tm, int y, int z, uint32_t zero) {
    const uint32_t i = slot(issued);
    fence_proxy_async_smem();
    __syncwarp();
    tma_load_3d_elect(base + kOwnBytes * i + zero, tm, bar + 8 * i + zero, kOwnBytes, 0, y, z);
    issued = step(issued);
  }
  // the oldest tile not yet used (its address), or 0 when the wait ran out
  __device__ __forceinline__ uint32_t wait() {
    const uint32_t i = slot(used);
    const bool ok = mbar_wait_warp(bar + 8 * i, used >= slots ? 1u : 0u, kRoleOwn);
    used = step(used);
    return ok ? base + kOwnBytes * i : 0u;
  }
  __device__ __forceinline__ void drain() {  // leave no copy in flight
    while (used != issued) wait();
  }
};

// Four 8 x 8 matrices of 16-bit elements, that is 8 rows of 16 bytes each:
// lane 8 i + j gives the address of row j of matrix i; thread (n8, t) gets bytes
// 4 t .. 4 t + 3 of row n8.
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Two 16 x 16 matrices of bytes, transposed: lane 16 i + j gives the address
// of row j of matrix i; thread (n8, t) gets of column n8 (r[2 i]) and n8 + 8 (r[2 i + 1]) the
// rows 4 t .. 4 t + 3.
__device__ __forceinline__ void ldmatrix2_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Shared address of 16-byte piece c of row r of a swizzled tile of D-byte rows.
template <int D>
__device__ __forceinline__ uint32_t tile_at(uint32_t tile, int r, int c) {
  return tile + r * D + 16 * (D == 128 ? (c ^ (r & 7)) : (c ^ ((r >> 1) & 3)));
}

// ---- phase A of the own rows: scores and row max of the share of cost n from w ----
// A = K: sixteen keys by 32 channels per product; B: the unit's queries.  A key
// past the sequence's last (in a started 16-key step) gets the lowest score, whose table
// entry is 0.  The loop is as short as it can be: with the next step's fragments read
// ahead (more code) LLaMA-7B heads, B64, 4001 shared and up to 777 own keys took 3 %
// longer.
template <int D>
__device__ __forceinline__ bool own_scores(const SharedArgs& a, bool k_u8, OwnRing& ring, Walk w, int n) {
  constexpr int kKeys = kOwnBytes / D;
  constexpr int kSub = kKeys / 16;     // 16-key steps per block
  constexpr int kK = D / 32;           // products per step
  const int lane = threadIdx.x & 31, n8 = lane >> 2, t = lane & 3;
  Walk ld = w;
  int left = n;  // not yet issued
  auto issue = [&](uint32_t read) {
    ring.issue(&a.tm_kc, ld.blk * kKeys, ld.b * a.Hkv + ld.hk, read & a.none);
    left = ld.skip(a, kKeys, left, 1);
  };
#pragma unroll 1
  for (uint32_t i = 0; i < ring.slots; ++i)
    if (left > 0) issue(0u);
  uint32_t tile = 0;
  while (n > 0) {
    Unit x;
    x.set(a, w);
    int32_t* sp = a.scores + static_cast<size_t>(x.row + 2 * t) * a.ld_s + n8;
    uint32_t q[kK][2];
    {
      const uint32_t* qp = reinterpret_cast<const uint32_t*>(a.q + static_cast<size_t>(x.row + min(n8, x.rows - 1)) * D) + t;
#pragma unroll
      for (int c = 0; c < kK; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i) q[c][i] = __ldg(qp + 8 * c + 4 * i);  // rows past the unit's are not stored
    }
    int32_t m[2] = {INT_MIN, INT_MIN};
    const int run = min(n, w.nb - w.blk);  // blocks of this unit
    const int s0 = w.blk * kSub, s1 = (w.blk + run) * kSub;
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
      const int in = s % kSub;
      if (in == 0 && (tile = ring.wait()) == 0) return false;
      uint32_t k[kK][4];
#pragma unroll
      for (int c = 0; c < kK; ++c) ldmatrix4(k[c], tile_at<D>(tile, 16 * in + (lane & 15), 2 * c + (lane >> 4)));
      int32_t d[2][4];  // two chains of products
#pragma unroll
      for (int c = 0; c < 2; ++c) d[c][0] = d[c][1] = d[c][2] = d[c][3] = 0;
#pragma unroll
      for (int c = 0; c < kK; ++c)
        mma16832(d[c & 1], k_u8, k[c][0], k[c][1], k[c][2], k[c][3], q[c][0], q[c][1]);
      if (in == kSub - 1 && left > 0) {
        uint32_t read = 0;
#pragma unroll
        for (int c = 0; c < kK; ++c) read |= k[c][0] | k[c][1] | k[c][2] | k[c][3];
        issue(read);
      }
      // d[..][0], [1]: key n8, rows 2t and 2t + 1; [2], [3]: key n8 + 8
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int32_t v = 16 * s + 8 * e + n8 < x.len ? d[0][2 * e + r] + d[1][2 * e + r] : INT_MIN;
          if (2 * t + r < x.rows) sp[static_cast<size_t>(r) * a.ld_s + 16 * s + 8 * e] = v;
          m[r] = imax(m[r], v);
        }
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      m[0] = imax(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
      m[1] = imax(m[1], __shfl_xor_sync(0xffffffffu, m[1], o));
    }
    if (n8 < 2 && 2 * t + n8 < x.rows) atomicMax(a.row_max + x.at + 2 * t + n8, bias(n8 ? m[1] : m[0]));
    n = w.skip(a, kKeys, n, run);
  }
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

// ---- phase B of the own rows: Z and the index bytes of the same blocks ----
// Thread t of four takes four scores of a 16-key step; the eight lane groups
// take the unit's rows, and with fewer than eight rows several steps.  The next
// step's scores are on their way while this one's are worked on.  One step per turn of
// the loop: with four unrolled (more loads in flight, more code to fetch)
// LLaMA-7B heads, B64, 4001 shared and up to 777 own keys took 3 % longer.
template <int D>
__device__ __forceinline__ void own_sums(const SharedArgs& a, const HeadParamsDev* hp_s, const uint32_t* lut_s, Walk w,
                                         int n) {
  constexpr int kKeys = kOwnBytes / D;
  constexpr int kSub = kKeys / 16;
  const int lane = threadIdx.x & 31, n8 = lane >> 2, t = lane & 3;
  while (n > 0) {
    const int run = min(n, w.nb - w.blk);  // blocks of this unit
    Unit x;
    x.set(a, w);
    const int rp = x.rows > 4 ? 8 : x.rows > 2 ? 4 : x.rows;  // lane groups per step
    const int par = 8 / rp;                                   // steps side by side
    const int mine = min(n8 % rp, x.rows - 1);
    const bool live = n8 % rp < x.rows;
    const int s1 = min((w.blk + run) * kSub, (x.len + 15) / 16);  // started steps
    const size_t row = static_cast<size_t>(x.row + mine) * a.ld_s + 4 * t;
    const int4* sp = reinterpret_cast<const int4*>(a.scores + row);
    uint32_t* ip = a.index + row / 4;
    auto load = [&](int s) { return s < s1 ? sp[4 * s] : make_int4(INT_MIN, INT_MIN, INT_MIN, INT_MIN); };
    int s = w.blk * kSub + n8 / rp;
    int4 v = load(s);
    const HeadParamsDev hp = hp_s[a.per_head ? x.head + mine : 0];
    const uint32_t* lut = lut_s + 32 * hp.lut;
    RowIndex index;
    index.set(hp, unbias(__ldcg(a.row_max + x.at + mine)));
    uint32_t z = 0;
#pragma unroll 1
    for (; s < s1; s += par) {
      const int4 nx = load(s + par);
      const uint32_t i0 = index(v.x), i1 = index(v.y), i2 = index(v.z), i3 = index(v.w);
      z += (lut[i0] + lut[i1]) + (lut[i2] + lut[i3]);
      if (live) ip[4 * s] = prefill::pack4(i0, i1, i2, i3);
      v = nx;
    }
    __syncwarp();
    z += __shfl_xor_sync(0xffffffffu, z, 1);
    z += __shfl_xor_sync(0xffffffffu, z, 2);
    for (int o = 4 * rp; o < 32; o <<= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if (t == 0 && n8 < x.rows) atomicAdd(a.row_z + x.at + n8, static_cast<int32_t>(z));
    n = w.skip(a, kKeys, n, run);
  }
}

// First V tiles of the share into the ring: they wait for nothing, so they
// start before the barrier that phase C waits for.  Leaves `ld` at the next one.
template <int D>
__device__ __forceinline__ int own_pv_start(const SharedArgs& a, OwnRing& ring, Walk& ld, int n) {
#pragma unroll 1
  for (uint32_t i = 0; i < ring.slots && n > 0; ++i) {
    ring.issue(&a.tm_vc, ld.blk * (kOwnBytes / D), ld.b * a.Hkv + ld.hk, 0u);
    n = ld.skip(a, kOwnBytes / D, n, 1);
  }
  return n;  // not yet issued
}

// ---- phase C of the own rows: P.V of the same blocks ----
// A = V^T: sixteen channels by 32 keys per product, transposed on the way from
// shared memory; B = P: query row n8, keys 4 t .. + 3 and 16 + 4 t .. + 3, made
// while V is read (made a step ahead, with more code: 2 % longer in the case above).
template <int D>
__device__ __forceinline__ bool own_pv(const SharedArgs& a, bool v_u8, OwnRing& ring, const HeadParamsDev* hp_s,
                                       const uint32_t* lut_s, Walk w, Walk ld, int left, int n) {
  constexpr int kKeys = kOwnBytes / D;
  constexpr int kStep = kKeys / 32;  // 32-key steps per block
  constexpr int kM = D / 16;         // products per step
  const int lane = threadIdx.x & 31, n8 = lane >> 2, t = lane & 3;
  while (n > 0) {
    Unit x;
    x.set(a, w);
    const int mine = min(n8, x.rows - 1);
    const uint32_t* ip = a.index + static_cast<size_t>(x.row + mine) * (a.ld_s / 4) + t;
    auto index_word = [&](int s) { return 16 * s < x.len ? ip[4 * s] : 0x1F1F1F1Fu; };  // of 16-key step s
    const int run = min(n, w.nb - w.blk);  // blocks of this unit
    const int s0 = w.blk * kStep, s1 = (w.blk + run) * kStep;
    // of the next 32 keys
    uint32_t iy0 = index_word(2 * s0), iy1 = index_word(2 * s0 + 1);
    const uint32_t R = static_cast<uint32_t>(exact_R(__ldcg(a.row_z + x.at + mine)));  // < 2^25: Z >= 2^15
    const uint32_t lut = smem_u32(lut_s) + 128 * hp_s[a.per_head ? x.head + mine : 0].lut;
    uint32_t psum = 0;
    int32_t o[kM][4];
#pragma unroll
    for (int c = 0; c < kM; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[c][i] = 0;
    // P of four keys (0 for rows the unit does not have)
    auto make_p = [&](uint32_t word) {
      uint32_t b[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        b[e] = static_cast<uint32_t>(
            (static_cast<unsigned long long>(lds_u32(lut + 4 * ((word >> (8 * e)) & 255u))) * R + (1ull << 31)) >> 32);
      const uint32_t p = n8 < x.rows ? prefill::pack4(b[0], b[1], b[2], b[3]) : 0u;
      psum = __dp4a(p, 0x01010101u, psum);
      return p;
    };
    uint32_t tile = 0;
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
      const uint32_t ix0 = iy0, ix1 = iy1;
      iy0 = index_word(2 * s + 2);
      iy1 = index_word(2 * s + 3);
      const int in = s % kStep;
      if (in == 0 && (tile = ring.wait()) == 0) return false;
      uint32_t p0 = 0, p1 = 0, read = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // half of the channels at a time
        uint32_t v[kM / 2][4];
#pragma unroll
        for (int c = 0; c < kM / 2; ++c) ldmatrix2_trans(v[c], tile_at<D>(tile, 32 * in + lane, h * (kM / 2) + c));
        if (h == 0) {
          p0 = make_p(ix0);
          p1 = make_p(ix1);
        }
#pragma unroll
        for (int c = 0; c < kM / 2; ++c) {
          mma16832_pv(o[h * (kM / 2) + c], v_u8, v[c][0], v[c][1], v[c][2], v[c][3], p0, p1);
          read |= v[c][0] | v[c][1] | v[c][2] | v[c][3];
        }
      }
      if (in == kStep - 1 && left > 0) {
        ring.issue(&a.tm_vc, ld.blk * kKeys, ld.b * a.Hkv + ld.hk, read & a.none);
        left = ld.skip(a, kKeys, left, 1);
      }
    }
    if (v_u8) {
      psum += __shfl_xor_sync(0xffffffffu, psum, 1);
      psum += __shfl_xor_sync(0xffffffffu, psum, 2);
      if (t == 0 && n8 < x.rows) atomicAdd(a.row_p + x.at + n8, static_cast<int32_t>(psum));
    }
    // o[c][0], [1]: channel 16 c + n8, rows 2t and 2t + 1; [2], [3]: channel 16 c + 8 + n8
#pragma unroll
    for (int r = 0; r < 2; ++r)
      if (2 * t + r < x.rows) {
        float* dst = a.acc + static_cast<size_t>(x.at + 2 * t + r) * D + n8;
#pragma unroll
        for (int c = 0; c < kM; ++c)
#pragma unroll
          for (int e = 0; e < 2; ++e) atomicAdd(dst + 16 * c + 8 * e, static_cast<float>(o[c][2 * e + r]));
      }
    n = w.skip(a, kKeys, n, run);
  }
  return true;
}

// Requantised outputs of all rows, four channels per thread.
template <int D>
__device__ __forceinline__ void finish(const SharedArgs& a, const HeadParamsDev* hp_s, int thread, int threads) {
  const long long n = static_cast<long long>(a.Hkv) * a.R * (D / 4);
  for (long long i = thread; i < n; i += threads) {
    const int row = static_cast<int>(i / (D / 4)), c = 4 * static_cast<int>(i % (D / 4));
    const int hk = row / a.R, r = row - hk * a.R, b = r / a.G, h = hk * a.G + (r - b * a.G);
    bool skip = false;
    if (a.lengths != nullptr) {
      const int len = __ldg(a.lengths + b);
      skip = len < 0 || len > a.Lmax;
      if (skip && !a.zero_left_out) continue;
    }
    const float4 v = __ldcg(reinterpret_cast<const float4*>(a.acc + static_cast<size_t>(row) * D + c));
    const HeadParamsDev hp = hp_s[a.per_head ? h : 0];
    const int32_t fix = hp.zv != 0 ? hp.zv * __ldcg(a.row_p + row) : 0;  // sum P (v - z_v)
    const float f[4] = {v.x, v.y, v.z, v.w};
    int32_t y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      y[k] = skip ? 0 : static_cast<int8_t>(prefill::requant_byte(static_cast<int32_t>(f[k]) - fix, hp.Mo, hp.so));
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

// ZP: the instance for K or V codes with zero-points (u8); the other takes int8 only.
template <int D, bool ZP>
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
  // A ring slot holds K tiles and V tiles in turn.  Each kind has a full barrier
  // of its own: its consumer then waits for every phase of that barrier, one
  // after the other, as a wait for a parity has to.
  auto bar_full = [&](int v, int i) { return bar(kBarKvFull + v * C::kMaxStages + i); };
  auto bar_kv_empty = [&](int i) { return bar(kBarKvFull + 2 * C::kMaxStages + i); };

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  if (smem + C::kUsed > smem_raw + C::kSmemBytes) {  // the alignment took more than its share: nothing runs
    if (tid == 0) atomicOr(&g_device_error, kErrTimeout);
    return;
  }
  const bool k_u8 = ZP && args.k_u8, v_u8 = ZP && args.v_u8;
  const int F = args.fold;
  const int RF = kBM / F;       // lanes per fold
  const uint32_t stages = args.stages;  // at least 4: the key tiles of a tile fit the ring
  const int psets = kPBufs / F; // sets of F P buffers
  const int set_bits = F == 1 ? 2 : F == 2 ? 1 : 0;
  // this CTA's tiles
  const int t0 = first_tile(args, blockIdx.x), t1 = first_tile(args, blockIdx.x + 1);

  // The queries of at most two segments stay in the two Q buffers through all
  // phases, loaded by the softmax warps; of more, one warp loads them again in every phase.
  const bool q_stays = t0 < t1 && (t1 - 1) / args.seg_tiles - t0 / args.seg_tiles < 2;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarQFull + i), q_stays ? kSoftWarps : 1);
      mbar_init(bar(kBarQEmpty + i), 1);
      mbar_init(bar(kBarSFull + i), 1);
      mbar_init(bar(kBarSEmpty + i), kTeamWarps);
    }
    for (int i = 0; i < kPBufs; ++i) {
      mbar_init(bar(kBarPFull + i), kTeamWarps);
      mbar_init(bar(kBarPEmpty + i), 1);
    }
    mbar_init(bar(kBarOFull), 1);
    mbar_init(bar(kBarOEmpty), kSoftWarps);
    mbar_init(bar(kBarDrain), 1);
    mbar_init(bar(kBarDrain + 1), 1);
    for (int i = 0; i < kOwnWarps * kMaxOwnSlots; ++i) mbar_init(bar(kBarOwn + i), 1);
    for (int i = 0; i < C::kMaxStages; ++i) {
      mbar_init(bar_full(0, i), 1);
      mbar_init(bar_full(1, i), 1);
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

  // Grid-wide barrier k, reached by all softmax and own warps: whether every
  // warp's work so far was done and every CTA arrived in time.
  auto grid_sync = [&](int k, bool ok) {
    const bool v = bar_red_and(kNbBoth, 32 * (kSoftWarps + kOwnWarps), ok);
    if (tid == 0) {
      uint32_t good = 0;
      if (v) {
        // release and acquire at gpu scope by one thread cover the CTA's
        // other threads, which the named barriers order with it
        asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(args.ctr + k) : "memory");
        good = quant::wait_count(args.ctr + k, gridDim.x) ? 1u : 0u;
      }
      *verdict = good;
    }
    bar_red_and(kNbBoth, 32 * (kSoftWarps + kOwnWarps), true);
    return *verdict != 0u;
  };
  bool complete = false;  // softmax and own warps: acc holds every sum
  constexpr int kPieces = D / 16;  // of a row
  // piece i of the query rows of a segment (16-byte pieces, row by row)
  auto q_piece = [&](const Segment& sg, int i) {
    const int row = sg.rt * kBM + i / kPieces;
    if (i >= RF * kPieces || row >= args.R) return make_uint4(0, 0, 0, 0);
    const int b = row / args.G, g = row - b * args.G;
    return __ldg(reinterpret_cast<const uint4*>(args.q + (static_cast<size_t>(b) * args.H + sg.hk * args.G + g) * D +
                                                16 * (i % kPieces)));
  };
  auto q_store = [&](uint32_t qb, int i, uint4 v) {
    if (i >= RF * kPieces) return;
    const int row = kBM - RF + kBM * static_cast<int>(qb) + i / kPieces, c = i % kPieces;
    const int piece = D == 128 ? (c ^ (row & 7)) : (c ^ ((row >> 1) & 3));  // the TMA's swizzle
    *reinterpret_cast<uint4*>(smem + C::kOffQ + row * D + 16 * piece) = v;
  };
  auto q_zero = [&](int worker, int workers) {  // the padding rows: zero for good
    for (int i = worker; i < C::kQRows * kPieces; i += workers)
      *reinterpret_cast<uint4*>(smem + C::kOffQ + 16 * i) = make_uint4(0, 0, 0, 0);
  };
  // Registers: 896 threads are launched with 72 each; the softmax warps give 8
  // each (4096 in all), which is what the own warps take (16 each).
  if (warp < kSoftWarps) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
  else if (warp >= kOwnWarp0) asm volatile("setmaxnreg.inc.sync.aligned.u32 88;");

  if (warp < kSoftWarps) {
    // ======================= softmax warps =======================
    const int sw = warp;
    const int quad = warp & 3;
    const int half = (sw >> 2) & 1;
    const int team = sw / kTeamWarps;
    const int grp = team * 2 + half;
    const int r = quad * 32 + lane;  // TMEM lane
    const int f = r / RF;            // its fold (uniform over the warp)
    const int rr = r - f * RF;       // its row of the tile
    const uint32_t tlane = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t trow = tlane + half * kCols;
    const uint32_t prow = smem_u32(tab) + 4u * r;
    bool ok = true;
    uint32_t sc = 0;  // tiles so far
    uint32_t pc = 0;  // P tiles so far
    uint32_t no = 0;  // O segments so far
    if (F > 1 && sw < 4) {
      // the lanes of the other folds in every P buffer: zero for good
      const uint32_t zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      for (int b = 0; b < kPBufs; ++b)
        if (b % F != f)
          for (int c = 0; c < 4; ++c) tmem_st8(tlane + kColP + b * 32 + 8 * c, zero);
      tmem_wait_st();
      tc_fence_before();
    }
    auto soft_sync = [&](bool mine) { return bar_red_and(kNbSoft, 32 * kSoftWarps, mine); };
    auto arrive_warp = [&](uint32_t b) {
      __syncwarp();
      if (lane == 0) mbar_arrive(b);
    };
    if (q_stays) {
      const Segment sg = segment_at(args, t0, t1);
      const bool two = t0 + sg.n < t1;
      const Segment sh = two ? segment_at(args, t0 + sg.n, t1) : sg;
      constexpr int kPer = kBM * kPieces / (32 * kSoftWarps);  // 1 or 2 pieces per thread and segment
      uint4 v[2][kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        v[0][k] = q_piece(sg, tid + 32 * kSoftWarps * k);
        v[1][k] = q_piece(sh, tid + 32 * kSoftWarps * k);
      }
      if (F > 1) {
        q_zero(tid, 32 * kSoftWarps);
        soft_sync(true);
      }
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        q_store(0, tid + 32 * kSoftWarps * k, v[0][k]);
        if (two) q_store(1, tid + 32 * kSoftWarps * k, v[1][k]);
      }
      fence_proxy_async_smem();
      arrive_warp(bar(kBarQFull));
      if (two) arrive_warp(bar(kBarQFull + 1));
    }
    // The scores of tile `idx`, kChunk columns at a time; columns from nv on are
    // `low`.  One copy of the body in a rolled loop: the phases' code has to
    // stay small (instruction fetches were a third of the stalls with both
    // halves unrolled and a masked copy beside them).
    auto walk_s = [&](uint32_t idx, int nv, uint32_t low, auto&& body) {
      const uint32_t buf = idx & 1;
      if (!mbar_wait_warp(bar(kBarSFull + buf), (idx >> 1) & 1, kRoleSoftmax)) return false;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < kCols / kChunk; ++c) {
        uint32_t v[kChunk];
        tmem_ld16(trow + kColS + buf * kBN + kChunk * c, v);
        tmem_wait_ld();
        if (c == kCols / kChunk - 1) {
          tc_fence_before();
          arrive_warp(bar(kBarSEmpty + buf));
        }
        if (nv < kCols) {
#pragma unroll
          for (int k = 0; k < kChunk; ++k)
            if (kChunk * c + k >= nv) v[k] = low;
        }
        body(v, c);
      }
      return true;
    };
    auto first_j = [&](uint32_t s0) { return static_cast<int>((static_cast<uint32_t>(team) - s0) & 1u); };
    // keys of this thread's half of its key tile in tile j that exist: a prefix
    auto nvalid = [&](int j) { return min(max(args.Lp - ((j * F + f) * kBN + half * kCols), 0), kCols); };

    quant::griddep_wait();  // the counters and row maxima are zeroed

    // ---- phase A ----
    for (int t = t0; t < t1 && ok;) {
      const Segment sg = segment_at(args, t, t1);
      int32_t m = INT_MIN;
      for (int j = first_j(sc); j < sg.n; j += kTeams) {
        int32_t m4[4] = {INT_MIN, INT_MIN, INT_MIN, INT_MIN};
        const bool got = walk_s(sc + j, nvalid(sg.j0 + j), 0x80000000u, [&](const uint32_t (&v)[kChunk], int) {
#pragma unroll
          for (int k = 0; k < kChunk; k += 8) {
            m4[0] = __vimax3_s32(m4[0], static_cast<int32_t>(v[k + 0]), static_cast<int32_t>(v[k + 1]));
            m4[1] = __vimax3_s32(m4[1], static_cast<int32_t>(v[k + 2]), static_cast<int32_t>(v[k + 3]));
            m4[2] = __vimax3_s32(m4[2], static_cast<int32_t>(v[k + 4]), static_cast<int32_t>(v[k + 5]));
            m4[3] = __vimax3_s32(m4[3], static_cast<int32_t>(v[k + 6]), static_cast<int32_t>(v[k + 7]));
          }
        });
        if (!got) { ok = false; break; }
        m = imax(m, imax(imax(m4[0], m4[1]), imax(m4[2], m4[3])));
      }
      sc += sg.n;
      const int row = sg.rt * kBM + rr;
      if (row < args.R && m != INT_MIN) atomicMax(args.row_max + static_cast<size_t>(sg.hk) * args.R + row, bias(m));
      t += sg.n;
    }
    ok = grid_sync(0, ok);

    // index code of a score (see the prefill kernel): the bits of
    // 0x4B000000 + k, k = idx + 1 (idx <= 30) or 32 (clipped)
    uint32_t Cx = 0;
    float Ms32 = 0.f, c1 = 0.f;
    const uint32_t* lut_h = lut_s;
    auto row_index = [&](const Segment& sg) {
      const int row = min(sg.rt * kBM + rr, args.R - 1);  // rows past R repeat the last one and are dropped
      const int h = sg.hk * args.G + row % args.G;
      const HeadParamsDev hp = hp_s[args.per_head ? h : 0];
      lut_h = lut_s + 32 * hp.lut;
      Cx = 0x4B000000u + static_cast<uint32_t>(unbias(__ldcg(args.row_max + static_cast<size_t>(sg.hk) * args.R + row)));
      const float Mf = __int2float_rn(hp.M);
      Ms32 = Mf * __uint_as_float(static_cast<uint32_t>(127 - 5 - hp.s) << 23);
      c1 = (1.5f - Mf * __uint_as_float(static_cast<uint32_t>(127 + 23 - hp.s) << 23)) * 0.03125f;
      return static_cast<size_t>(sg.hk) * args.R + row;
    };
    // the "score" of a masked key: its X is a huge float, so its code is 32
    auto masked = [&]() { return Cx - 0x7F000000u; };
    auto idx_bits2 = [&](uint32_t s0, uint32_t s1, uint32_t& b0, uint32_t& b1) {
      const float y0 = fma_rz_sat(__uint_as_float(Cx - s0), Ms32, c1);
      const float y1 = fma_rz_sat(__uint_as_float(Cx - s1), Ms32, c1);
      float k0, k1;
      fma2_rz(y0, y1, pack2(32.0f), pack2(8388608.0f), k0, k1);
      b0 = __float_as_uint(k0);
      b1 = __float_as_uint(k1);
    };

    // ---- phase B ----
    if (ok) {
      for (int t = t0; t < t1;) {
        const Segment sg = segment_at(args, t, t1);
        const size_t at = row_index(sg);
#pragma unroll
        for (int i = grp * 8; i < grp * 8 + 8; ++i) tab[(i + 1) * kBM + r] = lut_h[i];
        if (!soft_sync(ok)) { ok = false; break; }
        int32_t Z = 0;
        for (int j = first_j(sc); j < sg.n; j += kTeams) {
          int32_t z4[4] = {0, 0, 0, 0};
          const bool got = walk_s(sc + j, nvalid(sg.j0 + j), masked(), [&](const uint32_t (&v)[kChunk], int) {
#pragma unroll
            for (int k = 0; k < kChunk; k += 2) {
              uint32_t b0, b1;
              idx_bits2(v[k], v[k + 1], b0, b1);
              z4[k & 3] += static_cast<int32_t>(lds_u32(b0 * 512u + prow));
              z4[(k + 1) & 3] += static_cast<int32_t>(lds_u32(b1 * 512u + prow));
            }
          });
          if (!got) { ok = false; break; }
          Z += (z4[0] + z4[1]) + (z4[2] + z4[3]);
        }
        sc += sg.n;
        if (sg.rt * kBM + rr < args.R && Z != 0) atomicAdd(args.row_z + at, Z);
        t += sg.n;
        if (!soft_sync(ok)) { ok = false; break; }  // the table may be written again
      }
      ok = grid_sync(1, ok);
      if (ok) {
        // ---- phase C ----
        for (int t = t0; t < t1;) {
          const Segment sg = segment_at(args, t, t1);
          const size_t at = row_index(sg);
          const unsigned long long R = exact_R(__ldcg(args.row_z + at));
#pragma unroll
          for (int i = grp * 8; i < grp * 8 + 8; ++i) {
            const uint32_t P = static_cast<uint32_t>((static_cast<unsigned long long>(lut_h[i]) * R + (1ull << 31)) >> 32);
            tab[(i + 1) * kBM + r] = P;
            tab[C::kTabBytes / 4 + (i + 1) * kBM + r] = P << 8;
          }
          if (!soft_sync(ok)) { ok = false; break; }
          uint32_t psum = 0;
          for (int j = first_j(sc); j < sg.n; j += kTeams) {
            const uint32_t pi = pc + j;
            const uint32_t set = pi & (psets - 1);
            const uint32_t pb = set * F + f;  // this fold's buffer of the set
            const bool got = walk_s(sc + j, nvalid(sg.j0 + j), masked(), [&](const uint32_t (&v)[kChunk], int c) {
              uint32_t pw[kChunk / 4];
#pragma unroll
              for (int q = 0; q < kChunk / 4; ++q) {
                uint32_t kb[4], p[4];
                idx_bits2(v[q * 4], v[q * 4 + 1], kb[0], kb[1]);
                idx_bits2(v[q * 4 + 2], v[q * 4 + 3], kb[2], kb[3]);
#pragma unroll
                for (int b = 0; b < 4; ++b) p[b] = lds_u32(kb[b] * 512u + prow + (b & 1) * C::kTabBytes);
                pw[q] = (p[0] + p[1]) + ((p[2] + p[3]) << 16);
              }
              if (v_u8) {
#pragma unroll
                for (int q = 0; q < kChunk / 4; ++q) psum = __dp4a(pw[q], 0x01010101u, psum);
              }
              // The set's last P.V has read it.  With one set (F = 4) that was the
              // other team's, tile pi - 1, and the P.V of even and of odd tiles complete
              // a barrier each: a parity tells only two states apart, and at this
              // point the P.V of tile pi - 2 may be done or not.
              if (c == 0) {
                const uint32_t e = psets == 1 ? (pi & 1) ^ 1 : set;
                const uint32_t phase = psets == 1 ? ((pi + 1) >> 1) - 1 : (pi >> set_bits) - 1;  // pi = 0 .. psets - 1: none yet
                if (!mbar_wait_warp(bar(kBarPEmpty + e), phase & 1, kRoleSoftmax)) ok = false;
              }
              tmem_st4(tlane + kColP + pb * 32 + half * (kCols / 4) + c * (kChunk / 4), pw[0], pw[1], pw[2], pw[3]);
            });
            if (!got) ok = false;
            if (!ok) break;
            tmem_wait_st();
            tc_fence_before();
            arrive_warp(bar(kBarPFull + set));
          }
          sc += sg.n;
          pc += sg.n;
          const int row = sg.rt * kBM + rr;
          if (psum != 0 && row < args.R) atomicAdd(args.row_p + at, static_cast<int32_t>(psum));
          // O (int32, TMEM) of the segment -> acc: this thread's lane, a quarter of the channels
          if (ok && !mbar_wait_warp(bar(kBarOFull), no & 1, kRoleSoftmax)) ok = false;
          if (ok) {
            tc_fence_after();
            float* dst = args.acc + at * D + grp * (D / 4);
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
              uint32_t v[16];
              tmem_ld16(tlane + kColO + grp * (D / 4) + 16 * c, v);
              tmem_wait_ld();
              if (row < args.R) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  red_add4(dst + 16 * c + 4 * q, __int2float_rn(static_cast<int32_t>(v[4 * q])),
                           __int2float_rn(static_cast<int32_t>(v[4 * q + 1])),
                           __int2float_rn(static_cast<int32_t>(v[4 * q + 2])),
                           __int2float_rn(static_cast<int32_t>(v[4 * q + 3])));
              }
            }
            tc_fence_before();
            arrive_warp(bar(kBarOEmpty));
          }
          ++no;
          t += sg.n;
          if (!soft_sync(ok)) { ok = false; break; }
        }
        complete = grid_sync(2, ok);
      }
    }
  } else if (warp >= kOwnWarp0) {
    // ========================== own rows ==========================
    const int ow = warp - kOwnWarp0;
    {
      // what the later phases add to: row_z, row_p and acc are consecutive words
      const size_t rows = static_cast<size_t>(args.Hkv) * args.R;
      const size_t n = 2 * rows + rows * D;
      for (size_t i = static_cast<size_t>(blockIdx.x) * (32 * kOwnWarps) + (tid - 32 * kOwnWarp0); i < n;
           i += static_cast<size_t>(gridDim.x) * (32 * kOwnWarps))
        args.row_z[i] = 0;
    }
    if (args.lengths != nullptr && blockIdx.x == 0 && ow == 0)
      for (int b = lane; b < args.B; b += 32) {
        const int n = __ldg(args.lengths + b);
        if (n < 0 || n > args.Lmax) atomicOr(&g_device_error, kErrParamRange);
      }
    Walk w;
    // neighbouring shares on different CTAs
    const int n = args.Lmax > 0 ? w.share(args, kOwnBytes / D, ow * gridDim.x + blockIdx.x, kOwnWarps * gridDim.x)
                                : 0;
    const uint32_t own_slots = args.own_slots;
    OwnRing ring{sKV + stages * C::kTileBytes + kOwnBytes * own_slots * ow, bar(kBarOwn + kMaxOwnSlots * ow), own_slots, 0u,
                 0u};
    quant::griddep_wait();
    bool ok = own_scores<D>(args, k_u8, ring, w, n);
    if ((ok = grid_sync(0, ok))) {
      Walk ld = w;
      const int left = own_pv_start<D>(args, ring, ld, n);
      own_sums<D>(args, hp_s, lut_s, w, n);
      if ((ok = grid_sync(1, true))) {
        ok = own_pv<D>(args, v_u8, ring, hp_s, lut_s, w, ld, left, n);
        complete = grid_sync(2, ok);
      }
    }
    ring.drain();
  } else if (warp == kProducerWarp) {
    // ============================ TMA producer ============================
    // lane s owns ring slot s (see the prefill kernel)
    if (lane == 0 && t0 < t1) {
      tma_prefetch_desc(&args.tm_k);
      tma_prefetch_desc(&args.tm_v);
    }
    __syncwarp();
    if (static_cast<uint32_t>(lane) < stages) {
      const uint32_t slot = static_cast<uint32_t>(lane);
      const uint32_t dst = sKV + slot * C::kTileBytes;
      uint32_t n = 0, mine = 0;       // the next load's slot; loads of this lane
      uint32_t kinds[2] = {0, 0};     // of them K and V
      bool ok = true;
      // the key tiles of tile j
      auto load = [&](int v, int j, int hk) {
        const int nf = folds_at(args, j);
        for (int x = 0; x < nf; ++x) {
          const bool other = n != slot;
          if (++n == stages) n = 0;
          if (!ok || other) continue;
          if (!mbar_wait(bar_kv_empty(slot), (mine & 1) ^ 1, kRoleProducer)) {
            ok = false;
          } else {
            mbar_arrive_expect_tx(bar_full(v, slot), C::kTileBytes);
            tma_load_3d(dst, v ? &args.tm_v : &args.tm_k, bar_full(v, slot), 0, (j * F + x) * kBN, hk);
            ++mine;
            kinds[0] += 1 - v;
            kinds[1] += v;
          }
        }
      };
      // in the order the MMA warp takes them
#pragma unroll 1
      for (int phase = 0; phase < 3; ++phase)
        for (int t = t0; t < t1 && ok;) {
          const Segment sg = segment_at(args, t, t1);
          const int turns = 2 * sg.n + (phase == 2 ? 4 : 0);  // K of tile e, V of tile e - 2
#pragma unroll 1
          for (int y = 0; y < turns; ++y) {
            const int j = (y >> 1) - ((y & 1) ? 2 : 0);
            if (j < 0 || j >= sg.n || ((y & 1) && phase < 2)) continue;
            load(y & 1, sg.j0 + j, sg.hk);
          }
          t += sg.n;
        }
      for (int v = 0; v < 2; ++v)  // no copy left in flight
        if (kinds[v] > 0) mbar_wait(bar_full(v, slot), (kinds[v] - 1) & 1, kRoleProducer);
    }
    __syncwarp();
  } else if (warp == kMmaWarp || warp == kPvWarp) {
    // ============================= MMA issuers =============================
    // One thread issues S = Q.K^T, another O += P.V.  Both walk the ring's load
    // sequence (K of tile e, then in phase C V of tile e - 2), each past the
    // other's slots.  What lies between two tiles' products is the latency of a few
    // dependent instructions, in which the tensor pipe stands still: so one
    // thread runs the whole loop, and waits for a K or V tile only before its
    // own products, while those of the one before it run (warp-wide loops: B9
    // L50000 2 % longer).  Two issuers instead of one took 3 % from B64 L8192 and left the other cases where they were.
    if (elect_one()) {
      const bool pv = warp == kPvWarp;
      const uint64_t kv_desc0 = smem_desc(sKV, 16, C::kSBO, C::kSwizzle);
      constexpr uint32_t kSlotDesc = C::kTileBytes >> 4;
      bool ok = true;
      uint32_t slot = 0;
      uint32_t par = 0;  // bit s: parity of the next phase of slot s's barrier of this warp's kind
      auto past = [&](uint32_t n) {  // n slots on (n <= 2 F, F <= stages)
        slot += n;
        if (slot >= stages) slot -= stages;
      };
      // the K or V tile in the next slot; with its products issued, `taken` moves on
      auto arrived = [&]() { return mbar_wait(bar_full(pv ? 1 : 0, slot), (par >> slot) & 1, kRoleMma); };
      auto taken = [&]() {
        mma_commit(bar_kv_empty(slot));
        par ^= 1u << slot;
        past(1);
      };
      if (!pv) {
        const uint32_t idesc = idesc_i8(kBM, kBN, 1, k_u8 ? 0u : 1u, 0);
        const uint64_t q_desc0 = smem_desc(s_base + C::kOffQ, 16, C::kSBO, C::kSwizzle);
        uint32_t sc = 0, nq = 0;
        for (int phase = 0; phase < 3 && ok; ++phase) {
          if (q_stays) nq = 0;
          for (int t = t0; t < t1 && ok; ++nq) {
            const Segment sg = segment_at(args, t, t1);
            const uint32_t qb = nq & 1;
            if (!mbar_wait(bar(kBarQFull + qb), q_stays ? 0u : (nq >> 1) & 1, kRoleMma)) { ok = false; break; }
            const uint64_t q_desc = q_desc0 + ((static_cast<uint32_t>(kBM - RF + kBM * qb) * D) >> 4);
#pragma unroll 1
            for (int e = 0; e < sg.n; ++e) {
              const int nf = folds_at(args, sg.j0 + e);
              const uint32_t buf = sc & 1;
              if (!(ok = mbar_wait(bar(kBarSEmpty + buf), ((sc >> 1) & 1) ^ 1, kRoleMma))) break;
              tc_fence_after();
              // the queries in the lanes of fold x against key tile x
#pragma unroll 1
              for (int x = 0; x < nf; ++x) {
                if (!(ok = arrived())) break;
                const uint64_t k_desc = kv_desc0 + slot * kSlotDesc;
                const uint64_t a_desc = q_desc - ((static_cast<uint32_t>(x * RF) * D) >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk)
                  mma_i8_ss(tmem + kColS + buf * kBN, a_desc + 2 * kk, k_desc + 2 * kk, idesc, (x > 0 || kk > 0) ? 1u : 0u);
                taken();
              }
              if (!ok) break;
              mma_commit(bar(kBarSFull + buf));
              ++sc;
              if (phase == 2 && e >= 2) past(F);  // V of tile e - 2, not the head's last: a full one
            }
            // V of the segment's last two tiles
            if (phase == 2)
              for (int e = max(sg.n - 2, 0); e < sg.n; ++e) past(folds_at(args, sg.j0 + e));
            if (!ok) break;
            if (!q_stays) mma_commit(bar(kBarQEmpty + qb));
            t += sg.n;
          }
        }
      } else {
        const uint32_t idesc = idesc_i8(kBM, D, 0, v_u8 ? 0u : 1u, 1);
        uint32_t pc = 0, no = 0;
        // K tiles of phases A and B
        uint32_t before = 0;
        for (int t = t0; t < t1;) {
          const Segment sg = segment_at(args, t, t1);
          before += 2 * (min((sg.j0 + sg.n) * F, args.key_tiles) - sg.j0 * F);
          t += sg.n;
        }
        slot = before % stages;
        for (int t = t0; t < t1 && ok; ++no) {
          const Segment sg = segment_at(args, t, t1);
          for (int e = 0; e < min(sg.n, 2); ++e) past(folds_at(args, sg.j0 + e));  // K of the first two tiles
#pragma unroll 1
          for (int j = 0; j < sg.n; ++j) {
            if (j + 2 < sg.n) past(folds_at(args, sg.j0 + j + 2));
            const int nf = folds_at(args, sg.j0 + j);
            const uint32_t set = pc & (psets - 1);
            // the first P.V of a segment: O of the previous one has been read
            ok = (j > 0 || mbar_wait(bar(kBarOEmpty), (no & 1) ^ 1, kRoleMma)) &&
                 mbar_wait(bar(kBarPFull + set), (pc >> set_bits) & 1, kRoleMma);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int x = 0; x < nf; ++x) {
              if (!(ok = arrived())) break;
              const uint64_t v_desc = kv_desc0 + slot * kSlotDesc;
#pragma unroll
              for (int kk = 0; kk < kBN / 32; ++kk)
                mma_i8_ts(tmem + kColO, tmem + kColP + (set * F + x) * 32 + kk * 8, v_desc + ((32u * D * kk) >> 4), idesc,
                          (j > 0 || x > 0 || kk > 0) ? 1u : 0u);
              taken();
            }
            if (!ok) break;
            mma_commit(bar(kBarPEmpty + (psets == 1 ? pc & 1 : set)));
            if (j == sg.n - 1) mma_commit(bar(kBarOFull));
            ++pc;
          }
          t += sg.n;
        }
      }
      mma_commit(bar(kBarDrain + (pv ? 1 : 0)));
      mbar_wait(bar(kBarDrain + (pv ? 1 : 0)), 0, kRoleMma);
    }
    __syncwarp();
  } else {
    // ============================== Q rows ==============================
    // more than two segments: eight loads in flight per lane
    if (!q_stays && t0 < t1) {
      constexpr int kBatch = 8;
      if (F > 1) {
        q_zero(lane, 32);
        __syncwarp();  // before the first rows
      }
      uint32_t nq = 0;
      bool ok = true;
#pragma unroll 1
      for (int phase = 0; phase < 3 && ok; ++phase)
#pragma unroll 1
        for (int t = t0; t < t1; ++nq) {
          const Segment sg = segment_at(args, t, t1);
          const uint32_t qb = nq & 1;
          if (!mbar_wait_warp(bar(kBarQEmpty + qb), ((nq >> 1) & 1) ^ 1, kRoleQ)) { ok = false; break; }
#pragma unroll 1
          for (int i0 = 0; i0 < RF * kPieces; i0 += 32 * kBatch) {
            uint4 v[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) v[k] = q_piece(sg, i0 + 32 * k + lane);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) q_store(qb, i0 + 32 * k + lane, v[k]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarQFull + qb));
          t += sg.n;
        }
    }
  }

  if (complete) {
    constexpr int kFinishers = 32 * (kSoftWarps + kOwnWarps);
    finish<D>(args, hp_s, blockIdx.x * kFinishers + (warp < kSoftWarps ? tid : tid - 32 * (kOwnWarp0 - kSoftWarps)),
              gridDim.x * kFinishers);
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
