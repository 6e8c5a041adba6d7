// Attention over the 8-bit key/value cache, few query rows per kv head
// (decode, drafted tokens): the cache is streamed once and bounds the time.
//
//   s_ij = scale * q_i . k_j,  L_i = ln sum_j exp(s_ij),  O_i = sum_j exp(s_ij - L_i) v_j
//
// over the visible keys j of query i.  The rows of one (request, kv head) are
// its new tokens times the Hq / Hkv query heads that share the kv head, in
// tiles of ROWS, 8 or 16; a work unit is one such tile over all of the request's
// keys.
//
// Work.  The keys of every unit are cut into tiles of 32, and the tiles of
// all units, in order and with a fixed cost for each piece, into one equal range
// per CTA, so any mix of lengths fills the GPU evenly.  A CTA covers whole units
// and at most two pieces of units, which it leaves as normalised partials with
// their logsumexp; a second, dependent kernel merges those per row in CTA order.
//
// A CTA.  One producer warp walks the range: it publishes a descriptor and the
// query rows of each unit piece, reads block tables and scales for 32 tiles at
// a time, of one piece or of many, and moves the tiles (32 keys of K and of V
// as codes) through a ring of TMA loads.  A piece belongs to 1, 2, 4 or 8 of
// the eight other warps, a few tiles each while it is short, so that short pieces
// run side by side; its warps take the tiles in turn, each with a softmax of
// its own, and merge through shared memory at the end.  In a warp a tile goes
//   codes -> f16 (exact) -> S = Q K^T -> P -> O += P V
// by m16n8k16 f16 products, with 8 rows S^T = K Q^T and O^T = V^T P^T, half as
// many (64 requests of 30 to 8192 tokens, 4 rows per kv head: 123 us with 16
// rows, 113 with 8, before the pieces' cost was set): each warp reads its own
// keys straight from shared memory in the product's operand layout, which a
// choice of which key and which head-dim index each lane takes makes 16-byte
// reads without bank conflicts (tok() below).  tcgen05 would need the codes
// converted in shared memory first: twice the traffic of the conversion for
// rows that fill an eighth of its 128.
//
// What bounds it.  DRAM for long keys: 24 requests of 20000 to 32768 tokens, 8
// kv heads of 128, in 200 us, 6.3 TB/s; the pieces' starts and ends and the
// last CTA for shorter ones: 64 requests of 30 to 8192 in 101 us (5.5 TB/s).
// Latency for little work: one request of 1000 in 10.7 us, two launches.
// (Times beside a choice are those of the kernel as it then was, with and
// without it.)
//
// Numbers.  A query row is divided by the power of two of its largest element
// and held in f16, three bits more than its bf16 has: exact but for elements
// below 2^-17 of the row's largest, whose error is at most 2^-25 of it.  Sums
// are fp32.  The row keeps two references: m, the largest s (log2 units), for
// l = sum 2^(s - m); and E, the largest s + floor(log2 v_scale), for the
// output's weights 2^(14 + s - E) v_scale, which lie below 2^15 and are
// rounded to f16 (11 bits), so that neither a block of small values nor one
// of zeros costs the others precision.  Where a block's scale lies far above 2^E
// the two factors of such a weight leave fp32's range; those tiles take a branch
// of their own (up to 2 % of the others' time, for asking).  E is kept as
// its distance from m: beside a large m a sum with log2 v_scale would be lost.
//
// Four bits (E2M1Codes; fa_cache4.cuh has the layout).  The walk, the ring, the
// pieces and their merge are the same.  A tile is 64 keys, one bulk copy for each of
// its blocks with the scales inside, and two warps take half of it each.  In a warp
//   codes -> f16, times their scales (exact) -> S -> P -> O += P V
// and as no value's range needs a second reference, E is 0.  It is the taking apart
// that bounds it: 520 instructions for 32 keys, 128 conversions and 128
// multiplications among them.  24 requests of 20000 to 32768 tokens, 8 kv heads of
// 128, take 139 us, 5.1 TB/s (114 us with the loads alone, 121 without either
// product); 64 of 30 to 8192 80 us; one of 1000 10.4 us.
#pragma once
#include <cuda_bf16.h>

#include "fa_cache.cuh"
#include "fa_cache4.cuh"
#include "sm103_ptx.cuh"

namespace fa {

// What a cache holds its rows as.
struct E4M3Codes {  // a scale per block and head, beside the codes
  static constexpr bool k4 = false;
  struct Maps {
    CUtensorMap k, v;
  };
};
struct E2M1Codes {  // a scale for 16 elements, in granules with the codes
  static constexpr bool k4 = true;
  struct Maps {};
};

namespace dec {

constexpr int kKeys = 32;                    // keys of a tile, or part of one, that a warp takes
constexpr int kWarpScan = 128;               // requests that one warp sums
// References before the first key: -FLT_MAX, as scores may lie anywhere above.
// What is subtracted from it or from a score may then be -inf, which ends as a
// weight of 0; it is never added to +inf.
constexpr float kInit = -3.402823466e38f;

enum : unsigned { kSiteStageFull = 501, kSiteStageEmpty = 502, kSiteSegFull = 503, kSiteSegEmpty = 504,
                  kSiteMergeW = 505, kSiteMergeR = 506, kSiteIssued = 507 };

struct Seg {
  int r, h, row0;      // request, kv head, first row of the tile
  int nv;              // rows of the tile that exist
  int c0, n, len;      // the request's first query row, new tokens, cached tokens
  int t0, nt;          // first key tile of the piece and their number (0: end)
  int mode;            // 0: the whole unit; 1: leaves a partial in slot
  int slot, base;      // base: ring position of the first tile
  int w0, nw;          // its warps (few rows per kv head only)
};

// ROWS query rows a unit, 16 or 8.  8 rows at d = 64 leave registers and room
// for two CTAs per SM with half the ring each.
constexpr int ctas_per_sm(int d, int rows) { return d == 64 && rows == 8 ? 2 : 1; }
template <int D, int ROWS, class F>
struct Layout {
  static constexpr int kCtas = ctas_per_sm(D, ROWS);
  // Consumer warps, and the numbers of them that a piece may have: 1, 2, 4 and 8.
  // Taking 4-bit codes apart is more instructions a byte, whose latencies more warps
  // hide: 15, with the producer as many as have 128 registers a thread, of which a
  // piece has 1, 3 or all (24 requests of 20000 to 32768 tokens: 145 us, 154 with 8;
  // 143 with two CTAs of 8 warps, which have 96 registers and spill).
  static constexpr bool kMany = F::k4 && D == 128 && ROWS == 8;
  static constexpr int kWarps = kMany ? 15 : 8;
  static constexpr int kThreads = 32 * (kWarps + 1);            // and the producer
  static constexpr int kSmall = kMany ? 3 : 2, kMiddle = kMany ? 15 : 4;
  static constexpr int kSmalls = kWarps / kSmall, kMiddles = kMany ? 0 : 2;
  static constexpr int kMerges = kSmalls + kMiddles + 1;        // groups that merge
  __device__ static int next_size(int nw) { return nw == 1 ? kSmall : nw == kSmall ? kMiddle : kWarps; }
  // 1, 2, 4: a bit for each size above one.
  __device__ static uint32_t kind_of(int nw) { return nw == kSmall ? 1u : nw == kWarps ? 4u : 2u; }
  // Offset of the merge barrier of the warps of a group that `warp` is one of.
  __device__ static int merge_bar(int warp, uint32_t kind) {
    return 8 * (kind == 1u ? warp / kSmall : kind == 2u ? kSmalls + warp / kMiddle : kMerges - 1);
  }
  static constexpr int kSegs = 8;                               // unit pieces in flight
  // Keys of a tile: what one load brings of each of its blocks.  Of 4-bit codes two
  // warps share one, as the producer takes about 100 cycles a load and 32 keys
  // arrive every 196 (24 requests of 20000 to 32768 tokens: 143 us with 32 keys).
  static constexpr int kParts = F::k4 ? 2 : 1;
  static constexpr int kTile = kParts * kKeys;
  // A piece's fixed cost, in tiles (64 requests of 30 to 8192 tokens, 8 bits, 5: 114 us,
  // 12: 104).  4 bits, us with 8 / 12 / 16 / 20 / 28 (8 kv heads of 128, then of 64):
  //   64 requests of 30 to 8192 tokens    84.0 / 80.5 / 77.9 / 77.5 / 79.5   51.4 / 50.0 / 50.1 / 50.7 / 52.0
  //   200 of 30 to 2000                   94.3 / 94.8 / 95.2 / 98.9 / 102    55.8 / 55.4 / 57.0 / 58.2 / 60.3
  //   24 of 20000 to 32768                137 within 0.4                     87.8 / 87.9 / 88.2 / 88.4 / 90.1
  //   32 of 4000, 4 kv heads; 16 of 1 to 1024, 32
  //                                       30.6 / 30.4 / 29.3 / 29.5 / 29.0   19.9 / 19.4 / 19.5 / 20.1 / 20.9
  static constexpr int kUnitCost = F::k4 ? (D == 64 ? 10 : 16) : 12;
  static constexpr int kMinCost = F::k4 ? 6 : 12;               // least cost of a CTA's range
  static constexpr int kHalf = kKeys * D;                       // codes of K (or V) of a tile; 4 bits: unused
  static constexpr int kPart = 2 * c4::Granule<D>::kBytes;      // 4 bits: of a warp's keys
  static constexpr int kStage = F::k4 ? kParts * kPart : 2 * kHalf;
  static constexpr int kStages = (kMany ? 139264 : 131072) / kCtas / kStage * kParts / kWarps * kWarps / kParts;
  static constexpr int kIssue = kStages / 2 < 32 ? kStages / 2 : 32;  // lanes that issue loads
  // Tiles whose blocks and scales are held.  An entry is reused so many tiles
  // later: before the first of 32 tiles is looked up, all but the last ring's
  // worth has been consumed.
  static constexpr int kMeta = kStages + 32 <= 64 ? 64 : 128;
  static_assert(kMeta >= kStages + 32, "entries of tiles in flight");
  static constexpr int kMerge = kStages * kStage;
  static constexpr int kQ = kMerge + kWarps * 8 * D * 4;        // bf16 [segs][rows][D]
  static constexpr int kStats = kQ + kSegs * ROWS * D * 2;      // float4 [warps][8]
  static constexpr int kScales = kStats + kWarps * 8 * 16;      // float4 [meta]
  // int4 [meta]: blocks, row in the block, valid; 4 bits: blocks, and in an int
  // each in the place of the scales the granule in the block and 16 times valid
  static constexpr int kBlk = kScales + kMeta * 16;
  static constexpr int kSeg = kBlk + kMeta * 16;
  static constexpr int kBar = (kSeg + kSegs * static_cast<int>(sizeof(Seg)) + 15) & ~15;
  static constexpr int kFull = kBar;                    // [stages]
  static constexpr int kEmpty = kFull + 8 * kStages;    // [stages]
  static constexpr int kSegFull = kEmpty + 8 * kStages; // [segs]
  static constexpr int kSegEmpty = kSegFull + 8 * kSegs;
  static constexpr int kMergeW = kSegEmpty + 8 * kSegs; // [merges] small groups, middle ones, all
  static constexpr int kMergeR = kMergeW + 8 * kMerges;
  static constexpr int kIssued = kMergeR + 8 * kMerges; // int [stages]: position last issued
  static constexpr int kAbort = (kIssued + 4 * kStages + 7) & ~7;
  static constexpr int kScan = kAbort + 8;              // long long [33]
  // (a stage's tiles then belong to one warp of a piece for all: it has seen the
  // one before land when it waits for the next)
  static_assert(kStages * kParts % kWarps == 0, "stages");
  static constexpr int kStart = (kScan + 33 * 8 + 15) & ~15;  // int4
  static constexpr int kBytes = kStart + 16;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kCtas * (kAlloc + 1024) <= 228 * 1024, "shared memory of an SM");
};

// Which key of a 32-key tile is column n (0..7) of score tile j (0..3), and
// where its bytes lie.  TMA stores 128-byte rows with the 16-byte chunks of
// row y XORed by y & 7.  A K read takes, over eight lanes (n = 2i, 2i+1; four
// chunks each), a V read columns 2t of four t and two (d = 128) adjacent
// chunks: both touch all 32 banks once for the row orders 0 2 5 7 (even
// columns) and 4 6 1 3 (odd), as rows 2i and 2i+1 differ in bit 2 and the four
// rows of a V read in bits 1-2.  At d = 64 a row holds two keys, the columns
// 2i and 2i+1, and the two orders belong to score tiles 2j and 2j+1.
template <int D>
__device__ __forceinline__ int tok(int j, int n) {
  if constexpr (D == 128) {
    return 8 * j + ((0x37156240u >> (4 * n)) & 7u);
  } else {
    const uint32_t rows = (j & 1) ? 0x3164u : 0x7520u;
    return 16 * (j >> 1) + 2 * static_cast<int>((rows >> (4 * (n >> 1))) & 7u) + (n & 1);
  }
}
// Byte offset of 16-byte chunk c of key `t`.
template <int D>
__device__ __forceinline__ uint32_t code_at(int t, int c) {
  const int row = D == 128 ? t : t >> 1;
  const int ch = D == 128 ? c : (t & 1) * 4 + c;
  return static_cast<uint32_t>(row * 128 + ((ch ^ (row & 7)) << 4));
}

// Waits for a phase until the time `end` at most, whether or not the CTA is
// giving up: for copies in flight that must not outlive it.
__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity, uint64_t end) {
  while (!mbar_try_wait(bar, parity) && globaltimer_ns() < end) {
  }
}

// Waits until ring position p has been issued.  A barrier's parity tells only
// the phase before from the one after: a warp that knows of a tile more than
// one round of the ring before the tile is issued would take the phase of two
// rounds ago for its own.
__device__ __forceinline__ bool issue_wait(uint32_t tag, int p, const WaitCtx& w, unsigned site) {
  uint64_t t0 = 0;
  for (uint32_t it = 0;; ++it) {
    int v;
    asm volatile("ld.acquire.cta.shared.s32 %0, [%1];" : "=r"(v) : "r"(tag) : "memory");
    if (v == p) return true;
    if (it == 0) t0 = globaltimer_ns();
    if ((it & 31u) == 31u) {
      if (*w.cta_abort) return false;
      if (globaltimer_ns() - t0 > w.timeout_ns) {
        if (atomicCAS(&w.err->code, 0u, 1u) == 0u) {
          w.err->site = site;
          w.err->block = blockIdx.x;
          w.err->tile = p;
          __threadfence();
        }
        *w.cta_abort = 1;
        return false;
      }
    }
  }
}
__device__ __forceinline__ void issue_mark(uint32_t tag, int p) {
  asm volatile("st.release.cta.shared.s32 [%0], %1;" ::"r"(tag), "r"(p) : "memory");
}

// True in one thread of the (converged) warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// Four E4M3 codes to two pairs of f16 (exact).
__device__ __forceinline__ void e4m3_to_f16(uint32_t c, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(c));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Largest value over the lanes that hold one row's keys: a quad where the rows
// come first in the score product, else the eight lanes of equal t4.
template <bool WIDE>
__device__ __forceinline__ float row_max(float x) {
  if constexpr (WIDE) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
  } else {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
  }
}

// The 8 x 8 matrix of 16-bit elements that a warp holds (lane l: row l / 4,
// elements 2 (l % 4), + 1), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// floor(log2 x) of a normal positive x (smaller ones: -127).
__device__ __forceinline__ float floor_log2(float x) {
  return static_cast<float>(static_cast<int>((__float_as_uint(x) >> 23) & 0xffu) - 127);
}

// The power of two just below a row's largest |element| (as fp32 bits), kept
// where both it and its reciprocal are normal.
__device__ __forceinline__ int row_exponent(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 23) - 127;
  return max(-120, min(120, e));
}
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

}  // namespace dec

struct CacheFwdArgs {
  const __nv_bfloat16* q;  // [T][Hq][D] with a token stride
  long long q_stride;
  const float* ks;         // [blocks][Hkv]
  const float* vs;
  const uint8_t* data;     // 4 bits: [blocks][Hkv][P / 16][18 D]
  const int* table;        // [R][M]
  const int* seq_lens;     // [R]
  const int* cu_q;         // [R + 1]
  const long long* slot_map;  // [T] or null
  __nv_bfloat16* o;        // [T][Hq][D]
  float* lse;              // [T][Hq]
  float* part_o;           // [2 grid][rows][D]
  float* part_l;           // [2 grid][rows], log2 units
  int4* desc;              // [grid]: the unit begun and not finished by each CTA: its request's
                           // first query row (-1: none), kv head, row tile, rows
  int* cont;               // [grid]: 1, 2: holds (the end of) a unit begun before it
  int R, T, Hq, Hkv, g, sh, M, blocks, causal;
  float scale_log2;        // scale * log2(e) / k_unit
  float k_unit;            // a power of two that K's scales are multiplied by
  float v_unit;            // 4 bits: what V's values are multiplied by
  DevError* err;
  DevError* index_err;
  unsigned long long timeout_ns;
};

namespace dec {

// A block's scales lie in 0 .. 2^120: the two kernels would take others differently,
// and the K scale times k_unit has to be finite.  What is larger, infinity, NaN and
// what has a sign are the bit patterns behind 2^120's (0 with a sign is made one
// without).
constexpr uint32_t kBadScale = ((120u + 127u) << 23) + 1u;
__device__ __forceinline__ uint32_t scale_bits(float x) { return __float_as_uint(x + 0.f); }

struct Req {
  int c0, n, len, nrt, kt;
};
// A request's rows and keys, with what is out of range cut off.
template <int ROWS, int KEYS>
__device__ __forceinline__ Req request(const CacheFwdArgs& a, int r) {
  Req q;
  const int c0 = a.cu_q[r], c1 = a.cu_q[r + 1], len = a.seq_lens[r];
  q.c0 = max(0, min(a.T, c0));
  q.n = max(0, min(a.T, c1) - q.c0);
  const long long cap = static_cast<long long>(a.M) << a.sh;
  q.len = static_cast<int>(max(0ll, min(cap, static_cast<long long>(len))));
  q.nrt = static_cast<int>((static_cast<long long>(q.n) * a.g + ROWS - 1) / ROWS);
  q.kt = max(1, (q.len + KEYS - 1) / KEYS);
  return q;
}
// Keys that a request with rows is let see: none if its tokens got no slots.  (Its
// tiles are counted all the same: with the slots looked up wherever request() is,
// one short request took 11.1 us for 10.8, also without a slot map.)
__device__ __forceinline__ int keys_of(const CacheFwdArgs& a, const Req& q) {
  return a.slot_map && a.slot_map[q.c0] < 0 ? 0 : q.len;
}
// Reports what request() cuts off.
__device__ __forceinline__ void check_request(const CacheFwdArgs& a, int r) {
  const int len = a.seq_lens[r], c0 = a.cu_q[r], c1 = a.cu_q[r + 1];
  if (len < 0 || len > (static_cast<long long>(a.M) << a.sh)) record_index_error(a.index_err, kSiteFwdLen, r);
  if (c0 < 0 || c1 < c0 || c1 > a.T) record_index_error(a.index_err, kSiteFwdRows, r);
}
__device__ __forceinline__ long long cost_of(const CacheFwdArgs& a, const Req& q, int unit_cost) {
  return static_cast<long long>(a.Hkv) * q.nrt * (q.kt + unit_cost);
}

}  // namespace dec

template <int D, int ROWS, class F>
__global__ void __launch_bounds__(dec::Layout<D, ROWS, F>::kThreads, dec::ctas_per_sm(D, ROWS))
    fa_cache_fwd_kernel(const __grid_constant__ typename F::Maps maps, const __grid_constant__ CacheFwdArgs a) {
  using namespace dec;
  using Ly = Layout<D, ROWS, F>;
  constexpr int kRows = ROWS, kSegs = Ly::kSegs, kWarps = Ly::kWarps, kThreads = Ly::kThreads;
  constexpr int kTile = Ly::kTile, kParts = Ly::kParts, kUnitCost = Ly::kUnitCost, kMinCost = Ly::kMinCost;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  griddep_launch_dependents();  // the merge's CTAs may line up; they wait for this grid
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + Ly::kAbort);
  Seg* segs = reinterpret_cast<Seg*>(sm + Ly::kSeg);
  float4* s_scales = reinterpret_cast<float4*>(sm + Ly::kScales);
  int4* s_blk = reinterpret_cast<int4*>(sm + Ly::kBlk);
  int* s_in = reinterpret_cast<int*>(sm + Ly::kScales);  // 4 bits
  if (warp == kWarps) {
    for (int i = lane; i < Ly::kStages; i += 32) {
      mbar_init(base + Ly::kFull + 8 * i, F::k4 ? 1 : 2);  // its loads, and its scales
      mbar_init(base + Ly::kEmpty + 8 * i, kParts);
      issue_mark(base + Ly::kIssued + 4 * i, -1);
    }
    if (lane < kSegs) {
      mbar_init(base + Ly::kSegFull + 8 * lane, 1);
      mbar_init(base + Ly::kSegEmpty + 8 * lane, kWarps);
    }
    if (lane < Ly::kMerges) {
      const int n = lane < Ly::kSmalls ? Ly::kSmall : lane < Ly::kMerges - 1 ? Ly::kMiddle : kWarps;
      mbar_init(base + Ly::kMergeW + 8 * lane, n);
      mbar_init(base + Ly::kMergeR + 8 * lane, n);
    }
    fence_mbar_init();
    if (lane == 0) {
      *abort_flag = 0;
      if constexpr (!F::k4) {
        prefetch_tensormap(&maps.k);
        prefetch_tensormap(&maps.v);
      }
      a.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
      a.cont[blockIdx.x] = 0;
    }
  }

  // This CTA's range of the total cost: its length, and the request, kv head,
  // row tile and place in it that it starts at.  A small batch is summed by the
  // producer alone, a large one by the whole CTA.
  long long left = 0;
  int4 at = make_int4(0, 0, 0, 0);
  auto range = [&](long long total, long long& x0, long long& len) {
    const long long want = (total + kMinCost - 1) / kMinCost;
    const int parts = static_cast<int>(min(static_cast<long long>(gridDim.x), max(1ll, want)));
    const int c = min(static_cast<int>(blockIdx.x), parts);
    x0 = total * c / parts;
    len = c < parts ? total * (c + 1) / parts - x0 : 0;
  };
  auto place = [&](int r, long long in) {
    const Req q = request<kRows, kTile>(a, r);
    const int unit = q.kt + kUnitCost;
    const int u = static_cast<int>(in / unit);
    return make_int4(r, u / q.nrt, u % q.nrt, static_cast<int>(in - static_cast<long long>(u) * unit));
  };
  if (a.R <= kWarpScan) {
    if (warp == kWarps) {
      long long c[kWarpScan / 32], total = 0;
#pragma unroll
      for (int i = 0; i < kWarpScan / 32; ++i) {
        const int r = i * 32 + lane;
        c[i] = 0;
        if (r < a.R) {
          c[i] = cost_of(a, request<kRows, kTile>(a, r), kUnitCost);
          if (blockIdx.x == 0) check_request(a, r);
        }
      }
#pragma unroll
      for (int i = 0; i < kWarpScan / 32; ++i) total += c[i];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
      long long x0;
      range(total, x0, left);
      if (left > 0) {
        long long before = 0;
        int found = -1;
        long long in = 0;
#pragma unroll
        for (int i = 0; i < kWarpScan / 32; ++i) {
          if (found < 0 && i * 32 < a.R) {
            long long incl = c[i];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const long long v = __shfl_up_sync(0xffffffffu, incl, o);
              if (lane >= o) incl += v;
            }
            incl += before;
            const uint32_t past = __ballot_sync(0xffffffffu, incl > x0);
            if (past) {
              const int l = __ffs(past) - 1;
              found = i * 32 + l;
              in = x0 - __shfl_sync(0xffffffffu, incl - c[i], l);
            }
            before = __shfl_sync(0xffffffffu, incl, 31);
          }
        }
        at = place(found, in);
      }
    }
    __syncthreads();
  } else {
    const int per = (a.R + kThreads - 1) / kThreads;
    const int ra = min(a.R, tid * per), rb = min(a.R, ra + per);
    long long mine = 0, total, x0;
    for (int r = ra; r < rb; ++r) {
      mine += cost_of(a, request<kRows, kTile>(a, r), kUnitCost);
      if (blockIdx.x == 0) check_request(a, r);
    }
    const long long before = cta_scan(mine, reinterpret_cast<long long*>(sm + Ly::kScan), total) - mine;
    range(total, x0, left);
    if (left > 0 && before <= x0 && x0 < before + mine) {
      long long x = before;
      int r = ra;
      for (;; ++r) {
        const long long c = cost_of(a, request<kRows, kTile>(a, r), kUnitCost);
        if (x0 < x + c) break;  // ends: this thread's requests hold x0
        x += c;
      }
      *reinterpret_cast<int4*>(sm + Ly::kStart) = place(r, x0 - x);
    }
    __syncthreads();
    at = *reinterpret_cast<const int4*>(sm + Ly::kStart);
  }
  const WaitCtx wc{abort_flag, a.err, a.timeout_ns};
  auto full = [&](int s) { return base + Ly::kFull + 8 * s; };
  auto empty = [&](int s) { return base + Ly::kEmpty + 8 * s; };

  if (warp == kWarps) {
    // ------------------------------------------------------------ producer
    int r = at.x, h = at.y, rt = at.z, y = at.w;  // the walk: unit, and place in its cost
    // tiles that a short piece leaves a warp: as many as the ring holds for
    // each, or one where there is too little work for all of them
    const int per_warp = left * kParts >= 40 ? Ly::kStages * kParts / kWarps : 1;
    int pos = 0, nseg = 0;  // ring positions used, pieces published
    int issued = 0;         // positions up to this lane's last load
    int next_warp = 0;      // first warp of the next piece
    int held = -1;          // first request of the 32 in the lanes' registers
    Req mineq{}, q{};
    const int P = 1 << a.sh;
    const int boxes = P < kTile ? kTile / P : 1;  // blocks of a tile
    // the piece whose tiles are being fetched
    int pr = 0, ph = 0, plen = 0, pt = 0, pend = 0;
    bool ok = true, fresh = true;  // fresh: the request's sizes are still to be looked up
    for (;;) {
      // 32 tiles: what is left of the piece, and further ones
      int fill = 0, mr = -1, mh = 0, mlen = 0, mt = 0;
      while (fill < 32) {
        if (pt == pend) {
          if (left <= 0) break;
          const int si = nseg % kSegs;
          if (nseg >= kSegs) {
            // a place for its descriptor; waited for only with no tile at hand,
            // as the pieces before may need those to end
            const uint32_t bar = base + Ly::kSegEmpty + 8 * si, ph_ = ((nseg / kSegs) - 1) & 1;
            if (fill > 0) {
              if (!__all_sync(0xffffffffu, mbar_test_wait(bar, ph_))) break;
            } else {
              ok = __all_sync(0xffffffffu, mbar_wait(bar, ph_, wc, kSiteSegEmpty, nseg));
              if (!ok) break;
            }
          }
          // the next piece: the walk goes on until one has tiles
          int t0 = 0, t1 = 0;
          while (left > 0) {
            if (fresh || rt >= q.nrt) {
              if (!fresh) {
                rt = 0;
                if (++h == a.Hkv) {
                  h = 0;
                  ++r;
                  fresh = true;
                }
              }
              if (fresh) {
                for (;; ++r) {  // ends: cost is left
                  if (held < 0 || r >= held + 32) {
                    held = r;
                    mineq = Req{};
                    if (r + lane < a.R) mineq = request<kRows, kTile>(a, r + lane);
                  }
                  q.c0 = __shfl_sync(0xffffffffu, mineq.c0, r - held);
                  q.n = __shfl_sync(0xffffffffu, mineq.n, r - held);
                  q.len = __shfl_sync(0xffffffffu, mineq.len, r - held);
                  q.nrt = __shfl_sync(0xffffffffu, mineq.nrt, r - held);
                  q.kt = __shfl_sync(0xffffffffu, mineq.kt, r - held);
                  if (q.nrt > 0) break;
                }
                fresh = false;
              }
            }
            const int take = static_cast<int>(min(static_cast<long long>(q.kt + kUnitCost - y), left));
            t0 = max(0, y - kUnitCost);
            t1 = max(0, y + take - kUnitCost);
            left -= take;
            y = 0;
            if (t1 > t0) break;
            if (left > 0) ++rt;  // a unit's cost is never cut before its first tile but at the end
          }
          if (t1 <= t0) break;
          pr = r;
          ph = h;
          plen = q.len;
          pt = t0;
          pend = t1;
          const int nv = min(kRows, q.n * a.g - rt * kRows);
          if (lane == 0) {
            const int nt = t1 - t0;
            const bool begins = t0 == 0, ends = t1 == q.kt;
            Seg* s = segs + si;
            int nw = 1;
            while (nw < kWarps && nw * per_warp < nt * kParts) nw = Ly::next_size(nw);
            const int w0 = nw == kWarps ? 0 : ((next_warp + nw - 1) / nw * nw) % kWarps;
            next_warp = (w0 + nw) % kWarps;
            s->r = r;
            s->h = h;
            s->row0 = rt * kRows;
            s->nv = nv;
            s->c0 = q.c0;
            s->n = q.n;
            s->len = keys_of(a, q);
            s->t0 = t0;
            s->nt = nt;
            s->mode = begins && ends ? 0 : 1;
            s->slot = 2 * blockIdx.x + (begins ? 1 : 0);
            s->base = pos + fill;
            s->w0 = w0;
            s->nw = nw;
            mbar_arrive_expect_tx(base + Ly::kSegFull + 8 * si, static_cast<uint32_t>(nv * D * 2));
            if (begins && !ends) a.desc[blockIdx.x] = make_int4(q.c0, h, rt, nv);
            if (!begins) a.cont[blockIdx.x] = ends ? 2 : 1;
          }
          __syncwarp();
          // its query rows: those of a token lie together
          if (lane < nv) {
            const int rr = rt * kRows + lane, tk = rr / a.g, in = rr - tk * a.g;
            if (lane == 0 || in == 0) {
              const int n = min(nv - lane, a.g - in);
              bulk_load_1d(base + Ly::kQ + (si * kRows + lane) * D * 2,
                           a.q + (q.c0 + tk) * a.q_stride + static_cast<long long>(h * a.g + in) * D,
                           static_cast<uint32_t>(n * D * 2), base + Ly::kSegFull + 8 * si);
            }
          }
          ++nseg;
          ++rt;
        }
        const int take = min(32 - fill, pend - pt);
        if (lane >= fill && lane < fill + take) {
          mr = pr;
          mh = ph;
          mlen = plen;
          mt = pt + lane - fill;
        }
        fill += take;
        pt += take;
      }
      if (fill == 0) break;
      // their blocks and scales, a lane each, then the loads, by some lanes
      int blk[2 * kParts];
#pragma unroll
      for (int i = 0; i < 2 * kParts; ++i) blk[i] = -1;
      if (mr >= 0) {
        const int* row = a.table + static_cast<long long>(mr) * a.M;
#pragma unroll
        for (int i = 0; i < 2 * kParts; ++i) {
          const int key = mt * kTile + i * (F::k4 ? P : 16);
          if (i < boxes && key < mlen) {
            blk[i] = row[key >> a.sh];
            if (blk[i] < 0 || blk[i] >= a.blocks) {
              record_index_error(a.index_err, kSiteFwdBlock, mr);
              blk[i] = -1;
            } else {
              blk[i] = blk[i] * a.Hkv + mh;
            }
          }
        }
        const int in = (mt * kTile) & (P - 1);  // its place in the block
        if constexpr (F::k4) {
          int valid = 0;  // of its four granules
#pragma unroll
          for (int i = 0; i < 4; ++i) valid |= blk[boxes == 1 ? 0 : boxes == 2 ? i >> 1 : i] >= 0 ? 1 << i : 0;
          s_blk[(pos + lane) % Ly::kMeta] = make_int4(blk[0], blk[1], blk[2], blk[3]);
          s_in[(pos + lane) % Ly::kMeta] = in / c4::kTokens + 16 * valid;
        } else {
          const int valid = boxes == 1 ? (blk[0] >= 0 ? 3 : 0) : (blk[0] >= 0 ? 1 : 0) | (blk[1] >= 0 ? 2 : 0);
          s_blk[(pos + lane) % Ly::kMeta] = make_int4(blk[0], blk[1], in * D / 128, valid);
        }
      }
      // on their way while the loads are issued
      float ks[2] = {0.f, 0.f}, vs[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (!F::k4 && blk[i] >= 0) {
          ks[i] = __ldg(a.ks + blk[i]);
          vs[i] = __ldg(a.vs + blk[i]);
        }
      __syncwarp();
      // Several lanes issue the loads, each on a tile of its own: a load of 2
      // or 4 KB took 270 cycles from one lane, 105 from eight, and 73 from 32;
      // half the ring at most, as the lanes go on together.
      for (int i0 = 0; i0 < fill; i0 += Ly::kIssue) {
        const int p = pos + i0 + lane;
        if (lane < Ly::kIssue && i0 + lane < fill) {
          const int st = p % Ly::kStages, round = p / Ly::kStages;
          if (round > 0) ok = mbar_wait(empty(st), (round - 1) & 1, wc, kSiteStageEmpty, p);
          if (ok) {
            issued = p + 1;
            issue_mark(base + Ly::kIssued + 4 * st, p);
            const int4 bl = s_blk[p % Ly::kMeta];
            const uint32_t kb = base + st * Ly::kStage, vb = kb + Ly::kHalf;
            if constexpr (F::k4) {
              // four granules: together, or one or two of each of its blocks
              constexpr int kBytes = c4::Granule<D>::kBytes;
              const int each = min(P, kTile) / c4::kTokens, in = s_in[p % Ly::kMeta] & 15;
              const long long per = P / c4::kTokens;
              const int b[4] = {bl.x, bl.y, bl.z, bl.w};
              uint32_t n = 0;
#pragma unroll
              for (int i = 0; i < 4; ++i) n += i < boxes && b[i] >= 0 ? 1 : 0;
              mbar_arrive_expect_tx(full(st), n * each * kBytes);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (i < boxes && b[i] >= 0)
                  bulk_load_1d(kb + i * each * kBytes, a.data + (b[i] * per + in) * kBytes, each * kBytes, full(st));
            } else if (boxes == 1) {
              if (bl.x >= 0) {
                mbar_arrive_expect_tx(full(st), Ly::kStage);
                tma_load_3d(kb, &maps.k, full(st), 0, bl.z, bl.x);
                tma_load_3d(vb, &maps.v, full(st), 0, bl.z, bl.x);
              } else {
                mbar_arrive(full(st));
              }
            } else {
              const uint32_t nbox = (bl.x >= 0 ? 1u : 0u) + (bl.y >= 0 ? 1u : 0u);
              mbar_arrive_expect_tx(full(st), nbox * Ly::kHalf);
              if (bl.x >= 0) {
                tma_load_3d(kb, &maps.k, full(st), 0, 0, bl.x);
                tma_load_3d(vb, &maps.v, full(st), 0, 0, bl.x);
              }
              if (bl.y >= 0) {
                tma_load_3d(kb + Ly::kHalf / 2, &maps.k, full(st), 0, 0, bl.y);
                tma_load_3d(vb + Ly::kHalf / 2, &maps.v, full(st), 0, 0, bl.y);
              }
            }
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        // the scales of these tiles, by the lanes that have them
        if (!F::k4 && ok && lane >= i0 && lane < min(fill, i0 + Ly::kIssue)) {
          const int e = pos + lane;
          if (max(max(scale_bits(ks[0]), scale_bits(vs[0])), max(scale_bits(ks[1]), scale_bits(vs[1]))) >= kBadScale) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (max(scale_bits(ks[i]), scale_bits(vs[i])) >= kBadScale) {  // as if it had no block
                record_index_error(a.index_err, kSiteFwdScale, mr);
                ks[i] = vs[i] = 0.f;
                s_blk[e % Ly::kMeta].w &= boxes == 1 ? 0 : ~(1 << i);
              }
          }
          ks[0] *= a.k_unit;
          ks[1] *= a.k_unit;
          s_scales[e % Ly::kMeta] = boxes == 1 ? make_float4(ks[0], ks[0], vs[0], vs[0])
                                           : make_float4(ks[0], ks[1], vs[0], vs[1]);
          mbar_arrive(full(e % Ly::kStages));
        }
        if (!ok) break;
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      pos += fill;
    }
    // the end, also after a wait that gave up (the others then stop by the flag)
    if (ok) {
      const int si = nseg % kSegs;
      if (nseg >= kSegs)
        ok = mbar_wait(base + Ly::kSegEmpty + 8 * si, ((nseg / kSegs) - 1) & 1, wc, kSiteSegEmpty, nseg);
      if (lane == 0 && ok) {
        segs[si].nt = 0;
        mbar_arrive(base + Ly::kSegFull + 8 * si);
      }
    }
    // every load issued has landed before this warp exits, also where the
    // consumers gave up
    issued = __reduce_max_sync(0xffffffffu, issued);
    if (lane == 0) {
      const uint64_t end = globaltimer_ns() + a.timeout_ns;
      for (int p = max(0, issued - Ly::kStages); p < issued; ++p)
        mbar_drain(full(p % Ly::kStages), (p / Ly::kStages) & 1, end);
      for (int n = max(0, nseg - kSegs); n < nseg; ++n)
        if (n % kSegs != nseg % kSegs || !ok)  // that one is the end's now
          mbar_drain(base + Ly::kSegFull + 8 * (n % kSegs), (n / kSegs) & 1, end);
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  constexpr int kK = D / 16;   // score products per 8 keys
  float* merge = reinterpret_cast<float*>(sm + Ly::kMerge);
  float4* stats = reinterpret_cast<float4*>(sm + Ly::kStats);
  // Merges of this warp's small, middle and whole group: bits 0-2 are the phase of the
  // next; bits 3-5 tell which of the three the last one was, if any.
  uint32_t merges = 0;
  auto unit = [&](float x) { return F::k4 ? x * a.v_unit : x; };
  // Where output row `row` of piece s goes, as a row of [T][Hq].
  auto out_row = [&](const Seg& s, int row) {
    const int rr = s.row0 + row, tk = rr / a.g;
    return static_cast<long long>(s.c0 + tk) * a.Hq + s.h * a.g + (rr - tk * a.g);
  };
  for (int ns = 0;; ++ns) {
    const int si = ns % kSegs;
    bool ok = mbar_wait(base + Ly::kSegFull + 8 * si, (ns / kSegs) & 1, wc, kSiteSegFull, ns);
    if (!__all_sync(0xffffffffu, ok)) return;
    const Seg& s = segs[si];
    if (s.nt == 0) return;
    const int w0 = s.w0, nw = s.nw;
    if (warp < w0 || warp >= w0 + nw) {  // not this warp's
      if (lane == 0) mbar_arrive(base + Ly::kSegEmpty + 8 * si);
      continue;
    }

    // the lane's place in the products; opaque where two CTAs share the
    // registers, so that offsets made from it are not kept between pieces
    int ln = lane;
    if constexpr (Ly::kCtas == 2) asm volatile("" : "+r"(ln));
    const int g4 = ln >> 2, t4 = ln & 3;
    // ROWS = 16: S = Q K^T and O = P V with the 16 query rows first; a lane
    //   holds rows g4, g4 + 8 and columns (2 t4 + e) D/8 + i in o[i][2 y + e].
    // ROWS = 8: S^T = K Q^T and O^T = V^T P^T, 16 keys or columns first and the
    //   8 rows second, half the products; a lane holds rows 2 t4 + y and columns
    //   g4 D/8 + i in o[i / 2][2 (i & 1) + y].
    constexpr bool kWide = ROWS == 16;
    constexpr int kO = kWide ? D / 8 : D / 16;
    float o[kO][4];
    float m[2] = {kInit, kInit}, E[2] = {0.f, 0.f}, l[2] = {0.f, 0.f};  // E: the second reference less m
    const bool busy = warp - w0 < s.nt * kParts;
    auto row_of = [&](int y) { return kWide ? g4 + 8 * y : 2 * t4 + y; };  // a lane's two rows
    if (busy) {
#pragma unroll
      for (int i = 0; i < kO; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
      // Q rows g4 (and g4 + 8) in operand layout: product kk takes, in lane
      // t4, the four elements 4 (kk % 4) .. + 3 of chunk t4 + 4 (kk / 4)
      constexpr int kY = kWide ? 2 : 1;
      uint32_t qa[kK][2 * kY];
      float c[2];     // scale of the scores of each row
      int lim[2];     // keys visible to it
#pragma unroll
      for (int y = 0; y < kY; ++y) {
        const bool real = g4 + 8 * y < s.nv;
        const uint32_t src = base + Ly::kQ + (si * kRows + g4 + 8 * y) * D * 2 + t4 * 32;
        uint4 w[D / 32];  // 2 vectors of 8 per chunk
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
          w[e] = lds128(src + (e >> 1) * 128 + (e & 1) * 16);
          if (!real) w[e] = make_uint4(0u, 0u, 0u, 0u);
        }
        uint32_t am = 0;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) am = amax2(w[e].x, amax2(w[e].y, amax2(w[e].z, amax2(w[e].w, am))));
        am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
        am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
        const int ex = row_exponent(am << 16);
        const float inv = pow2i(-ex);
        c[y] = a.scale_log2 * pow2i(ex);
#pragma unroll
        for (int kk = 0; kk < kK; ++kk) {
          const uint4 v = w[2 * (kk >> 2) + ((kk & 3) >> 1)];
          const uint32_t p0 = (kk & 1) ? v.z : v.x, p1 = (kk & 1) ? v.w : v.y;
          qa[kk][y] = pack_f16(__uint_as_float(p0 << 16) * inv, __uint_as_float(p0 & 0xffff0000u) * inv);
          qa[kk][kY + y] = pack_f16(__uint_as_float(p1 << 16) * inv, __uint_as_float(p1 & 0xffff0000u) * inv);
        }
      }
      if constexpr (!kWide) {
        const float mine = c[0];
        c[0] = __shfl_sync(0xffffffffu, mine, 8 * t4);
        c[1] = __shfl_sync(0xffffffffu, mine, 8 * t4 + 4);
      }
#pragma unroll
      for (int y = 0; y < 2; ++y)
        lim[y] = row_of(y) >= s.nv ? 0 : (a.causal ? min(s.len, s.len - s.n + (s.row0 + row_of(y)) / a.g + 1) : s.len);
      // keys visible to every real row of the tile
      const int all = a.causal ? min(s.len, s.len - s.n + s.row0 / a.g + 1) : s.len;

      for (int k = warp - w0; k < s.nt * kParts; k += nw) {
        const int p = s.base + k / kParts, part = k % kParts, st = p % Ly::kStages;
        // the piece's first round: the stage may be further behind than a phase
        ok = k >= Ly::kStages * kParts || issue_wait(base + Ly::kIssued + 4 * st, p, wc, kSiteIssued);
        ok = ok && mbar_wait(full(st), (p / Ly::kStages) & 1, wc, kSiteStageFull, p);
        if (!__all_sync(0xffffffffu, ok)) break;
        const int key0 = s.t0 * kTile + k * kKeys;
        if (F::k4 && key0 >= s.len) {  // none of its keys
          if (lane == 0) mbar_arrive(empty(st));
          continue;
        }
        const uint32_t kb = base + st * Ly::kStage + part * Ly::kPart, vb = kb + Ly::kHalf;
        const float4 sc = F::k4 ? make_float4(a.k_unit, a.k_unit, 1.f, 1.f) : s_scales[p % Ly::kMeta];
        // bit i: the 16-key group i has a block
        const int valid = F::k4 ? (s_in[p % Ly::kMeta] >> (4 + 2 * part)) & 3 : s_blk[p % Ly::kMeta].w;
        const bool careful = key0 + kKeys > all || valid != 3;
        // scores in log2 units, x[z][..] of row y: of key column(z, y)'s token
        // wide: tiles of 8 keys z = 0..3, [2 y + e], key 2 t4 + e of the tile;
        // else: groups of 16 keys z = 0, 1, [2 e + y], key g4 of tile 2 z + e
        constexpr int kZ = kWide ? 4 : 2;
        float x[kZ][4];
#pragma unroll
        for (int z = 0; z < kZ; ++z)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[z][e] = 0.f;
        auto at = [](int y, int e) { return kWide ? 2 * y + e : 2 * e + y; };
        // columns of score tiles: of 4 bits, the keys as they come
        auto key_of = [](int j, int n) { return F::k4 ? 8 * j + n : tok<D>(j, n); };
        auto token = [&](int z, int e) { return kWide ? key_of(z, 2 * t4 + e) : key_of(2 * z + e, g4); };
        // two score tiles at a time: chains of dependent products side by side
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          if constexpr (F::k4) {
            using G = c4::Granule<D>;
            const uint32_t gr = kb + (j >> 1) * G::kBytes;
            uint32_t w[2][D / 32], f[2][D / 64];  // codes; scales of the lane's groups, twice each
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int t = g4 + 8 * y;
              if constexpr (D == 128) {
                const uint4 v = lds128(gr + t * G::kRow + t4 * 16);
                w[y][0] = v.x; w[y][1] = v.y; w[y][2] = v.z; w[y][3] = v.w;
                const uint32_t both = c4::e4m3x2_to_f16(lds16(gr + G::kKScales + t * 8 + t4 * 2));
                f[y][0] = __byte_perm(both, 0u, 0x1010);
                f[y][1] = __byte_perm(both, 0u, 0x3232);
              } else {
                const uint2 v = lds64(gr + t * G::kRow + t4 * 8);
                w[y][0] = v.x; w[y][1] = v.y;
                f[y][0] = __byte_perm(c4::e4m3x2_to_f16(lds8(gr + G::kKScales + t * 4 + t4)), 0u, 0x1010);
              }
            }
#pragma unroll
            for (int e = 0; e < kK; e += 2) {
              uint32_t b[2][4];
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                c4::e2m1_to_f16(w[y][e / 2], b[y][0], b[y][1], b[y][2], b[y][3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) b[y][i] = c4::mul_f16x2(b[y][i], f[y][e / 4]);
              }
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                if constexpr (kWide) {
                  mma16816(x[j], qa[e + i], b[0][2 * i], b[0][2 * i + 1]);
                  mma16816(x[j + 1], qa[e + i], b[1][2 * i], b[1][2 * i + 1]);
                } else {
                  const uint32_t ka[4] = {b[0][2 * i], b[1][2 * i], b[0][2 * i + 1], b[1][2 * i + 1]};
                  mma16816(x[j / 2], ka, qa[e + i][0], qa[e + i][1]);
                }
              }
            }
          } else {
            uint32_t w[2][D / 16];
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const int t = tok<D>(j + f, g4);
#pragma unroll
              for (int hc = 0; hc < D / 64; ++hc) {
                const uint4 v = lds128(kb + code_at<D>(t, t4 + 4 * hc));
                w[f][4 * hc] = v.x;
                w[f][4 * hc + 1] = v.y;
                w[f][4 * hc + 2] = v.z;
                w[f][4 * hc + 3] = v.w;
              }
            }
#pragma unroll
            for (int e = 0; e < kK; ++e) {
              uint32_t b[2][2];
              e4m3_to_f16(w[0][e], b[0][0], b[0][1]);
              e4m3_to_f16(w[1][e], b[1][0], b[1][1]);
              if constexpr (kWide) {
                mma16816(x[j], qa[e], b[0][0], b[0][1]);
                mma16816(x[j + 1], qa[e], b[1][0], b[1][1]);
              } else {
                const uint32_t ka[4] = {b[0][0], b[1][0], b[0][1], b[1][1]};
                mma16816(x[j / 2], ka, qa[e][0], qa[e][1]);
              }
            }
          }
        }
#pragma unroll
        for (int z = 0; z < kZ; ++z)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float f = c[y] * (z < kZ / 2 ? sc.x : sc.y);
#pragma unroll
            for (int e = 0; e < 2; ++e) x[z][at(y, e)] *= f;
          }
        if (careful) {
#pragma unroll
          for (int z = 0; z < kZ; ++z)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int t = token(z, e);
              const bool there = (valid >> (t >> 4)) & 1;
#pragma unroll
              for (int y = 0; y < 2; ++y)
                if (!there || key0 + t >= lim[y]) x[z][at(y, e)] = -INFINITY;
            }
        }
        // weights, as f16 operands of the product with V
        uint32_t pa[2][4];
        auto weigh = [&](auto value) {  // of scores x[z] of row y: 2^(x - m), and what it counts in l
#pragma unroll
          for (int z = 0; z < kZ; ++z) {
            float p[2][2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
#pragma unroll
              for (int e = 0; e < 2; ++e) p[y][e] = x[z][at(y, e)] - m[y];
              l[y] += value(z < kZ / 2 ? 0 : 1, y, p[y]);
            }
            if constexpr (kWide) {
              pa[z >> 1][2 * (z & 1)] = pack_f16(p[0][0], p[0][1]);
              pa[z >> 1][2 * (z & 1) + 1] = pack_f16(p[1][0], p[1][1]);
            } else {
              // key g4, rows 2 t4, 2 t4 + 1 -> row g4, keys 2 t4, 2 t4 + 1
              pa[z][0] = transpose8(pack_f16(p[0][0], p[1][0]));
              pa[z][1] = transpose8(pack_f16(p[0][1], p[1][1]));
            }
          }
        };
        if constexpr (F::k4) {
          // one reference: no value is more than 2^18 times another's step
          float up[2];
          bool grew = false;
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float top = x[0][at(y, 0)];
#pragma unroll
            for (int z = 0; z < kZ; ++z) top = fmax3(top, x[z][at(y, 0)], x[z][at(y, 1)]);
            const float m1 = fmaxf(m[y], row_max<kWide>(top));
            up[y] = ex2(m[y] - m1);
            l[y] *= up[y];
            grew = grew || up[y] != 1.f;
            m[y] = m1;
          }
          if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
            for (int i = 0; i < kO; ++i)
#pragma unroll
              for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int e = 0; e < 2; ++e) o[i][at(y, e)] *= up[y];
          }
          weigh([&](int, int, float (&p)[2]) {
#pragma unroll
            for (int e = 0; e < 2; ++e) p[e] = ex2(p[e]);
            const float sum = p[0] + p[1];
#pragma unroll
            for (int e = 0; e < 2; ++e) p[e] *= 16384.f;
            return sum;
          });
        } else {
          float gm[2][2];  // largest score of each row in each group of 16 keys
#pragma unroll
          for (int gr = 0; gr < 2; ++gr)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              gm[gr][y] = fmaxf(x[gr * (kZ / 2)][at(y, 0)], x[gr * (kZ / 2)][at(y, 1)]);
              if constexpr (kWide) gm[gr][y] = fmaxf(gm[gr][y], fmaxf(x[2 * gr + 1][at(y, 0)], x[2 * gr + 1][at(y, 1)]));
            }
          // over the lanes that hold a row's keys; of both groups together where
          // they have one scale
          const bool same = sc.z == sc.w;
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            if (same) {
              gm[0][y] = gm[1][y] = row_max<kWide>(fmaxf(gm[0][y], gm[1][y]));
            } else {
              gm[0][y] = row_max<kWide>(gm[0][y]);
              gm[1][y] = row_max<kWide>(gm[1][y]);
            }
          }
          const float lv[2] = {floor_log2(sc.z), floor_log2(sc.w)};
          float wgt[2][2], up[2];
          bool grew = false, apart = false;
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float m1 = fmaxf(m[y], fmaxf(gm[0][y], gm[1][y])), dm = m[y] - m1;
            const float E1 = fmaxf(E[y] + dm, fmaxf(gm[0][y] - m1 + lv[0], gm[1][y] - m1 + lv[1]));
            l[y] *= ex2(dm);
            up[y] = ex2(E[y] + dm - E1);
            grew = grew || up[y] != 1.f;
            m[y] = m1;
            E[y] = E1;
            apart = apart || E1 < fmaxf(fmaxf(lv[0], lv[1]) - 86.f, -106.f);
            const float f = ex2(14.f - E1);
            wgt[0][y] = f * sc.z;
            wgt[1][y] = f * sc.w;
          }
          if (__any_sync(0xffffffffu, grew || apart)) {
            apart = __any_sync(0xffffffffu, apart);
#pragma unroll
            for (int i = 0; i < kO; ++i)
#pragma unroll
              for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int e = 0; e < 2; ++e) o[i][at(y, e)] *= up[y];
          }
          if (!apart) {
            weigh([&](int gr, int y, float (&p)[2]) {
#pragma unroll
              for (int e = 0; e < 2; ++e) p[e] = ex2(p[e]);
              const float sum = p[0] + p[1];
#pragma unroll
              for (int e = 0; e < 2; ++e) p[e] *= wgt[gr][y];
              return sum;
            });
          } else {
            // A group whose V scale is 2^86 or more above 2^E: its weights' factor
            // may leave fp32's range, and so may the exponentials, which only
            // together are below 2^15.  What the factor has above 2^100 goes into
            // their arguments.  (The scales are read again: held until here, they
            // would not fit in the registers of two CTAs.)
            weigh([&](int gr, int y, float (&v)[2]) {
              const float4 again = s_scales[p % Ly::kMeta];
              const float size = gr == 0 ? again.z : again.w, lv = floor_log2(size);
              const float a = 14.f - E[y] + lv, over = fmaxf(a - 100.f, 0.f);
              // size / 2^lv; lv is -127 for 0 and what lies below the normal numbers
              const uint32_t mantissa = (__float_as_uint(size) & 0x7fffffu) | 0x3f800000u;
              const float w = ex2(a - over) * (lv == -127.f ? size * 0x1p127f : __uint_as_float(mantissa));
#pragma unroll
              for (int e = 0; e < 2; ++e) v[e] = ex2(v[e] + over);
              const float sum = (v[0] + v[1]) * ex2(-over);
#pragma unroll
              for (int e = 0; e < 2; ++e) v[e] *= w;
              return sum;
            });
          }
        }
        // O += P V: lane g4 takes output columns g4 D/8 .. of the keys 2 t4, 2 t4 + 1
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          if constexpr (F::k4) {
            using G = c4::Granule<D>;
            const uint32_t gr = kb + ks * G::kBytes;
            const int flip = D == 128 ? g4 & 1 : (g4 >> 1) & 1;
            // piece g4 of tokens 2 t4, 2 t4 + 1 and of those + 8
            const uint32_t v0 = gr + G::kV + g4 * D + ((t4 * 2) ^ (flip * 8)) * G::kPiece, v1 = v0 ^ (8 * G::kPiece);
            uint32_t w[4][D / 64 == 2 ? 2 : 1];
            if constexpr (D == 128) {
              const uint4 c = lds128(v0), d = lds128(v1);
              w[0][0] = c.x; w[0][1] = c.y; w[1][0] = c.z; w[1][1] = c.w;
              w[2][0] = d.x; w[2][1] = d.y; w[3][0] = d.z; w[3][1] = d.w;
            } else {
              const uint2 c = lds64(v0), d = lds64(v1);
              w[0][0] = c.x; w[1][0] = c.y; w[2][0] = d.x; w[3][0] = d.y;
            }
            uint32_t f = lds32(gr + G::kVScales + (D == 128 ? g4 : g4 >> 1) * 16 + t4 * 4);
            if (careful) {  // what lies behind the last token may be anything, a scale that is no number too
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (key0 + 16 * ks + 2 * t4 + (e & 1) + 8 * (e >> 1) >= s.len || !((valid >> ks) & 1))
                  f &= ~(0xffu << (8 * e));
            }
            const uint32_t f0 = c4::e4m3x2_to_f16(f), f1 = c4::e4m3x2_to_f16(f >> 16);
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
              // codes of two tokens side by side: even elements, then odd ones
              constexpr uint32_t kLow = 0x0f0f0f0fu;
              uint32_t b0[8], b1[8];
              auto pairs = [&](uint32_t u, uint32_t v, uint32_t f, uint32_t (&b)[8]) {
                c4::e2m1_to_f16((u & kLow) | ((v << 4) & ~kLow), b[0], b[2], b[4], b[6]);
                c4::e2m1_to_f16(((u >> 4) & kLow) | (v & ~kLow), b[1], b[3], b[5], b[7]);
#pragma unroll
                for (int e = 0; e < 8; ++e) b[e] = c4::mul_f16x2(b[e], f);
              };
              pairs(w[0][i], w[1][i], f0, b0);
              pairs(w[2][i], w[3][i], f1, b1);
              if constexpr (kWide) {
#pragma unroll
                for (int e = 0; e < 8; ++e) mma16816(o[8 * i + e], pa[ks], b0[e], b1[e]);
              } else {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                  const uint32_t va[4] = {b0[e], b0[e + 1], b1[e], b1[e + 1]};
                  mma16816(o[4 * i + e / 2], va, pa[ks][0], pa[ks][1]);
                }
              }
            }
          } else {
            constexpr int kW = D / 32;
            uint32_t w[4][kW];  // keys: score tile 2 ks (even, odd column), 2 ks + 1
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int t = tok<D>(2 * ks + (e >> 1), 2 * t4 + (e & 1));
              if constexpr (kW == 4) {
                const uint4 v = lds128(vb + code_at<D>(t, g4));
                w[e][0] = v.x; w[e][1] = v.y; w[e][2] = v.z; w[e][3] = v.w;
              } else {
                const uint2 v = lds64(vb + code_at<D>(t, g4 >> 1) + (g4 & 1) * 8);
                w[e][0] = v.x; w[e][1] = v.y;
              }
              // what lies behind the last token may be anything, NaN too
              if (careful && (key0 + t >= s.len || !((valid >> (t >> 4)) & 1))) {
#pragma unroll
                for (int f = 0; f < kW; ++f) w[e][f] = 0u;
              }
            }
#pragma unroll
            for (int f = 0; f < kW; ++f) {
              uint32_t b0[4], b1[4];
              e4m3_to_f16(__byte_perm(w[0][f], w[1][f], 0x5140), b0[0], b0[1]);
              e4m3_to_f16(__byte_perm(w[0][f], w[1][f], 0x7362), b0[2], b0[3]);
              e4m3_to_f16(__byte_perm(w[2][f], w[3][f], 0x5140), b1[0], b1[1]);
              e4m3_to_f16(__byte_perm(w[2][f], w[3][f], 0x7362), b1[2], b1[3]);
              if constexpr (kWide) {
#pragma unroll
                for (int e = 0; e < 4; ++e) mma16816(o[4 * f + e], pa[ks], b0[e], b1[e]);
              } else {
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                  const uint32_t va[4] = {b0[e], b0[e + 1], b1[e], b1[e + 1]};
                  mma16816(o[2 * f + e / 2], va, pa[ks][0], pa[ks][1]);
                }
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty(st));
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        if constexpr (kWide) {
          l[y] += __shfl_xor_sync(0xffffffffu, l[y], 1);
          l[y] += __shfl_xor_sync(0xffffffffu, l[y], 2);
        } else {
          l[y] += __shfl_xor_sync(0xffffffffu, l[y], 4);
          l[y] += __shfl_xor_sync(0xffffffffu, l[y], 8);
          l[y] += __shfl_xor_sync(0xffffffffu, l[y], 16);
        }
      }
    }
    // column i of the lane's run `e` (wide: two runs a row) of row y
    auto out = [&](int y, int e, int i) { return kWide ? o[i % kO][2 * y + e] : o[(i / 2) % kO][2 * (i & 1) + y]; };
    auto run_at = [&](int e) { return (kWide ? 2 * t4 + e : g4) * (D / 8); };  // its first column
    constexpr int kRuns = kWide ? 2 : 1;
    const bool first = kWide ? t4 == 0 : g4 == 0;  // the lane that writes a row's statistics


    if (nw == 1) {  // nothing to merge
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int row = row_of(y);
        if (row < s.nv) {
          // a row without a visible key: O = 0, L = -inf
          const float fin = l[y] == 0.f ? 0.f : unit(ex2(E[y] - 14.f) / l[y]);
          const float lg = l[y] == 0.f ? -INFINITY : m[y] + log2f(l[y]);
          const long long to = s.mode == 0 ? out_row(s, row) : static_cast<long long>(s.slot) * kRows + row;
#pragma unroll
          for (int e = 0; e < kRuns; ++e) {
            const long long col = to * D + run_at(e);
#pragma unroll
            for (int i = 0; i < D / 8; i += 8) {
              float f[8];
#pragma unroll
              for (int z = 0; z < 8; ++z) f[z] = out(y, e, i + z) * fin;
              if (s.mode == 0) {
                *reinterpret_cast<uint4*>(a.o + col + i) = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                                                      pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
              } else {
                *reinterpret_cast<float4*>(a.part_o + col + i) = make_float4(f[0], f[1], f[2], f[3]);
                *reinterpret_cast<float4*>(a.part_o + col + i + 4) = make_float4(f[4], f[5], f[6], f[7]);
              }
            }
          }
          if (first) {
            if (s.mode == 0) a.lse[to] = lg * 0.6931471805599453f;
            else a.part_l[to] = lg;
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(base + Ly::kSegEmpty + 8 * si);
      continue;
    }

    // merge of its warps, eight rows at a time
    const uint32_t kind = Ly::kind_of(nw);
    const int bar = Ly::merge_bar(warp, kind);
    const int active = min(nw, s.nt * kParts);
    // 16-byte chunks are XORed so that the eight lanes of a store fall on
    // different banks
    auto chunk_at = [](int row, int ch) {
      int sw;
      if constexpr (kWide) sw = D == 128 ? ((ch >> 3) & 3) | ((row & 1) << 2) : ((ch >> 3) & 1) | ((row & 1) << 1);
      else sw = D == 128 ? (row >> 1) & 3 : ((row & 2) << 1) | ((row >> 2) & 1);
      return ch ^ sw;
    };
#pragma unroll
    for (int y = 0; y < ROWS / 8; ++y) {
      if (8 * y >= s.nv) break;
      // this warp's buffer is free once the last merge that it was part of,
      // of whatever size, has been read
      if (merges >> 3) {
        const uint32_t last = merges >> 3;  // its phase is the one before that size's next
        ok = mbar_wait(base + Ly::kMergeR + Ly::merge_bar(warp, last), (merges & last) ? 0 : 1, wc, kSiteMergeR, ns);
        if (!__all_sync(0xffffffffu, ok)) return;
      }
      const uint32_t use = (merges & kind) ? 1 : 0;
      merges = ((merges & 7) ^ kind) | kind << 3;
      if (busy) {
#pragma unroll
        for (int z = 0; z < 2 / (ROWS / 8); ++z) {  // wide: row g4 of this pass, else both rows
          const int yy = kWide ? y : z, row = kWide ? g4 : 2 * t4 + z;
          if (8 * y + row < s.nv) {
            float* mw = merge + (warp * 8 + row) * D;
#pragma unroll
            for (int e = 0; e < kRuns; ++e)
#pragma unroll
              for (int i = 0; i < D / 8; i += 4) {
                const int ch = (run_at(e) + i) >> 2;
                *reinterpret_cast<float4*>(mw + 4 * chunk_at(row, ch)) =
                    make_float4(out(yy, e, i), out(yy, e, i + 1), out(yy, e, i + 2), out(yy, e, i + 3));
              }
            if (first) stats[warp * 8 + row] = make_float4(m[yy], l[yy], E[yy], 0.f);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(base + Ly::kMergeW + bar);
      ok = mbar_wait(base + Ly::kMergeW + bar, use, wc, kSiteMergeW, ns);
      if (!__all_sync(0xffffffffu, ok)) return;
      const int rows = min(8, s.nv - 8 * y);
      for (int it = (warp - w0) * 32 + lane; it < rows * (D / 4); it += 32 * nw) {
        const int row = it / (D / 4), ch = it % (D / 4);
        float4 q[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
          q[w] = w < active ? stats[(w0 + w) * 8 + row] : make_float4(kInit, 0.f, 0.f, 0.f);
        float M = kInit, Em = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, q[w].x);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          q[w].z = w < active ? q[w].z + (q[w].x - M) : -INFINITY;
          Em = fmaxf(Em, q[w].z);
        }
        float L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          if (w < active) {
            const float f = ex2(q[w].z - Em);
            const float4 v = *reinterpret_cast<const float4*>(merge + ((w0 + w) * 8 + row) * D + 4 * chunk_at(row, ch));
            L += q[w].y * ex2(q[w].x - M);
            acc.x += f * v.x;
            acc.y += f * v.y;
            acc.z += f * v.z;
            acc.w += f * v.w;
          }
        }
        // a row without a visible key: O = 0, L = -inf
        const float fin = L == 0.f ? 0.f : unit(ex2(Em - 14.f) / L);
        const float lg = L == 0.f ? -INFINITY : M + log2f(L);
        acc.x *= fin;
        acc.y *= fin;
        acc.z *= fin;
        acc.w *= fin;
        if (s.mode == 0) {
          const long long to = out_row(s, row + 8 * y);
          *reinterpret_cast<uint2*>(a.o + to * D + 4 * ch) =
              make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
          if (ch == 0) a.lse[to] = lg * 0.6931471805599453f;
        } else {
          const long long to = static_cast<long long>(s.slot) * kRows + row + 8 * y;
          *reinterpret_cast<float4*>(a.part_o + to * D + 4 * ch) = acc;
          if (ch == 0) a.part_l[to] = lg;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(base + Ly::kMergeR + bar);
    }
    if (lane == 0) mbar_arrive(base + Ly::kSegEmpty + 8 * si);
  }
}

// Merges the partials of each unit that more than one CTA worked on, in CTA
// order: L = log2 sum 2^(L_s), O = sum 2^(L_s - L) O_s.  One CTA (or more, in
// y, for large units) per CTA of the forward: it takes the unit that one began
// and did not finish.  Each warp looks up the parts itself, 32 CTAs at a time,
// and four parts are loaded together: two rounds of loads behind the wait, where
// a list in shared memory took five and 1.5 to 2 us more.
template <int D, int ROWS, class F>
__global__ void __launch_bounds__(512) fa_cache_merge_kernel(const __grid_constant__ CacheFwdArgs a, int grid) {
  const int c = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  griddep_wait();
  const int4 d = a.desc[c];
  const int mark0 = c + 1 + lane < grid ? a.cont[c + 1 + lane] : 0;
  if (d.x < 0) return;
  for (int it0 = blockIdx.y * 512 + (tid & ~31); it0 < d.w * (D / 4); it0 += 512 * gridDim.y) {
    const int it = min(it0 + lane, d.w * (D / 4) - 1);  // (a warp's last lanes may do its last item again)
    const int row = it / (D / 4), ch = it % (D / 4);
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    // the part that was begun here, then those behind up to the one that ends:
    // CTAs in between may have had nothing to do
    int first = c, mark = mark0;
    uint32_t own = 1u;
    for (bool more = true; more;) {
      const uint32_t end = __ballot_sync(0xffffffffu, mark == 2);
      uint32_t parts = __ballot_sync(0xffffffffu, mark != 0);
      if (end) parts &= (end & (0u - end)) * 2u - 1u;  // up to the first that ends
      more = end == 0u && first + 33 < grid;
      while (own | parts) {
        float l[4];
        float4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          l[i] = -INFINITY;
          v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          int slot = -1;
          if (own) {
            slot = 2 * c + 1;
            own = 0u;
          } else if (parts) {
            slot = 2 * (first + __ffs(parts));
            parts &= parts - 1u;
          }
          if (slot >= 0) {
            const long long p = static_cast<long long>(slot) * ROWS + row;
            l[i] = a.part_l[p];
            v[i] = *reinterpret_cast<const float4*>(a.part_o + p * D + 4 * ch);
          }
        }
        const float m = fmaxf(fmaxf(M, fmaxf(l[0], l[1])), fmaxf(l[2], l[3]));
        if (m == -INFINITY) continue;  // rows without a visible key so far
        const float f = ex2(M - m);
        M = m;
        L *= f;
        acc.x *= f;
        acc.y *= f;
        acc.z *= f;
        acc.w *= f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float g = ex2(l[i] - m);
          L += g;
          acc.x += g * v[i].x;
          acc.y += g * v[i].y;
          acc.z += g * v[i].z;
          acc.w += g * v[i].w;
        }
      }
      first += 32;
      mark = more && first + 1 + lane < grid ? a.cont[first + 1 + lane] : 0;
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const int rr = d.z * ROWS + row, tk = rr / a.g;
    const long long to = static_cast<long long>(d.x + tk) * a.Hq + d.y * a.g + (rr - tk * a.g);
    *reinterpret_cast<uint2*>(a.o + to * D + 4 * ch) =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    if (ch == 0) a.lse[to] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
  }
}

}  // namespace fa
