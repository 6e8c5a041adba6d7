// Attention over the 4-bit key/value cache, many query rows per kv head
// (prompts, chunks of them): bound by the tensor cores.
//
// Units, the cut into ranges, tensor memory, the halves A and B and the loop of
// scores, softmax and weights are those of the 8-bit cache's kernel
// (fa_cache_prompt.cuh), with other operands: a value, code times scale, is exact
// in f16 and in nothing shorter, so both products are f16's, and K and V are
// both made in shared memory by four warps, from granules that one bulk copy
// per block brings.  A score product takes 16 of the head dimension and as
// long as one of 32 in 8 bits (either reads 6 KB of shared memory), and as the
// queries were two 8-bit parts there, S costs the same.
//
// Everything turns by steps of 64 keys: rings of three for granules, K and V.
//
// Softmax: one reference m, the weights 2^(10 + s - m), moved only when a
// step exceeds it by more than 4, so that they stay below 2^15.
//
// Prompts of 1500 to 4096 tokens of 3 requests behind up to 10000, 32 heads on 8 of
// 128, take 1227 us, 1.22 PFLOP/s (8 bits: 1129).  A step of 64 keys takes 1840
// cycles: the loop is that of the 8-bit kernel, and of shared memory's time K's
// values, written and read as f16, take 250 more: 1350 of the 1840 in all.
#pragma once
#include <cuda_bf16.h>

#include "fa_cache4.cuh"
#include "fa_cache_prompt.cuh"

namespace fa {

namespace prm4 {

using prm::kBias;
using prm::kHalf;
using prm::kInit;
using prm::kKeys;
using prm::kLazy;
using prm::kRows;
using prm::kSegs;
using prm::kStepKeys;
using prm::kThreads;
constexpr int kRing = 3;    // steps of granules, K, V
// Steps whose keys' presence is held: a step is loaded at most kRing granules,
// kRing of K and two scores before the softmax takes it.
constexpr int kSeen = 16;

enum : unsigned { kSiteSegFull = 541, kSiteSegEmpty = 542, kSiteQFull = 543, kSiteQEmpty = 544, kSiteKFull = 545,
                  kSiteKEmpty = 546, kSiteVFull = 547, kSiteVEmpty = 548, kSiteS = 549, kSiteP = 550, kSitePV = 551,
                  kSiteSeen = 552, kSiteRawFull = 553, kSiteRawEmpty = 554, kSiteJoin = 555 };

template <int D>
struct Layout {
  static constexpr int kBlocks = D / 64;                // 64-element column blocks of a row
  static constexpr int kQHalf = kHalf * D * 2;          // f16 rows of a half, block by block
  static constexpr int kTile = kStepKeys * D * 2;       // K or V of a step, f16
  static constexpr int kBlock = kStepKeys * 128;        // a column block of it
  static constexpr int kGranules = kStepKeys / c4::kTokens;
  static constexpr int kRawStep = kGranules * c4::Granule<D>::kBytes;
  static constexpr int kStagedPart = 64 * D * 2;        // bf16 rows of Q
  static constexpr int kQ = 0;
  static constexpr int kK = 2 * kQHalf;                 // [ring]
  static constexpr int kV = kK + kRing * kTile;         // [ring]
  static constexpr int kStaged = kV + kRing * kTile;    // [2]
  static constexpr int kScan = kStaged;                 // before the first: long long [33]
  static constexpr int kRaw = kStaged + 2 * kStagedPart;  // [ring]
  static constexpr int kRowScale = kRaw + kRing * kRawStep;  // float [256]
  static constexpr int kSeenAt = kRowScale + kRows * 4;      // int [seen]: bit i: granule i of the step is there
  static constexpr int kStat = kSeenAt + kSeen * 4;          // float4 [2][128]: a row's statistics, of either half
  static constexpr int kSeg = kStat + 2 * kHalf * 16;
  static constexpr int kBar = (kSeg + kSegs * static_cast<int>(sizeof(dec::Seg)) + 15) & ~15;
  static constexpr int kSegFull = kBar;
  static constexpr int kSegEmpty = kSegFull + 8 * kSegs;
  static constexpr int kQFull = kSegEmpty + 8 * kSegs;
  static constexpr int kQEmpty = kQFull + 8;
  static constexpr int kKFull = kQEmpty + 8;            // [ring] each
  static constexpr int kKEmpty = kKFull + 8 * kRing;
  static constexpr int kVFull = kKEmpty + 8 * kRing;
  static constexpr int kVEmpty = kVFull + 8 * kRing;
  static constexpr int kRawFull = kVEmpty + 8 * kRing;
  static constexpr int kRawEmpty = kRawFull + 8 * kRing;
  static constexpr int kSeenBar = kRawEmpty + 8 * kRing;  // [seen]
  static constexpr int kSFull = kSeenBar + 8 * kSeen;     // [2] A, B [2] score buffers
  static constexpr int kPFull = kSFull + 32;              // [2][2]
  static constexpr int kPvDone = kPFull + 32;             // [2][2]
  static constexpr int kJoin = kPvDone + 32;              // [4] pairs of softmax warps
  static constexpr int kFin = kJoin + 32;
  static constexpr int kTmemSlot = kFin + 16;
  static constexpr int kAbort = kTmemSlot + 8;
  static constexpr int kStart = (kAbort + 8 + 15) & ~15;  // int4
  static constexpr int kBytes = kStart + 16;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kAlloc <= 227 * 1024, "shared memory of a CTA");
};

// Eight codes times f (a scale twice) to 16 bytes of f16.
__device__ __forceinline__ uint4 values8(uint32_t w, uint32_t f) {
  uint4 r;
  c4::e2m1_to_f16(w, r.x, r.y, r.z, r.w);
  return make_uint4(c4::mul_f16x2(r.x, f), c4::mul_f16x2(r.y, f), c4::mul_f16x2(r.z, f), c4::mul_f16x2(r.w, f));
}
__device__ __forceinline__ uint32_t low_twice(uint32_t w) { return __byte_perm(w, 0u, 0x1010); }
__device__ __forceinline__ uint32_t high_twice(uint32_t w) { return __byte_perm(w, 0u, 0x3232); }

// A unit's end for a softmax thread and its row: the halves' sums joined where
// both have the same rows, O and L written, or left as a partial.  (Written into
// the kernel instead, prompts took 1265 us for 1227; the 8-bit kernel the other way
// about.)
template <int D, typename W>
__device__ __forceinline__ bool finish(const CacheFwdArgs& a, const dec::Seg& s, int x, int row, int warp, int lane,
                                       float m, float l, uint32_t tO, float4* stat, uint32_t joined,
                                       W&& wait) {
  const bool two = s.nv > kHalf;
  const bool real = row < s.nv;
  // The halves' statistics, through shared memory; then each of the two
  // warps that have a row combines and writes one half of its columns.
  const bool join = !two && s.base > 1;
  float f = 1.f, f2 = 0.f;  // what this half's sums and the other's count
  if (join) {
    const uint32_t bar = joined + 8 * (warp & 3);
    stat[x * kHalf + row] = make_float4(m, l, 0.f, 0.f);
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
    if (!__all_sync(0xffffffffu, wait(bar, 0))) return false;
    tc_fence_after();
    const float4 b = stat[(1 - x) * kHalf + row];
    const float m1 = fmaxf(m, b.x);
    f = ex2(m - m1);
    f2 = ex2(b.x - m1);
    l = l * f + b.y * f2;
    m = m1;
  }
  const float inv = l == 0.f ? 0.f : ex2(-kBias) / l * a.v_unit;
  const float lg = l == 0.f ? -INFINITY : m + log2f(l);
  f *= inv;
  f2 *= inv;
  const int rr = s.row0 + row, tk = rr / a.g;
  const long long at = static_cast<long long>(s.c0 + tk) * a.Hq + s.h * a.g + (rr - tk * a.g);
  const long long pat = static_cast<long long>(s.slot) * kRows + row;
#pragma unroll 1
  for (int q = join ? x * (D / 64) : 0; q < (join && x == 0 ? D / 64 : D / 32); ++q) {
    uint32_t o[32];
    tmem_ld32(tO + 32 * q, o);
    tmem_ld_wait32(o);
#pragma unroll
    for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
    if (join) {
      uint32_t o2[32];
      tmem_ld32(tO + (kHalf - 2 * x * kHalf) + 32 * q, o2);
      tmem_ld_wait32(o2);
#pragma unroll
      for (int y = 0; y < 32; ++y)
        o[y] = __float_as_uint(fmaf(__uint_as_float(o2[y]), f2, __uint_as_float(o[y])));
    }
    if (real) {
      if (s.mode == 0) {
        uint4* dst = reinterpret_cast<uint4*>(a.o + at * D + 32 * q);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          dst[e] = make_uint4(
              pack_bf16(__uint_as_float(o[8 * e]), __uint_as_float(o[8 * e + 1])),
              pack_bf16(__uint_as_float(o[8 * e + 2]), __uint_as_float(o[8 * e + 3])),
              pack_bf16(__uint_as_float(o[8 * e + 4]), __uint_as_float(o[8 * e + 5])),
              pack_bf16(__uint_as_float(o[8 * e + 6]), __uint_as_float(o[8 * e + 7])));
      } else {
        // a row a lane: 32 bytes a store, as every row takes a pass of its own
#pragma unroll
        for (int e = 0; e < 32; e += 8) prm::stg256(a.part_o + pat * D + 32 * q + e, o + e);
      }
    }
  }
  if (real && (two || x == 0)) {
    if (s.mode == 0) a.lse[at] = lg * 0.6931471805599453f;
    else a.part_l[pat] = lg;
  }
  tc_fence_before();  // O has been read: the next piece's first product may overwrite it
  __syncwarp();
  if (join) {  // by the other warp, too
    if (lane == 0) mbar_arrive(joined + 8 * (warp & 3));
    if (!__all_sync(0xffffffffu, wait(joined + 8 * (warp & 3), 1))) return false;
  }
  return true;
}

}  // namespace prm4

template <int D>
__global__ void __launch_bounds__(prm4::kThreads, 1) fa_cache4_prompt_kernel(const __grid_constant__ CacheFwdArgs a) {
  using namespace prm4;
  using dec::Seg;
  using Ly = Layout<D>;
  using G = c4::Granule<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  griddep_launch_dependents();
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + Ly::kAbort);
  Seg* segs = reinterpret_cast<Seg*>(sm + Ly::kSeg);
  if (tid == 0) {
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(base + Ly::kSegFull + 8 * i, 1);
      mbar_init(base + Ly::kSegEmpty + 8 * i, 15);  // 8 softmax warps, 4 converters, 2 issuers, loader
    }
    mbar_init(base + Ly::kQFull, 4);
    mbar_init(base + Ly::kQEmpty, 10);  // both issuers' products, and each softmax warp's reads of the row scales
    for (int i = 0; i < kRing; ++i) {
      mbar_init(base + Ly::kKFull + 8 * i, 4);
      mbar_init(base + Ly::kKEmpty + 8 * i, 2);
      mbar_init(base + Ly::kVFull + 8 * i, 4);
      mbar_init(base + Ly::kVEmpty + 8 * i, 2);
      mbar_init(base + Ly::kRawFull + 8 * i, 1);
      mbar_init(base + Ly::kRawEmpty + 8 * i, 4);
    }
    for (int i = 0; i < kSeen; ++i) mbar_init(base + Ly::kSeenBar + 8 * i, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(base + Ly::kSFull + 8 * i, 1);
      mbar_init(base + Ly::kPFull + 8 * i, 4);
      mbar_init(base + Ly::kPvDone + 8 * i, 1);
      mbar_init(base + Ly::kJoin + 8 * i, 2);
    }
    mbar_init(base + Ly::kFin, 1);
    mbar_init(base + Ly::kFin + 8, 1);
    *abort_flag = 0;
    fence_mbar_init();
    a.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
    a.cont[blockIdx.x] = 0;
  }

  long long x0, x1;
  if (!prm::range_of(a, reinterpret_cast<long long*>(sm + Ly::kScan), reinterpret_cast<int4*>(sm + Ly::kStart), x0, x1))
    return;
  if (warp == 12) {
    tmem_alloc(base + Ly::kTmemSlot, 512);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + Ly::kTmemSlot);
  auto wait = [&](int at, uint32_t parity, unsigned site, int item) {
    return mbar_wait(base + at, parity & 1u, WaitCtx{abort_flag, a.err, a.timeout_ns}, site, item);
  };

  // Steps are counted over all pieces: step s has place s % kRing of the rings,
  // there for the (s / kRing)th time.
  if (warp >= 12) {
    prm::reg_dec<80>();
    if (warp == 13) {
      prm::walk(a, *reinterpret_cast<const int4*>(sm + Ly::kStart), x1 - x0, segs, base + Ly::kSegFull,
                base + Ly::kSegEmpty,
                [&](uint32_t bar, uint32_t parity, int item) { return wait(bar - base, parity, kSiteSegEmpty, item); });
    } else if (warp == 14) {
      // ------------------------------------------------------- the loader
      // A step's granules as they lie, one copy for those of a block.
      const int P = 1 << a.sh, unit = min(P, kStepKeys);  // tokens that lie together
      int step = 0;
      bool ok = true;
      for (int ns = 0;; ++ns) {
        const int si = ns % kSegs;
        ok = __all_sync(0xffffffffu, wait(Ly::kSegFull + 8 * si, ns / kSegs, kSiteSegFull, ns));
        if (!ok) break;
        const Seg& s = segs[si];
        const int nt = s.nt, h = s.h, len = s.len, key0 = s.t0 * kKeys, steps = s.base;
        if (nt == 0) break;
        const int* table = a.table + static_cast<long long>(s.r) * a.M;
        // block of this lane's granule (4 lanes) in step i; -1: none, -2: no keys
        auto block_of = [&](int i) {
          const int key = key0 + i * kStepKeys + lane * c4::kTokens;
          return lane < Ly::kGranules && i < steps && key < len ? max(-1, table[key >> a.sh]) : -2;
        };
        int next = block_of(0);
        for (int i = 0; i < steps; ++i, ++step) {
          const int b = next, st = step % kRing;
          next = block_of(i + 1);
          const bool real = b >= 0 && b < a.blocks;
          if (b != -2 && !real) record_index_error(a.index_err, kSiteFwdBlock, s.r);
          const uint32_t there = __ballot_sync(0xffffffffu, real);
          const bool issue = real && ((lane * c4::kTokens) & (unit - 1)) == 0;
          const uint32_t copies = __ballot_sync(0xffffffffu, issue);
          const uint32_t bytes = static_cast<uint32_t>(unit / c4::kTokens * G::kBytes);
          ok = step < kRing || wait(Ly::kRawEmpty + 8 * st, step / kRing - 1, kSiteRawEmpty, step);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) {
            reinterpret_cast<volatile int*>(sm + Ly::kSeenAt)[step % kSeen] = static_cast<int>(there);
            mbar_arrive(base + Ly::kSeenBar + 8 * (step % kSeen));
            mbar_arrive_expect_tx(base + Ly::kRawFull + 8 * st, __popc(copies) * bytes);
          }
          __syncwarp();
          if (issue) {
            const int in = ((key0 + i * kStepKeys + lane * c4::kTokens) & (P - 1)) / c4::kTokens;
            const long long at = (static_cast<long long>(b) * a.Hkv + h) * (P / c4::kTokens) + in;
            bulk_load_1d(base + Ly::kRaw + st * Ly::kRawStep + lane * G::kBytes, a.data + at * G::kBytes, bytes,
                         base + Ly::kRawFull + 8 * st);
          }
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(base + Ly::kSegEmpty + 8 * si);
      }
      // no copy outlives the CTA, also where a wait gave up
      if (lane == 0) {
        const uint64_t end = globaltimer_ns() + a.timeout_ns;
        for (int t = max(0, step - kRing); t < step; ++t)
          dec::mbar_drain(base + Ly::kRawFull + 8 * (t % kRing), (t / kRing) & 1, end);
      }
    } else {
      // ------------------------------------------------ the issuers, 12 and 15
      constexpr uint32_t idS = prm::idesc_f16_f32(kHalf, kStepKeys, false), idPV = prm::idesc_f16_f32(kHalf, D, true);
      constexpr uint32_t kHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // as fa_cache_prompt.cuh
      auto desc = [](uint32_t lo) { return (static_cast<uint64_t>(kHi) << 32) | lo; };
      auto low = [](uint32_t addr, uint32_t lbo) { return ((addr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16); };
      const int x = __shfl_sync(0xffffffffu, warp == 15 ? 1 : 0, 0);
      const uint32_t dS = tmem + prm::kColS + x * kHalf, dO = tmem + prm::kColO + x * kHalf;
      auto all_wait = [&](int at, uint32_t parity, unsigned site, int item) {
        return __all_sync(0xffffffffu, wait(at, parity, site, item)) != 0;
      };
      int step0 = 0, cnt = 0;  // the piece's first step, this half's steps
      for (int ns = 0;; ++ns) {
        const int si = ns % kSegs;
        if (!all_wait(Ly::kSegFull + 8 * si, ns / kSegs, kSiteSegFull, ns)) break;
        const int nt = __shfl_sync(0xffffffffu, segs[si].nt, 0), steps = __shfl_sync(0xffffffffu, segs[si].base, 0);
        const bool two = __shfl_sync(0xffffffffu, segs[si].nv, 0) > kHalf;
        if (nt == 0) break;
        // (Q is full: all steps of the pieces before are in the rings, so that
        // the waits below for K and V are one phase ahead at most)
        bool ok = all_wait(Ly::kQFull, ns, kSiteQFull, ns);
        // rows for both halves: each takes every step; else every other one,
        // with the same rows
        const int own = two ? steps : (steps + 1 - x) >> 1;
        const uint32_t q = low(base + Ly::kQ + (two ? x * Ly::kQHalf : 0), 16);
        auto step_of = [&](int k) { return step0 + (two ? k : 2 * k + x); };
        // a step's operand has been read by this half: by both, or alone
        auto freed = [&](uint32_t bar) {
          tc_commit(bar);
          if (!two) tc_commit(bar);
        };
        if (ok && own > 0 && cnt > 0)
          ok = all_wait(Ly::kPvDone + 8 * (2 * x + ((cnt - 1) & 1)), (cnt - 1) >> 1, kSitePV, step0);
        // i = -1: the first scores only
#pragma unroll 1
        for (int i = -1; ok && i < own; ++i) {
          const int n = i + 1;
          if (n < own) {
            const int g = step_of(n), st = g % kRing, buf = (cnt + n) & 1;
            ok = all_wait(Ly::kKFull + 8 * st, g / kRing, kSiteKFull, g);
            // the buffer's weights, of two steps before, have been multiplied
            if (ok && i >= 1) ok = all_wait(Ly::kPvDone + 8 * (2 * x + buf), (cnt + i - 1) >> 1, kSitePV, g);
            if (!ok) break;
            tc_fence_after();
            const uint32_t k = low(base + Ly::kK + st * Ly::kTile, 16);
            const uint32_t d = dS + buf * kStepKeys;
            if (dec::elect_one()) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)  // 16 elements of each row
                mma_ss(d, desc(q + (kk >> 2) * ((kHalf * 128) >> 4) + 2 * (kk & 3)),
                       desc(k + (kk >> 2) * (Ly::kBlock >> 4) + 2 * (kk & 3)), idS, kk > 0 ? 1u : 0u);
              tc_commit(base + Ly::kSFull + 8 * (2 * x + buf));
              freed(base + Ly::kKEmpty + 8 * st);
              if (n + 1 == own) tc_commit(base + Ly::kQEmpty);  // the last read of Q
            }
            __syncwarp();
          }
          if (i >= 0) {
            const int g = step_of(i), st = g % kRing, buf = (cnt + i) & 1;
            ok = all_wait(Ly::kVFull + 8 * st, g / kRing, kSiteVFull, g);
            if (ok) ok = all_wait(Ly::kPFull + 8 * (2 * x + buf), (cnt + i) >> 1, kSiteP, g);
            if (!ok) break;
            tc_fence_after();
            const uint32_t v = low(base + Ly::kV + st * Ly::kTile, Ly::kBlock);
            const uint32_t first = i == 0 ? 0u : 1u, p = dS + buf * kStepKeys;
            if (dec::elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kStepKeys / 16; ++kk)
                mma_ts(dO, p + 8 * kk, desc(v + static_cast<uint32_t>(kk * 128)), idPV, kk == 0 ? first : 1u);
              tc_commit(base + Ly::kPvDone + 8 * (2 * x + buf));
              freed(base + Ly::kVEmpty + 8 * st);
            }
            __syncwarp();
          }
        }
        if (!ok) break;
        if (own == 0 && lane == 0) mbar_arrive(base + Ly::kQEmpty);
        cnt += own;
        step0 += steps;
        if (lane == 0) mbar_arrive(base + Ly::kSegEmpty + 8 * si);
      }
      // nothing that reads shared or tensor memory outlives the CTA
      if (dec::elect_one()) {
        tc_commit(base + Ly::kFin + 8 * x);
        dec::mbar_drain(base + Ly::kFin + 8 * x, 0, globaltimer_ns() + a.timeout_ns);
      }
      __syncwarp();
    }
  } else if (warp >= 8) {
    prm::reg_dec<96>();
    // ------------------------------------- granules to K and V, queries to f16
    const int cw = warp - 8, ct = tid - 256;
    int step = 0;
    for (int ns = 0;; ++ns) {
      const int si = ns % kSegs;
      bool ok = wait(Ly::kSegFull + 8 * si, ns / kSegs, kSiteSegFull, ns);
      if (!__all_sync(0xffffffffu, ok)) break;
      const Seg& s = segs[si];
      if (s.nt == 0) break;
      const int steps = s.base, h = s.h;

      // Q, 64 rows at a time: the bf16 rows to the staging buffers, each to where
      // only the thread that copied it reads; then divided by the power of two of
      // the row's largest element and rounded to f16, with the next 64 on their way.
      {
        constexpr int kLanes = D / 8, kAt = 32 / kLanes;  // lanes per row (8 elements each), rows per warp
        constexpr int kEach = 64 / (4 * kAt);             // rows of a lane
        const int col = lane % kLanes, row_w = cw * kAt + lane / kLanes;
        const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
        const int nv = s.nv, chunks = nv > kHalf ? 4 : 2;
        const int tk0 = s.row0 / a.g, in0 = s.row0 - tk0 * a.g;
        const float per_g = 1.f / static_cast<float>(a.g);
        const __nv_bfloat16* q0 = a.q + (s.c0 + tk0) * a.q_stride + static_cast<long long>(h * a.g) * D + col * 8;
        auto copy = [&](int c) {
          if (c < chunks) {
#pragma unroll 4
            for (int i = 0; i < kEach; ++i) {
              const int row = c * 64 + row_w + i * 4 * kAt, y = in0 + row;
              // y / g, of y < g + 256
              const int tk = a.g > 256 ? (y >= a.g ? 1 : 0) : static_cast<int>((static_cast<float>(y) + 0.5f) * per_g);
              const bool real = row < nv;
              const long long at = real ? tk * a.q_stride + static_cast<long long>(y - tk * a.g) * D : 0;
              prm::copy16(base + Ly::kStaged + (c & 1) * Ly::kStagedPart + ct * 16 + i * 2048, q0 + at, real);
            }
          }
          prm::copies_end();
        };
        copy(0);
        copy(1);
        ok = ns == 0 || wait(Ly::kQEmpty, ns - 1, kSiteQEmpty, ns);
        ok = __all_sync(0xffffffffu, ok);
        for (int c = 0; ok && c < chunks; ++c) {
          prm::copies_but_last();
          const uint32_t from = base + Ly::kStaged + (c & 1) * Ly::kStagedPart + ct * 16;
          const uint32_t to = base + Ly::kQ + (c >> 1) * Ly::kQHalf + (col >> 3) * (kHalf * 128) + (c & 1) * (64 * 128) +
                              row_w * 128 + (((col & 7) ^ (row_w & 7)) << 4);
          float* row_scale = reinterpret_cast<float*>(sm + Ly::kRowScale) + c * 64 + row_w;
#pragma unroll 1
          for (int i0 = 0; i0 < kEach; i0 += 4) {
            uint4 w[4];
            uint32_t am[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = dec::lds128(from + (i0 + i) * 2048);
#pragma unroll
            for (int i = 0; i < 4; ++i) am[i] = amax2(w[i].x, amax2(w[i].y, amax2(w[i].z, amax2(w[i].w, 0u))));
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1)
#pragma unroll
              for (int i = 0; i < 4; ++i) am[i] = max(am[i], __shfl_xor_sync(0xffffffffu, am[i], o));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int ex = dec::row_exponent(am[i] << 16);
              const float inv = dec::pow2i(-ex);
              auto two = [&](uint32_t u) {
                return dec::pack_f16(rope::low(u ^ flip) * inv, rope::high(u ^ flip) * inv);
              };
              const int r = (i0 + i) * 4 * kAt;  // rows: multiples of 8 apart
              static_assert((4 * kAt) % 8 == 0, "the swizzle of a lane's rows");
              prm::sts128(to + r * 128, make_uint4(two(w[i].x), two(w[i].y), two(w[i].z), two(w[i].w)));
              if (col == 0) row_scale[r] = c * 64 + row_w + r < nv ? fabsf(a.scale_log2) * dec::pow2i(ex) : 0.f;
            }
          }
          copy(c + 2);
        }
        if (!ok) break;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(base + Ly::kQFull);

      const int len = s.len, key0 = s.t0 * kKeys;
      for (int i = 0; i < steps; ++i, ++step) {
        const int st = step % kRing;
        ok = wait(Ly::kRawFull + 8 * st, step / kRing, kSiteRawFull, step) &&
             (step < kRing || wait(Ly::kKEmpty + 8 * st, step / kRing - 1, kSiteKEmpty, step));
        if (!__all_sync(0xffffffffu, ok)) break;
        const uint32_t from = base + Ly::kRaw + st * Ly::kRawStep;
        // K: rows of a key, 16-element groups to two chunks each of its row,
        // XORed with the row's low bits
        {
          const uint32_t to = base + Ly::kK + st * Ly::kTile;
          if constexpr (D == 128) {  // groups t and t + 4: the same place in both column blocks
            const int t = ct & 3;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int key = (ct >> 2) + 32 * u;
              const uint32_t gr = from + (key >> 4) * G::kBytes;
              const uint4 c = dec::lds128(gr + (key & 15) * G::kRow + t * 16);
              const uint32_t f = c4::e4m3x2_to_f16(dec::lds16(gr + G::kKScales + (key & 15) * 8 + t * 2));
              const uint32_t f0 = low_twice(f), f1 = high_twice(f);
              const uint32_t at0 = to + key * 128 + (((2 * t) ^ (key & 7)) << 4), at1 = at0 ^ 16u;
              prm::sts128(at0, values8(c.x, f0));
              prm::sts128(at1, values8(c.y, f0));
              prm::sts128(at0 + Ly::kBlock, values8(c.z, f1));
              prm::sts128(at1 + Ly::kBlock, values8(c.w, f1));
            }
          } else {  // groups 2 u and 2 u + 1
            const int u = ct & 1, key = ct >> 1;
            const uint32_t gr = from + (key >> 4) * G::kBytes;
            const uint4 c = dec::lds128(gr + (key & 15) * G::kRow + u * 16);
            const uint32_t f = c4::e4m3x2_to_f16(dec::lds16(gr + G::kKScales + (key & 15) * 4 + u * 2));
            const uint32_t f0 = low_twice(f), f1 = high_twice(f), row = to + key * 128, sw = (key & 7) << 4;
            prm::sts128(row + ((u * 64) ^ sw), values8(c.x, f0));
            prm::sts128(row + ((u * 64 + 16) ^ sw), values8(c.y, f0));
            prm::sts128(row + ((u * 64 + 32) ^ sw), values8(c.z, f1));
            prm::sts128(row + ((u * 64 + 48) ^ sw), values8(c.w, f1));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(base + Ly::kKFull + 8 * st);
        ok = step < kRing || wait(Ly::kVEmpty + 8 * st, step / kRing - 1, kSiteVEmpty, step);
        if (!__all_sync(0xffffffffu, ok)) break;
        // V: pieces of several tokens; what no token lies in may be anything, a
        // scale that is no number too: it counts as 0
        {
          const uint32_t to = base + Ly::kV + st * Ly::kTile;
          const int there = reinterpret_cast<const volatile int*>(sm + Ly::kSeenAt)[step % kSeen];
          const int left = len - (key0 + i * kStepKeys);
          auto keys_there = [&](int g) { return (there >> g) & 1 ? left - 16 * g : 0; };
          if constexpr (D == 128) {
            // tokens 2 u, 2 u + 1 of piece p, group p: two chunks of a row in column
            // block p / 4, the lanes of the upper tokens the odd one first
            const int u = ct & 7, p = (ct >> 3) & 7, odd = u >> 2;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int g = (ct >> 6) + 2 * y;
              const uint32_t gr = from + g * G::kBytes;
              const uint4 c = dec::lds128(gr + G::kV + p * D + ((u * 16) ^ ((p & 1) * 64)));
              uint32_t s2 = dec::lds16(gr + G::kVScales + p * 16 + c4::scale_place(2 * u));
              const int n = keys_there(g) - 2 * u;
              if (n < 2) s2 &= n < 1 ? 0u : 0xffu;
              const uint32_t f = c4::e4m3x2_to_f16(s2);
              const uint32_t f0 = low_twice(f), f1 = high_twice(f);
              const int key = 16 * g + 2 * u;
              const uint32_t at0 = to + (p >> 2) * Ly::kBlock + key * 128 + (((2 * (p & 3) + odd) ^ (key & 7)) << 4);
              const uint32_t at1 = at0 ^ 16u;  // the other chunk; + 128, ^ 16 the next row's
              prm::sts128(at0, values8(odd ? c.y : c.x, f0));
              prm::sts128(at1, values8(odd ? c.x : c.y, f0));
              prm::sts128(at1 + 128, values8(odd ? c.w : c.z, f1));
              prm::sts128(at0 + 128, values8(odd ? c.z : c.w, f1));
            }
          } else {
            // tokens 4 u .. 4 u + 3 of piece p, a chunk of a row
            const int u = (ct & 1) + 2 * ((ct >> 3) & 1), p = ((ct >> 1) & 3) + 4 * ((ct >> 4) & 1), g = ct >> 5;
            const uint32_t gr = from + g * G::kBytes;
            const uint4 c = dec::lds128(gr + G::kV + p * D + ((u * 16) ^ (((p >> 1) & 1) * 32)));
            const uint32_t sc = gr + G::kVScales + (p >> 1) * 16 + c4::scale_place(4 * u);
            uint32_t s4 = dec::lds16(sc) | dec::lds16(sc + 4) << 16;
            const int n = keys_there(g) - 4 * u;
            if (n < 4) s4 = n < 1 ? 0u : s4 & (0xffffffffu >> (8 * (4 - n)));
            const uint32_t f = c4::e4m3x2_to_f16(s4), e = c4::e4m3x2_to_f16(s4 >> 16);
            const uint32_t w[4] = {c.x, c.y, c.z, c.w};
            const uint32_t fs[4] = {low_twice(f), high_twice(f), low_twice(e), high_twice(e)};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int key = 16 * g + 4 * u + j;
              prm::sts128(to + key * 128 + ((p ^ (key & 7)) << 4), values8(w[j], fs[j]));
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(base + Ly::kRawEmpty + 8 * st);
          mbar_arrive(base + Ly::kVFull + 8 * st);
        }
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      if (lane == 0) mbar_arrive(base + Ly::kSegEmpty + 8 * si);
    }
    prm::copies_done();  // none outlives the CTA, also where a wait gave up
  } else {
    prm::reg_inc<168>();
    // ------------------------------------------------ softmax and epilogue
    const int x = warp >> 2;  // half
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + prm::kColS + x * kHalf, tO = tmem + lane_off + prm::kColO + x * kHalf;
    int cnt = 0, step0 = 0;  // steps of this half, the piece's first step
    for (int ns = 0;; ++ns) {
      const int si = ns % kSegs;
      bool ok = wait(Ly::kSegFull + 8 * si, ns / kSegs, kSiteSegFull, ns);
      if (!__all_sync(0xffffffffu, ok)) break;
      const Seg& s = segs[si];
      if (s.nt == 0) break;
      const int steps = s.base;
      // Rows for both halves: each takes every step, of its own rows.  Else
      // both have the same rows, A the even steps and B the odd ones, and join
      // at the end.
      const bool two = s.nv > kHalf;
      const int own = two ? steps : (steps + 1 - x) >> 1;
      const int row = two ? tid : tid & (kHalf - 1);  // of the unit
      // no wait is left out for a piece without a step of this half: a phase
      // that a warp never saw could pass for a later one of the same parity
      ok = wait(Ly::kQFull, ns, kSiteQFull, ns);
      if (!__all_sync(0xffffffffu, ok)) break;
      // a score's factor; never 0, as masked scores stay -inf
      const float f = fmaxf(prm::lds_f32(base + Ly::kRowScale + 4 * row) * a.k_unit, prm::kTiny);
      __syncwarp();
      if (lane == 0) mbar_arrive(base + Ly::kQEmpty);
      if (own == 0) {
        step0 += steps;
        if (lane == 0) mbar_arrive(base + Ly::kSegEmpty + 8 * si);
        continue;
      }
      // keys visible to this row, and to every row of this warp
      const int lim = a.causal ? min(s.len, s.len - s.n + (s.row0 + row) / a.g + 1) : s.len;
      const int all = __reduce_min_sync(0xffffffffu, lim);
      float m = kInit, l = 0.f;
      bool far = false;
      for (int i = 0; i < own; ++i, ++cnt) {
        const int in = two ? i : 2 * i + x, step = step0 + in, buf = 2 * x + (cnt & 1);
        ok = wait(Ly::kSFull + 8 * buf, cnt >> 1, kSiteS, step) &&
             wait(Ly::kSeenBar + 8 * (step % kSeen), step / kSeen, kSiteSeen, step);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        const uint32_t tSb = tS + (cnt & 1) * kStepKeys;
        uint32_t v[2][32];
        float mx[2];  // of each 32 keys
        const int key0 = s.t0 * kKeys + in * kStepKeys;
        const int there = reinterpret_cast<const volatile int*>(sm + Ly::kSeenAt)[step % kSeen];
        const bool careful = key0 + kStepKeys > all || there != (1 << Ly::kGranules) - 1;
        tmem_ldred_max32(tSb, v[0], mx[0]);
        tmem_ldred_max32(tSb + 32, v[1], mx[1]);
        tmem_ldred_wait32(v[0], mx[0]);
        tmem_ldred_dep32(v[1], mx[1]);
        if (careful) {
          constexpr uint32_t kNegInf = 0xff800000u;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            // keys of the granule below this are visible
            const int end = (there >> y) & 1 ? lim - (key0 + 16 * y) : 0;
#pragma unroll
            for (int z = 0; z < 16; ++z)
              if (z >= end) v[y >> 1][(y & 1) * 16 + z] = kNegInf;
          }
          mx[0] = prm::max32(v[0], 0, 32);
          mx[1] = prm::max32(v[1], 0, 32);
        }
        const float mb = fmaxf(mx[0], mx[1]) * f;
        const bool bump = mb > m + kLazy;
        float up = 1.f;
        if (bump) {
          up = ex2(m - mb);
          l *= up;
          m = mb;
        }
        const bool moved = __any_sync(0xffffffffu, bump);
        // The exponent is one fused product and sum, whose product is not
        // rounded as m's was: above 2^17 (log2 units) that difference counts,
        // and the scores are reduced in two steps instead.
        if (moved) far = __any_sync(0xffffffffu, fabsf(m) > 131072.f && m != kInit);
        if (far) {
#pragma unroll
          for (int y = 0; y < 64; ++y) {
            uint32_t& w = v[y >> 5][y & 31];
            w = __float_as_uint(__fsub_rn(__fmul_rn(__uint_as_float(w), f), m));
          }
        }
        const float ff = far ? 1.f : f, nm = far ? kBias : kBias - m;
        const uint64_t f2 = f2_pack(ff, ff), n2 = f2_pack(nm, nm);
        uint64_t sum[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          uint32_t w[16];
#pragma unroll
          for (int y = 0; y < 32; y += 2) {
            float a0, a1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(v[ch][y]), __uint_as_float(v[ch][y + 1])), f2, n2), a0, a1);
            a0 = ex2(a0);
            a1 = ex2(a1);
            sum[(y >> 1) & 1] = f2_add(sum[(y >> 1) & 1], f2_pack(a0, a1));
            w[y >> 1] = dec::pack_f16(a0, a1);
          }
          tmem_st16(tSb + 16 * ch, w);
        }
        float s0, s1;
        f2_unpack(f2_add(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
        if (moved && i > 0) {  // O to the new reference, once it has every weight before
          ok = __all_sync(0xffffffffu, wait(Ly::kPvDone + 8 * (buf ^ 1), (cnt - 1) >> 1, kSitePV, step));
          tc_fence_after();
#pragma unroll 1
          for (int z = 0; z < D / 32; ++z) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * z, o);
            tmem_ld_wait32(o);
#pragma unroll
            for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * up);
            tmem_st32(tO + 32 * z, o);
          }
        }
        tmem_st_wait();
        if (!ok) break;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(base + Ly::kPFull + 8 * buf);
      }
      step0 += steps;
      if (!__all_sync(0xffffffffu, ok)) break;
      ok = wait(Ly::kPvDone + 8 * (2 * x + ((cnt - 1) & 1)), (cnt - 1) >> 1, kSitePV, step0);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      l *= 1.f / (1 << static_cast<int>(kBias));  // the sum of 2^(s - m)
      ok = finish<D>(
          a, s, x, row, warp, lane, m, l, tO, reinterpret_cast<float4*>(sm + Ly::kStat), base + Ly::kJoin,
          [&](uint32_t bar, uint32_t parity) { return wait(bar - base, parity, kSiteJoin, step0); });
      if (!__all_sync(0xffffffffu, ok)) break;
      if (lane == 0) mbar_arrive(base + Ly::kSegEmpty + 8 * si);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace fa
