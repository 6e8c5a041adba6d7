// Attention over the 8-bit key/value cache, many query rows per kv head
// (prompts, chunks of them): bound by the tensor cores.
//
// The rows of one (request, kv head), new tokens times the query heads that
// share the kv head, come in tiles of 256: two halves of 128 rows, A and B,
// each a single-SM tcgen05 tile with a softmax warpgroup of its own, over the
// same keys in tiles of 128.  As in the few-row kernel (fa_cache_fwd.cuh) the
// key tiles of all units, in order, are cut into one equal range per CTA, and
// units that more than one CTA works on leave partials for the merge; here
// a unit's number of key tiles follows its last row's position.
//
// Products.  S is taken in 8 bits: a query row, divided by a power of two of
// its own, is the sum of two E4M3 numbers per element, the rounded value and
// the rest (bf16 has 8 significant bits, E4M3 four: exact down to 2^-9 of the
// row's largest element, and off by at most 2^-17 of that below; exact in rows
// whose largest is below 2^-116), so that
//   S = Q_hi K^T + Q_lo K^T
// costs what one f16 product would, and K goes from the cache to the tensor
// cores as it is.  P stays f16, as two parts of it would cost the softmax more
// than they save; tcgen05 has no product of f16 with E4M3, so four warps turn
// V's codes into f16 (exact) on their way: bulk copies bring the next tiles'
// to buffers, as the blocks hold them, and these warps write them out in the
// 128-byte-swizzled layout of an MN-major operand.
//
// TMEM (512 columns): of each half two buffers of scores, fp32 [128][64], A at
// [0,128) and B at [128,256), P over the first half of each as f16 pairs; O of
// A [256,384) and of B [384,512).
// A key tile is two steps of 64 keys.  For each half one thread issues S(0),
// then for step i S(i+1) and PV(i): the scores of a step are made while the
// softmax does the one before, so that it never waits for its own weights to be
// multiplied.  (With steps of 128 keys and one buffer, scores, softmax and
// weights followed one another: 4100 cycles per tile and half, of which the
// softmax took 1800.)  S(i+1) takes the buffer of P(i-1) and waits until PV(i-1)
// is done: that the products of a thread run in order is promised for one
// accumulator only.  What happens once a step (scores made, weights written,
// weights multiplied) has a barrier for even and one for odd steps: a wait by
// parity tells one phase from the next, and those who skip some would be two
// behind on a single one.
//
// A unit with rows for A only (a few tokens, a prompt's end) gives both halves
// the same rows and alternate steps; at its end they join their sums, each warp
// reading both accumulators (drafts of 16 requests: 48.5 us with B idle, then 44.2;
// 38 now.  Times beside a choice are those of the kernel as it then was.)
//
// What bounds it: the loop from weights to the scores that take their buffer.
// Prompts of 1500 to 4096 tokens of 3 requests behind up to 10000, 32 heads on 8
// of 128, take 1129 us, 1.32 PFLOP/s of bf16's 1.92 (978 us with heads of 64).
// Of 1690 cycles a step of 64 keys, taken at 1116 us, the products of both halves
// take 1260 by themselves (S 48 cycles each, the time to read 6 KB of shared
// memory, where the sums take 32; PV 64), the softmax 1150 while both run.  But
// S(i+2) waits for PV(i): 512 cycles for both halves' PV, 270 to learn of it, 770
// for both S and 100 to learn of that are 1650.  A third score buffer does not fit
// tensor memory; halves kept half a step apart, taking turns at the softmax or at
// issuing, were slower (1140, 1300 and 1305 us).
//
// Warps: 0-3 softmax and epilogue of A, 4-7 of B, 8-11 codes to f16 (and Q),
// 12 and 15 issue A's and B's products, 13 walks the range, 14 loads.
//
// Softmax: as in the few-row kernel a row has two references, m for l = sum
// 2^(s - m) and E for the weights 2^(10 + s - E) v_scale of the product, both
// moved only when a tile exceeds one by more than 4 (so the weights stay below
// 2^15; O is rescaled then).  The exponentials give the weights directly,
// log2 v_scale being in their argument, and l takes each block's sum times
// the inverse of what its weights carry.
#pragma once
#include <cuda_bf16.h>

#include "fa_cache_fwd.cuh"
#include "sm103_ptx.cuh"
#include "tmem_ldst.cuh"

namespace fa {

namespace prm {

constexpr int kThreads = 512;
constexpr int kRows = 256;       // query rows of a unit
constexpr int kHalf = 128;
constexpr int kKeys = 128;       // keys of a tile
constexpr int kStepKeys = 64;    // of a step: scores, softmax, weights
constexpr int kSegs = 4;
constexpr int kUnitCost = 5;     // a piece's fixed cost, in tiles (3: 1140 us for prompts of 3 requests, 5: 1124)
constexpr int kMinCost = 6;      // least cost of a CTA's range
constexpr float kLazy = 4.f;     // log2 a reference may be exceeded by
constexpr float kBias = 10.f;    // log2 the weights are scaled by
using dec::kInit;
constexpr float kTiny = 1.17549435e-38f;
constexpr uint32_t kColS = 0, kColO = 256;  // + 128 for B

enum : unsigned { kSiteSegFull = 521, kSiteSegEmpty = 522, kSiteQFull = 523, kSiteQEmpty = 524, kSiteKFull = 525,
                  kSiteKEmpty = 526, kSiteVFull = 527, kSiteVEmpty = 528, kSiteS = 529, kSiteP = 530, kSitePV = 531,
                  kSiteScales = 532, kSiteRawFull = 533, kSiteRawEmpty = 534, kSiteJoin = 535 };

template <int D>
struct Layout {
  static constexpr int kPart = kHalf * 128;      // one half's rows, high or low parts (d = 64: half of each row used)
  static constexpr int kQHalf = 2 * kPart;
  static constexpr int kKTile = kKeys * 128;     // K codes, rows as for Q
  static constexpr int kVTile = kKeys * D * 2;   // V, f16
  static constexpr int kQ = 0;
  static constexpr int kK = 2 * kQHalf;          // [2]
  static constexpr int kV = kK + 2 * kKTile;     // [2]
  static constexpr int kRawTile = kKeys * D;                  // codes of a tile of V, as they lie
  static constexpr int kRaw = kV + 2 * kVTile;                // [3]
  static constexpr int kStaged = kRaw;                        // over two of them: bf16 rows of one half of Q
  static constexpr int kScan = kRaw + 2 * kRawTile;           // before the first: long long [33]
  static constexpr int kRowScale = kRaw + 3 * kRawTile;       // float [256]
  static_assert(kHalf * D * 2 == 2 * kRawTile, "the staged rows' place");
  static constexpr int kKs = kRowScale + kRows * 4;        // float [4][8]: K scale, -1: no block
  static constexpr int kLv = kKs + 4 * 8 * 4;                 // float [4][8]: log2 of the V scale
  static constexpr int kClean = kLv + 4 * 8 * 4;              // int [4]: every key of the tile is one to see
  static constexpr int kStat = kClean + 4 * 4;                // float4 [2][128]: a row's statistics, of either half
  static constexpr int kSeg = kStat + 2 * kHalf * 16;
  static constexpr int kBar = (kSeg + kSegs * static_cast<int>(sizeof(dec::Seg)) + 15) & ~15;
  static constexpr int kSegFull = kBar;
  static constexpr int kSegEmpty = kSegFull + 8 * kSegs;
  static constexpr int kQFull = kSegEmpty + 8 * kSegs;
  static constexpr int kQEmpty = kQFull + 8;
  static constexpr int kKFull = kQEmpty + 8;      // [2]
  static constexpr int kKEmpty = kKFull + 16;
  static constexpr int kVFull = kKEmpty + 16;
  static constexpr int kVEmpty = kVFull + 16;
  static constexpr int kSFull = kVEmpty + 16;     // [2] A, B [2] score buffers
  static constexpr int kPFull = kSFull + 32;      // [2][2]
  static constexpr int kPvDone = kPFull + 32;     // [2][2]
  static constexpr int kScales = kPvDone + 32;    // [4]
  static constexpr int kRawFull = kScales + 32;
  static constexpr int kRawEmpty = kRawFull + 24;
  static constexpr int kJoin = kRawEmpty + 24;    // [4] pairs of softmax warps
  static constexpr int kFin = kJoin + 32;
  static constexpr int kTmemSlot = kFin + 16;
  static constexpr int kAbort = kTmemSlot + 8;
  static constexpr int kStart = (kAbort + 8 + 15) & ~15;  // int4
  static constexpr int kBytes = kStart + 16;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kAlloc <= 227 * 1024, "shared memory of a CTA");
};

// F(n, m, a, b) = sum of floor((a i + b) / m) over i < n; n >= 0, m > 0, a, b >= 0.
// Two steps, taken in turn as in Euclid's algorithm (sums of floors as counts of
// lattice points: Graham, Knuth, Patashnik, Concrete Mathematics, 3.5):
//   the whole parts of a / m and b / m: F(n, m, a, b) =
//     floor(a / m) n (n - 1) / 2 + floor(b / m) n + F(n, m, a mod m, b mod m);
//   then, a, b < m, K = floor((a (n - 1) + b) / m) the last and largest term: for
//     each j < K the i with a term of j at most are the first
//     ceil(((j + 1) m - b) / a), and the others count one each, so that
//     F(n, m, a, b) = n K - F(K, a, m, a + m - b - 1).
// K < n and all of a step's values are at most the first's a n + b + m.
template <typename T>
__device__ __forceinline__ long long floor_sum_in(T n, T m, T a, T b) {
  long long sum = 0;
  for (bool minus = false; n > 0; minus = !minus) {
    const long long terms = n, whole = static_cast<long long>(a / m) * (terms * (terms - 1) / 2) + b / m * terms;
    a %= m;
    b %= m;
    const T last = (a * (n - 1) + b) / m;
    sum += minus ? -(whole + terms * last) : whole + terms * last;
    if (last == 0) break;
    const T from = a + m - b - 1, by = a;
    n = last;
    a = m;
    m = by;
    b = from;
  }
  return sum;
}
__device__ __noinline__ long long floor_sum(long long n, long long m, long long a, long long b) {
  // divisions of 64 bits take several times as long: a third of what a CTA
  // does before its first load
  if (a * n + b + m < (1ll << 31))
    return floor_sum_in<unsigned>(static_cast<unsigned>(n), static_cast<unsigned>(m), static_cast<unsigned>(a),
                                  static_cast<unsigned>(b));
  return floor_sum_in<long long>(n, m, a, b);
}

// Keys that the last row of row tile rt sees.
__device__ __forceinline__ int seen_of(const CacheFwdArgs& a, const dec::Req& q, int rt) {
  int seen = q.len;
  if (a.causal && q.n <= q.len) {
    const unsigned last = min(static_cast<unsigned>(rt) * kRows + kRows, static_cast<unsigned>(q.n) * a.g) - 1;
    seen = q.len - q.n + static_cast<int>(last / a.g) + 1;
  }
  return seen;
}
__device__ __forceinline__ int tiles_of(const CacheFwdArgs& a, const dec::Req& q, int rt) {
  return max(1, (seen_of(a, q, rt) + kKeys - 1) / kKeys);
}
// Cost of the row tiles before rt (< nrt): all of them full, so tile i sees
// base + floor((256 (i + 1) - 1) / g) + 1 keys, base = len - n, and has
// floor((256 i + 255 + g (base + 128)) / (128 g)) key tiles.
__device__ __forceinline__ long long cost_before(const CacheFwdArgs& a, const dec::Req& q, int rt) {
  if (!(a.causal && q.n <= q.len)) return static_cast<long long>(rt) * (tiles_of(a, q, 0) + kUnitCost);
  const long long base = q.len - q.n;
  return floor_sum(rt, static_cast<long long>(kKeys) * a.g, kRows, a.g * (base + kKeys) + kRows - 1) +
         static_cast<long long>(rt) * kUnitCost;
}
__device__ __forceinline__ long long head_cost(const CacheFwdArgs& a, const dec::Req& q) {
  return q.nrt == 0 ? 0 : cost_before(a, q, q.nrt - 1) + tiles_of(a, q, q.nrt - 1) + kUnitCost;
}

template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N) : "memory");
}

// kind::f16 with f16 A and B (format 0), fp32 D.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Sixteen codes to sixteen f16, two 16-byte pieces.
__device__ __forceinline__ void codes16(uint4 c, uint4& lo, uint4& hi) {
  dec::e4m3_to_f16(c.x, lo.x, lo.y);
  dec::e4m3_to_f16(c.y, lo.z, lo.w);
  dec::e4m3_to_f16(c.z, hi.x, hi.y);
  dec::e4m3_to_f16(c.w, hi.z, hi.w);
}

// 16 bytes from global to shared memory, or zeros; for the thread that waits
// for its own copies.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Those before the last copies_end, or all.
__device__ __forceinline__ void copies_but_last() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void sts128(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ void sts64(uint32_t at, uint2 v) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(v.x), "r"(v.y) : "memory");
}

// 32 bytes to global memory, aligned.
__device__ __forceinline__ void stg256(float* at, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// The power of two that a row is divided by, given its largest |element| as
// bf16 bits.  It takes that one to [2^7, 2^8), as E4M3 holds up to 448; for the
// smallest rows it stays at 2^-124, so that it and the row's scale are normal:
// their elements, multiples of 2^-133, are then multiples of 2^-9 with 8 bits at
// most, which two E4M3 numbers hold exactly.
__device__ __forceinline__ int split_exponent(uint32_t bf16_abs) {
  return max(static_cast<int>(bf16_abs >> 7) - 127 - 7, -124);
}

// Four bf16 times `inv` as the sum of two E4M3 numbers each.
__device__ __forceinline__ void split4(uint32_t w0, uint32_t w1, float inv, uint32_t& hi, uint32_t& lo) {
  const float f[4] = {__uint_as_float(w0 << 16) * inv, __uint_as_float(w0 & 0xffff0000u) * inv,
                      __uint_as_float(w1 << 16) * inv, __uint_as_float(w1 & 0xffff0000u) * inv};
  hi = pack_e4m3x4(f[0], f[1], f[2], f[3]);
  float g[4];
  e4m3x4_to_f32(hi, g);
  lo = pack_e4m3x4(f[0] - g[0], f[1] - g[1], f[2] - g[2], f[3] - g[3]);
}

__device__ __forceinline__ float lds_f32(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ float max32(const uint32_t (&r)[32], int lo, int hi) {
  float m = -INFINITY;
#pragma unroll
  for (int i = lo; i < hi; i += 2) m = fmax3(m, __uint_as_float(r[i]), __uint_as_float(r[i + 1]));
  return m;
}

}  // namespace prm

// G: keys of a step that share their scales, a block's or, of larger ones, all 64.
template <int D, int G>
__global__ void __launch_bounds__(prm::kThreads, 1)
    fa_cache_prompt_kernel(const __grid_constant__ CUtensorMap tmK, const uint8_t* __restrict__ v8,
                           const __grid_constant__ CacheFwdArgs a) {
  using namespace prm;
  using dec::Req;
  using dec::Seg;
  using Ly = Layout<D>;
  static_assert(G == 16 || G == 32 || G == kStepKeys, "keys that share a scale");
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
    for (int i = 0; i < 2; ++i) {
      mbar_init(base + Ly::kKFull + 8 * i, 1);
      mbar_init(base + Ly::kKEmpty + 8 * i, 2);
      mbar_init(base + Ly::kVFull + 8 * i, 4);
      mbar_init(base + Ly::kVEmpty + 8 * i, 2);
      for (int b = 0; b < 2; ++b) {
        mbar_init(base + Ly::kSFull + 8 * (2 * i + b), 1);
        mbar_init(base + Ly::kPFull + 8 * (2 * i + b), 4);
        mbar_init(base + Ly::kPvDone + 8 * (2 * i + b), 1);
      }
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(base + Ly::kRawFull + 8 * i, 1);
      mbar_init(base + Ly::kRawEmpty + 8 * i, 4);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(base + Ly::kScales + 8 * i, 1);
      mbar_init(base + Ly::kJoin + 8 * i, 2);
    }
    mbar_init(base + Ly::kFin, 1);
    mbar_init(base + Ly::kFin + 8, 1);
    *abort_flag = 0;
    fence_mbar_init();
    a.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
    a.cont[blockIdx.x] = 0;
  }

  const int per = (a.R + kThreads - 1) / kThreads;
  const int ra = min(a.R, tid * per), rb = min(a.R, ra + per);
  long long mine = 0, total;
  for (int r = ra; r < rb; ++r) {
    mine += a.Hkv * head_cost(a, dec::request<kRows, kKeys>(a, r));
    if (blockIdx.x == 0) dec::check_request(a, r);
  }
  const long long before = cta_scan(mine, reinterpret_cast<long long*>(sm + Ly::kScan), total) - mine;
  const long long want = (total + kMinCost - 1) / kMinCost;
  const int parts = static_cast<int>(min(static_cast<long long>(gridDim.x), max(1ll, want)));
  if (static_cast<int>(blockIdx.x) >= parts) return;
  const long long x0 = total * blockIdx.x / parts, x1 = total * (blockIdx.x + 1) / parts;
  if (x0 >= x1) return;
  if (before <= x0 && x0 < before + mine) {
    long long x = before;
    int r = ra;
    for (;; ++r) {
      const long long c = a.Hkv * head_cost(a, dec::request<kRows, kKeys>(a, r));
      if (x0 < x + c) break;  // ends: this thread's requests hold x0
      x += c;
    }
    // and the kv head; the walker finds the row tile
    const long long per_head = head_cost(a, dec::request<kRows, kKeys>(a, r));
    const int h = static_cast<int>((x0 - x) / per_head);
    const long long y = x0 - x - h * per_head;
    *reinterpret_cast<int4*>(sm + Ly::kStart) =
        make_int4(r, h, static_cast<int>(y & 0xffffffffll), static_cast<int>(y >> 32));
  }
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

  if (warp >= 12) {
    reg_dec<80>();
    if (warp == 13) {
      // --------------------------------------------------------- the walker
      const int4 at = *reinterpret_cast<const int4*>(sm + Ly::kStart);
      int r = at.x, h = at.y, rt = 0;
      Req q = dec::request<kRows, kKeys>(a, r);
      long long into = static_cast<long long>(at.w) << 32 | static_cast<unsigned>(at.z);
      // the last row tile whose cost begins at or before it, 32 at a time
      for (int end = q.nrt; end - rt > 1;) {
        const int each = (end - rt + 31) / 32, mine = rt + lane * each;
        const bool before = lane == 0 || (mine < end && cost_before(a, q, mine) <= into);
        rt += (31 - __clz(__ballot_sync(0xffffffffu, before))) * each;
        end = min(end, rt + each);
      }
      if (lane == 0) {
        int y = static_cast<int>(into - cost_before(a, q, rt));
        long long left = x1 - x0;
        int nseg = 0;
        bool ok = true;
        while (left > 0) {
          if (rt >= q.nrt) {  // the next kv head, the next request with rows
            rt = 0;
            if (++h == a.Hkv) {
              h = 0;
              do q = dec::request<kRows, kKeys>(a, ++r); while (q.nrt == 0);  // ends: cost is left
            }
          }
          const int kt = tiles_of(a, q, rt);
          const int take = static_cast<int>(min(static_cast<long long>(kt + kUnitCost - y), left));
          const int t0 = max(0, y - kUnitCost), t1 = max(0, y + take - kUnitCost);
          left -= take;
          if (t1 > t0) {
            const int si = nseg % kSegs;
            if (nseg >= kSegs && !wait(Ly::kSegEmpty + 8 * si, nseg / kSegs - 1, kSiteSegEmpty, nseg)) {
              ok = false;
              break;
            }
            const bool begins = t0 == 0, ends = t1 == kt;
            Seg* s = segs + si;
            s->r = r;
            s->h = h;
            s->row0 = rt * kRows;
            s->nv = min(kRows, q.n * a.g - rt * kRows);
            s->c0 = q.c0;
            s->n = q.n;
            s->len = dec::keys_of(a, q);
            s->t0 = t0;
            s->nt = t1 - t0;
            s->mode = begins && ends ? 0 : 1;
            s->slot = 2 * blockIdx.x + (begins ? 1 : 0);
            // steps: without the second half of a last tile that no row sees
            s->base = max(1, min(2 * (t1 - t0), (seen_of(a, q, rt) - t0 * kKeys + kStepKeys - 1) / kStepKeys));
            mbar_arrive(base + Ly::kSegFull + 8 * si);
            if (begins && !ends) a.desc[blockIdx.x] = make_int4(q.c0, h, rt, min(kRows, q.n * a.g - rt * kRows));
            if (!begins) a.cont[blockIdx.x] = ends ? 2 : 1;
            ++nseg;
          }
          ++rt;
          y = 0;
        }
        if (ok) {
          const int si = nseg % kSegs;
          if (nseg < kSegs || wait(Ly::kSegEmpty + 8 * si, nseg / kSegs - 1, kSiteSegEmpty, nseg)) {
            segs[si].nt = 0;
            mbar_arrive(base + Ly::kSegFull + 8 * si);
          }
        }
      }
    } else if (warp == 14) {
      // ------------------------------------------------------- the loader
      // Codes of a tile's blocks, K's to their place, V's as they lie into a
      // raw buffer; its scales, fetched while the tile before is loaded.  A
      // piece's tiles take raw buffers 2, 0, 1, 2, ...; 0 and 1 once its
      // queries, which are staged there, have been read.
      const int unit = min(1 << a.sh, kKeys);  // tokens that lie together
      fence_proxy_async_smem();  // the scan's use of the raw buffer
      if (lane == 0) prefetch_tensormap(&tmK);
      int jt = 0;
      uint32_t turn = 0;  // bit i: phase of raw buffer i's next use
      bool ok = true;
      for (int ns = 0;; ++ns) {
        const int si = ns % kSegs;
        ok = __all_sync(0xffffffffu, wait(Ly::kSegFull + 8 * si, ns / kSegs, kSiteSegFull, ns));
        if (!ok) break;
        const Seg& s = segs[si];
        const int nt = s.nt, h = s.h, len = s.len, t0 = s.t0;
        const bool two = s.nv > kHalf;
        if (nt == 0) break;
        const int* table = a.table + static_cast<long long>(s.r) * a.M;
        // block of this lane's 16 keys (8 lanes) in tile j; -1: none, -2: no keys
        auto block_of = [&](int j) {
          const int key = (t0 + j) * kKeys + lane * 16;
          return lane < 8 && j < nt && key < len ? max(-1, table[key >> a.sh]) : -2;
        };
        int next = block_of(0);
        for (int j = 0; j < nt; ++j, ++jt) {
          const int b = next;
          const bool real = b >= 0 && b < a.blocks;
          const long long bh = static_cast<long long>(b) * a.Hkv + h;
          float ks = -1.f, lv = 0.f;
          if (real) {
            ks = a.ks[bh];
            lv = a.vs[bh];
          }
          next = block_of(j + 1);
          const bool issue = real && ((lane * 16) & (unit - 1)) == 0;
          const uint32_t bytes = static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, issue)) * unit * D);
          const int st = jt & 1, in_block = ((t0 + j) * kKeys + lane * 16) & ((1 << a.sh) - 1);
          ok = jt < 2 || wait(Ly::kKEmpty + 8 * st, (jt >> 1) - 1, kSiteKEmpty, jt);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(base + Ly::kKFull + 8 * st, bytes / D * 128);
          __syncwarp();
          // rows of keys without a block keep what they held: their scores
          // are masked
          if (issue)
            tma_load_3d(base + Ly::kK + st * Ly::kKTile + lane * 16 * 128, &tmK, base + Ly::kKFull + 8 * st, 0,
                        in_block, static_cast<int>(bh));
          if (real && max(dec::scale_bits(ks), dec::scale_bits(lv)) >= dec::kBadScale) {  // as if it had no block
            ks = -1.f;
            lv = 0.f;
          }
          // (one report for both: a second one's code took prompts from 1122 to 1285 us)
          if (b != -2 && ks < 0.f) record_index_error(a.index_err, real ? kSiteFwdScale : kSiteFwdBlock, s.r);
          const bool clean = __popc(__ballot_sync(0xffffffffu, ks >= 0.f)) == 8 && (t0 + j + 1) * kKeys <= len;
          if (lane < 8) {
            reinterpret_cast<float*>(sm + Ly::kKs)[(jt & 3) * 8 + lane] = ks * a.k_unit;
            reinterpret_cast<float*>(sm + Ly::kLv)[(jt & 3) * 8 + lane] = fmaxf(log2f(lv), -200.f);
          }
          if (lane == 0) reinterpret_cast<int*>(sm + Ly::kClean)[jt & 3] = clean;
          __syncwarp();
          if (lane == 0) mbar_arrive(base + Ly::kScales + 8 * (jt & 3));
          const int rb = (j + 2) % 3, prev = (j + 1) % 3;
          // Two tiles ahead, but one with rows for both halves: the
          // conversions then fall between the softmax's steps (1212 us for
          // prompts of 3 requests, else 1268; for drafts of 16 44.1 and 40.5).
          // (A piece of one tile leaves out the wait for its queries.  The next
          // one's cannot mistake the phase: buffer 2, used in between, was
          // freed after them.)
          ok = wait(Ly::kRawEmpty + 8 * rb, (turn >> rb) ^ 1, kSiteRawEmpty, jt) &&
               (j != 1 || wait(Ly::kQFull, ns, kSiteQFull, ns)) &&
               (!two || j == 0 || wait(Ly::kRawEmpty + 8 * prev, (turn >> prev) ^ 1, kSiteRawEmpty, jt));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(base + Ly::kRawFull + 8 * rb, bytes);
          __syncwarp();
          if (issue)
            bulk_load_1d(base + Ly::kRaw + rb * Ly::kRawTile + lane * 16 * D, v8 + (bh << a.sh) * D + in_block * D,
                         static_cast<uint32_t>(unit * D), base + Ly::kRawFull + 8 * rb);
          turn ^= 1u << rb;
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(base + Ly::kSegEmpty + 8 * si);
      }
      // no copy outlives the CTA, also where a wait gave up (the K tile then
      // may be one ahead of V's: a phase that never began ends by its time)
      if (lane == 0 && jt > 0) {
        const uint64_t end = globaltimer_ns() + a.timeout_ns;
        for (int i = 0; i < 3; ++i) dec::mbar_drain(base + Ly::kRawFull + 8 * i, ((turn >> i) ^ 1) & 1, end);
        for (int t = max(0, jt - 2); t < jt; ++t) dec::mbar_drain(base + Ly::kKFull + 8 * (t & 1), (t >> 1) & 1, end);
      }
      if (lane == 0 && !ok)
        dec::mbar_drain(base + Ly::kKFull + 8 * (jt & 1), (jt >> 1) & 1, globaltimer_ns() + 1000000);
    } else {
      // ------------------------------------------------ the issuers, 12 and 15
      // One for each half: the tensor pipe queues little, so whatever one
      // thread waits for between its products would be lost (about 120 cycles
      // a wait).  A whole warp runs along and elects a thread to issue, so
      // that addresses and descriptors stay in uniform registers: from a
      // branch of one lane every product moved its descriptors there first,
      // and a key tile took 3000 cycles to issue against 2048 to run.
      constexpr uint32_t idS = idesc_e4m3_f32(kHalf, kStepKeys), idPV = idesc_f16_f32(kHalf, D, true);
      // operand descriptors (sw128_desc) by their low word; the high word,
      // stride 1024 and the swizzle, is the same for all
      constexpr uint32_t kHi = (1024u >> 4) | (1u << 14) | (2u << 29);
      auto desc = [](uint32_t lo) { return (static_cast<uint64_t>(kHi) << 32) | lo; };
      auto low = [](uint32_t addr, uint32_t lbo) { return ((addr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16); };
      const int x = __shfl_sync(0xffffffffu, warp == 15 ? 1 : 0, 0);
      const uint32_t dS = tmem + kColS + x * kHalf, dO = tmem + kColO + x * kHalf;
      auto all_wait = [&](int at, uint32_t parity, unsigned site, int item) {
        return __all_sync(0xffffffffu, wait(at, parity, site, item)) != 0;
      };
      int jt = 0, cnt = 0;  // the piece's first tile, this half's steps
      for (int ns = 0;; ++ns) {
        const int si = ns % kSegs;
        if (!all_wait(Ly::kSegFull + 8 * si, ns / kSegs, kSiteSegFull, ns)) break;
        const int nt = __shfl_sync(0xffffffffu, segs[si].nt, 0), steps = __shfl_sync(0xffffffffu, segs[si].base, 0);
        const bool two = __shfl_sync(0xffffffffu, segs[si].nv, 0) > kHalf;
        if (nt == 0) break;
        bool ok = all_wait(Ly::kQFull, ns, kSiteQFull, ns);
        // rows for both halves: each takes every step; else every other one,
        // with the same rows
        const int own = two ? steps : (steps + 1 - x) >> 1;
        const uint32_t q = low(base + Ly::kQ + (two ? x * Ly::kQHalf : 0), 16);
        auto step_of = [&](int k) { return two ? k : 2 * k + x; };
        if (ok && own > 0 && cnt > 0)
          ok = all_wait(Ly::kPvDone + 8 * (2 * x + ((cnt - 1) & 1)), (cnt - 1) >> 1, kSitePV, jt);
        // i = -1: the first scores only
#pragma unroll 1
        for (int i = -1; ok && i < own; ++i) {
          const int n = i + 1;
          if (n < own) {
            const int g = step_of(n), tk = jt + (g >> 1), buf = (cnt + n) & 1;
            if (!two || (g & 1) == 0) ok = all_wait(Ly::kKFull + 8 * (tk & 1), tk >> 1, kSiteKFull, tk);
            // the buffer's weights, of two steps before, have been multiplied
            if (ok && i >= 1) ok = all_wait(Ly::kPvDone + 8 * (2 * x + buf), (cnt + i - 1) >> 1, kSitePV, tk);
            if (!ok) break;
            tc_fence_after();
            const uint32_t k = low(base + Ly::kK + (tk & 1) * Ly::kKTile + (g & 1) * (kStepKeys * 128), 16);
            const uint32_t d = dS + buf * kStepKeys;
            if (dec::elect_one()) {
#pragma unroll
              for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk)  // 32 codes of each row
                  mma_ss_f8(d, desc(q + ((part * Ly::kPart) >> 4) + 2 * kk), desc(k + 2 * kk), idS,
                            part + kk > 0 ? 1u : 0u);
              tc_commit(base + Ly::kSFull + 8 * (2 * x + buf));
              if (!two || (g & 1) == 1 || g + 1 == steps) tc_commit(base + Ly::kKEmpty + 8 * (tk & 1));
              if (n + 1 == own) tc_commit(base + Ly::kQEmpty);  // the last read of Q
            }
            __syncwarp();
          }
          if (i >= 0) {
            const int g = step_of(i), tv = jt + (g >> 1), buf = (cnt + i) & 1;
            if (!two || (g & 1) == 0) ok = all_wait(Ly::kVFull + 8 * (tv & 1), tv >> 1, kSiteVFull, tv);
            if (ok) ok = all_wait(Ly::kPFull + 8 * (2 * x + buf), (cnt + i) >> 1, kSiteP, tv);
            if (!ok) break;
            tc_fence_after();
            const uint32_t v = low(base + Ly::kV + (tv & 1) * Ly::kVTile + (g & 1) * (kStepKeys * 128), 16384);
            const uint32_t first = i == 0 ? 0u : 1u, p = dS + buf * kStepKeys;
            if (dec::elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kStepKeys / 16; ++kk)
                mma_ts(dO, p + 8 * kk, desc(v + static_cast<uint32_t>(kk * 128)), idPV, kk == 0 ? first : 1u);
              tc_commit(base + Ly::kPvDone + 8 * (2 * x + buf));
              if (!two || (g & 1) == 1 || g + 1 == steps) tc_commit(base + Ly::kVEmpty + 8 * (tv & 1));
            }
            __syncwarp();
          }
        }
        if (ok && !two && x == 1 && (steps & 1)) {
          // a last tile without a step of this half, freed in its own phase
          const int t = jt + (steps >> 1);
          ok = all_wait(Ly::kKFull + 8 * (t & 1), t >> 1, kSiteKFull, t);
          if (ok && lane == 0) mbar_arrive(base + Ly::kKEmpty + 8 * (t & 1));
          if (ok && lane == 0 && own == 0) mbar_arrive(base + Ly::kQEmpty);
          ok = ok && all_wait(Ly::kVFull + 8 * (t & 1), t >> 1, kSiteVFull, t);
          if (ok && lane == 0) mbar_arrive(base + Ly::kVEmpty + 8 * (t & 1));
        }
        if (!ok) break;
        cnt += own;
        jt += nt;
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
    reg_dec<96>();
    // ----------------------------------------- V's codes to f16, Q in parts
    // A thread turns 16 codes of a row into two 16-byte pieces, of rows kStep
    // apart.  Eight lanes read 128 bytes in a row.  Their pieces go to the
    // places 0 2 4 6 of a 128-byte row, XORed with the row's low bits: at
    // d = 64 of two rows, on different banks; at d = 128 of two column blocks
    // of one, so the lanes of the upper write their odd pieces first.
    constexpr int kPer = kKeys * D / 16 / 128;      // per thread and tile
    constexpr int kStep = kKeys / kPer;
    const int cw = warp - 8, ct = tid - 256;
    const int c16 = ct & (D / 16 - 1), row_lo = ct / (D / 16);
    const bool odd_first = D == 128 && (c16 & 4);
    const uint32_t piece = static_cast<uint32_t>((c16 >> 2) * 16384 + row_lo * 128 +
                                                 ((((c16 & 3) * 2 + (odd_first ? 1 : 0)) ^ (row_lo & 7)) << 4));
    // one tile; loads four at a time, as one after the other each would wait
    // for its own
    auto put = [&](int st, int jt, int keys_left, uint32_t raw_at) {
      const uint32_t to0 = base + Ly::kV + st * Ly::kVTile + piece, to1 = to0 ^ 16u;
      const bool clean = reinterpret_cast<const volatile int*>(sm + Ly::kClean)[jt & 3] != 0;
#pragma unroll
      for (int b = 0; b < kPer; b += 4) {
        uint4 c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = dec::lds128(raw_at + (b + i) * 2048);
        if (!clean) {  // what no token lies in may be anything, NaN too
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = row_lo + kStep * (b + i);
            if (row >= keys_left || lds_f32(base + Ly::kKs + (jt & 3) * 32 + 4 * (row >> 4)) < 0.f)
              c[i] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4 p, q;
          if (odd_first) c[i] = make_uint4(c[i].z, c[i].w, c[i].x, c[i].y);
          codes16(c[i], p, q);
          sts128(to0 + (b + i) * (kStep * 128), p);
          sts128(to1 + (b + i) * (kStep * 128), q);
        }
      }
    };
    int jt = 0;
    uint32_t turn = 0;  // bit i: phase of raw buffer i's next use
    for (int ns = 0;; ++ns) {
      const int si = ns % kSegs;
      bool ok = wait(Ly::kSegFull + 8 * si, ns / kSegs, kSiteSegFull, ns);
      if (!__all_sync(0xffffffffu, ok)) break;
      const Seg& s = segs[si];
      const int nt = s.nt;
      if (nt == 0) break;
      const int h = s.h;

      // Q, 64 rows at a time: the bf16 rows to raw buffers 0 and 1, once every
      // warp has read those, each to where only the thread that copied it
      // reads; then in two parts to their places, with the next 64 on their way.
      // (128 at a time and without the second copies ahead, two or three rows
      // of a warp at once: 23000 cycles for 256 rows, a sixth of a piece.)
      ok = wait(Ly::kRawEmpty, turn ^ 1, kSiteRawEmpty, jt) &&
           wait(Ly::kRawEmpty + 8, (turn >> 1) ^ 1, kSiteRawEmpty, jt);
      if (!__all_sync(0xffffffffu, ok)) break;
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
              copy16(base + Ly::kStaged + (c & 1) * (64 * D * 2) + ct * 16 + i * 2048, q0 + at, real);
            }
          }
          copies_end();
        };
        copy(0);
        copy(1);
        ok = ns == 0 || wait(Ly::kQEmpty, ns - 1, kSiteQEmpty, ns);
        ok = __all_sync(0xffffffffu, ok);
        for (int c = 0; ok && c < chunks; ++c) {
          copies_but_last();
          const uint32_t from = base + Ly::kStaged + (c & 1) * (64 * D * 2) + ct * 16;
          const uint32_t to = base + Ly::kQ + (c >> 1) * Ly::kQHalf + (c & 1) * (64 * 128) + row_w * 128 +
                              (((col >> 1) ^ (row_w & 7)) << 4) + (col & 1) * 8;
          float* row_scale = reinterpret_cast<float*>(sm + Ly::kRowScale) + c * 64 + row_w;
#pragma unroll 1
          for (int i0 = 0; i0 < kEach; i0 += 4) {
            const uint32_t to4 = to + i0 * (4 * kAt * 128);
            uint4 w[4];
            uint32_t am[4];
            if (c * 64 + cw * kAt + i0 * 4 * kAt >= nv) {  // none of the warp's rows exists
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                sts64(to4 + 4 * kAt * 128 * i, make_uint2(0u, 0u));
                sts64(to4 + 4 * kAt * 128 * i + Ly::kPart, make_uint2(0u, 0u));
                if (col == 0) row_scale[(i0 + i) * 4 * kAt] = 0.f;
              }
              continue;
            }
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
              const int ex = split_exponent(am[i]);
              const float inv = dec::pow2i(-ex);
              uint2 hi, lo;
              split4(w[i].x ^ flip, w[i].y ^ flip, inv, hi.x, lo.x);
              split4(w[i].z ^ flip, w[i].w ^ flip, inv, hi.y, lo.y);
              sts64(to4 + 4 * kAt * 128 * i, hi);
              sts64(to4 + 4 * kAt * 128 * i + Ly::kPart, lo);
              if (col == 0) row_scale[(i0 + i) * 4 * kAt] = fabsf(a.scale_log2) * dec::pow2i(ex);
            }
          }
          copy(c + 2);
        }
        if (!ok) break;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(base + Ly::kQFull);

      for (int j = 0; j < nt; ++j, ++jt) {
        const int st = jt & 1, left = s.len - (s.t0 + j) * kKeys;
        const int rb = (j + 2) % 3;
        ok = wait(Ly::kRawFull + 8 * rb, turn >> rb, kSiteRawFull, jt) &&
             (jt < 2 || wait(Ly::kVEmpty + 8 * st, (jt >> 1) - 1, kSiteVEmpty, jt));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        put(st, jt, left, base + Ly::kRaw + rb * Ly::kRawTile + ct * 16);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(base + Ly::kRawEmpty + 8 * rb);
          mbar_arrive(base + Ly::kVFull + 8 * st);
        }
        turn ^= 1u << rb;
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      if (lane == 0) mbar_arrive(base + Ly::kSegEmpty + 8 * si);
    }
    copies_done();  // none outlives the CTA, also where a wait gave up
  } else {
    reg_inc<168>();
    // ------------------------------------------------ softmax and epilogue
    const int x = warp >> 2;  // half
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + kColS + x * kHalf, tO = tmem + lane_off + kColO + x * kHalf;
    constexpr int kGroups = kStepKeys / G;          // groups of a step
    constexpr int kStepG = 4 / kGroups;             // a group's place among the scales
    int cnt = 0, jt = 0;  // steps of this half, the piece's first tile
    for (int ns = 0;; ++ns) {
      const int si = ns % kSegs;
      bool ok = wait(Ly::kSegFull + 8 * si, ns / kSegs, kSiteSegFull, ns);
      if (!__all_sync(0xffffffffu, ok)) break;
      const Seg& s = segs[si];
      const int nt = s.nt;
      if (nt == 0) break;
      // Rows for both halves: each takes every step, of its own rows.  Else
      // both have the same rows, A the even steps and B the odd ones, and join
      // at the end.
      const bool two = s.nv > kHalf;
      const int own = two ? s.base : (s.base + 1 - x) >> 1;
      const int row = two ? tid : tid & (kHalf - 1);  // of the unit
      // no wait is left out for a piece without a step of this half: a phase
      // that a warp never saw could pass for a later one of the same parity
      ok = wait(Ly::kQFull, ns, kSiteQFull, ns);
      if (!__all_sync(0xffffffffu, ok)) break;
      const float c = lds_f32(base + Ly::kRowScale + 4 * row);
      __syncwarp();
      if (lane == 0) mbar_arrive(base + Ly::kQEmpty);
      if (own == 0) {
        jt += nt;
        if (lane == 0) mbar_arrive(base + Ly::kSegEmpty + 8 * si);
        continue;
      }
      // keys visible to this row, and to every row of this warp
      const int lim = a.causal ? min(s.len, s.len - s.n + (s.row0 + row) / a.g + 1) : s.len;
      const int all = __reduce_min_sync(0xffffffffu, lim);
      float m = kInit, e = 0.f, l = 0.f;  // e: the second reference less the first
      bool far = false;
      for (int i = 0; i < own; ++i, ++cnt) {
        const int step = two ? i : 2 * i + x, tile = jt + (step >> 1), buf = 2 * x + (cnt & 1);
        // (the scales of a tile are never replaced before its scores are read)
        ok = wait(Ly::kSFull + 8 * buf, cnt >> 1, kSiteS, tile) &&
             wait(Ly::kScales + 8 * (tile & 3), tile >> 2, kSiteScales, tile);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        const uint32_t tSb = tS + (cnt & 1) * kStepKeys;
        uint32_t v[2][32];
        float mx[2];  // of each 32 keys
        // scales of 16-key group y
        const uint32_t scales = base + Ly::kKs + (tile & 3) * 32 + (step & 1) * 16;
        auto ks_at = [&](int y) { return lds_f32(scales + 4 * y); };
        auto lv_at = [&](int y) { return lds_f32(scales + (Ly::kLv - Ly::kKs) + 4 * y); };
        const int key0 = s.t0 * kKeys + step * kStepKeys;
        bool careful = key0 + kStepKeys > all;
        float fk[kGroups], lv[kGroups];
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          const float ks = ks_at(g * kStepG);
          careful = careful | (ks < 0.f);
          fk[g] = fmaxf(c * ks, kTiny);
          lv[g] = lv_at(g * kStepG);
        }
        if constexpr (G >= 32) {
          tmem_ldred_max32(tSb, v[0], mx[0]);
          tmem_ldred_max32(tSb + 32, v[1], mx[1]);
          tmem_ldred_wait32(v[0], mx[0]);
          tmem_ldred_dep32(v[1], mx[1]);
        } else {
          tmem_ld32(tSb, v[0]);
          tmem_ld32(tSb + 32, v[1]);
          tmem_ld_wait32(v[0]);
          tmem_ld_dep32(v[1]);
        }
        if (careful) {
          constexpr uint32_t kNegInf = 0xff800000u;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            // keys of the group below this are visible
            const int end = ks_at(y) < 0.f ? 0 : lim - (key0 + 16 * y);
#pragma unroll
            for (int z = 0; z < 16; ++z)
              if (z >= end) v[y >> 1][(y & 1) * 16 + z] = kNegInf;
          }
        }
        // the step's references, eb relative to mb
        float mb = kInit, eb = -INFINITY;
        auto see = [&](int g, float top) {
          const float t = top * fk[g], m1 = fmaxf(mb, t);
          eb = fmaxf(eb + (mb - m1), t - m1 + lv[g]);
          mb = m1;
        };
        if constexpr (G == 16) {
#pragma unroll
          for (int g = 0; g < 4; ++g) see(g, max32(v[g >> 1], (g & 1) * 16, (g & 1) * 16 + 16));
        } else {
          if (careful) {
            mx[0] = max32(v[0], 0, 32);
            mx[1] = max32(v[1], 0, 32);
          }
          if constexpr (G == 32) {
            see(0, mx[0]);
            see(1, mx[1]);
          } else {
            see(0, fmaxf(mx[0], mx[1]));
          }
        }
        const bool bump = mb > m + kLazy || eb + (mb - m) > e + kLazy;
        float up = 1.f;
        if (bump) {
          const float m1 = fmaxf(m, mb), e1 = fmaxf(e + (m - m1), eb + (mb - m1));
          l *= ex2(m - m1);
          up = ex2(e + (m - m1) - e1);
          m = m1;
          e = e1;
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
            w = __float_as_uint(__fsub_rn(__fmul_rn(__uint_as_float(w), fk[y / G]), m));
          }
        }
        float sums = 0.f;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          // 2^up_g: what the weights of this group carry beside 2^(s - m).
          // Below 2^-60 they are 0 in f16 whatever it is.  It has no upper
          // bound: together with s - m it is at most kBias + kLazy, and a group
          // beyond 2^126 counts nothing in l, as its s - m are below -112.
          const float up_g = fmaxf(lv[g] + kBias - e, -60.f);
          const float f = far ? 1.f : fk[g], nm = far ? up_g : up_g - m;
          const uint64_t f2 = f2_pack(f, f), n2 = f2_pack(nm, nm);
          uint64_t sum[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
          for (int z = 0; z < (G + 31) / 32; ++z) {
            const int ch = g * G / 32 + z, lo = (g * G) % 32;
            constexpr int n = G < 32 ? G : 32;
            uint32_t w[n / 2];
#pragma unroll
            for (int y = 0; y < n; y += 2) {
              float a0, a1;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(v[ch][lo + y]), __uint_as_float(v[ch][lo + y + 1])), f2, n2), a0,
                        a1);
              a0 = ex2(a0);
              a1 = ex2(a1);
              sum[(y >> 1) & 1] = f2_add(sum[(y >> 1) & 1], f2_pack(a0, a1));
              w[y >> 1] = dec::pack_f16(a0, a1);
            }
            if constexpr (G < 32) tmem_st8(tSb + 8 * g, w);
            else tmem_st16(tSb + 16 * ch, w);
          }
          float s0, s1;
          f2_unpack(f2_add(sum[0], sum[1]), s0, s1);
          sums = fmaf(s0 + s1, ex2(-up_g), sums);
        }
        l += sums;
        if (moved && i > 0) {  // O to the new reference, once it has every weight before
          ok = __all_sync(0xffffffffu, wait(Ly::kPvDone + 8 * (buf ^ 1), (cnt - 1) >> 1, kSitePV, tile));
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
      jt += nt;
      if (!__all_sync(0xffffffffu, ok)) break;
      ok = wait(Ly::kPvDone + 8 * (2 * x + ((cnt - 1) & 1)), (cnt - 1) >> 1, kSitePV, jt);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const bool real = row < s.nv;
      // The halves' statistics, through shared memory; then each of the two
      // warps that have a row combines and writes one half of its columns.
      const bool join = !two && s.base > 1;
      float f = 1.f, f2 = 0.f;  // what this half's sums and the other's count
      if (join) {
        const uint32_t bar = base + Ly::kJoin + 8 * (warp & 3);
        float4* stat = reinterpret_cast<float4*>(sm + Ly::kStat);
        stat[x * kHalf + row] = make_float4(m, e, l, 0.f);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
        ok = wait(Ly::kJoin + 8 * (warp & 3), 0, kSiteJoin, jt);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        const float4 b = stat[(1 - x) * kHalf + row];
        const float m1 = fmaxf(m, b.x), e0 = e + (m - m1), eb = b.y + (b.x - m1), e1 = fmaxf(e0, eb);
        l = l * ex2(m - m1) + b.z * ex2(b.x - m1);
        f = ex2(e0 - e1);
        f2 = ex2(eb - e1);
        m = m1;
        e = e1;
      }
      const float inv = l == 0.f ? 0.f : ex2(e - kBias) / l;
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
            for (int e = 0; e < 32; e += 8) stg256(a.part_o + pat * D + 32 * q + e, o + e);
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
        if (lane == 0) mbar_arrive(base + Ly::kJoin + 8 * (warp & 3));
        ok = wait(Ly::kJoin + 8 * (warp & 3), 1, kSiteJoin, jt);
        if (!__all_sync(0xffffffffu, ok)) break;
      }
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
