// The 8-bit key/value cache: appends.
//
// Cache: codes uint8 [blocks][Hkv][P][d] for K and for V (P tokens per block,
// E4M3), scales fp32 [blocks][Hkv]; the value a code stands for is
// E4M3(code) * scale.  A block's scale is a power of two: a block fills token
// by token, so its scale has to grow after codes were written, and dividing a
// code by a power of two only moves its exponent (nothing is rounded a second
// time until a value falls below E4M3's smallest normal, 2^-6), while a
// floating-point code loses no precision from a scale that is up to twice the
// smallest one that fits.
#pragma once
#include <cuda_bf16.h>

#include "fa_index.cuh"
#include "sm103_ptx.cuh"

namespace fa {

// ------------------------------------------------------------------ append

namespace app {
constexpr int kMaxChunk = 64;  // most tokens a CTA looks at for starts of runs
}  // namespace app

struct AppendArgs {
  const __nv_bfloat16* x[2];   // K, V rows: [T][Hkv][d] with a token stride
  long long stride[2];         // elements between tokens
  uint8_t* codes[2];
  float* scale[2];
  const long long* slot_map;   // [T]
  long long slots;             // blocks * P
  int T, Hkv, sh;              // blocks of P = 2^sh tokens
  int chunk, group;            // tokens and rows (heads of K, then of V) of a CTA
  DevError* err;
};

// The smallest power of two s with a <= 448 s, its exponent within
// [-100, 120], for a >= 0 given as bf16 bits: 448 = 1.75 * 2^8, so it is the
// exponent of a less 8, one more where a's mantissa is above 1.75.  (-100
// keeps 1 / s and every product with it normal; a block of zeros gets it.)
__device__ __forceinline__ float scale_of(uint32_t bf16_abs) {
  int e = static_cast<int>(bf16_abs >> 7) - 127 - 8 + ((bf16_abs & 0x7fu) > 0x60u ? 1 : 0);
  e = max(-100, min(120, e));
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Largest |x| of eight bf16, as bf16 bits (they order like the values).
__device__ __forceinline__ uint32_t amax2(uint32_t w, uint32_t m) {
  return max(m, max(w & 0x7fffu, (w >> 16) & 0x7fffu));
}

__device__ __forceinline__ uint32_t quant4(uint32_t w0, uint32_t w1, float inv) {
  return pack_e4m3x4(__uint_as_float(w0 << 16) * inv, __uint_as_float(w0 & 0xffff0000u) * inv,
                     __uint_as_float(w1 << 16) * inv, __uint_as_float(w1 & 0xffff0000u) * inv);
}

// Four codes' values.
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t c, float (&f)[4]) {
  asm("{\n\t.reg .b16 lo, hi, a, b, c, d;\n\t.reg .b32 x, y;\n\t"
      "mov.b32 {lo, hi}, %4;\n\t"
      "cvt.rn.f16x2.e4m3x2 x, lo;\n\t"
      "cvt.rn.f16x2.e4m3x2 y, hi;\n\t"
      "mov.b32 {a, b}, x;\n\t"
      "mov.b32 {c, d}, y;\n\t"
      "cvt.f32.f16 %0, a;\n\t"
      "cvt.f32.f16 %1, b;\n\t"
      "cvt.f32.f16 %2, c;\n\t"
      "cvt.f32.f16 %3, d;\n}"
      : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3])
      : "r"(c));
}
// Four codes times `ratio` (a power of two below 1), rounded to nearest even.
__device__ __forceinline__ uint32_t rescale4(uint32_t c, float ratio) {
  float f[4];
  e4m3x4_to_f32(c, f);
  return pack_e4m3x4(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
}

// New K and V rows into the cache.  A run is a maximal stretch of consecutive
// tokens in consecutive slots of one block; grid (chunks of tokens, groups of
// rows: kv heads of K, then of V).  Each CTA handles the runs that start in its
// chunk: a warp takes a run of one token (decode), the whole CTA a longer one
// (prompts), whose rows it holds in registers between the maximum and the
// rounding, so that they are read once, with the next head's already on their
// way.  A run that starts inside a block keeps the rows before it: the scale is
// the larger of the block's and its own, and if it grows those rows' codes are
// divided by the growth.
//
// NV: 16-byte vectors per thread of the longest run, P * D / 8 / THREADS.
//
// Bound by memory for prompts: 24 of 1 to 4096 tokens, 8 kv heads of 128 in
// blocks of 64, in 58.7 us, 5.4 TB/s (152 us with one head a CTA and 16 tokens;
// 62 with four CTAs per SM instead of five).
// By latency for single tokens: 32 of them in 2.4 us, 500 of 16 heads in 5.8 us.
template <int D, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS, 640 / THREADS) fa_cache_append_kernel(AppendArgs a) {
  constexpr int kWarps = THREADS / 32;
  __shared__ long long s_slot[app::kMaxChunk + 2];
  __shared__ uint32_t s_max[2][kWarps];
  __shared__ int s_len[kWarps];
  __shared__ uint8_t s_single[app::kMaxChunk];  // the runs of one token
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t0 = blockIdx.x * a.chunk;
  const int g0 = blockIdx.y * a.group, g1 = min(2 * a.Hkv, g0 + a.group);
  const int P = 1 << a.sh;
  // slots of the chunk and its two neighbours; an unusable slot reads as -1
  if (tid < a.chunk + 2) {
    const int t = t0 - 1 + tid;
    long long s = t >= 0 && t < a.T ? a.slot_map[t] : -1;
    if (s < -1 || s >= a.slots) {
      if (g0 == 0) record_index_error(a.err, kSiteAppendSlot, t);
      s = -1;
    }
    s_slot[tid] = s;
  }
  __syncthreads();
  uint64_t starts = 0, singles = 0;  // bit i: a run starts at token t0 + i; it has one token
#pragma unroll
  for (int w = 0; w < app::kMaxChunk / 32; ++w) {
    const int i = 32 * w + lane;
    bool start = false, more = false;
    if (i < a.chunk) {
      const long long s = s_slot[i + 1];
      start = s >= 0 && !(s_slot[i] >= 0 && s_slot[i] + 1 == s && (s & (P - 1)) != 0);
      more = s_slot[i + 2] == s + 1 && ((s + 1) & (P - 1)) != 0;
    }
    starts |= static_cast<uint64_t>(__ballot_sync(0xffffffffu, start)) << (32 * w);
    singles |= static_cast<uint64_t>(__ballot_sync(0xffffffffu, start && !more)) << (32 * w);
  }
  if (tid < app::kMaxChunk && ((singles >> tid) & 1u))
    s_single[__popcll(singles & ((1ull << tid) - 1ull))] = static_cast<uint8_t>(tid);
  __syncthreads();

  // runs of one token: a warp for each and head, four at a time so that their
  // loads are in flight together
  const int ng = g1 - g0, items = __popcll(singles) * ng;
  for (int k0 = warp; k0 < items; k0 += 4 * kWarps) {
    uint32_t w[4][D / 64];
    float old[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = k0 + u * kWarps;
      if (k < items) {
        const int i = s_single[k / ng], gi = g0 + k % ng, z = gi >= a.Hkv ? 1 : 0, h = gi - z * a.Hkv;
        const long long s = s_slot[i + 1];
        const uint32_t* src = reinterpret_cast<const uint32_t*>(
            (z ? a.x[1] : a.x[0]) + (t0 + i) * (z ? a.stride[1] : a.stride[0]) + static_cast<long long>(h) * D);
        old[u] = (s & (P - 1)) ? (z ? a.scale[1] : a.scale[0])[(s >> a.sh) * a.Hkv + h] : 0.f;
#pragma unroll
        for (int e = 0; e < D / 64; ++e) w[u][e] = __ldg(src + lane * (D / 64) + e);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = k0 + u * kWarps;
      if (k < items) {
        const int gi = g0 + k % ng, z = gi >= a.Hkv ? 1 : 0, h = gi - z * a.Hkv;
        const long long s = s_slot[s_single[k / ng] + 1], bh = (s >> a.sh) * a.Hkv + h;
        const int off = static_cast<int>(s & (P - 1));
        uint8_t* blk = (z ? a.codes[1] : a.codes[0]) + bh * P * D;
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < D / 64; ++e) m = amax2(w[u][e], m);
        m = __reduce_max_sync(0xffffffffu, m);
        const float now = fmaxf(old[u], scale_of(m));
        const float inv = __fdiv_rn(1.f, now);
        if (D == 128)
          reinterpret_cast<uint32_t*>(blk + off * D)[lane] = quant4(w[u][0], w[u][D / 64 - 1], inv);
        else
          reinterpret_cast<uint16_t*>(blk + off * D)[lane] = static_cast<uint16_t>(quant4(w[u][0], 0u, inv));
        if (off > 0 && now > old[u]) {
          const float ratio = __fdiv_rn(old[u], now);
          uint4* v = reinterpret_cast<uint4*>(blk);
          for (int j = lane; j < off * (D / 16); j += 32) {
            const uint4 c = v[j];
            v[j] = make_uint4(rescale4(c.x, ratio), rescale4(c.y, ratio), rescale4(c.z, ratio),
                              rescale4(c.w, ratio));
          }
        }
        if (lane == 0 && now != old[u]) (z ? a.scale[1] : a.scale[0])[bh] = now;
      }
    }
  }

  // longer runs: the CTA, one after the other, head by head
  int par = 0;
  for (uint64_t todo = starts & ~singles; todo; todo &= todo - 1) {
    const int i = __ffsll(static_cast<long long>(todo)) - 1;
    const long long s = s_slot[i + 1];
    const int off = static_cast<int>(s & (P - 1)), t = t0 + i;
    // its length: tokens while the slots go on (P <= 128 <= THREADS)
    const bool in = off + tid < P && t + tid < a.T && a.slot_map[t + tid] == s + tid;
    const uint32_t bal = __ballot_sync(0xffffffffu, in);
    __syncthreads();  // s_len of the run before has been read
    if (lane == 0) s_len[warp] = bal == 0xffffffffu ? 32 : __ffs(~bal) - 1;
    __syncthreads();
    int len = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      len += s_len[w];
      if (s_len[w] < 32) break;
    }
    constexpr int kRow = D / 8;  // vectors per row
    uint4 next[NV];
    float next_old = 0.f;
    auto fetch = [&](int gi) {
      const int z = gi >= a.Hkv ? 1 : 0, h = gi - z * a.Hkv;
      const long long stride = z ? a.stride[1] : a.stride[0];
      const __nv_bfloat16* src = (z ? a.x[1] : a.x[0]) + t * stride + static_cast<long long>(h) * D;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int k = tid + j * THREADS;
        next[j] = make_uint4(0u, 0u, 0u, 0u);
        if (k < len * kRow) next[j] = __ldg(reinterpret_cast<const uint4*>(src + (k / kRow) * stride) + k % kRow);
      }
      if (off > 0) next_old = (z ? a.scale[1] : a.scale[0])[(s >> a.sh) * a.Hkv + h];
    };
    fetch(g0);
    for (int gi = g0; gi < g1; ++gi, par ^= 1) {
      uint4 v[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) v[j] = next[j];
      const float old = next_old;
      if (gi + 1 < g1) fetch(gi + 1);
      const int z = gi >= a.Hkv ? 1 : 0, h = gi - z * a.Hkv;
      const long long bh = (s >> a.sh) * a.Hkv + h;
      uint8_t* blk = (z ? a.codes[1] : a.codes[0]) + bh * P * D;
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j) m = amax2(v[j].x, amax2(v[j].y, amax2(v[j].z, amax2(v[j].w, m))));
      m = __reduce_max_sync(0xffffffffu, m);
      if (lane == 0) s_max[par][warp] = m;
      __syncthreads();  // and s_max[par ^ 1] has been read by all
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = max(m, s_max[par][w]);
      const float now = fmaxf(old, scale_of(m));
      const float inv = __fdiv_rn(1.f, now);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int k = tid + j * THREADS;
        if (k < len * kRow)
          reinterpret_cast<uint2*>(blk + off * D)[k] =
              make_uint2(quant4(v[j].x, v[j].y, inv), quant4(v[j].z, v[j].w, inv));
      }
      if (off > 0 && now > old) {
        const float ratio = __fdiv_rn(old, now);
        uint4* c4 = reinterpret_cast<uint4*>(blk);
        for (int j = tid; j < off * (D / 16); j += THREADS) {
          const uint4 c = c4[j];
          c4[j] = make_uint4(rescale4(c.x, ratio), rescale4(c.y, ratio), rescale4(c.z, ratio),
                             rescale4(c.w, ratio));
        }
      }
      if (tid == 0 && now != old) (z ? a.scale[1] : a.scale[0])[bh] = now;
    }
  }
}

}  // namespace fa
