// Rotary positions: pairs of a row's elements turned by the angles of its
// position.
//
//   half:        (x_i, x_{i + rot/2}) -> (x_i c_i - x_{i + rot/2} s_i, x_{i + rot/2} c_i + x_i s_i)
//   interleaved: the same of (x_{2i}, x_{2i+1}),    i < rot / 2
//
// with (c_i, s_i) the position's row of a table; elements from rot on pass.  The
// gradient is the transposed rotation, s_i negated.
//
// A result is the exact value, with the table's entries as they are, rounded
// once to bf16.  Its products have 32 bits, so a fp32 sum is off by about one
// unit of its last place; where that is too near a border of bf16's rounding
// to tell (5 values of 65536), it is taken again in 64 bits.  So a key that the
// cache's append turns on the way is bit for bit one turned before, and its 4-bit
// code never hangs on how a sum was ordered.
#pragma once
#include <cuda_bf16.h>

#include "fa_index.cuh"
#include "sm103_ptx.cuh"

namespace fa {

namespace rope {

constexpr int kThreads = 256;

// x c + y s to within about one unit in its last place: the product's own error
// is added, so that cancellation does not raise it.
__device__ __forceinline__ float turn(float x, float c, float y, float s) {
  const float p = y * s, e = fmaf(y, s, -p);
  return fmaf(x, c, p) + e;
}
// Too near the middle of two bf16 numbers, or not a number (an infinity's error is none).
__device__ __forceinline__ bool unsure(float r) {
  return ((__float_as_uint(r) - 0x7ffeu) & 0xffffu) <= 4u || r != r;
}
// The same in 64 bits, as a fp32 number that rounds to bf16 as the exact one
// does: cut off, its last bit set where bits were lost.
__device__ __forceinline__ float turn_exactly(float x, float c, float y, float s) {
  const double v = static_cast<double>(x) * c + static_cast<double>(y) * s;
  const float f = __double2float_rz(v);
  return static_cast<double>(f) == v ? f : __uint_as_float(__float_as_uint(f) | 1u);
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Eight elements x with their partners y, cs[i] their (cos, +-sin): x_i c_i + y_i s_i.
__device__ __forceinline__ uint4 turn8(uint4 x, uint4 y, const float2 (&cs)[8]) {
  const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
  uint32_t r[4];
  bool again = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = turn(low(xw[i]), cs[2 * i].x, low(yw[i]), cs[2 * i].y);
    const float b = turn(high(xw[i]), cs[2 * i + 1].x, high(yw[i]), cs[2 * i + 1].y);
    again = again || unsure(a) || unsure(b);
    r[i] = pack_bf16(a, b);
  }
  if (again) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r[i] = pack_bf16(turn_exactly(low(xw[i]), cs[2 * i].x, low(yw[i]), cs[2 * i].y),
                       turn_exactly(high(xw[i]), cs[2 * i + 1].x, high(yw[i]), cs[2 * i + 1].y));
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}
// Elements exchanged with their neighbours.
__device__ __forceinline__ uint4 swap_pairs(uint4 x) {
  return make_uint4(__byte_perm(x.x, 0u, 0x1032), __byte_perm(x.y, 0u, 0x1032), __byte_perm(x.z, 0u, 0x1032),
                    __byte_perm(x.w, 0u, 0x1032));
}
// Four pairs' (cos, sin) as those of eight interleaved elements.
__device__ __forceinline__ void spread(const float2 (&p)[4], float2 (&cs)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    cs[2 * i] = make_float2(p[i].x, -p[i].y);
    cs[2 * i + 1] = p[i];
  }
}
// N pairs of a table row.
template <int N>
__device__ __forceinline__ void load_pairs(const float2* from, float sign, float2 (&p)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(from + i));
    p[i] = make_float2(v.x, sign * v.y);
    p[i + 1] = make_float2(v.z, sign * v.w);
  }
}

}  // namespace rope

struct RopeArgs {
  const __nv_bfloat16* x;
  __nv_bfloat16* out;
  long long xb, xh, xn, ob, oh, on;  // elements between batches, heads and tokens
  const int* positions;
  long long pb;                      // positions between batches, 0: the same for all
  const float2* table;               // [length][rot / 2] (cos, sin)
  int length, B, H, N, rot;
  int group;                         // heads of a thread
  float sign;                        // -1: transposed
  DevError* err;
};

// D / 16 lanes take a token's row, each two vectors of eight elements that turn
// among themselves (or pass): i and i + rot / 16, or 2 i and 2 i + 1 where pairs
// are neighbours.  A lane keeps its pairs' cos and sin for its group of heads.
template <int D, bool PAIRS>
__global__ void __launch_bounds__(rope::kThreads) fa_rope_kernel(RopeArgs a) {
  using namespace rope;
  constexpr int kLanes = D / 16;
  const long long at = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) / kLanes;
  if (at >= static_cast<long long>(a.B) * a.N) return;
  const int i = threadIdx.x % kLanes;
  const int b = static_cast<int>(at / a.N), n = static_cast<int>(at - static_cast<long long>(b) * a.N);
  const int h0 = blockIdx.y * a.group, h1 = min(a.H, h0 + a.group);
  const int pos = a.positions[b * a.pb + n];
  if (pos >= a.length && i == 0 && h0 == 0) record_index_error(a.err, kSiteRopePosition, n);
  const int items = a.rot / 16;
  const bool turns = i < items && pos >= 0 && pos < a.length;
  const bool apart = !PAIRS && i < items;  // the two vectors do not lie together
  const int v0 = apart ? i : 2 * i, v1 = apart ? i + items : 2 * i + 1;
  float2 cs[8];
  if (turns) load_pairs<8>(a.table + static_cast<long long>(pos) * (a.rot / 2) + 8 * i, a.sign, cs);
  const __nv_bfloat16* x = a.x + b * a.xb + n * a.xn;
  __nv_bfloat16* out = a.out + b * a.ob + n * a.on;
#pragma unroll 4
  for (int h = h0; h < h1; ++h) {
    const uint4* from = reinterpret_cast<const uint4*>(x + h * a.xh);
    uint4* to = reinterpret_cast<uint4*>(out + h * a.oh);
    uint4 p = from[v0], q = from[v1];
    if (turns) {
      if constexpr (PAIRS) {
        const float2 c0[4] = {cs[0], cs[1], cs[2], cs[3]}, c1[4] = {cs[4], cs[5], cs[6], cs[7]};
        float2 e[8];
        spread(c0, e);
        p = turn8(p, swap_pairs(p), e);
        spread(c1, e);
        q = turn8(q, swap_pairs(q), e);
      } else {
        float2 e[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k] = make_float2(cs[k].x, -cs[k].y);
        const uint4 p1 = turn8(p, q, e);
        q = turn8(q, p, cs);
        p = p1;
      }
    }
    to[v0] = p;
    to[v1] = q;
  }
}

}  // namespace fa
