// Rotary positions: pairs of a row's elements turned by the angles of its
// position.
//
//   half:        (x_i, x_{i + rot/2}) -> (x_i c_i - x_{i + rot/2} s_i, x_{i + rot/2} c_i + x_i s_i)
//   interleaved: the same of (x_{2i}, x_{2i+1}),    i < rot / 2
//
// with (c_i, s_i) the position's row of a table; elements from rot on pass.  The
// gradient is the transposed rotation, s_i negated.
//
// A result is the exact value, with the table's entries as they are, rounded once to
// bf16.  Its products have 32 bits, so a fp32 sum is off by about one unit of its last
// place; where that is too near a border of bf16's rounding to tell (8 values of
// 65536), it is taken again with the rests of its roundings.  So a key that the cache's
// append turns on the way is bit for bit one turned before, and its 4-bit code never
// hangs on how a sum was ordered.
#pragma once
#include <cuda_bf16.h>

#include "fa_index.cuh"
#include "sm103_ptx.cuh"

namespace fa {

namespace rope {

constexpr int kThreads = 128;

__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Products and sums of two, subnormals as they are (in sm103_ptx.cuh they count as 0).
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Two (cos, sin), for the two-wide arithmetic.
struct Pair {
  uint64_t c, s;
};

// a + b, and what its rounding left.
__device__ __forceinline__ float add_rest(float a, float b, float& rest) {
  const float h = __fadd_rn(a, b), z = __fsub_rn(h, a);
  rest = __fadd_rn(__fsub_rn(a, __fsub_rn(h, z)), __fsub_rn(b, z));
  return h;
}
// A fp32 number cut off from t, and whether something (of `left`'s sign, less than t's
// last bit) is left of it, as a number that rounds to bf16 as both together do: with
// its last bit set where bits were lost.  t is 0 only with nothing or its sign left.
__device__ __forceinline__ float with_rest(float t, float left) {
  uint32_t bits = __float_as_uint(t);
  if (left != 0.f) bits = (bits - ((bits ^ __float_as_uint(left)) >> 31)) | 1u;
  return __uint_as_float(bits);
}
// Whether a result with this lower half is too near a border (0x8000) to tell.
__device__ __forceinline__ bool in_doubt(uint32_t half) { return half - 0x7ffdu <= 7u; }
// Whether a product's rest is a fp32 number: factors of 8 and 24 bits lose none of
// them from 2^-100 on.
__device__ __forceinline__ bool kept(float product, float x, float c) {
  return fabsf(product) >= 0x1p-100f || x == 0.f || c == 0.f;
}
// x c + y s as a fp32 number that rounds to bf16 as the exact one does.  Most that
// come here do so with another value in doubt, and turn2's own result serves (all of
// them taken again, rope of 9001 tokens took 38.6 us for 35.7).  Of the others products
// and sums are kept as pairs of fp32 numbers, rounded value and rest (the rest of a
// sum: Knuth, The Art of Computer Programming 2, 4.2.2, theorem B), where two of them
// hold all; else they are taken in 64 bits, in which the products are exact.  (All
// of them in 64 bits, of which a warp's operation takes an SM 16 cycles, took half of
// the time: 140 us for 93.)
__device__ __forceinline__ float turn_exactly(float x, float c, float y, float s) {
  const float p = __fmul_rn(x, c), q = __fmul_rn(y, s), pe = fmaf(x, c, -p), qe = fmaf(y, s, -q);
  const float fast = __fadd_rn(fmaf(x, c, q), qe);
  if (!in_doubt(__float_as_uint(fast) & 0xffffu) && fast == fast) return fast;
  float he, ue, ve, left;
  const float h = add_rest(p, q, he), u = add_rest(pe, qe, ue), v = add_rest(he, u, ve), t = add_rest(h, v, left);
  if (fabsf(t) < INFINITY && ue == 0.f && ve == 0.f && kept(p, x, c) && kept(q, y, s)) return with_rest(t, left);
  const double P = static_cast<double>(x) * c, Q = static_cast<double>(y) * s, H = P + Q, Z = H - P;
  if (!(fabs(H) < INFINITY)) return static_cast<float>(H);  // of no finite factors
  const double E = (P - (H - Z)) + (Q - Z);
  const float T = __double2float_rz(H);
  // what is cut off has H's sign, and E less than its last bit
  return with_rest(T, H != T ? copysignf(1.f, T) : E < 0 ? -1.f : E > 0 ? 1.f : 0.f);
}

// Whether some of the results r is too near a border: of their lower halves, two by
// two and less 0x7ffd each, `near` is the smallest so far; `sum` their sum.
struct Doubt {
  uint32_t near = 0xffffffffu;
  uint64_t sum = 0;  // two zeros

  __device__ __forceinline__ void see(uint64_t r) {
    float a, b;
    f2_unpack(r, a, b);
    near = __vminu2(near, __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x5410) - 0x7ffd7ffdu);
    sum = f2_add(sum, r);
  }
  // Lower halves of 0x7ffe to 0x8002 give 1 to 5 (the upper of two perhaps one less,
  // a borrow of the lower); a result that is no number makes the sum none.
  __device__ __forceinline__ bool any() const {
    float a, b;
    f2_unpack(sum, a, b);
    return (near & 0xffffu) <= 7u || (near >> 16) <= 7u || a + b != a + b;
  }
};

// x c + y s, twice.  The product's own error is added to the sum, so that
// cancellation does not raise it: it is off by less than two units in its last place
// (a half by either sum, in the larger sum's units, and 2^-150 where the product's
// error lies below fp32).
__device__ __forceinline__ uint64_t turn2(uint64_t x, uint64_t y, uint64_t c, uint64_t s, Doubt& doubt) {
  const uint64_t minus = f2_pack(-1.f, -1.f);
  const uint64_t p = mul2(y, s), e = fma2(y, mul2(s, minus), p);  // the product, less its error
  const uint64_t r = fma2(e, minus, fma2(x, c, p));
  doubt.see(r);
  return r;
}
__device__ __forceinline__ uint32_t pack2(uint64_t r) {
  float a, b;
  f2_unpack(r, a, b);
  return pack_bf16(a, b);
}
__device__ __forceinline__ uint64_t both(uint32_t w) { return f2_pack(low(w), high(w)); }
__device__ __forceinline__ uint32_t negated(uint32_t w) { return w ^ 0x80008000u; }

// The same of four words' elements.  Few come here: a loop over arrays in local
// memory, as registers would be taken from everyone (112 a thread for 80: rope of
// 32768 tokens 130 us for 101).
__device__ __forceinline__ void turn_again(const uint32_t (&x)[4], const uint32_t (&y)[4], const Pair (&cs)[4],
                                           uint32_t (&r)[4]) {
  uint32_t w[12];
  Pair p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = x[i];
    w[4 + i] = y[i];
    p[i] = cs[i];
  }
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    float c0, c1, s0, s1;
    f2_unpack(p[i].c, c0, c1);
    f2_unpack(p[i].s, s0, s1);
    const uint32_t u = w[i], v = w[4 + i];
    w[8 + i] = pack_bf16(turn_exactly(low(u), c0, low(v), s0), turn_exactly(high(u), c1, high(v), s1));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = w[8 + i];
}

// Eight pairs, in place: the first elements in p and the second in q or, PAIRS,
// neighbours; the first become x c - y s, the second y c + x s.
template <bool PAIRS>
__device__ __forceinline__ void turn_pairs(uint4& p, uint4& q, const Pair (&cs)[4]) {
  uint32_t w[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
  uint32_t r[8];
  // pairs 2 i and 2 i + 1: words i and i + 4, or 2 i and 2 i + 1 with the lower
  // halves' elements the first
  auto first = [&](int i) { return PAIRS ? __byte_perm(w[2 * i], w[2 * i + 1], 0x5410) : w[i]; };
  auto second = [&](int i) { return PAIRS ? __byte_perm(w[2 * i], w[2 * i + 1], 0x7632) : w[i + 4]; };
  auto put = [&](int i, uint32_t x, uint32_t y) {
    r[PAIRS ? 2 * i : i] = PAIRS ? __byte_perm(x, y, 0x5410) : x;
    r[PAIRS ? 2 * i + 1 : i + 4] = PAIRS ? __byte_perm(x, y, 0x7632) : y;
  };
  Doubt doubt;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t x = both(first(i)), y = both(second(i)), ny = both(negated(second(i)));
    put(i, pack2(turn2(x, ny, cs[i].c, cs[i].s, doubt)), pack2(turn2(y, x, cs[i].c, cs[i].s, doubt)));
  }
  if (doubt.any()) {
    uint32_t x[4], y[4], ny[4], xr[4], yr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = first(i);
      y[i] = second(i);
      ny[i] = negated(y[i]);
    }
    turn_again(x, ny, cs, xr);
    turn_again(y, x, cs, yr);
#pragma unroll
    for (int i = 0; i < 4; ++i) put(i, xr[i], yr[i]);
  }
  p = make_uint4(r[0], r[1], r[2], r[3]);
  q = make_uint4(r[4], r[5], r[6], r[7]);
}

// The two vectors of eight elements that lane i of a row takes: i and i + rot / 16 or,
// where they pass or neighbours are pairs, 2 i and 2 i + 1.  They turn among
// themselves, by the row's eight (cos, sin) from 8 i on.
struct Vectors {
  int first, second;
};
template <bool PAIRS>
__device__ __forceinline__ Vectors vectors_of(int i, int rot) {
  const int items = rot / 16;
  return !PAIRS && i < items ? Vectors{i, i + items} : Vectors{2 * i, 2 * i + 1};
}

// Eight (cos, sin) of a table's row, sines times `sign`.
__device__ __forceinline__ void load_angles(const float2* from, float sign, Pair (&cs)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(from + 2 * i));
    cs[i] = {f2_pack(v.x, v.z), f2_pack(sign * v.y, sign * v.w)};
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

// D / 16 lanes take a token's row, each two vectors, and keep their cos and sin for
// their group of heads.  A head's elements are on their way while the one before is
// turned, the first ones before the position is known.
//
// Bound by DRAM: 32768 rows of 32 heads of 128 (the gradient's) in 96 us, 5.7 TB/s;
// 9001 tokens of 40 heads, half of each in neighbours, in 38 us.  Seven CTAs per SM:
// with four heads' elements on their way a thread had 112 registers, and the first
// took 130 us.  Latency for few: 64 tokens in 2.9 us, with the position, then its row
// of the table to wait for.
template <int D, bool PAIRS>
__global__ void __launch_bounds__(rope::kThreads, 7) fa_rope_kernel(RopeArgs a) {
  using namespace rope;
  constexpr int kLanes = D / 16;
  const long long at = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) / kLanes;
  if (at >= static_cast<long long>(a.B) * a.N) return;
  const int i = threadIdx.x % kLanes;
  const int b = static_cast<int>(at / a.N), n = static_cast<int>(at - static_cast<long long>(b) * a.N);
  const int h0 = blockIdx.y * a.group, h1 = min(a.H, h0 + a.group);
  const Vectors v = vectors_of<PAIRS>(i, a.rot);
  const __nv_bfloat16* x = a.x + b * a.xb + n * a.xn;
  __nv_bfloat16* out = a.out + b * a.ob + n * a.on;
  uint4 p, q;
  auto load = [&](int h) {
    const uint4* from = reinterpret_cast<const uint4*>(x + h * a.xh);
    p = from[v.first];
    q = from[v.second];
  };
  load(h0);
  const int pos = a.positions[b * a.pb + n];
  if (pos >= a.length && i == 0 && h0 == 0) record_index_error(a.err, kSiteRopePosition, n);
  const bool turns = 16 * i < a.rot && pos >= 0 && pos < a.length;
  Pair cs[4];
  if (turns) load_angles(a.table + static_cast<long long>(pos) * (a.rot / 2) + 8 * i, a.sign, cs);
#pragma unroll 1
  for (int h = h0; h < h1; ++h) {
    uint4 p0 = p, q0 = q;
    if (h + 1 < h1) load(h + 1);  // (out may be x: another head's row)
    if (turns) turn_pairs<PAIRS>(p0, q0, cs);
    uint4* to = reinterpret_cast<uint4*>(out + h * a.oh);
    to[v.first] = p0;
    to[v.second] = q0;
  }
}

}  // namespace fa
