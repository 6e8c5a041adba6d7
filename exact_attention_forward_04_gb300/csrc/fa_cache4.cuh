// The 4-bit key/value cache: its layout, appends and reads.
//
// A row (one token and kv head of K or of V) is d codes of 4 bits, E2M1 (0, .5, 1,
// 1.5, 2, 3, 4, 6 and a sign), and an E4M3 scale for each 16 of them; the value
// is E2M1(code) * E4M3(scale) * unit, the unit a power of two for all of the
// cache's K or V.  A value without its unit has six significant bits between
// 2^-10 and 2688: f16 holds it exactly, so the products of attention take it as
// it is and a scale costs one multiplication of two values.  Scales belong to one
// token each, so an append writes its own bytes and nothing else: it reads
// nothing back, and no two tokens of a call can be in each other's way.
//
// Granules.  The rows of 16 tokens of a block and head lie together, K codes, K
// scales, V codes, V scales, 18 d bytes, so that a tile of the attention is one
// bulk copy, and in the order in which a warp's products take them, so that
// its reads need neither a swizzle by a tensor map nor a shuffle:
//   K codes   token by token; a lane of a quad takes groups t and t + 4 (d = 64:
//             t), so the groups of a row come in the order 0 4 1 5 2 6 3 7
//   V codes   eight pieces of d / 8 elements, in each token by token: a lane
//             takes one piece of tokens 2 t, 2 t + 1, 2 t + 8, 2 t + 9.  The pieces
//             of half the lanes have tokens 0-7 and 8-15 exchanged, so that
//             eight lanes' reads touch every bank once.
//   V scales  group by group, tokens 0 1 8 9 2 3 10 11 ..: a lane's four in a word
#pragma once
#include <cuda_bf16.h>

#include "fa_cache.cuh"
#include "fa_rope.cuh"

namespace fa {

namespace c4 {

constexpr int kTokens = 16;  // of a granule
template <int D>
struct Granule {
  static constexpr int kRow = D / 2;          // bytes of a row's codes
  static constexpr int kKScales = 8 * D;      // where each part begins
  static constexpr int kV = 9 * D;
  static constexpr int kVScales = 17 * D;
  static constexpr int kBytes = 18 * D;
  static constexpr int kPiece = D / 16;       // bytes of a token in a piece of V
};
// Place of a K row's 16-element group.
template <int D>
__device__ __forceinline__ int k_place(int group) {
  return D == 128 ? (group & 3) * 2 + (group >> 2) : group;
}
// Offset, among V's codes, of a token's bytes of piece p.
template <int D>
__device__ __forceinline__ int v_place(int p, int token) {
  const int flip = D == 128 ? p & 1 : (p >> 1) & 1;
  return p * D + (token ^ (flip * 8)) * Granule<D>::kPiece;
}
// Place of a token's V scale among its group's.
__device__ __forceinline__ int scale_place(int token) {
  return ((token & 7) >> 1) * 4 + (token >> 3) * 2 + (token & 1);
}

// Eight values to eight codes, the first in the lowest bits; rounded to nearest
// even, at most 6.
__device__ __forceinline__ uint32_t pack_e2m1x8(const float (&f)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}
// Eight codes to four pairs of f16, exact.  (2 cycles a pair for a quarter of an SM;
// placing the bits by shifts and masks took 5.)
__device__ __forceinline__ void e2m1_to_f16(uint32_t w, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n}"
      : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
      : "r"(w));
}
// Two E4M3 numbers to f16, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float f16_low(uint32_t w) {
  float f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, a;\n}" : "=f"(f) : "r"(w));
  return f;
}
__device__ __forceinline__ float f16_high(uint32_t w) { return f16_low(w >> 16); }

// A group's scale and codes of its elements x:
//   s = E4M3(max |x| / (6 unit)), nearest even, at most 448;  code = E2M1(x / (s unit)), 0 where s = 0.
// Both quotients are taken as products with reciprocals, off by 2^-22 of them, and
// rounded to multiples of fewer bits: x has 8 bits and 6 or s times a border
// between two codes or scales at most 7, so that a quotient is the border itself or
// 2^-9 of it away, and the product ends on the border exactly where the quotient
// lies on it.

// The scale's code, of the largest |x| as bf16 bits; `inv` is 1 / (s unit) or 0.
__device__ __forceinline__ uint32_t scale_code(uint32_t amax, float inv_unit, float& inv) {
  const float x = __uint_as_float(min(amax, 0x7f80u) << 16);  // not a number: as infinity
  const float want = __uint_as_float((__float_as_uint(x * inv_unit * (1.f / 6.f)) + 0x80u) & 0xffffff00u);
  uint32_t code;
  asm("{\n\t.reg .b16 a;\n\tcvt.rn.satfinite.e4m3x2.f32 a, %1, %2;\n\tcvt.u32.u16 %0, a;\n}"
      : "=r"(code)
      : "f"(0.f), "f"(want));
  const float s = f16_low(e4m3x2_to_f16(code));
  asm("rcp.approx.f32 %0, %1;" : "=f"(inv) : "f"(s));
  inv = s > 0.f ? inv * inv_unit : 0.f;
  return code;
}
// Eight elements' codes.  A quotient (about 6 at most, borders from 1/4 on) is rounded
// to multiples of 2^-13 by adding 1024 and taking it away again, in pairs.
__device__ __forceinline__ uint32_t codes8(uint4 v, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const uint64_t inv2 = f2_pack(inv, inv), up = f2_pack(1024.f, 1024.f), down = f2_pack(-1024.f, -1024.f);
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f2_unpack(f2_add(f2_fma(rope::both(w[i]), inv2, up), down), f[2 * i], f[2 * i + 1]);
  return pack_e2m1x8(f);
}
// The largest |x| of eight, as bf16 bits.
__device__ __forceinline__ uint32_t amax8(uint4 v) {
  const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                              __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
  return max(m & 0xffffu, m >> 16);
}

constexpr int kThreads = 128;

}  // namespace c4

struct Append4Args {
  const __nv_bfloat16* k;     // [T][Hkv][D] with a token stride
  const __nv_bfloat16* v;
  long long k_stride, v_stride;
  uint8_t* data;              // [blocks][Hkv][P / 16][18 D]
  const long long* slot_map;  // [T]
  long long slots;            // blocks * P
  int T, Hkv, sh;             // blocks of P = 2^sh tokens
  int group;                  // rows (heads of K, then of V) of a warp
  float k_inv, v_inv;         // 1 / unit
  const int* positions;       // [T]; null: K is not turned
  const float2* table;        // [length][rot / 2] (cos, sin)
  int length, rot;
  DevError* err;
};

// New K and V rows into the cache.  D / 16 lanes take a row, two vectors of eight
// elements each: of V, and of K's elements that pass, one group of 16; of those that
// turn the two that turn among themselves, so that a lane keeps eight cos and sin for
// all heads, and a vector's group has its other half in a lane that a shuffle asks for
// its largest element.  A warp takes 4 tokens (8 at d = 64) and a run of rows, heads of
// K, then of V, so that K's bytes are stored 256 and V's 32 in a row; a row's elements
// are on their way while the one before is written.
//
// 24 prompts, 51072 tokens of 8 kv heads of 128 in blocks of 64: 67 us with all of K
// turned, 4.0 TB/s, 55 without; ALU 54 %, issue slots 61 %, DRAM 57 %.  What it takes
// beyond 40 us of bytes: where halves turn, two scale codes a lane in place of one and
// four shuffles for their maxima, and stores of 1 to 8 bytes.  Seven CTAs per SM (78 us
// with six, and 104 with four rows' elements on their way in four; 92 with cos and sin
// read again for every head).  32 tokens in 3.3 us, 500 of 16 heads of 64 in 3.7, a
// microsecond of it for position and table one after the other.
template <int D, bool PAIRS>
__global__ void __launch_bounds__(c4::kThreads, 7) fa_cache4_append_kernel(Append4Args a) {
  using namespace c4;
  using G = Granule<D>;
  constexpr int kLanes = D / 16;
  const int t = static_cast<int>((static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) / kLanes);
  const int c = threadIdx.x % kLanes;
  const int g0 = blockIdx.y * a.group, g1 = min(2 * a.Hkv, g0 + a.group);
  const bool token_there = t < a.T;
  const int tt = token_there ? t : a.T - 1;
  // the vectors of K (rot is 0 where nothing turns)
  const rope::Vectors kv = rope::vectors_of<PAIRS>(c, a.rot);
  const __nv_bfloat16 *krow = a.k + tt * a.k_stride, *vrow = a.v + tt * a.v_stride;
  const int k0 = min(g0, a.Hkv), k1 = min(g1, a.Hkv), v0 = max(g0, a.Hkv) - a.Hkv, v1 = max(g1, a.Hkv) - a.Hkv;
  const uint4* from = reinterpret_cast<const uint4*>(k0 < k1 ? krow + static_cast<long long>(k0) * D
                                                             : vrow + static_cast<long long>(v0) * D);
  uint4 x[2];
  auto load = [&](const uint4* row, int first, int second) {
    x[0] = __ldg(row + first);
    x[1] = __ldg(row + second);
  };
  if (k0 < k1) load(from, kv.first, kv.second);
  else load(from, 2 * c, 2 * c + 1);
  const long long slot = a.slot_map[tt];
  const bool there = token_there && slot >= 0 && slot < a.slots;
  if (token_there && !there && slot != -1 && c == 0 && g0 == 0) record_index_error(a.err, kSiteAppendSlot, t);
  const int P = 1 << a.sh, token = static_cast<int>(slot) & 15;
  const long long head = static_cast<long long>(P / 16) * G::kBytes;  // bytes of a block's head
  uint8_t* block = a.data + (slot >> a.sh) * a.Hkv * head +
                   static_cast<long long>((static_cast<int>(slot) & (P - 1)) >> 4) * G::kBytes;
  rope::Pair cs[4];
  bool turns = false;
  if (a.positions && g0 < a.Hkv && 16 * c < a.rot) {
    const int pos = a.positions[tt];
    if (there && pos >= a.length && c == 0 && g0 == 0) record_index_error(a.err, kSiteRopePosition, t);
    turns = pos >= 0 && pos < a.length;
    if (turns) rope::load_angles(a.table + static_cast<long long>(pos) * (a.rot / 2) + 8 * c, 1.f, cs);
  }
  // where the other halves of the vectors' groups are: five bits of a lane and one of
  // which of its two vectors, for each
  const bool apart = kv.second != kv.first + 1 || (kv.first & 1);
  int other = 0;
  if (apart) {
    const int items = a.rot / 16;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int u = (e ? kv.second : kv.first) ^ 1;
      const int lane = (threadIdx.x & 31) - c + (u < items ? u : u < 2 * items ? u - items : u >> 1);
      other |= (lane | (u < items ? 0 : u < 2 * items ? 32 : (u & 1) * 32)) << (8 * e);
    }
  }
  const bool any_apart = !PAIRS && a.rot > 16;
  uint8_t* gr = block + k0 * head;
  int at0 = token * G::kRow + k_place<D>(kv.first >> 1) * 8 + (kv.first & 1) * 4;
  int at1 = token * G::kRow + k_place<D>(kv.second >> 1) * 8 + (kv.second & 1) * 4;
  // a group's scale by the lane with its first vector
  int scale0 = kv.first & 1 ? 0 : G::kKScales + token * (D / 16) + k_place<D>(kv.first >> 1);
  const int scale1 = kv.second & 1 ? 0 : G::kKScales + token * (D / 16) + k_place<D>(kv.second >> 1);
#pragma unroll 1
  for (int h = k0; h < k1; ++h, gr += head) {
    uint4 v[2] = {x[0], x[1]};
    from += D / 8;
    if (h + 1 < k1) load(from, kv.first, kv.second);
    else if (v0 < v1) load(reinterpret_cast<const uint4*>(vrow), 2 * c, 2 * c + 1);
    if (turns) rope::turn_pairs<PAIRS>(v[0], v[1], cs);
    uint32_t m0 = amax8(v[0]), m1 = amax8(v[1]);
    if (any_apart) {
      uint32_t o[2][2];  // the largest of both vectors of the lanes asked
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        o[e][0] = __shfl_sync(0xffffffffu, m0, other >> (8 * e));
        o[e][1] = __shfl_sync(0xffffffffu, m1, other >> (8 * e));
      }
      if (apart) {
        m0 = max(m0, other & 32 ? o[0][1] : o[0][0]);
        m1 = max(m1, other & (32 << 8) ? o[1][1] : o[1][0]);
      }
    }
    if (!apart) m0 = m1 = max(m0, m1);
    if (!there) continue;
    float i0, i1;
    const uint32_t s0 = scale_code(m0, a.k_inv, i0), s1 = scale_code(m1, a.k_inv, i1);
    *reinterpret_cast<uint32_t*>(gr + at0) = codes8(v[0], i0);
    *reinterpret_cast<uint32_t*>(gr + at1) = codes8(v[1], i1);
    if (scale0 > 0) gr[scale0] = static_cast<uint8_t>(s0);
    if (scale1 > 0) gr[scale1] = static_cast<uint8_t>(s1);
  }
  from = reinterpret_cast<const uint4*>(vrow + static_cast<long long>(v0) * D);
  gr = block + v0 * head;
  at0 = G::kV + v_place<D>(D == 128 ? c : 2 * c, token);
  at1 = G::kV + v_place<D>(D == 128 ? c : 2 * c + 1, token);
  scale0 = G::kVScales + c * 16 + scale_place(token);
#pragma unroll 1
  for (int h = v0; h < v1; ++h, gr += head) {
    uint4 v[2] = {x[0], x[1]};
    from += D / 8;
    if (h + 1 < v1) load(from, 2 * c, 2 * c + 1);
    if (!there) continue;
    float inv;
    const uint32_t s = scale_code(max(amax8(v[0]), amax8(v[1])), a.v_inv, inv);
    const uint32_t c0 = codes8(v[0], inv), c1 = codes8(v[1], inv);
    if constexpr (D == 128) {
      *reinterpret_cast<uint2*>(gr + at0) = make_uint2(c0, c1);
    } else {
      *reinterpret_cast<uint32_t*>(gr + at0) = c0;
      *reinterpret_cast<uint32_t*>(gr + at1) = c1;
    }
    gr[scale0] = static_cast<uint8_t>(s);
  }
}

struct Read4Args {
  const uint8_t* data;
  const long long* slot_map;  // [T]
  long long slots;
  __nv_bfloat16* k;           // [T][Hkv][D]
  __nv_bfloat16* v;
  int T, Hkv, sh, group;
  float k_unit, v_unit;
  DevError* err;
};

// The rows at some slots as bf16, which holds every value exactly; zeros where
// there is none.  A lane takes one group.  Bound by DRAM: the rows of 24 prompts in
// 47 us, 5.7 TB/s.
template <int D>
__global__ void __launch_bounds__(c4::kThreads) fa_cache4_read_kernel(Read4Args a) {
  using namespace c4;
  using G = Granule<D>;
  constexpr int kLanes = D / 16;
  const int t = static_cast<int>((static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) / kLanes);
  const int c = threadIdx.x % kLanes;
  const int g0 = blockIdx.y * a.group, g1 = min(2 * a.Hkv, g0 + a.group);
  if (t >= a.T) return;
  const long long slot = a.slot_map[t];
  const bool there = slot >= 0 && slot < a.slots;
  if (!there && slot != -1 && c == 0 && g0 == 0) record_index_error(a.err, kSiteReadSlot, t);
  const int P = 1 << a.sh, token = static_cast<int>(slot) & 15;
  const uint8_t* block = a.data + (there ? (slot >> a.sh) * a.Hkv * (P / 16) * G::kBytes +
                                               static_cast<long long>((static_cast<int>(slot) & (P - 1)) >> 4) * G::kBytes
                                         : 0);
#pragma unroll 2
  for (int g = g0; g < g1; ++g) {
    const bool is_v = g >= a.Hkv;
    const int h = is_v ? g - a.Hkv : g;
    uint4 r[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    if (there) {
      const uint8_t* gr = block + static_cast<long long>(h) * (P / 16) * G::kBytes;
      uint2 code;
      uint32_t scale;
      if (!is_v) {
        code = *reinterpret_cast<const uint2*>(gr + token * G::kRow + k_place<D>(c) * 8);
        scale = gr[G::kKScales + token * (D / 16) + k_place<D>(c)];
      } else {
        if constexpr (D == 128) {
          code = *reinterpret_cast<const uint2*>(gr + G::kV + v_place<D>(c, token));
        } else {
          code = make_uint2(*reinterpret_cast<const uint32_t*>(gr + G::kV + v_place<D>(2 * c, token)),
                            *reinterpret_cast<const uint32_t*>(gr + G::kV + v_place<D>(2 * c + 1, token)));
        }
        scale = gr[G::kVScales + c * 16 + scale_place(token)];
      }
      const float s = f16_low(e4m3x2_to_f16(scale)) * (is_v ? a.v_unit : a.k_unit);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t f[4], o[4];
        e2m1_to_f16(e ? code.y : code.x, f[0], f[1], f[2], f[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pack_bf16(f16_low(f[i]) * s, f16_high(f[i]) * s);
        r[e] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    uint4* to = reinterpret_cast<uint4*>((is_v ? a.v : a.k) + (static_cast<long long>(t) * a.Hkv + h) * D);
    to[2 * c] = r[0];
    to[2 * c + 1] = r[1];
  }
}

}  // namespace fa
