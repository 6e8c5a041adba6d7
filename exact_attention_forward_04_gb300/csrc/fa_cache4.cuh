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

// Sixteen bf16 to codes and their scale:
//   s = E4M3(max |x| / (6 unit)), nearest even, at most 448;  code = E2M1(x / (s unit)), 0 where s = 0.
// A quotient is taken as a product with a reciprocal, off by 2^-23 of it, and
// rounded to 16 bits: x has 8 bits and s times a border between two codes at most
// 7, so that their quotient is the border itself or 2^-9 of it away, and the
// product ends on the border exactly where the quotient lies on it.
__device__ __forceinline__ uint2 quantise16(const uint32_t (&w)[8], float inv_unit, uint32_t& scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = amax2(w[i], m);
  m = min(m, 0x7f80u);  // not a number: as infinity
  const float want = __fdiv_rn(__uint_as_float(m << 16) * inv_unit, 6.f);
  asm("{\n\t.reg .b16 a;\n\tcvt.rn.satfinite.e4m3x2.f32 a, %1, %2;\n\tcvt.u32.u16 %0, a;\n}"
      : "=r"(scale)
      : "f"(0.f), "f"(want));
  const float s = f16_low(e4m3x2_to_f16(scale));
  const float inv = s > 0.f ? __fdiv_rn(1.f, s) * inv_unit : 0.f;
  uint32_t r[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = (i & 1) ? rope::high(w[4 * e + i / 2]) : rope::low(w[4 * e + i / 2]);
      f[i] = __uint_as_float((__float_as_uint(x * inv) + 0x80u) & 0xffffff00u);
    }
    r[e] = pack_e2m1x8(f);
  }
  return make_uint2(r[0], r[1]);
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

// New K and V rows into the cache.  A lane takes 16 elements of a row, one group:
// their scale needs nobody else's.  A warp takes 4 tokens (8 at d = 64) and a run of
// heads, so that K's bytes are stored 256 and V's 32 in a row and a position's cos
// and sin are read once for several heads.  Halves to be turned together lie in
// two lanes; each reads the other's elements from L1.
template <int D, bool PAIRS>
__global__ void __launch_bounds__(c4::kThreads) fa_cache4_append_kernel(Append4Args a) {
  using namespace c4;
  using G = Granule<D>;
  constexpr int kLanes = D / 16;
  const int t = (blockIdx.x * kThreads + threadIdx.x) / kLanes, c = threadIdx.x % kLanes;
  const int g0 = blockIdx.y * a.group, g1 = min(2 * a.Hkv, g0 + a.group);
  if (t >= a.T) return;
  const long long slot = a.slot_map[t];
  if (slot < 0 || slot >= a.slots) {
    if (slot != -1 && c == 0 && g0 == 0) record_index_error(a.err, kSiteAppendSlot, t);
    return;
  }
  const int P = 1 << a.sh, token = static_cast<int>(slot) & 15;
  uint8_t* block = a.data + (slot >> a.sh) * a.Hkv * (P / 16) * G::kBytes +
                   static_cast<long long>((static_cast<int>(slot) & (P - 1)) >> 4) * G::kBytes;
  // the angles of this lane's elements: those of vectors 2 c and 2 c + 1
  float2 cs[2][8];
  int partner[2] = {-1, -1};  // vector that each turns with; -1: it passes
  if (a.positions && g0 < a.Hkv && 16 * c < a.rot) {
    const int pos = a.positions[t];
    if (pos >= a.length && c == 0 && g0 == 0) record_index_error(a.err, kSiteRopePosition, t);
    if (pos >= 0 && pos < a.length) {
      const float2* row = a.table + static_cast<long long>(pos) * (a.rot / 2);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int v = 2 * c + e, half = a.rot / 16;
        if constexpr (PAIRS) {
          float2 p[4];
          rope::load_pairs<4>(row + 4 * v, 1.f, p);
          rope::spread(p, cs[e]);
          partner[e] = v;
        } else {
          const bool first = v < half;
          rope::load_pairs<8>(row + 8 * (first ? v : v - half), first ? -1.f : 1.f, cs[e]);
          partner[e] = first ? v + half : v - half;
        }
      }
    }
  }
  const bool turns = partner[0] >= 0;
#pragma unroll 1
  for (int g = g0; g < g1; ++g) {
    const bool is_v = g >= a.Hkv;
    const int h = is_v ? g - a.Hkv : g;
    const uint4* row = reinterpret_cast<const uint4*>((is_v ? a.v + t * a.v_stride : a.k + t * a.k_stride) +
                                                      static_cast<long long>(h) * D);
    uint4 x[2] = {__ldg(row + 2 * c), __ldg(row + 2 * c + 1)};
    if (!is_v && turns) {
      if constexpr (PAIRS) {
#pragma unroll
        for (int e = 0; e < 2; ++e) x[e] = rope::turn8(x[e], rope::swap_pairs(x[e]), cs[e]);
      } else {
        const uint4 y[2] = {__ldg(row + partner[0]), __ldg(row + partner[1])};
#pragma unroll
        for (int e = 0; e < 2; ++e) x[e] = rope::turn8(x[e], y[e], cs[e]);
      }
    }
    const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    uint32_t scale;
    const uint2 code = quantise16(w, is_v ? a.v_inv : a.k_inv, scale);
    uint8_t* gr = block + static_cast<long long>(h) * (P / 16) * G::kBytes;
    if (!is_v) {
      *reinterpret_cast<uint2*>(gr + token * G::kRow + k_place<D>(c) * 8) = code;
      gr[G::kKScales + token * (D / 16) + k_place<D>(c)] = static_cast<uint8_t>(scale);
    } else {
      if constexpr (D == 128) {
        *reinterpret_cast<uint2*>(gr + G::kV + v_place<D>(c, token)) = code;
      } else {
        *reinterpret_cast<uint32_t*>(gr + G::kV + v_place<D>(2 * c, token)) = code.x;
        *reinterpret_cast<uint32_t*>(gr + G::kV + v_place<D>(2 * c + 1, token)) = code.y;
      }
      gr[G::kVScales + c * 16 + scale_place(token)] = static_cast<uint8_t>(scale);
    }
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
// there is none.  Lanes as in the append.
template <int D>
__global__ void __launch_bounds__(c4::kThreads) fa_cache4_read_kernel(Read4Args a) {
  using namespace c4;
  using G = Granule<D>;
  constexpr int kLanes = D / 16;
  const int t = (blockIdx.x * kThreads + threadIdx.x) / kLanes, c = threadIdx.x % kLanes;
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
