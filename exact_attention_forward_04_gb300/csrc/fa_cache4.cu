// C ABI of the 4-bit key/value cache (declared in include/fa_fwd.h): argument
// validation and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "fa_cache4.cuh"
#include "fa_cache4_prompt.cuh"
#include "fa_cache_fwd.cuh"
#include "fa_cache_host.h"
#include "fa_fwd.h"
#include "fa_host.h"

namespace fa {
namespace {

using namespace cachehost;

size_t cache_bytes(int Hkv, int d, int blocks, int P) {
  return static_cast<size_t>(blocks) * Hkv * (P / c4::kTokens) * 18 * d;
}

// A power of two of 2^-64 to 2^64: it and a scale's reciprocal, and every product
// of the two, are normal.
bool unit_ok(float u) {
  int e = 0;
  return std::isfinite(u) && std::frexp(u, &e) == 0.5f && e >= -63 && e <= 65;
}

// ------------------------------------------------------------------ append

int cache4_append(const void* k, const void* v, long long k_stride, long long v_stride, void* data, float k_unit,
                  float v_unit, const long long* slot_map, const int* positions, const float* table, int length,
                  int rot, int interleaved, int T, int Hkv, int d, int blocks, int P, cudaStream_t s) {
  int st = check_cache(Hkv, d, blocks, P);
  if (st != FA_OK) return st;
  if (T < 0 || !unit_ok(k_unit) || !unit_ok(v_unit)) return FA_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return FA_ERR_INVALID_ARG;
  if (positions) {
    if (!table || length <= 0) return FA_ERR_INVALID_ARG;
    if (rot <= 0 || rot > d || rot % 16 != 0) return FA_ERR_UNSUPPORTED;
  }
  if (T == 0) return FA_OK;
  if (!k || !v || !data || !slot_map) return FA_ERR_INVALID_ARG;
  const long long row = static_cast<long long>(Hkv) * d;
  if (T > 1 && (k_stride < row || v_stride < row)) return FA_ERR_INVALID_ARG;
  if ((k_stride | v_stride) & 7) return FA_ERR_MISALIGNED;
  if (k_stride > (1ll << 40) || v_stride > (1ll << 40)) return FA_ERR_UNSUPPORTED;
  if (misaligned(k, 16) || misaligned(v, 16) || misaligned(data, 16) || misaligned(slot_map, 8) ||
      misaligned(positions, 4) || (positions && misaligned(table, 16)))
    return FA_ERR_MISALIGNED;
  const size_t n = static_cast<size_t>(T), nx = 2 * static_cast<size_t>(row);
  if (overlapping({{data, cache_bytes(Hkv, d, blocks, P)}},
                  {{k, (n - 1) * k_stride * 2 + nx},
                   {v, (n - 1) * v_stride * 2 + nx},
                   {slot_map, 8 * n},
                   {positions, positions ? 4 * n : 0},
                   {table, positions ? static_cast<size_t>(length) * rot * 4 : 0}}))
    return FA_ERR_INVALID_ARG;
  host::Device dev;
  if ((st = host::device(&dev)) != FA_OK) return st;
  Append4Args a{};
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.data = static_cast<uint8_t*>(data);
  a.slot_map = slot_map;
  a.slots = static_cast<long long>(blocks) * P;
  a.T = T;
  a.Hkv = Hkv;
  a.sh = block_shift(P);
  a.k_inv = 1.f / k_unit;
  a.v_inv = 1.f / v_unit;
  a.positions = positions;
  a.table = reinterpret_cast<const float2*>(table);
  a.length = length;
  a.rot = positions ? rot : 0;
  a.err = dev.index_err;
  // Rows of a thread, by the lanes that one each would give an SM.  Measured (us, K
  // turned; tokens of 8 kv heads of 128, as many of 16 of 64 within 5 %), rows 1 / 2 / 4 / 8 / 16:
  //   1000 (842)      4.4 / 5.4 / 6.5 / 8.6 / 10.2     8000 (6736)    18.9 / 15.1 / 13.9 / 14.9 / 18.8
  //   2000 (1684)     6.1 / 6.3 / 7.2 / 9.3 / 13.2     16000 (13473)  34.9 / 27.2 / 24.4 / 23.7 / 26.1
  //   4000 (3368)    10.9 / 9.1 / 9.5 / 12.1 / 16.4    51000 (42947)  106.7 / 81.9 / 71.8 / 67.1 / 67.6
  const long long lanes = static_cast<long long>(T) * (d / 16), per_sm = lanes * 2 * Hkv / dev.sms;
  a.group = per_sm <= 2048 ? 1 : per_sm <= 8192 ? 4 : 8;
  while ((2 * Hkv + a.group - 1) / a.group > 65535) a.group *= 2;
  const dim3 grid(static_cast<unsigned>((lanes + c4::kThreads - 1) / c4::kThreads),
                  static_cast<unsigned>((2 * Hkv + a.group - 1) / a.group));
  if (d == 128) {
    if (interleaved) fa_cache4_append_kernel<128, true><<<grid, c4::kThreads, 0, s>>>(a);
    else fa_cache4_append_kernel<128, false><<<grid, c4::kThreads, 0, s>>>(a);
  } else {
    if (interleaved) fa_cache4_append_kernel<64, true><<<grid, c4::kThreads, 0, s>>>(a);
    else fa_cache4_append_kernel<64, false><<<grid, c4::kThreads, 0, s>>>(a);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FA_OK : host::fail(e);
}

// -------------------------------------------------------------------- read

int cache4_read(const void* data, float k_unit, float v_unit, const long long* slot_map, void* k, void* v, int T,
                int Hkv, int d, int blocks, int P, cudaStream_t s) {
  int st = check_cache(Hkv, d, blocks, P);
  if (st != FA_OK) return st;
  if (T < 0 || !unit_ok(k_unit) || !unit_ok(v_unit)) return FA_ERR_INVALID_ARG;
  if (T == 0) return FA_OK;
  if (!data || !slot_map || !k || !v) return FA_ERR_INVALID_ARG;
  if (misaligned(data, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(slot_map, 8))
    return FA_ERR_MISALIGNED;
  const size_t n = static_cast<size_t>(T) * Hkv * d * 2;
  if (overlapping({{k, n}, {v, n}}, {{data, cache_bytes(Hkv, d, blocks, P)}, {slot_map, 8 * static_cast<size_t>(T)}}))
    return FA_ERR_INVALID_ARG;
  host::Device dev;
  if ((st = host::device(&dev)) != FA_OK) return st;
  Read4Args a{};
  a.data = static_cast<const uint8_t*>(data);
  a.slot_map = slot_map;
  a.slots = static_cast<long long>(blocks) * P;
  a.k = static_cast<__nv_bfloat16*>(k);
  a.v = static_cast<__nv_bfloat16*>(v);
  a.T = T;
  a.Hkv = Hkv;
  a.sh = block_shift(P);
  a.k_unit = k_unit;
  a.v_unit = v_unit;
  a.err = dev.index_err;
  // as the append:
  //   2000 (1684)     3.8 / 3.9 / 3.9 / 5.1 / 7.3      16000 (13473)  16.7 / 16.1 / 17.6 / 19.6 / 17.3
  //   8000 (6736)     9.4 / 9.5 / 10.5 / 9.9 / 13.5    51000 (42947)  51.7 / 47.1 / 47.4 / 50.7 / 58.0
  const long long lanes = static_cast<long long>(T) * (d / 16), per_sm = lanes * 2 * Hkv / dev.sms;
  a.group = per_sm <= 8192 ? 1 : 2;
  while ((2 * Hkv + a.group - 1) / a.group > 65535) a.group *= 2;
  const dim3 grid(static_cast<unsigned>((lanes + c4::kThreads - 1) / c4::kThreads),
                  static_cast<unsigned>((2 * Hkv + a.group - 1) / a.group));
  if (d == 128) fa_cache4_read_kernel<128><<<grid, c4::kThreads, 0, s>>>(a);
  else fa_cache4_read_kernel<64><<<grid, c4::kThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FA_OK : host::fail(e);
}

// ----------------------------------------------------------------- forward

// Query rows of a unit, and with them the kernel, by the average rows a request
// has per kv head: the few-row kernel with 8 or, at d = 128, 16, which reads the keys
// again for every so many, or the many-row one with 256.  Measured (us; lengths evenly
// up to 4000 for 64 requests of 8 kv heads, of 8000 for one), rows of 8 / 16 / 256 a
// unit:
//   rows per kv head          8               16                24                32                48
//   64 requests, d = 128  54 / 68 / 111   91 / 75 / 111   130 / 127 / 112   163 / 131 / 112   241 / 187 / 115
//                d = 64   35 / 52 / 89    56 / 56 / 89     77 / 89 / 89      99 / 94 / 90     142 / 132 / 91
//   one request, d = 128  17 / 17 / 25    17 / 19 / 25     19 / 21 / 25      19 / 21 / 25      23 / 23 / 26
//                d = 64   17 / 15 / 22    17 / 17 / 23     17 / 17 / 23      17 / 17 / 23      19 / 19 / 23
int unit_rows4(int R, int T, int Hq, int Hkv, int d, int sms) {
  const long long rows = static_cast<long long>(T) * (Hq / Hkv);
  const bool few = static_cast<long long>(R) * Hkv * 8 <= sms;
  if (rows <= (few ? 48ll : d == 64 ? 24ll : 8ll) * R) return 8;
  return d == 128 && rows <= 16ll * R ? 16 : prm4::kRows;
}

size_t cache4_workspace(int R, int T, int Hq, int Hkv, int d) {
  if ((d != 64 && d != 128) || R <= 0 || T <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return 0;
  host::Device dev;
  if (host::device(&dev) != FA_OK) return 0;
  const int rows = unit_rows4(R, T, Hq, Hkv, d, dev.sms);
  return workspace_bytes(fwd_grid(dev.sms, rows, d), rows, d);
}

// By device and d (64, 128): 8 rows, 16 rows, many.
bool g_ready[64][2][3] = {};

template <int D, int ROWS>
int launch_few(CacheFwdArgs& a, int P, int grid, bool& done, cudaStream_t s) {
  using Ly = dec::Layout<D, ROWS, E2M1Codes>;
  const int st = ready(fa_cache_fwd_kernel<D, ROWS, E2M1Codes>, Ly::kAlloc, done);
  if (st != FA_OK) return st;
  fa_cache_fwd_kernel<D, ROWS, E2M1Codes><<<grid, Ly::kThreads, Ly::kAlloc, s>>>(E2M1Codes::Maps{}, a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return host::fail(e);
  // a unit of one tile is never split: nothing to merge
  if (static_cast<long long>(a.M) * P <= Ly::kTile) return FA_OK;
  return launch_merge<D, ROWS, E2M1Codes>(a, grid, 1, s);
}

template <int D>
int launch_cache4_fwd(CacheFwdArgs& a, int P, char* ws, const host::Device& dev, cudaStream_t s) {
  const int unit = unit_rows4(a.R, a.T, a.Hq, a.Hkv, D, dev.sms), grid = fwd_grid(dev.sms, unit, D);
  set_workspace(a, ws, grid, unit, D);
  bool* set = g_ready[dev.dev][D == 128];
  if (unit == prm4::kRows) {
    using Ly = prm4::Layout<D>;
    const int st = ready(fa_cache4_prompt_kernel<D>, Ly::kAlloc, set[2], 128);
    if (st != FA_OK) return st;
    fa_cache4_prompt_kernel<D><<<grid, prm4::kThreads, Ly::kAlloc, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return host::fail(e);
    if (static_cast<long long>(a.M) * P <= prm4::kKeys) return FA_OK;
    return launch_merge<D, prm4::kRows, E2M1Codes>(a, grid, 4, s);
  }
  if constexpr (D == 128) {
    if (unit == 16) return launch_few<D, 16>(a, P, grid, set[1], s);
  }
  return launch_few<D, 8>(a, P, grid, set[0], s);
}

int cache4_fwd(const FwdCall& c, const void* data, float k_unit, float v_unit, cudaStream_t s) {
  if (!unit_ok(k_unit) || !unit_ok(v_unit)) return FA_ERR_INVALID_ARG;
  CacheFwdArgs a;
  host::Device dev;
  const int st = forward_args(c, {{data, cache_bytes(c.Hkv, c.d, c.blocks, c.P), 16}}, cache4_workspace, &a, &dev);
  if (st != FA_OK || a.T == 0) return st;
  a.data = static_cast<const uint8_t*>(data);
  a.k_unit *= k_unit;
  a.v_unit = v_unit;
  char* w = static_cast<char*>(c.ws);
  return c.d == 128 ? launch_cache4_fwd<128>(a, c.P, w, dev, s) : launch_cache4_fwd<64>(a, c.P, w, dev, s);
}

}  // namespace
}  // namespace fa

extern "C" {

int fa_cache_append_e2m1(const void* k, const void* v, long long k_stride, long long v_stride, void* data,
                         float k_unit, float v_unit, const long long* slot_map, const int* positions,
                         const float* table, int length, int rot, int interleaved, int T, int Hkv, int d,
                         int num_blocks, int block_tokens, void* stream) {
  return fa::cache4_append(k, v, k_stride, v_stride, data, k_unit, v_unit, slot_map, positions, table, length, rot,
                           interleaved, T, Hkv, d, num_blocks, block_tokens, static_cast<cudaStream_t>(stream));
}

int fa_cache_read_e2m1(const void* data, float k_unit, float v_unit, const long long* slot_map, void* k, void* v,
                       int T, int Hkv, int d, int num_blocks, int block_tokens, void* stream) {
  return fa::cache4_read(data, k_unit, v_unit, slot_map, k, v, T, Hkv, d, num_blocks, block_tokens,
                         static_cast<cudaStream_t>(stream));
}

size_t fa_cache_fwd_e2m1_workspace_size(int R, int T, int Hq, int Hkv, int d) {
  return fa::cache4_workspace(R, T, Hq, Hkv, d);
}

int fa_cache_fwd_e2m1(const void* q, long long q_stride, const void* data, float k_unit, float v_unit,
                      const int* block_table, const int* seq_lens, const int* cu_q, const long long* slot_map,
                      void* o, float* lse, int R, int T, int Hq, int Hkv, int d, int num_blocks, int block_tokens,
                      int max_blocks, float scale, int causal, void* workspace, size_t workspace_bytes,
                      void* stream) {
  const fa::cachehost::FwdCall c{q, q_stride, block_table, seq_lens, cu_q, slot_map, o, lse, R, T, Hq, Hkv, d,
                                 num_blocks, block_tokens, max_blocks, scale, causal, workspace, workspace_bytes};
  return fa::cache4_fwd(c, data, k_unit, v_unit, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
