// C ABI of the 8-bit key/value cache (declared in include/fa_fwd.h): argument
// validation and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fa_cache.cuh"
#include "fa_cache_fwd.cuh"
#include "fa_cache_host.h"
#include "fa_cache_prompt.cuh"
#include "fa_cache_slots.cuh"
#include "fa_fwd.h"
#include "fa_host.h"

namespace fa {
namespace {

using namespace cachehost;

// ------------------------------------------------------------------- slots

int cache_slots(const SlotArgs& a, int P, cudaStream_t s) {
  if (a.R < 0 || a.T < 0 || a.F < 0 || a.M <= 0) return FA_ERR_INVALID_ARG;
  if (block_shift(P) < 0) return FA_ERR_UNSUPPORTED;
  if (!a.free_used || !a.cu_new || !a.free_used_out) return FA_ERR_INVALID_ARG;
  if (a.R > 0 && (!a.table || !a.seq_lens || !a.new_lens || !a.seq_lens_out)) return FA_ERR_INVALID_ARG;
  if ((a.T > 0 && !a.slot_map) || (a.F > 0 && !a.free_blocks)) return FA_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(a.table), static_cast<const void*>(a.seq_lens),
                        static_cast<const void*>(a.new_lens), static_cast<const void*>(a.free_blocks),
                        static_cast<const void*>(a.free_used), static_cast<const void*>(a.cu_new),
                        static_cast<const void*>(a.seq_lens_out), static_cast<const void*>(a.free_used_out),
                        static_cast<const void*>(a.positions)})
    if (misaligned(p, 4)) return FA_ERR_MISALIGNED;
  if (misaligned(a.slot_map, 8)) return FA_ERR_MISALIGNED;
  const size_t r = static_cast<size_t>(a.R);
  const std::initializer_list<Range> ins = {{a.seq_lens, 4 * r}, {a.new_lens, 4 * r}, {a.free_blocks, 4 * static_cast<size_t>(a.F)},
                       {a.free_used, 4}};
  const std::initializer_list<Range> outs = {{a.table, 4 * r * a.M}, {a.cu_new, 4 * (r + 1)}, {a.slot_map, 8 * static_cast<size_t>(a.T)},
                        {a.seq_lens_out, 4 * r}, {a.free_used_out, 4},
                        {a.positions, a.positions ? 4 * static_cast<size_t>(a.T) : 0}};
  if (overlapping(outs, ins)) return FA_ERR_INVALID_ARG;
  host::Device dev;
  const int st = host::device(&dev);
  if (st != FA_OK) return st;
  long long grid = (static_cast<long long>(a.T) + slots::kThreads - 1) / slots::kThreads;
  grid = grid < 1 ? 1 : (grid > 2 * dev.sms ? 2 * dev.sms : grid);
  fa_cache_slots_kernel<<<static_cast<unsigned>(grid), slots::kThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FA_OK : host::fail(e);
}

// ------------------------------------------------------------------ append

template <int D>
void launch_append(const AppendArgs& a, dim3 grid, cudaStream_t s) {
  const int nv = ((1 << a.sh) * D) / (8 * 128);  // 1 .. 16
  if (nv == 16) fa_cache_append_kernel<D, 8, 256><<<grid, 256, 0, s>>>(a);
  else if (nv == 8) fa_cache_append_kernel<D, 8, 128><<<grid, 128, 0, s>>>(a);
  else if (nv == 4) fa_cache_append_kernel<D, 4, 128><<<grid, 128, 0, s>>>(a);
  else if (nv == 2) fa_cache_append_kernel<D, 2, 128><<<grid, 128, 0, s>>>(a);
  else fa_cache_append_kernel<D, 1, 128><<<grid, 128, 0, s>>>(a);
}

int cache_append(const void* k, const void* v, long long k_stride, long long v_stride, void* k8, void* v8,
                 float* ks, float* vs, const long long* slot_map, int T, int Hkv, int d, int blocks, int P,
                 cudaStream_t s) {
  int st = check_cache(Hkv, d, blocks, P);
  if (st != FA_OK) return st;
  if (T < 0) return FA_ERR_INVALID_ARG;
  if (T == 0) return FA_OK;
  if (!k || !v || !k8 || !v8 || !ks || !vs || !slot_map) return FA_ERR_INVALID_ARG;
  const long long row = static_cast<long long>(Hkv) * d;
  if (T > 1 && (k_stride < row || v_stride < row)) return FA_ERR_INVALID_ARG;
  if ((k_stride | v_stride) & 7) return FA_ERR_MISALIGNED;
  if (k_stride > (1ll << 40) || v_stride > (1ll << 40)) return FA_ERR_UNSUPPORTED;
  for (const void* p : {k, v, static_cast<const void*>(k8), static_cast<const void*>(v8)})
    if (misaligned(p, 16)) return FA_ERR_MISALIGNED;
  if (misaligned(ks, 4) || misaligned(vs, 4) || misaligned(slot_map, 8)) return FA_ERR_MISALIGNED;
  const size_t nx = 2 * static_cast<size_t>(row), nc = static_cast<size_t>(blocks) * P * row;
  const size_t nk = static_cast<size_t>(T - 1) * k_stride * 2 + nx, nv = static_cast<size_t>(T - 1) * v_stride * 2 + nx;
  const size_t ns = static_cast<size_t>(blocks) * Hkv * 4;
  const std::initializer_list<Range> outs = {{k8, nc}, {v8, nc}, {ks, ns}, {vs, ns}};
  const std::initializer_list<Range> ins = {{k, nk}, {v, nv}, {slot_map, 8 * static_cast<size_t>(T)}};
  if (overlapping(outs, ins)) return FA_ERR_INVALID_ARG;
  host::Device dev;
  if ((st = host::device(&dev)) != FA_OK) return st;
  AppendArgs a{};
  a.x[0] = static_cast<const __nv_bfloat16*>(k);
  a.x[1] = static_cast<const __nv_bfloat16*>(v);
  a.stride[0] = k_stride;
  a.stride[1] = v_stride;
  a.codes[0] = static_cast<uint8_t*>(k8);
  a.codes[1] = static_cast<uint8_t*>(v8);
  a.scale[0] = ks;
  a.scale[1] = vs;
  a.slot_map = slot_map;
  a.slots = static_cast<long long>(blocks) * P;
  a.T = T;
  a.Hkv = Hkv;
  a.sh = block_shift(P);
  a.err = dev.index_err;
  // Tokens and rows of a CTA, by the rows there are for each SM: few of both where
  // latency counts, more of them where a CTA without a run's start, and the wait
  // for a run's first rows, cost more (us; 8 kv heads, d = 128, P = 64; single
  // tokens / prompts):
  //   tokens     4 x 1          16 x 1         64 x 1         64 x 4
  //     32      2.6 / 3.4      3.7 / 3.4      5.4 / 3.3      16 / 5.5
  //    512      7.0 / 6.1      4.6 / 4.6      9.1 / 3.6      30 / 5.9
  //   2048       21 / 14        13 / 7.5       12 / 4.9      30 / 6.1
  //  32768        - / 190        - / 79         - / 51        - / 39
  const long long per_sm = 2ll * T * Hkv / dev.sms;
  a.chunk = per_sm <= 24 ? 4 : per_sm <= 160 ? 16 : app::kMaxChunk;
  a.group = per_sm <= 600 ? (2 * Hkv > 65535 ? 2 : 1) : 4;
  const dim3 grid(static_cast<unsigned>((static_cast<long long>(T) + a.chunk - 1) / a.chunk),
                  static_cast<unsigned>((2 * Hkv + a.group - 1) / a.group));
  if (d == 128) launch_append<128>(a, grid, s);
  else launch_append<64>(a, grid, s);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FA_OK : host::fail(e);
}

// ----------------------------------------------------------------- forward

// Query rows of a unit, and with them the kernel, by the average rows a request
// has per kv head (tokens times the query heads that share it): the few-row
// kernel with 8 or 16, which reads the keys again for every so many, or the
// many-row one with 256.  Measured (us; d = 128, lengths evenly up to 4000 for
// 64 requests of 8 kv heads, of 8000 for one), rows of 8 / 16 / 256 a unit:
//   rows per kv head      8               16               24               48
//   64 requests     63 / 71 / 104   108 / 83 / 104   156 / 134 / 105  295 / 212 / 108
//   one request     18 / 19 / 23     18 / 22 / 24     19 / 21 / 24     25 / 23 / 25
// so with few units, where the many-row kernel's start counts, the step up to it
// comes later.
int unit_rows(int R, int T, int Hq, int Hkv, int sms) {
  const long long rows = static_cast<long long>(T) * (Hq / Hkv);
  const bool few = static_cast<long long>(R) * Hkv * 8 <= sms;
  return rows <= 8ll * R ? 8 : rows <= (few ? 48ll : 16ll) * R ? 16 : prm::kRows;
}

size_t cache_fwd_workspace(int R, int T, int Hq, int Hkv, int d) {
  if ((d != 64 && d != 128) || R <= 0 || T <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return 0;
  host::Device dev;
  if (host::device(&dev) != FA_OK) return 0;
  const int rows = unit_rows(R, T, Hq, Hkv, dev.sms);
  return workspace_bytes(fwd_grid(dev.sms, rows, d), rows, d);
}

// By device and d (64, 128): 8 rows, many rows with G 16, 32, 64, 16 rows.
bool g_cache_ready[64][2][5] = {};

template <int D>
int launch_cache_fwd(CacheFwdArgs& a, const void* k8, const void* v8, int P, char* ws, const host::Device& dev,
                     cudaStream_t s) {
  const int unit = unit_rows(a.R, a.T, a.Hq, a.Hkv, dev.sms), grid = fwd_grid(dev.sms, unit, D);
  set_workspace(a, ws, grid, unit, D);
  bool* set = g_cache_ready[dev.dev][D == 128];
  int st = FA_OK;
  if (unit == prm::kRows) {
    using Ly = prm::Layout<D>;
    // a key per 128-byte row, zeros behind the codes at d = 64
    CUtensorMap mk;
    st = host::tensor_map(&mk, CU_TENSOR_MAP_DATA_TYPE_UINT8, k8, D, static_cast<cuuint64_t>(P),
                          static_cast<cuuint64_t>(a.blocks) * a.Hkv, D, static_cast<cuuint64_t>(P) * D, 128,
                          static_cast<cuuint32_t>(P));
    if (st != FA_OK) return st;
    const uint8_t* vc = static_cast<const uint8_t*>(v8);
    auto launch = [&](auto kernel, bool& done) {
      if ((st = ready(kernel, Ly::kAlloc, done, 128)) == FA_OK) kernel<<<grid, prm::kThreads, Ly::kAlloc, s>>>(mk, vc, a);
    };
    if (P == 16) launch(fa_cache_prompt_kernel<D, 16>, set[1]);
    else if (P == 32) launch(fa_cache_prompt_kernel<D, 32>, set[2]);
    else launch(fa_cache_prompt_kernel<D, 64>, set[3]);
    if (st != FA_OK) return st;
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return host::fail(e);
    // a unit of one tile is never split: nothing to merge
    if (static_cast<long long>(a.M) * P <= prm::kKeys) return FA_OK;
    return launch_merge<D, prm::kRows, E4M3Codes>(a, grid, 4, s);
  }
  E4M3Codes::Maps maps;
  const cuuint64_t rows = static_cast<cuuint64_t>(P) * D / 128;
  const cuuint64_t bh = static_cast<cuuint64_t>(a.blocks) * a.Hkv;
  const cuuint32_t box = static_cast<cuuint32_t>((P < dec::kKeys ? P : dec::kKeys) * D / 128);
  st = host::tensor_map(&maps.k, CU_TENSOR_MAP_DATA_TYPE_UINT8, k8, 128, rows, bh, 128, rows * 128, 128, box);
  if (st != FA_OK) return st;
  st = host::tensor_map(&maps.v, CU_TENSOR_MAP_DATA_TYPE_UINT8, v8, 128, rows, bh, 128, rows * 128, 128, box);
  if (st != FA_OK) return st;
  if (unit == 8) {
    using Ly = dec::Layout<D, 8, E4M3Codes>;
    if ((st = ready(fa_cache_fwd_kernel<D, 8, E4M3Codes>, Ly::kAlloc, set[0])) != FA_OK) return st;
    fa_cache_fwd_kernel<D, 8, E4M3Codes><<<grid, Ly::kThreads, Ly::kAlloc, s>>>(maps, a);
  } else {
    using Ly = dec::Layout<D, 16, E4M3Codes>;
    if ((st = ready(fa_cache_fwd_kernel<D, 16, E4M3Codes>, Ly::kAlloc, set[4])) != FA_OK) return st;
    fa_cache_fwd_kernel<D, 16, E4M3Codes><<<grid, Ly::kThreads, Ly::kAlloc, s>>>(maps, a);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return host::fail(e);
  if (static_cast<long long>(a.M) * P <= dec::kKeys) return FA_OK;
  return unit == 8 ? launch_merge<D, 8, E4M3Codes>(a, grid, 1, s)
                   : launch_merge<D, 16, E4M3Codes>(a, grid, 1, s);
}

int cache_fwd(const FwdCall& c, const void* k8, const void* v8, const float* ks, const float* vs, cudaStream_t s) {
  CacheFwdArgs a;
  host::Device dev;
  const size_t nc = static_cast<size_t>(c.blocks) * c.P * c.Hkv * c.d, ns = static_cast<size_t>(c.blocks) * c.Hkv * 4;
  const int st = forward_args(c, {{k8, nc, 16}, {v8, nc, 16}, {ks, ns, 4}, {vs, ns, 4}}, cache_fwd_workspace, &a, &dev);
  if (st != FA_OK || a.T == 0) return st;
  a.ks = ks;
  a.vs = vs;
  char* w = static_cast<char*>(c.ws);
  return c.d == 128 ? launch_cache_fwd<128>(a, k8, v8, c.P, w, dev, s) : launch_cache_fwd<64>(a, k8, v8, c.P, w, dev, s);
}

}  // namespace
}  // namespace fa

extern "C" {

int fa_cache_slots(int* block_table, const int* seq_lens, const int* new_lens, const int* free_blocks,
                   const int* free_used, int* cu_new, long long* slot_map, int* seq_lens_out, int* free_used_out,
                   int R, int max_blocks, int num_free, int block_tokens, int num_tokens, void* stream) {
  fa::SlotArgs a{block_table, seq_lens, new_lens, free_blocks, free_used, cu_new, slot_map, seq_lens_out,
                 free_used_out, nullptr, R, max_blocks, num_free, fa::cachehost::block_shift(block_tokens), num_tokens};
  return fa::cache_slots(a, block_tokens, static_cast<cudaStream_t>(stream));
}

int fa_cache_slots_positions(int* block_table, const int* seq_lens, const int* new_lens, const int* free_blocks,
                             const int* free_used, int* cu_new, long long* slot_map, int* positions,
                             int* seq_lens_out, int* free_used_out, int R, int max_blocks, int num_free,
                             int block_tokens, int num_tokens, void* stream) {
  if (num_tokens > 0 && !positions) return FA_ERR_INVALID_ARG;
  fa::SlotArgs a{block_table, seq_lens, new_lens, free_blocks, free_used, cu_new, slot_map, seq_lens_out,
                 free_used_out, positions, R, max_blocks, num_free, fa::cachehost::block_shift(block_tokens), num_tokens};
  return fa::cache_slots(a, block_tokens, static_cast<cudaStream_t>(stream));
}

int fa_cache_append_e4m3(const void* k, const void* v, long long k_stride, long long v_stride, void* k8, void* v8,
                         float* k_scale, float* v_scale, const long long* slot_map, int T, int Hkv, int d,
                         int num_blocks, int block_tokens, void* stream) {
  return fa::cache_append(k, v, k_stride, v_stride, k8, v8, k_scale, v_scale, slot_map, T, Hkv, d, num_blocks,
                          block_tokens, static_cast<cudaStream_t>(stream));
}

size_t fa_cache_fwd_e4m3_workspace_size(int R, int T, int Hq, int Hkv, int d) {
  return fa::cache_fwd_workspace(R, T, Hq, Hkv, d);
}

int fa_cache_fwd_e4m3(const void* q, long long q_stride, const void* k8, const void* v8, const float* k_scale,
                      const float* v_scale, const int* block_table, const int* seq_lens, const int* cu_q, void* o,
                      float* lse, int R, int T, int Hq, int Hkv, int d, int num_blocks, int block_tokens,
                      int max_blocks, float scale, int causal, void* workspace, size_t workspace_bytes,
                      void* stream) {
  return fa_cache_fwd_e4m3_slots(q, q_stride, k8, v8, k_scale, v_scale, block_table, seq_lens, cu_q, nullptr, o, lse, R,
                                 T, Hq, Hkv, d, num_blocks, block_tokens, max_blocks, scale, causal, workspace,
                                 workspace_bytes, stream);
}

int fa_cache_fwd_e4m3_slots(const void* q, long long q_stride, const void* k8, const void* v8, const float* k_scale,
                            const float* v_scale, const int* block_table, const int* seq_lens, const int* cu_q,
                            const long long* slot_map, void* o, float* lse, int R, int T, int Hq, int Hkv, int d,
                            int num_blocks, int block_tokens, int max_blocks, float scale, int causal,
                            void* workspace, size_t workspace_bytes, void* stream) {
  const fa::cachehost::FwdCall c{q, q_stride, block_table, seq_lens, cu_q, slot_map, o, lse, R, T, Hq, Hkv, d,
                                 num_blocks, block_tokens, max_blocks, scale, causal, workspace, workspace_bytes};
  return fa::cache_fwd(c, k8, v8, k_scale, v_scale, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
