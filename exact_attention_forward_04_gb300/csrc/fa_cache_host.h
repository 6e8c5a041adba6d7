// What the host sides of the 8-bit and the 4-bit key/value cache share: checks
// of a call's sizes and arrays, launches.
#pragma once
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <mutex>

#include "fa_cache_fwd.cuh"
#include "fa_fwd.h"
#include "fa_host.h"

namespace fa {
namespace cachehost {

inline bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// log2 of the tokens per block, -1 where it is none of 16, 32, 64, 128.
inline int block_shift(int P) { return P == 16 ? 4 : P == 32 ? 5 : P == 64 ? 6 : P == 128 ? 7 : -1; }

// Sizes of a cache that fits 2^31 code rows of 128 bytes (the tensor maps'
// coordinates are 32-bit).
inline int check_cache(int Hkv, int d, int blocks, int P) {
  if (Hkv <= 0 || blocks <= 0) return FA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || block_shift(P) < 0 || Hkv > 65535) return FA_ERR_UNSUPPORTED;
  const long long bh = static_cast<long long>(blocks) * Hkv;
  if (bh > 0x7fffffffLL || static_cast<long long>(blocks) * P > (1ll << 40)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// An array of a call; one of no bytes may be null.
struct Range {
  const void* p;
  size_t n;
  int align = 1;
};

// Whether any of `outs` overlaps an input or another output.
inline bool overlapping(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    for (const Range& in : ins)
      if (host::overlap(o->p, o->n, in.p, in.n)) return true;
    for (auto p = o + 1; p != outs.end(); ++p)
      if (host::overlap(o->p, o->n, p->p, p->n)) return true;
  }
  return false;
}

// A forward's arguments beside the cache's arrays.
struct FwdCall {
  const void* q;
  long long q_stride;
  const int* table;
  const int* seq_lens;
  const int* cu_q;
  const long long* slot_map;
  void* o;
  float* lse;
  int R, T, Hq, Hkv, d, blocks, P, M;
  float scale;
  int causal;
  void* ws;
  size_t ws_bytes;
};

// Checks a forward and fills in what both caches' kernels take; `cache` are its
// arrays, `workspace` gives the bytes it needs.  FA_OK with a->T = 0: nothing to do.
inline int forward_args(const FwdCall& c, std::initializer_list<Range> cache,
                        size_t (*workspace)(int, int, int, int, int), CacheFwdArgs* args, host::Device* dev) {
  int st = check_cache(c.Hkv, c.d, c.blocks, c.P);
  if (st != FA_OK) return st;
  CacheFwdArgs& a = *args;
  a = CacheFwdArgs{};
  if (c.R < 0 || c.T < 0 || c.Hq <= 0 || c.M <= 0 || c.Hq % c.Hkv != 0) return FA_ERR_INVALID_ARG;
  if (c.causal != 0 && c.causal != 1) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(c.scale)) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(c.T) * c.Hq > 0x7fffffffLL || static_cast<long long>(c.M) * c.P > 0x7fffff00LL)
    return FA_ERR_UNSUPPORTED;
  if (c.T == 0 || c.R == 0) return FA_OK;
  if (!c.q || !c.table || !c.seq_lens || !c.cu_q || !c.o || !c.lse || !c.ws) return FA_ERR_INVALID_ARG;
  for (const Range& r : cache)
    if (!r.p) return FA_ERR_INVALID_ARG;
  const long long row = static_cast<long long>(c.Hq) * c.d;
  if (c.T > 1 && c.q_stride < row) return FA_ERR_INVALID_ARG;
  if (c.q_stride & 7) return FA_ERR_MISALIGNED;
  if (c.q_stride > (1ll << 40)) return FA_ERR_UNSUPPORTED;
  for (const void* p : {c.q, static_cast<const void*>(c.o), static_cast<const void*>(c.ws)})
    if (misaligned(p, 16)) return FA_ERR_MISALIGNED;
  for (const Range& r : cache)
    if (misaligned(r.p, r.align)) return FA_ERR_MISALIGNED;
  for (const void* p : {static_cast<const void*>(c.table), static_cast<const void*>(c.seq_lens),
                        static_cast<const void*>(c.cu_q), static_cast<const void*>(c.lse)})
    if (misaligned(p, 4)) return FA_ERR_MISALIGNED;
  if (misaligned(c.slot_map, 8)) return FA_ERR_MISALIGNED;
  if ((st = host::device(dev)) != FA_OK) return st;
  const size_t need = workspace(c.R, c.T, c.Hq, c.Hkv, c.d);
  if (need == 0) return FA_ERR_UNSUPPORTED;
  if (c.ws_bytes < need) return FA_ERR_INVALID_ARG;
  const size_t nq = (static_cast<size_t>(c.T - 1) * c.q_stride + row) * 2, no = static_cast<size_t>(c.T) * row * 2;
  const Range o{c.o, no}, lse{c.lse, static_cast<size_t>(c.T) * c.Hq * 4}, ws{c.ws, need};
  if (overlapping({o, lse, ws}, {{c.q, nq},
                                 {c.table, static_cast<size_t>(c.R) * c.M * 4},
                                 {c.seq_lens, static_cast<size_t>(c.R) * 4},
                                 {c.cu_q, (static_cast<size_t>(c.R) + 1) * 4},
                                 {c.slot_map, c.slot_map ? static_cast<size_t>(c.T) * 8 : 0}}) ||
      overlapping({o, lse, ws}, cache))
    return FA_ERR_INVALID_ARG;
  a.q = static_cast<const __nv_bfloat16*>(c.q);
  a.q_stride = c.q_stride;
  a.table = c.table;
  a.seq_lens = c.seq_lens;
  a.cu_q = c.cu_q;
  a.slot_map = c.slot_map;
  a.o = static_cast<__nv_bfloat16*>(c.o);
  a.lse = c.lse;
  a.R = c.R;
  a.T = c.T;
  a.Hq = c.Hq;
  a.Hkv = c.Hkv;
  a.g = c.Hq / c.Hkv;
  a.sh = block_shift(c.P);
  a.M = c.M;
  a.blocks = c.blocks;
  a.causal = c.causal;
  // A score's factor is a row's power of two (2^-124 to 2^120) times the scale,
  // times the K scale (2^-100 to 2^120): the scale is brought to [1/4, 1/2) and
  // the rest of it goes to the K scale, so that both parts stay normal.
  a.scale_log2 = c.scale * 1.4426950408889634f;
  int exponent = 0;
  std::frexp(a.scale_log2, &exponent);
  const int shift = std::min(26, std::max(-7, -1 - exponent));
  a.scale_log2 = std::ldexp(a.scale_log2, shift);
  a.k_unit = std::ldexp(1.f, -shift);
  a.v_unit = 1.f;
  a.err = dev->err;
  a.index_err = dev->index_err;
  a.timeout_ns = 2000ull * 1000 * 1000;
  return FA_OK;
}

// Workspace: the CTAs' marks, then two partials of a unit's query rows per CTA.
inline int fwd_grid(int sms, int rows, int d) { return sms * dec::ctas_per_sm(d, rows); }
inline size_t marks_bytes(int grid) { return static_cast<size_t>(grid) * 32 + 16; }  // and to the next 32 bytes
inline size_t workspace_bytes(int grid, int rows, int d) {
  return marks_bytes(grid) + static_cast<size_t>(2) * grid * rows * (d + 1) * 4;
}
inline void set_workspace(CacheFwdArgs& a, char* ws, int grid, int rows, int d) {
  a.desc = reinterpret_cast<int4*>(ws);
  a.cont = reinterpret_cast<int*>(ws + static_cast<size_t>(grid) * 16);
  // 32-byte stores; ws is aligned to 16
  const uintptr_t parts = reinterpret_cast<uintptr_t>(ws) + marks_bytes(grid);
  a.part_o = reinterpret_cast<float*>(parts & ~static_cast<uintptr_t>(31));
  a.part_l = a.part_o + static_cast<size_t>(2) * grid * rows * d;
}

// Dynamic shared memory of a kernel, set once per device.  `regs`: registers per
// thread that its warps' later shares (setmaxnreg) add up from, 0: any number; with
// others an increase would wait for ever.
template <typename K>
int ready(K kernel, int bytes, bool& done, int regs = 0) {
  static std::mutex mu;
  std::lock_guard<std::mutex> lock(mu);
  if (!done) {
    if (regs > 0) {
      cudaFuncAttributes attr;
      const cudaError_t e = cudaFuncGetAttributes(&attr, kernel);
      if (e != cudaSuccess) return host::fail(e);
      if (attr.numRegs != regs) return FA_ERR_UNSUPPORTED;
    }
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return host::fail(e);
    done = true;
  }
  return FA_OK;
}

// The merge as a programmatic dependent of the kernel before it.
template <int D, int ROWS, class F>
int launch_merge(const CacheFwdArgs& a, int grid, int split, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, split, 1);
  cfg.blockDim = dim3(512, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fa_cache_merge_kernel<D, ROWS, F>, a, grid);
  return e == cudaSuccess ? FA_OK : host::fail(e);
}

}  // namespace cachehost
}  // namespace fa
