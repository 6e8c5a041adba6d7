// C ABI of rotary positions (declared in include/fa_fwd.h): argument validation
// and launch.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fa_index.cuh"
#include "fa_rope.cuh"
#include "fa_fwd.h"
#include "fa_host.h"

namespace fa {
namespace {

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// Elements from a tensor's first to behind its last one.
long long span(int B, int H, int N, int d, long long sb, long long sh, long long sn) {
  return (B - 1) * sb + (H - 1) * sh + (N - 1) * sn + d;
}

// Whether no two rows of a tensor share an element: each axis steps over all that
// the axes of smaller steps reach.
bool rows_apart(const int (&n)[3], const long long* strides, int d) {
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int i, int j) { return strides[i] < strides[j]; });
  long long reach = d;
  for (int i : order) {
    if (n[i] == 1) continue;
    if (strides[i] < reach) return false;
    reach += strides[i] * (n[i] - 1);
  }
  return true;
}

int rope_run(const void* x, long long (&xs)[3], void* out, long long (&os)[3], const int* positions,
             long long positions_stride, const float* table, int length, int B, int H, int N, int d, int rot,
             int interleaved, int transposed, cudaStream_t s) {
  if (B < 0 || H <= 0 || N < 0 || length <= 0) return FA_ERR_INVALID_ARG;
  if ((interleaved != 0 && interleaved != 1) || (transposed != 0 && transposed != 1)) return FA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || rot <= 0 || rot > d || rot % 16 != 0) return FA_ERR_UNSUPPORTED;
  if (B == 0 || N == 0) return FA_OK;
  if (!x || !out || !positions || !table) return FA_ERR_INVALID_ARG;
  if (positions_stride != 0 && positions_stride < N) return FA_ERR_INVALID_ARG;
  const int n[3] = {B, H, N};
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 1) xs[i] = os[i] = 0;  // of no matter
    if (xs[i] < 0 || os[i] < 0) return FA_ERR_INVALID_ARG;
    if ((xs[i] | os[i]) & 7) return FA_ERR_MISALIGNED;
    if (xs[i] > (1ll << 31) || os[i] > (1ll << 31)) return FA_ERR_UNSUPPORTED;
    if ((n[i] - 1) * xs[i] > (1ll << 46) || (n[i] - 1) * os[i] > (1ll << 46)) return FA_ERR_UNSUPPORTED;
  }
  if (!rows_apart(n, os, d)) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * N > (1ll << 33)) return FA_ERR_UNSUPPORTED;
  if (misaligned(x, 16) || misaligned(out, 16) || misaligned(table, 16) || misaligned(positions, 4))
    return FA_ERR_MISALIGNED;
  const size_t nx = 2 * static_cast<size_t>(span(B, H, N, d, xs[0], xs[1], xs[2]));
  const size_t no = 2 * static_cast<size_t>(span(B, H, N, d, os[0], os[1], os[2]));
  // in place: the same rows, each read and written by the same threads
  bool same = x == out;
  for (int i = 0; i < 3; ++i) same = same && xs[i] == os[i];
  if (!same && host::overlap(out, no, x, nx)) return FA_ERR_INVALID_ARG;
  const size_t np = 4 * (static_cast<size_t>(B - 1) * positions_stride + N);
  if (host::overlap(out, no, positions, np)) return FA_ERR_INVALID_ARG;
  if (host::overlap(out, no, table, static_cast<size_t>(length) * rot * 4)) return FA_ERR_INVALID_ARG;
  host::Device dev;
  const int st = host::device(&dev);
  if (st != FA_OK) return st;
  RopeArgs a{};
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.xb = xs[0];
  a.xh = xs[1];
  a.xn = xs[2];
  a.ob = os[0];
  a.oh = os[1];
  a.on = os[2];
  a.positions = positions;
  a.pb = positions_stride;
  a.table = reinterpret_cast<const float2*>(table);
  a.length = length;
  a.B = B;
  a.H = H;
  a.N = N;
  a.rot = rot;
  a.sign = transposed ? -1.f : 1.f;
  a.err = dev.index_err;
  const long long lanes = static_cast<long long>(B) * N * (d / 16);
  const long long gx = (lanes + rope::kThreads - 1) / rope::kThreads;
  // Heads of a thread, by the lanes that one each would give an SM: one where rows are
  // few, many where its cos and sin are worth keeping.  Measured (us; tokens x heads of
  // 128, of 64 alike), heads 1 / 2 / 4 / 8 / 16:
  //   500 x 40 (1052)   5.9 / 5.6 / 6.5 / 9.1 / 14.2        4000 x 40 (8421)   22.5 / 19.1 / 18.7 / 20.9 / 20.4
  //   1000 x 40 (2105)  8.4 / 7.7 / 7.6 / 9.9 / 14.8        8000 x 40 (16842)  41.4 / 34.9 / 33.0 / 34.2 / 33.8
  //   2000 x 40 (4210)  13.0 / 11.4 / 12.3 / 11.8 / 16.4    16000 x 40 (33684) 79.1 / 66.9 / 63.1 / 62.7 / 61.5
  //   16000 x 8 (6736)  18.5 / 16.0 / 15.4 / 15.4           32000 x 40 (67368) 156 / 133 / 130 / 125 / 120
  const long long per_sm = lanes * H / dev.sms;
  a.group = per_sm <= 2048 ? 1 : per_sm <= 8192 ? 2 : per_sm <= 32768 ? 4 : 16;
  while ((H + a.group - 1) / a.group > 65535) a.group *= 2;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>((H + a.group - 1) / a.group));
  if (d == 128) {
    if (interleaved) fa_rope_kernel<128, true><<<grid, rope::kThreads, 0, s>>>(a);
    else fa_rope_kernel<128, false><<<grid, rope::kThreads, 0, s>>>(a);
  } else {
    if (interleaved) fa_rope_kernel<64, true><<<grid, rope::kThreads, 0, s>>>(a);
    else fa_rope_kernel<64, false><<<grid, rope::kThreads, 0, s>>>(a);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FA_OK : host::fail(e);
}

}  // namespace
}  // namespace fa

extern "C" int fa_rope(const void* x, long long x_batch, long long x_head, long long x_token, void* out,
                       long long out_batch, long long out_head, long long out_token, const int* positions,
                       long long positions_stride, const float* table, int length, int B, int H, int N, int d, int rot,
                       int interleaved, int transposed, void* stream) {
  long long xs[3] = {x_batch, x_head, x_token}, os[3] = {out_batch, out_head, out_token};
  return fa::rope_run(x, xs, out, os, positions, positions_stride, table, length, B, H, N, d, rot, interleaved,
                      transposed, static_cast<cudaStream_t>(stream));
}
