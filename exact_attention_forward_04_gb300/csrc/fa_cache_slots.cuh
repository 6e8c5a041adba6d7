// Slots of a paged key/value cache: block tables and slot maps from request
// lengths.
#pragma once
#include "fa_index.cuh"

namespace fa {

namespace slots {
constexpr int kThreads = 1024;
}

struct SlotArgs {
  int* table;             // [R][M]
  const int* seq_lens;    // [R]
  const int* new_lens;    // [R]
  const int* free_blocks; // [F]
  const int* free_used;   // [1]
  int* cu_new;            // [R + 1]
  long long* slot_map;    // [T]
  int* seq_lens_out;      // [R]
  int* free_used_out;     // [1]
  int* positions;         // [T] or null
  int R, M, F, sh, T;     // blocks of 2^sh tokens
};

// One request: tokens held and new, the blocks it needs and whether it fits its
// table row, the slot map and an int32 length (one that does not takes no block).
struct SlotReq {
  long long len, add, held, need;
  bool fits;
};
__device__ __forceinline__ SlotReq slot_req(const SlotArgs& a, int r, long long cu) {
  SlotReq q;
  q.len = max(0, a.seq_lens[r]);
  q.add = max(0, a.new_lens[r]);
  const int up = (1 << a.sh) - 1;
  q.held = (q.len + up) >> a.sh;
  const long long want = (q.len + q.add + up) >> a.sh;
  q.fits = want <= a.M && cu + q.add <= a.T && q.len + q.add <= 0x7fffffffll;
  q.need = q.fits ? want - q.held : 0;
  return q;
}

// Largest i < n with v[i] <= x (v ascending, v[0] <= x).
__device__ __forceinline__ int last_le(const long long* v, int n, long long x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// Block tables and slot maps from request lengths.  Every CTA scans all
// requests (two sums: new tokens, then blocks needed, whose refusals depend on
// the first), each thread a run of consecutive ones; then the CTAs share the
// slots and the granted table entries, each of which finds its request by a
// binary search over the threads' runs and a walk inside one.  Blocks are
// granted in request order, and the requests that get theirs form a prefix of
// those that need any, so one sum decides for all of them.
//
// Reads of the table are of entries below a request's held blocks, writes of
// entries from there on: CTAs need no order among themselves.
//
// Bound by latency: 4.9 us for 8 requests, 6.3 for 1000 and 5.9 for 64 prompts,
// where a launch with two dependent loads takes 2.4.  Here three depend on one
// another, the new lengths, the old ones behind the first scan, and the table or
// the free list, with two scans and a search of ten steps in between.
__global__ void __launch_bounds__(slots::kThreads) fa_cache_slots_kernel(SlotArgs a) {
  __shared__ long long s_cu[slots::kThreads], s_need[slots::kThreads], s_tmp[33];
  const int tid = threadIdx.x, nthr = blockDim.x;
  const int per = (a.R + nthr - 1) / nthr;
  const int r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);
  const long long used = max(0, *a.free_used);
  const long long avail = max(0ll, a.F - used);

  long long add = 0, total_new, total_need;
  for (int r = r0; r < r1; ++r) add += max(0, a.new_lens[r]);
  const long long cu0 = cta_scan(add, s_tmp, total_new) - add;
  long long need = 0, cu = cu0;
  for (int r = r0; r < r1; ++r) {
    const SlotReq q = slot_req(a, r, cu);
    need += q.need;
    cu += q.add;
  }
  const long long need0 = cta_scan(need, s_tmp, total_need) - need;
  s_cu[tid] = cu0;
  s_need[tid] = need0;
  __syncthreads();

  if (blockIdx.x == 0) {  // per-request outputs
    long long granted = 0, c = cu0, n = need0;
    for (int r = r0; r < r1; ++r) {
      const SlotReq q = slot_req(a, r, c);
      const bool ok = q.fits && (q.need == 0 || n + q.need <= avail);
      a.cu_new[r] = static_cast<int>(min(c, 0x7fffffffll));
      a.seq_lens_out[r] = static_cast<int>(q.len + (ok ? q.add : 0));
      c += q.add;
      n += q.need;
      granted += ok ? q.need : 0;
    }
    long long all;
    (void)cta_scan(granted, s_tmp, all);
    if (tid == 0) {
      a.cu_new[a.R] = static_cast<int>(min(total_new, 0x7fffffffll));
      *a.free_used_out = static_cast<int>(used + all);
    }
  }

  const long long stride = static_cast<long long>(gridDim.x) * nthr;
  const long long at = static_cast<long long>(blockIdx.x) * nthr + tid;
  for (long long t = at; t < a.T; t += stride) {
    long long slot = -1;
    int position = -1;
    if (t < total_new) {
      const int run = last_le(s_cu, nthr, t);
      long long c = s_cu[run], n = s_need[run];
      int r = run * per;
      SlotReq q = slot_req(a, r, c);
      while (t >= c + q.add) {  // ends: the run holds token t
        c += q.add;
        n += q.need;
        q = slot_req(a, ++r, c);
      }
      if (q.fits && (q.need == 0 || n + q.need <= avail)) {
        const long long pos = q.len + t - c, j = pos >> a.sh;
        position = static_cast<int>(pos);
        const int b = j < q.held ? a.table[static_cast<long long>(r) * a.M + j]
                                 : a.free_blocks[used + n + j - q.held];
        if (b >= 0) slot = (static_cast<long long>(b) << a.sh) + (pos & ((1 << a.sh) - 1));
      }
    }
    a.slot_map[t] = slot;
    if (a.positions) a.positions[t] = position;
  }
  for (long long i = at; i < min(total_need, avail); i += stride) {
    const int run = last_le(s_need, nthr, i);
    long long c = s_cu[run], n = s_need[run];
    int r = run * per;
    SlotReq q = slot_req(a, r, c);
    while (i >= n + q.need) {
      c += q.add;
      n += q.need;
      q = slot_req(a, ++r, c);
    }
    if (n + q.need <= avail)
      a.table[static_cast<long long>(r) * a.M + q.held + (i - n)] = a.free_blocks[used + i];
  }
}

}  // namespace fa
