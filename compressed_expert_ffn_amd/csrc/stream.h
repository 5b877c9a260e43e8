// Pieces shared by the kernels that stream weights once for a few rows: a
// register ring that keeps several units of loads in flight, and the loads of
// activation rows as MFMA operands.
#pragma once
#include "common.h"

namespace cefn {

// Run use(slot) on units 0 .. n-1 in order with R units' loads in flight:
// issue(i, slot) loads unit i into a register set, refilled as soon as its
// unit is used.  Past the end the last unit is loaded again (at most R - 1
// times, from cache) so that the loop has no branches between the loads.  The
// scheduling barriers keep one unit's decode from being hoisted over another's:
// all units' decoded operands at once do not fit the registers.
// between() runs once the first units' loads are under way (also where n is
// 0): what it reads arrives behind them.
template <int R, class Slot, class Issue, class Use, class Between>
__device__ __forceinline__ void stream_units(int n, Issue&& issue, Use&& use, Between&& between) {
  Slot ring[R];
  if (n > 0) {
#pragma unroll
    for (int p = 0; p < R; ++p) issue(p < n ? p : n - 1, ring[p]);
  }
  __builtin_amdgcn_sched_barrier(0);
  between();
  __builtin_amdgcn_sched_barrier(0);
  int i = 0;
  for (; i + R < n; i += R) {
#pragma unroll
    for (int p = 0; p < R; ++p) {
      use(ring[p]);
      __builtin_amdgcn_sched_barrier(0);
      const int nx = i + p + R;
      issue(nx < n ? nx : n - 1, ring[p]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int p = 0; p < R; ++p)
    if (i + p < n) {
      use(ring[p]);
      __builtin_amdgcn_sched_barrier(0);
    }
}

template <int R, class Slot, class Issue, class Use>
__device__ __forceinline__ void stream_units(int n, Issue&& issue, Use&& use) {
  stream_units<R, Slot>(n, issue, use, [] {});
}

// Eight consecutive 16-bit activations, k .. k + 7 of the row at p; from n on
// the row's last ones again, for products whose weights are zero there.
// ALIGNED: p is on a 16-byte boundary and n a multiple of 8.
template <bool ALIGNED>
__device__ __forceinline__ u4v load_row8(const uint16_t* p, int k, int n) {
  if constexpr (ALIGNED) return *reinterpret_cast<const u4v*>(p + min(k, n - 8));
  u4v r = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t v = p[min(k + e, n - 1)];
    r[e >> 1] |= v << (16 * (e & 1));
  }
  return r;
}

}  // namespace cefn
