// Top-k by one wavefront, shared by the routing kernels.
#pragma once
#include "common.h"

namespace cefn {

// Wavefront top-k (higher score first, ties to
// the lower index, NaN as -inf).  Up to 64 candidates: lane c ranks
// candidate c by counting the candidates ahead of it.  More: candidate c
// sits on lane c % 64 and each round takes the best remaining one by a
// butterfly over the lanes.  Selection r ends up in lane r's (myv, myi).
// k <= n, k <= 64.
__device__ inline void wave_topk(const float* sv, int n, int k, int lane, float& myv, int& myi) {
  if (n <= 64) {
    // one candidate per lane, ranked against all n in that same order (a
    // total order, so the ranks are 0 .. n-1): no cross-lane rounds
    float v = -INFINITY;
    if (lane < n) {
      v = sv[lane];
      v = (v == v) ? v : -INFINITY;
    }
    int rank = 0;
    for (int j = 0; j < n; ++j) {
      const float u = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), j));
      rank += (u > v || (u == v && j < lane)) ? 1 : 0;
    }
    myv = -INFINITY;
    myi = -1;
    for (int r = 0; r < k; ++r) {
      const unsigned long long m = __ballot(lane < n && rank == r);
      const int c = __ffsll((long long)m) - 1;
      const float u = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), c));
      if (lane == r) {
        myv = u;
        myi = c;
      }
    }
    return;
  }
  uint32_t used = 0;  // bit q: candidate lane + 64 q taken
  myv = -INFINITY;
  myi = -1;
  for (int r = 0; r < k; ++r) {
    float bv = -INFINITY;
    int bi = 0x7fffffff;
    int bok = 0;
    for (int q = 0; lane + 64 * q < n; ++q) {
      if ((used >> q) & 1u) continue;
      float v = sv[lane + 64 * q];
      v = (v == v) ? v : -INFINITY;
      if (!bok || v > bv) {
        bv = v;
        bi = lane + 64 * q;
        bok = 1;
      }
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const float ov = __shfl_xor(bv, m);
      const int oi = __shfl_xor(bi, m);
      const int ook = __shfl_xor(bok, m);
      if (ook && (!bok || ov > bv || (ov == bv && oi < bi))) {
        bv = ov;
        bi = oi;
        bok = 1;
      }
    }
    if (lane == r) {
      myv = bv;
      myi = bi;
    }
    if ((bi & 63) == lane) used |= 1u << (bi >> 6);
  }
}

}  // namespace cefn
