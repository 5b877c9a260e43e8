// Top-k by one wavefront, shared by the routing kernels.
#pragma once
#include "common.h"

namespace cefn {

// Largest value of a wavefront, by row shifts and row broadcasts (lane 63 ends
// with it; six dependent VALU steps, no LDS).  No NaNs.
__device__ __forceinline__ float wave_max(float v) {
  const int lowest = static_cast<int>(0xFF800000u);  // -inf where a step has no source
  auto step = [&](float x, auto ctrl, auto rows) {
    const int o = __builtin_amdgcn_update_dpp(lowest, __float_as_int(x), decltype(ctrl)::value, decltype(rows)::value,
                                              0xf, false);
    return fmaxf(x, __int_as_float(o));
  };
  using std::integral_constant;
  v = step(v, integral_constant<int, 0x111>{}, integral_constant<int, 0xf>{});  // row_shr:1
  v = step(v, integral_constant<int, 0x112>{}, integral_constant<int, 0xf>{});
  v = step(v, integral_constant<int, 0x114>{}, integral_constant<int, 0xf>{});
  v = step(v, integral_constant<int, 0x118>{}, integral_constant<int, 0xf>{});
  v = step(v, integral_constant<int, 0x142>{}, integral_constant<int, 0xa>{});  // row_bcast:15
  v = step(v, integral_constant<int, 0x143>{}, integral_constant<int, 0xc>{});  // row_bcast:31
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Wavefront top-k (higher score first, ties to the lower index, NaN as -inf).
// Up to 64 candidates: one per lane, and each round takes the lowest lane that
// holds the largest value left.  More: candidate c sits on lane c % 64 and
// each round takes the best remaining one by a butterfly over the lanes.
// Selection r ends up in lane r's (myv, myi).  k <= n, k <= 64.
__device__ inline void wave_topk(const float* sv, int n, int k, int lane, float& myv, int& myi) {
  if (n <= 64) {
    float v = -INFINITY;
    if (lane < n) {
      v = sv[lane];
      v = (v == v) ? v : -INFINITY;
    }
    bool left = lane < n;
    myv = -INFINITY;
    myi = -1;
#pragma unroll 1
    for (int r = 0; r < k; ++r) {
      const float best = wave_max(left ? v : -INFINITY);
      const int c = __ffsll(static_cast<long long>(__ballot(left && v == best))) - 1;
      if (lane == c) left = false;
      if (lane == r) {
        myv = best;
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
