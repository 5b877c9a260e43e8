// Internal interface of the few-token forward pass (few.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"

namespace cefn {

constexpr int FEW_MAX_T = 32;   // tokens a pass takes: two 16-row MFMA tiles
constexpr int FEW_WAVES = 16;   // wavefronts per workgroup (8 in the input projection's large grids)

struct FewArgs {
  const void* X;  // [T][d]
  void* Y;        // [T][d]
  int T, d, f, G, K, kg, ke, k, E, Pin;
  int resid, act;
  // router (layout in kernels.h)
  const float* Wr;
  int NCp, nsplit;
  const float* bias;  // [score columns]: group then expert biases
  uint32_t over_nc, over_kg, over_ke, over_k;  // ceil(2^32 / n) of the score columns, kg, ke and k (0 for n = 1)
  float* L;       // [nsplit][T][NCp] partial scores
  int* ticket;    // zero between passes
  // routing results, and the caller's lists (null where not asked for)
  int* idx;       // [T][k]
  float* w;       // [T][k]
  int* gidx;      // [T][kg]
  int *counts, *offsets, *perm, *gcounts, *goffsets, *gperm;
  int wants_lists;  // any of the six is asked for
  // touched groups: glist[0] of them, grec[a] the a-th's {group, its first
  // touched expert in elist, how many, its tokens}, and grow[a][t] the row
  // t*kg + rank of token t in it, or -1 (rows t < T)
  int* glist;
  int4* grec;
  int16_t* grow;  // [min(G, T*kg)][FEW_MAX_T]
  // the touched experts, group by group, with a residual: elist[0] of them,
  // and eslot[i][t] the slot t*k + b of token t that chose expert elist[1 + i], or -1
  int* elist;
  int16_t* eslot;  // [min(E, T*k)][FEW_MAX_T]
  // residual input factors
  const void* At;
  const uint16_t* At_s;
  long at_gs, at_sgs;
  float* U;       // [T][E][Pin][16]
  int u_all;      // U of every expert, in the scores' launch; 0: of the chosen ones, in a launch of its own
  // weights (layouts in kernels.h; 4-bit bases in q4.h)
  const void *W1, *W2;
  long w1_gs, w2_gs;             // per group: elements, or 32-bit words of a 4-bit base
  const uint16_t *W1_s, *W2_s;   // 4-bit base: scales
  long w1_sgs, w2_sgs;
  int w1_units;   // 4-bit base: units per tile of W1
  const void *B1, *Ad, *Bd;
  long bd_gs;
  int NV;
  const uint16_t *B1_s, *Ad_s, *Bd_s;
  float* Vp;      // [f blocks][T*k][16] partials of h A_down
  float* V;       // [T*k + 1][16]: their sums (v_sum), and a row of zeros at zero_slot
  int v_sum;      // 1: summed by a launch of its own; 0: by every workgroup of the down product
  int zero_slot;
  void* H;        // [T*kg][planes][f]: gate-weighted hidden sums, in fp32 or one or two 16-bit parts
  int zero_row;   // row of H that stays zero (the last of the workspace)
};

// k splits of the score product over workgroups.
int few_router_splits(int d);
// Whether the partials of h A_down are summed by a launch of their own.
bool few_v_sum(const FewArgs& a);
// The pass: activations xt, MFMAs ty, 4-bit base or not.
hipError_t launch_few(int xt, int ty, bool q4, const FewArgs& a, hipStream_t st);

// Base weights [rows n_in][cols] per group in device memory to the
// fragment-major order of kernels.h; es: element bytes.  src1: the second of
// two column-interleaved sources (SwiGLU's up projection) or null.
hipError_t launch_repack(int es, const void* src0, const void* src1, int groups, int n_in, int n_out, void* dst,
                         hipStream_t st);

}  // namespace cefn
