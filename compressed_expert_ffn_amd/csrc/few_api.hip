// moe_forward_few (include/moe.h): workspace, argument checks and launches of
// the few-token forward pass (few.hip).
#include <algorithm>
#include <new>

#include "api_internal.h"
#include "few.h"

using namespace cefn;
using namespace cefn_api;

namespace {

int col_blocks(const moe_handle* h) { return h->cfg.f * h->P_in / 32; }

// A row of H: fp32, or one or two 16-bit parts (few.hip's hidden_planes).
size_t hidden_row_bytes(const moe_handle* h) {
  const moe_config& c = h->cfg;
  const bool one = c.x_dtype == MOE_BF16 && c.base_dtype != MOE_BF16;
  return (one ? 2 : 4) * (size_t)c.f;
}

}  // namespace

namespace cefn_api {

int create_few(moe_handle* h) {
  const moe_config& c = h->cfg;
  h->few = new (std::nothrow) FewState();
  if (!h->few) return fail(MOE_ERR_OOM, "host memory");
  FewState& s = *h->few;
  s.T_cap = std::min<int>(c.T_max, FEW_MAX_T);
  if (s.T_cap == 0) return MOE_OK;
  const size_t T = s.T_cap, kg = c.top_groups;
  size_t off = 0;
  char* base = nullptr;
  auto take = [&](size_t bytes) {
    char* p = base ? base + off : nullptr;
    off += (bytes + 255) & ~(size_t)255;
    return p;
  };
  auto carve = [&]() {
    off = 0;
    s.ticket = reinterpret_cast<int*>(take(sizeof(int)));
    s.idx = reinterpret_cast<int*>(take(sizeof(int) * T * h->k));
    s.w = reinterpret_cast<float*>(take(sizeof(float) * T * h->k));
    s.gidx = reinterpret_cast<int*>(take(sizeof(int) * T * kg));
    s.glist = reinterpret_cast<int*>(take(sizeof(int)));
    s.grec = reinterpret_cast<int4*>(take(sizeof(int4) * std::min<size_t>(c.G, T * kg)));
    s.grow = reinterpret_cast<int16_t*>(take(sizeof(int16_t) * std::min<size_t>(c.G, T * kg) * FEW_MAX_T));
    s.bias = reinterpret_cast<float*>(take(sizeof(float) * h->NCp));
    s.L = reinterpret_cast<float*>(take(sizeof(float) * few_router_splits(c.d) * T * h->NCp));
    s.elist = reinterpret_cast<int*>(take(sizeof(int) * (1 + std::min<size_t>(h->E, T * h->k))));
    s.eslot = reinterpret_cast<int16_t*>(take(sizeof(int16_t) * std::min<size_t>(h->E, T * h->k) * FEW_MAX_T));
    if (c.r > 0) {
      s.V = reinterpret_cast<float*>(take(sizeof(float) * (T * h->k + 1) * RPAD));
      s.U = reinterpret_cast<float*>(take(sizeof(float) * T * h->E * h->P_in * RPAD));
      s.Vp = reinterpret_cast<float*>(take(sizeof(float) * col_blocks(h) * T * h->k * RPAD));
    }
    s.H = take(hidden_row_bytes(h) * (T * kg + 1));
  };
  carve();
  TRY(dalloc(h, &base, off));
  carve();
  // biases of the score columns, zeros where the layer has none
  if (hipMemset(s.bias, 0, sizeof(float) * h->NCp) != hipSuccess ||
      (h->gbias && hipMemcpy(s.bias, h->gbias, sizeof(float) * c.G, hipMemcpyDeviceToDevice) != hipSuccess) ||
      (h->ebias && hipMemcpy(s.bias + c.G, h->ebias, sizeof(float) * h->E, hipMemcpyDeviceToDevice) != hipSuccess)) {
    (void)hipGetLastError();
    return fail(MOE_ERR_HIP, "initialising the few-token workspace failed");
  }
  char* zero = static_cast<char*>(s.H) + hidden_row_bytes(h) * T * kg;
  if (hipMemset(s.ticket, 0, sizeof(int)) != hipSuccess || hipMemset(zero, 0, hidden_row_bytes(h)) != hipSuccess ||
      (s.V && hipMemset(s.V + T * h->k * RPAD, 0, RPAD * sizeof(float)) != hipSuccess)) {
    (void)hipGetLastError();
    return fail(MOE_ERR_HIP, "initialising the few-token workspace failed");
  }
  return MOE_OK;
}

}  // namespace cefn_api

extern "C" int moe_forward_few(moe_handle* h, const void* X, int32_t T, void* Y, const moe_route_out* routing,
                               void* stream) {
  if (!h) return fail(MOE_ERR_INVALID_ARG, "null handle");
  const moe_config& c = h->cfg;
  if (T < 0 || T > c.T_max) return fail(MOE_ERR_INVALID_ARG, "T=%d outside [0, T_max=%d]", T, c.T_max);
  if (T > FEW_MAX_T)
    return fail(MOE_ERR_INVALID_ARG, "T=%d is more than the %d tokens of a few-token pass", T, FEW_MAX_T);
  if (T == 0) return routing ? moe_route(h, X, 0, routing, stream) : MOE_OK;
  if (!X || !Y) return fail(MOE_ERR_INVALID_ARG, "null X or Y");
  if (X == Y) return fail(MOE_ERR_INVALID_ARG, "X and Y may not alias");
  if ((reinterpret_cast<uintptr_t>(X) & 15) || (reinterpret_cast<uintptr_t>(Y) & (c.x_dtype == MOE_F32 ? 3 : 1)))
    return fail(MOE_ERR_INVALID_ARG, "X must be on a 16-byte boundary, Y aligned to its type");
  if (h->off) return fail(MOE_ERR_UNSUPPORTED, "the handle's groups are offloaded: use moe_forward_offload");
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess) return fail(MOE_ERR_HIP, "no HIP device");
  if (dev != h->device)
    return fail(MOE_ERR_INVALID_ARG, "handle lives on device %d, device %d is current", h->device, dev);
  const FewState& s = *h->few;
  const bool q4 = c.base_dtype == MOE_INT4_G32;
  FewArgs a{};
  a.X = X;
  a.Y = Y;
  a.T = T;
  a.d = c.d;
  a.f = c.f;
  a.G = c.G;
  a.K = c.K;
  a.kg = c.top_groups;
  a.ke = c.top_experts;
  a.k = h->k;
  a.E = h->E;
  a.Pin = h->P_in;
  a.resid = c.resid;
  a.act = c.act == MOE_ACT_SWIGLU ? ACT_SWIGLU : ACT_GELU;
  a.Wr = h->Wr;
  a.NCp = h->NCp;
  a.nsplit = few_router_splits(c.d);
  a.bias = s.bias;
  auto over = [](int n) { return static_cast<uint32_t>(((1ull << 32) + n - 1) / n); };  // 0 for n = 1
  a.over_nc = over(c.G + (c.K > 1 ? h->E : 0));
  a.over_kg = over(c.top_groups);
  a.over_ke = over(c.top_experts);
  a.over_k = over(h->k);
  a.L = s.L;
  a.ticket = s.ticket;
  a.idx = routing && routing->idx ? routing->idx : s.idx;
  a.w = routing && routing->w ? routing->w : s.w;
  a.gidx = routing && routing->gidx ? routing->gidx : s.gidx;
  if (routing) {
    a.counts = routing->counts;
    a.offsets = routing->offsets;
    a.perm = routing->perm;
    a.gcounts = routing->gcounts;
    a.goffsets = routing->goffsets;
    a.gperm = routing->gperm;
    a.wants_lists = a.counts || a.offsets || a.perm || a.gcounts || a.goffsets || a.gperm;
  }
  a.glist = s.glist;
  a.grec = s.grec;
  a.grow = s.grow;
  a.At = h->At;
  a.At_s = h->At_s;
  a.at_gs = h->at_gs;
  a.at_sgs = h->at_sgs;
  a.U = s.U;
  // The input factors of every expert are read beside the selection while they
  // take no longer than it and the launch that reading the chosen ones' alone
  // costs.  Measured, one token, every / chosen: 19 MB 32.8 / 39.7 us a pass,
  // 67 MB 41.0 / 34.1, 75 MB in 4 bits 63 / 46, 134 MB 71 / 45.
  const size_t factors = (size_t)c.G * (c.resid == MOE_RESID_INT4_G32 ? 4 * h->at_gs + 2 * h->at_sgs
                                                                      : elem_bytes(h->mma) * h->at_gs);
  a.u_all = factors <= ((size_t)40 << 20) ? 1 : 0;
  a.W1 = h->W1;
  a.W2 = h->W2;
  a.w1_gs = h->w1_gs;
  a.w2_gs = h->w2_gs;
  a.W1_s = h->W1_s;
  a.W2_s = h->W2_s;
  a.w1_sgs = h->w1_sgs;
  a.w1_units = h->w1_units;
  a.w2_sgs = h->w2_sgs;
  a.B1 = h->B1;
  a.Ad = h->Ad;
  a.Bd = h->Bd;
  a.bd_gs = h->bd_gs;
  a.NV = h->NV;
  a.B1_s = h->B1_s;
  a.Ad_s = h->Ad_s;
  a.Bd_s = h->Bd_s;
  a.Vp = s.Vp;
  a.H = s.H;
  a.zero_row = s.T_cap * c.top_groups;
  a.V = s.V;
  a.zero_slot = s.T_cap * h->k;
  a.elist = s.elist;
  a.eslot = s.eslot;
  hipStream_t st = static_cast<hipStream_t>(stream);
  a.v_sum = few_v_sum(a) ? 1 : 0;
  const hipError_t e = launch_few(c.x_dtype, h->mma, q4, a, st);
  if (e != hipSuccess) return fail(MOE_ERR_HIP, "few-token launch: %s", hipGetErrorString(e));
  return MOE_OK;
}
