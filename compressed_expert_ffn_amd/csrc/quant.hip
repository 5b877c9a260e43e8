// Products of a few rows with a 4-bit matrix and group scales
// (include/moe_quant.h), and the packing of 4-bit matrices (q4.h).
//
// y = x W is bound by the bytes of W: half a byte per weight plus the scales,
// against at most 32 rows of x that stay in the caches.  Every code is read
// once, in 16-byte loads, for all rows together; the arithmetic runs on
// 16x16x32 MFMAs with the rows of x as the 16 rows of the A operand (q4.h has
// the decode and its exactness).
#include <hip/hip_runtime.h>

#include <memory>
#include <new>

#include "api_internal.h"
#include "moe_quant.h"
#include "q4.h"
#include "stream.h"

namespace cefn {

namespace {

// ------------------------------------------------------------- packing --
__device__ __forceinline__ float source_value(const Q4Source& s, int n_out, int k, int n) {
  int p = 0, col = n, cols = n_out;
  if (s.n_src == 2) {  // 16-column blocks of source 0, source 1, source 0, ...
    p = (n >> 4) & 1;
    col = (n >> 5) * 16 + (n & 15);
    cols = n_out / 2;
  }
  const long i = static_cast<long>(k) * cols + col;
  if (s.v_dtype == DT_F32) return static_cast<const float*>(s.v[p])[i];
  const uint16_t b = static_cast<const uint16_t*>(s.v[p])[i];
  return s.v_dtype == DT_F16 ? f16_bits_to_f32(b) : bf16_bits_to_f32(b);
}

// One thread per (scale row entry): the rows of one column that share a scale
// (or, where a group spans several units, all of them).
__global__ __launch_bounds__(256) void q4_pack_kernel(Q4Shape s, Q4Source src, int bit, uint32_t* words,
                                                      uint16_t* scales) {
  const int groups = (s.n_in + s.group - 1) / s.group;
  const int width = static_cast<int>(s.tiles()) * 16 * s.C;  // columns, padding included
  const long id = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int n = static_cast<int>(id % width);
  const int unit = s.unit();
  // groups that exist in the padded depth of the last unit
  const long gpad = (s.units() * unit + s.group - 1) / s.group;
  const long grp = id / width;
  if (grp >= gpad) return;
  const int k0 = static_cast<int>(grp) * s.group;
  const int k1 = min(k0 + s.group, s.n_in);
  const bool real = n < s.n_out && grp < groups;
  float scale = 0.f;
  uint16_t sbits = 0;
  if (real) {
    if (src.q) {
      sbits = src.scale[grp * s.n_out + n];
    } else {
      float amax = 0.f;
      for (int k = k0; k < k1; ++k) amax = fmaxf(amax, fabsf(source_value(src, s.n_out, k, n)));
      sbits = f32_to_f16_bits(amax / 7.0f);
      scale = f16_bits_to_f32(sbits);
    }
  }
  const int tile = n / (16 * s.C), c = (n >> 4) % s.C, l = n & 15;
  const long urow = k0 / unit;  // first unit of the group
  const int sg = s.group >= unit ? 0 : (k0 % unit) / s.group;
  scales[((static_cast<long>(tile) * s.srows() + urow / s.srow_units()) * 16 + l) * s.entries() + sg * s.C + c] = sbits;
  const int kend = static_cast<int>(min(static_cast<long>(k0) + s.group, s.units() * unit));
  for (int k = k0; k < kend; k += 8) {
    uint32_t nib = 0;
    for (int e = 0; e < 8; ++e) {
      int q = 0;
      if (real && k + e < s.n_in) {
        if (src.q) {
          q = src.q[static_cast<long>(k + e) * s.n_out + n];
        } else if (scale > 0.f) {
          const float v = rintf(source_value(src, s.n_out, k + e, n) / scale);
          q = static_cast<int>(fminf(fmaxf(v, -8.f), 7.f));
        }
      }
      nib |= static_cast<uint32_t>((q + 8) & 15) << (4 * e);
    }
    const long u = k / unit;
    const int r = k % unit;  // row inside the unit
    const int lane = l + 16 * ((r >> 3) & 3), j = (r >> 5) * s.C + c;
    words[((static_cast<long>(tile) * s.units() + u) * 64 + lane) * 4 + j] = q4_word(nib, bit);
  }
}

__global__ __launch_bounds__(256) void q4_unpack_kernel(Q4Shape s, int bit, const uint32_t* words,
                                                        const uint16_t* scales, int8_t* q, uint16_t* scale) {
  const long id = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (id >= static_cast<long>(s.n_in) * s.n_out) return;
  const int k = static_cast<int>(id / s.n_out), n = static_cast<int>(id % s.n_out);
  const int unit = s.unit();
  const int tile = n / (16 * s.C), c = (n >> 4) % s.C, l = n & 15;
  const long u = k / unit;
  const int r = k % unit;
  const uint32_t w = words[((static_cast<long>(tile) * s.units() + u) * 64 + l + 16 * ((r >> 3) & 3)) * 4 +
                           (r >> 5) * s.C + c];
  q[id] = static_cast<int8_t>(q4_code(w, r & 7, bit) - 8);
  if (k % s.group == 0) {
    const int sg = s.group >= unit ? 0 : r / s.group;
    scale[static_cast<long>(k / s.group) * s.n_out + n] =
        scales[((static_cast<long>(tile) * s.srows() + u / s.srow_units()) * 16 + l) * s.entries() + sg * s.C + c];
  }
}

__global__ __launch_bounds__(256) void q4_check_kernel(const int8_t* q, long n, int* bad) {
  const long i = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i < n && (q[i] < -8 || q[i] > 7)) *bad = 1;
}

// ------------------------------------------------------------- product --
struct MatvecArgs {
  Q4Shape s;
  const uint32_t* words;
  const uint16_t* scales;
  const uint16_t* X;
  long ldx;
  int T;  // rows, at most 16 MT
  uint16_t* Y;
  long ldy;
};

// grid: one workgroup per tile of 16 C columns; its NW wavefronts take
// consecutive ranges of 128-deep runs (C units each) and their sums meet in
// LDS.  GPU: groups per unit.  XI: loads of x per run, 4 rows each, so at most
// 4 XI rows.  ALIGNED: rows of X can be read 16 bytes at a time.
//
// A run of x is read the way memory holds it, 16 lanes to the 256 bytes of a
// row, and goes through the wavefront's own part of LDS to become operands
// (row on lane % 16).  Read as operands directly, 64 bytes of 16 rows, each
// load touches 16 lines for half of each; a compute unit takes about 2.5
// clocks a line, which bound every product of several rows (14336 x 4096,
// 32 rows: 31 us), and one row still cost the loads of 16.
template <int XT, int C, int GPU, int XI, int NW, int R, bool ALIGNED>
__global__ __launch_bounds__(NW * 64) void q4_matvec_kernel(MatvecArgs a) {
  using B = typename Frag<XT>::T;
  constexpr int MT = (4 * XI + 15) / 16;     // tiles of 16 rows
  constexpr int NS = 4 / C;                  // 32-row steps per unit
  constexpr int E = C * GPU;                 // scales per column and unit
  constexpr int SPG = NS / GPU;              // 32-row steps per group
  constexpr int PITCH = 272;                 // bytes of a row of x in LDS: 16 past a multiple of 128
  constexpr int XROWS = 16 * MT;
  extern __shared__ __attribute__((aligned(16))) char lds[];  // x [NW][XROWS][PITCH]; later sums [NW][C][MT][256]
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int l = lane & 15, q = lane >> 4;
  const int runs = static_cast<int>(a.s.units()) / C;
  const int u0 = static_cast<int>(static_cast<long>(runs) * wave / NW);
  const int u1 = static_cast<int>(static_cast<long>(runs) * (wave + 1) / NW);
  const uint32_t* wp = a.words + static_cast<long>(blockIdx.x) * a.s.units() * 256 + lane * 4;
  const uint16_t* sp = a.scales + (static_cast<long>(blockIdx.x) * a.s.srows() * 16 + l) * E;
  const int su = a.s.srow_units();
  // lane 16 r + c of load i: row 4 i + r, depths 8 c .. of the run
  const uint16_t* xp[XI];
#pragma unroll
  for (int i = 0; i < XI; ++i) xp[i] = a.X + min(4 * i + q, a.T - 1) * a.ldx;  // rows past T repeat the last one
  char* xw = lds + wave * XROWS * PITCH + q * PITCH + l * 16;
  const char* xr = lds + wave * XROWS * PITCH + min(l, 4 * XI - 1) * PITCH + q * 16;
  struct Slot {
    u4v w[C];
    u2v s[C];  // E fp16 scales
    u4v x[XI];
  };
  f4v acc[C][MT];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[c][m] = f4v{0.f, 0.f, 0.f, 0.f};
  const B ones = q4_ones<XT>();
  stream_units<ALIGNED ? R : 1, Slot>(
      u1 - u0,
      [&](int i, Slot& s) {
        const int run = u0 + i;
#pragma unroll
        for (int j = 0; j < C; ++j) {
          const int u = run * C + j;
          s.w[j] = *reinterpret_cast<const u4v*>(wp + static_cast<long>(u) * 256);
          s.s[j] = load_scales<E>(sp + static_cast<long>(u / su) * 16 * E);
        }
#pragma unroll
        for (int j = 0; j < XI; ++j) s.x[j] = load_row8<ALIGNED>(xp[j], run * 128 + 8 * l, a.s.n_in);
      },
      [&](const Slot& s) {
        // the wavefront's LDS operations run in order, so its reads see its
        // writes and the next run's writes come after them
#pragma unroll
        for (int j = 0; j < XI; ++j) *reinterpret_cast<u4v*>(xw + 4 * j * PITCH) = s.x[j];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < C; ++j) {
#pragma unroll
          for (int g = 0; g < GPU; ++g) {
            B x[SPG][MT];
            f4v part[C][MT];
            // sum of the group's activations, in every column of the tile
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              f4v sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int st = 0; st < SPG; ++st) {
                const int step = j * NS + g * SPG + st;
                x[st][m] = __builtin_bit_cast(B, *reinterpret_cast<const u4v*>(xr + 16 * m * PITCH + step * 64));
                sum = mfma16<XT>(x[st][m], ones, sum);
              }
#pragma unroll
              for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) part[c][m][i] = -kQ4Offset * sum[i];
            }
#pragma unroll
            for (int st = 0; st < SPG; ++st)
#pragma unroll
              for (int c = 0; c < C; ++c) {
                const uint32_t word = s.w[j][(g * SPG + st) * C + c];
                const B b = q4_frag<XT>(word);
#pragma unroll
                for (int m = 0; m < MT; ++m) part[c][m] = mfma16<XT>(x[st][m], b, part[c][m]);
              }
#pragma unroll
            for (int c = 0; c < C; ++c) {
              const float sc = scale_at(s.s[j], g * C + c);
#pragma unroll
              for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[c][m][i] += sc * part[c][m][i];
            }
          }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      });
  __syncthreads();  // every wavefront is done with its x: the sums take its place
  float* red = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int m = 0; m < MT; ++m)
      *reinterpret_cast<f4v*>(red + ((wave * C + c) * MT + m) * 256 + lane * 4) = acc[c][m];
  __syncthreads();
  // row 4 (lane / 16) + i of a block, column lane % 16: consecutive threads
  // take consecutive columns
  constexpr int COLS = C * 16;
  for (int v = threadIdx.x; v < COLS * a.T; v += NW * 64) {
    const int row = v / COLS, col = v % COLS;
    const int n = blockIdx.x * COLS + col;
    if (n >= a.s.n_out) continue;
    const int r = row & 15;
    const int at = ((col >> 4) * MT + (row >> 4)) * 256 + (16 * (r >> 2) + (col & 15)) * 4 + (r & 3);
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) sum += red[w * C * MT * 256 + at];
    a.Y[row * a.ldy + n] = from_f32<XT>(sum * Q4Type<XT>::undo);
  }
}

template <int XT, int C, int GPU, int XI, int NW, int R>
hipError_t launch_mv3(const MatvecArgs& a, bool aligned, hipStream_t st) {
  constexpr int MT = (4 * XI + 15) / 16;
  const dim3 grid(static_cast<unsigned>(a.s.tiles())), block(NW * 64);
  constexpr size_t xb = static_cast<size_t>(NW) * 16 * MT * 272, sb = sizeof(float) * NW * C * MT * 256;
  constexpr size_t lds = xb > sb ? xb : sb;
  auto go = [&](auto kernel) -> hipError_t {
    if (lds > 64 * 1024) {
      const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kernel, grid, block, lds, st, a);
    return hipGetLastError();
  };
  return aligned ? go(q4_matvec_kernel<XT, C, GPU, XI, NW, R, true>)
                 : go(q4_matvec_kernel<XT, C, GPU, XI, NW, R, false>);
}

template <int XT, int C, int GPU>
hipError_t launch_mv2(const MatvecArgs& a, bool aligned, hipStream_t st) {
  // Narrow tiles: about one workgroup per compute unit, which 16 wavefronts
  // fill; wide ones: more workgroups or more loads per run, 8 wavefronts and
  // deeper rings.  Measured (us, 8 / 16 wavefronts): 4096 x 4096, 1 row 5.3 /
  // 4.9, 32 rows 9.9 / 8.6; 4096 x 14336, 1 row 10.0 / 10.1, 32 rows 15.8 / 21.4.
  constexpr int W = C == 1 ? 16 : 8;
  if (a.T <= 4) return launch_mv3<XT, C, GPU, 1, W, C == 4 ? 2 : C == 2 ? 4 : 3>(a, aligned, st);
  if (a.T <= 8) return launch_mv3<XT, C, GPU, 2, W, C == 4 ? 2 : C == 2 ? 4 : 2>(a, aligned, st);
  if (a.T <= 16) return launch_mv3<XT, C, GPU, 4, W, C == 4 ? 2 : C == 2 ? 3 : 1>(a, aligned, st);
  return launch_mv3<XT, C, GPU, 8, W, C == 4 ? 2 : C == 2 ? 3 : 1>(a, aligned, st);
}

template <int XT>
hipError_t launch_mv(const MatvecArgs& a, bool aligned, hipStream_t st) {
  const int gpu = a.s.gpu();
  switch (a.s.C) {
    case 1:
      return gpu == 4 ? launch_mv2<XT, 1, 4>(a, aligned, st)
                      : gpu == 2 ? launch_mv2<XT, 1, 2>(a, aligned, st) : launch_mv2<XT, 1, 1>(a, aligned, st);
    case 2: return gpu == 2 ? launch_mv2<XT, 2, 2>(a, aligned, st) : launch_mv2<XT, 2, 1>(a, aligned, st);
    case 4: return launch_mv2<XT, 4, 1>(a, aligned, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_q4_pack(const Q4Shape& s, const Q4Source& src, int ty, uint32_t* words, uint16_t* scales,
                          hipStream_t st) {
  const long gpad = (s.units() * s.unit() + s.group - 1) / s.group;
  const long n = s.tiles() * 16 * s.C * gpad;
  hipLaunchKernelGGL(q4_pack_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, st, s, src,
                     q4_bit(ty), words, scales);
  return hipGetLastError();
}

hipError_t launch_q4_unpack(const Q4Shape& s, int ty, const uint32_t* words, const uint16_t* scales, int8_t* q,
                            uint16_t* scale, hipStream_t st) {
  const long n = static_cast<long>(s.n_in) * s.n_out;
  hipLaunchKernelGGL(q4_unpack_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, st, s, q4_bit(ty),
                     words, scales, q, scale);
  return hipGetLastError();
}

}  // namespace cefn

// -------------------------------------------------------------------- C ABI --
using namespace cefn;
using namespace cefn_api;

struct moe_quant {
  moe_quant_config cfg{};
  Q4Shape shape{};
  int device = 0;
  uint32_t* words = nullptr;
  uint16_t* scales = nullptr;
};

namespace {

int validate_quant(const moe_quant_config* c) {
  if (!c) return fail(MOE_ERR_INVALID_ARG, "null config");
  if (c->n_in < 1 || c->n_out < 1) return fail(MOE_ERR_INVALID_ARG, "n_in and n_out must be positive");
  if (c->x_dtype < 0 || c->x_dtype > 2) return fail(MOE_ERR_INVALID_ARG, "unknown x_dtype %d", c->x_dtype);
  if (c->group != 32 && c->group != 64 && c->group != 128)
    return fail(MOE_ERR_UNSUPPORTED, "group %d is not 32, 64 or 128", c->group);
  if (c->x_dtype == MOE_F32) return fail(MOE_ERR_UNSUPPORTED, "x_dtype must be F16 or BF16");
  if (c->n_in > (1 << 24) || c->n_out > (1 << 24) || static_cast<int64_t>(c->n_in) * c->n_out > (1LL << 31))
    return fail(MOE_ERR_UNSUPPORTED, "n_in, n_out <= 2^24 and n_in * n_out <= 2^31");
  return MOE_OK;
}

// Columns per tile (16 C): the widest tile that still gives most compute units
// a workgroup, since a wide tile re-uses the activations' fragments.  8192 x
// 28672 in tiles of 64 / 32 / 16 columns: 46 / 58 / 76 us for 24 rows, 27.7 /
// 26.4 / 25.3 us for one; 4096 x 14336: 15.9 / 22.1 / 31.8 us for 32 rows,
// 9.8 / 9.1 / 9.6 us for one.
int pick_c(int n_out) {
  for (int C : {4, 2})
    if ((n_out + 16 * C - 1) / (16 * C) >= 192) return C;
  return 1;
}

struct DeviceBuffers {
  void* p[3] = {};
  ~DeviceBuffers() {
    for (void* q : p)
      if (q) (void)hipFree(q);
  }
};

}  // namespace

extern "C" {

int moe_quant_destroy(moe_quant* h) {
  if (!h) return MOE_OK;
  int cur = -1;
  const bool other = hipGetDevice(&cur) == hipSuccess && cur != h->device && hipSetDevice(h->device) == hipSuccess;
  (void)hipDeviceSynchronize();
  if (h->words) (void)hipFree(h->words);
  if (h->scales) (void)hipFree(h->scales);
  if (other) (void)hipSetDevice(cur);
  delete h;
  return MOE_OK;
}

int moe_quant_create(const moe_quant_config* cfg, const moe_quant_weights* w, void* stream, moe_quant** out) {
  if (out) *out = nullptr;
  TRY(validate_quant(cfg));
  if (!w || !out) return fail(MOE_ERR_INVALID_ARG, "null weights or output handle");
  if ((w->q != nullptr) == (w->values != nullptr))
    return fail(MOE_ERR_INVALID_ARG, "give either q with scale, or values");
  if (w->q && !w->scale) return fail(MOE_ERR_INVALID_ARG, "q needs scale");
  if (w->values && (w->values_dtype < 0 || w->values_dtype > 2))
    return fail(MOE_ERR_INVALID_ARG, "unknown values_dtype %d", w->values_dtype);
  struct Guard {
    moe_quant* h;
    ~Guard() { (void)moe_quant_destroy(h); }
  } g{new (std::nothrow) moe_quant()};
  moe_quant* h = g.h;
  if (!h) return fail(MOE_ERR_OOM, "host memory");
  if (hipGetDevice(&h->device) != hipSuccess) {
    (void)hipGetLastError();
    return fail(MOE_ERR_HIP, "no HIP device");
  }
  h->cfg = *cfg;
  h->shape = Q4Shape{cfg->n_in, cfg->n_out, pick_c(cfg->n_out), cfg->group};
  const Q4Shape& s = h->shape;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const size_t n = static_cast<size_t>(cfg->n_in) * cfg->n_out;
  const size_t ns = static_cast<size_t>((cfg->n_in + cfg->group - 1) / cfg->group) * cfg->n_out;
  DeviceBuffers tmp;
  auto place = [&](const void* p, size_t bytes, void** keep, const void** at) -> int {
    *at = p;
    if (w->on_device || !p) return MOE_OK;
    if (hipMalloc(keep, bytes) != hipSuccess) {
      (void)hipGetLastError();
      return fail(MOE_ERR_OOM, "hipMalloc of %zu bytes failed", bytes);
    }
    if (hipMemcpy(*keep, p, bytes, hipMemcpyHostToDevice) != hipSuccess) {
      (void)hipGetLastError();
      return fail(MOE_ERR_HIP, "copy to device failed");
    }
    *at = *keep;
    return MOE_OK;
  };
  Q4Source src{};
  src.n_src = 1;
  src.v_dtype = w->values_dtype;
  const void* at = nullptr;
  TRY(place(w->q, n, &tmp.p[0], &at));
  src.q = static_cast<const int8_t*>(at);
  TRY(place(w->q ? w->scale : nullptr, ns * 2, &tmp.p[1], &at));
  src.scale = static_cast<const uint16_t*>(at);
  TRY(place(w->values, n * (w->values_dtype == MOE_F32 ? 4 : 2), &tmp.p[0], &at));
  src.v[0] = at;
  if (hipMalloc(&tmp.p[2], sizeof(int)) != hipSuccess ||
      hipMalloc(reinterpret_cast<void**>(&h->words), s.words() * 4) != hipSuccess ||
      hipMalloc(reinterpret_cast<void**>(&h->scales), s.scales() * 2) != hipSuccess) {
    (void)hipGetLastError();
    return fail(MOE_ERR_OOM, "hipMalloc of %ld bytes failed", s.words() * 4 + s.scales() * 2);
  }
  int bad = 0;
  hipError_t e = launch_zero(static_cast<int*>(tmp.p[2]), 1, st);
  if (e == hipSuccess && src.q) {
    hipLaunchKernelGGL(q4_check_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, st, src.q,
                       static_cast<long>(n), static_cast<int*>(tmp.p[2]));
    e = hipGetLastError();
  }
  if (e == hipSuccess) e = launch_q4_pack(s, src, cfg->x_dtype, h->words, h->scales, st);
  if (e == hipSuccess) e = hipStreamSynchronize(st);
  if (e == hipSuccess) e = hipMemcpy(&bad, tmp.p[2], sizeof(int), hipMemcpyDeviceToHost);
  if (e != hipSuccess) return fail(MOE_ERR_HIP, "packing: %s", hipGetErrorString(e));
  if (bad) return fail(MOE_ERR_INVALID_ARG, "q holds a code outside [-8, 7]");
  *out = h;
  g.h = nullptr;
  return MOE_OK;
}

int moe_quant_matvec(const moe_quant* h, const void* X, int64_t ldx, int32_t T, void* Y, int64_t ldy, void* stream) {
  if (!h) return fail(MOE_ERR_INVALID_ARG, "null handle");
  if (T < 0) return fail(MOE_ERR_INVALID_ARG, "T=%d is negative", T);
  if (ldx < h->cfg.n_in || ldy < h->cfg.n_out)
    return fail(MOE_ERR_INVALID_ARG, "ldx=%lld < n_in=%d or ldy=%lld < n_out=%d", (long long)ldx, h->cfg.n_in,
                (long long)ldy, h->cfg.n_out);
  if (T == 0) return MOE_OK;
  if (!X || !Y) return fail(MOE_ERR_INVALID_ARG, "null X or Y");
  if (X == Y) return fail(MOE_ERR_INVALID_ARG, "X and Y may not overlap");
  if ((reinterpret_cast<uintptr_t>(X) | reinterpret_cast<uintptr_t>(Y)) & 1)
    return fail(MOE_ERR_INVALID_ARG, "X and Y must be aligned to their type");
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess) return fail(MOE_ERR_HIP, "no HIP device");
  if (dev != h->device)
    return fail(MOE_ERR_INVALID_ARG, "handle lives on device %d, device %d is current", h->device, dev);
  const bool aligned = !(reinterpret_cast<uintptr_t>(X) & 15) && ldx % 8 == 0 && h->cfg.n_in % 8 == 0;
  for (int32_t t = 0; t < T; t += Q4_ROWS) {
    MatvecArgs a{h->shape, h->words, h->scales, static_cast<const uint16_t*>(X) + t * ldx, ldx,
                 T - t < Q4_ROWS ? T - t : Q4_ROWS, static_cast<uint16_t*>(Y) + t * ldy, ldy};
    const hipError_t e = h->cfg.x_dtype == MOE_F16
                             ? launch_mv<DT_F16>(a, aligned, static_cast<hipStream_t>(stream))
                             : launch_mv<DT_BF16>(a, aligned, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(MOE_ERR_HIP, "matvec launch: %s", hipGetErrorString(e));
  }
  return MOE_OK;
}

int moe_quant_read(const moe_quant* h, int8_t* q, uint16_t* scale) {
  if (!h) return fail(MOE_ERR_INVALID_ARG, "null handle");
  const size_t n = static_cast<size_t>(h->cfg.n_in) * h->cfg.n_out;
  const size_t ns = static_cast<size_t>((h->cfg.n_in + h->cfg.group - 1) / h->cfg.group) * h->cfg.n_out;
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess) return fail(MOE_ERR_HIP, "no HIP device");
  if (dev != h->device)
    return fail(MOE_ERR_INVALID_ARG, "handle lives on device %d, device %d is current", h->device, dev);
  DeviceBuffers tmp;
  if (hipMalloc(&tmp.p[0], n) != hipSuccess || hipMalloc(&tmp.p[1], ns * 2) != hipSuccess) {
    (void)hipGetLastError();
    return fail(MOE_ERR_OOM, "read buffers");
  }
  hipError_t e = launch_q4_unpack(h->shape, h->cfg.x_dtype, h->words, h->scales, static_cast<int8_t*>(tmp.p[0]),
                                  static_cast<uint16_t*>(tmp.p[1]), nullptr);
  if (e == hipSuccess) e = hipDeviceSynchronize();
  if (e == hipSuccess && q) e = hipMemcpy(q, tmp.p[0], n, hipMemcpyDeviceToHost);
  if (e == hipSuccess && scale) e = hipMemcpy(scale, tmp.p[1], ns * 2, hipMemcpyDeviceToHost);
  if (e != hipSuccess) return fail(MOE_ERR_HIP, "read: %s", hipGetErrorString(e));
  return MOE_OK;
}

int64_t moe_quant_bytes(const moe_quant* h) {
  return h ? static_cast<int64_t>(h->shape.words()) * 4 + h->shape.scales() * 2 : 0;
}

}  // extern "C"
