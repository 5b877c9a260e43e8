// The whole layer for a few tokens (moe_forward_few): 1 to 32 rows.
//
// With so few rows the layer is a stream of weights: every byte of the
// touched groups' bases is read once, for all tokens together, and the rows
// sit in the registers as the 16 rows of a 16x16x32 MFMA operand (two tiles
// beyond 16 tokens).  What is left to save is launches and latency, so the
// pass has three kernels, four or five for some shapes, cut into workgroups of
// 16 columns of output (32 of a 4-bit base) whose 4 to 16 wavefronts split
// the depth of the product:
//   route  router scores; the last workgroup to finish them selects groups
//          and experts for every token and lists the touched groups; beside
//          it, u = x A for every expert where that is less than a launch
//          (else for the chosen ones, in a launch of its own)
//   up     z = x W1 of each touched group, then per (token, chosen expert)
//          z + u B, the activation, the gate weight, the sum over the
//          group's experts, and partials of h A_down over the columns
//   down   y = sum over the touched groups of hbar W2, plus the residual
//          tail (sum of the partials, taken by a launch of its own before
//          this one where they are many) B_down
// The sum over a token's groups is made where the down product is (in the
// accumulator or the workgroup's own memory), so no combine pass is left.
//
// Everything between the kernels is held in 32 bits, or, where it feeds a
// 16-bit MFMA (the hidden sums), as two 16-bit parts of a 32-bit number or as
// one of an eighth of the result's step (hidden_planes below), and residual
// codes multiply as integers with their scale applied to the sum.
#include <type_traits>

#include "few.h"
#include "kernels.h"
#include "q4.h"
#include "stream.h"
#include "topk.h"

namespace cefn {

namespace {

constexpr int NW = FEW_WAVES;
constexpr int NT = NW * 64;
constexpr int UW = NW / 2;  // wavefronts per block of input factors

// The value a wavefront's lane r (the same for all lanes) holds.
__device__ __forceinline__ float lane_value(float v, int r) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), r));
}

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Eight consecutive activations as loaded, and as operands.
template <int XT>
struct Raw {
  u4v v[XT == DT_F32 ? 2 : 1];
};
template <int XT>
__device__ __forceinline__ Raw<XT> load_raw(const typename Elem<XT>::T* p) {
  Raw<XT> r;
  r.v[0] = reinterpret_cast<const u4v*>(p)[0];
  if constexpr (XT == DT_F32) r.v[1] = reinterpret_cast<const u4v*>(p)[1];
  return r;
}
template <int XT>
__device__ __forceinline__ void raw_to_f32(const Raw<XT>& r, float (&o)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (XT == DT_F32) {
      const uint32_t u = r.v[e >> 2][e & 3];
      o[e] = __uint_as_float(u);
    } else {
      const uint32_t u = r.v[0][e >> 1];
      const uint16_t b = static_cast<uint16_t>((u >> (16 * (e & 1))) & 0xFFFFu);
      o[e] = XT == DT_F16 ? f16_bits_to_f32(b) : bf16_bits_to_f32(b);
    }
  }
}
template <int XT, int TY>
__device__ __forceinline__ typename Frag<TY>::T raw_to_frag(const Raw<XT>& r) {
  if constexpr (XT == TY && TY != DT_F32) {
    return __builtin_bit_cast(typename Frag<TY>::T, r.v[0]);
  } else {
    float v[8];
    raw_to_f32<XT>(r, v);
    return to_frag<TY>(v);
  }
}
// fp32 to a 16-bit MFMA type by the hardware's conversions (nearest, ties to even).
template <int TY>
__device__ __forceinline__ typename Frag<TY>::T round_frag(const float (&v)[8]) {
  typename Frag<TY>::T r;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (TY == DT_BF16) r[i] = static_cast<__bf16>(v[i]);
    else if constexpr (TY == DT_F16) r[i] = static_cast<_Float16>(v[i]);
    else r[i] = v[i];
  }
  return r;
}
template <int TY>
__device__ __forceinline__ uint16_t round_bits(float v) {
  if constexpr (TY == DT_BF16) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  else return f32_to_f16_bits(v);
}

// Type and 16-bit parts the gate-weighted hidden sums (and V) are held in for
// the down product.  An fp16 number is exact to 2^-11, an eighth of what a
// bf16 result is rounded by, so bf16 activations on fp16 MFMAs need one part;
// where the result has the MFMAs' own precision the sums keep two, 22 or 16
// bits, so that y is rounded once.  A 4-bit base takes either MFMA type, hence
// fp16 for its down product.
__host__ __device__ constexpr int hidden_type(int ty, bool q4) {
  return q4 ? DT_F16 : ty;
}
__host__ __device__ constexpr int hidden_planes(int xt, int ht) {
  return ht == DT_F32 || (xt == DT_BF16 && ht == DT_F16) ? 1 : 2;
}

// v + A_down^T h over 16 columns of f: lane (l, q) holds rank column l of the
// factor at columns 4 q .. + 3 and h of its token there; lane (l, q) of v:
// rank columns 4 q .. of token l.  h goes in as two 16-bit parts.
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef short s4 __attribute__((ext_vector_type(4)));
template <int TY>
__device__ __forceinline__ f4v mfma16k16(const uint16_t (&x)[4], const uint16_t (&y)[4], f4v c) {
  s4 p, r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    p[i] = static_cast<short>(x[i]);
    r[i] = static_cast<short>(y[i]);
  }
  if constexpr (TY == DT_F16)
    return __builtin_amdgcn_mfma_f32_16x16x16f16(__builtin_bit_cast(h4, p), __builtin_bit_cast(h4, r), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(p, r, c, 0, 0, 0);
}
// Its operand: four values (or the word holding four codes) of eight `at`, half `half`.
template <int TY, int RS>
__device__ __forceinline__ u4v load_down_factor(const void* Ad, long at, int half) {
  u4v r = {0u, 0u, 0u, 0u};
  if constexpr (TY == DT_F32) {
    r = *reinterpret_cast<const u4v*>(static_cast<const float*>(Ad) + at * 8 + 4 * half);
  } else if constexpr (RS == RS_INT4) {
    r[0] = static_cast<const uint32_t*>(Ad)[at] >> (16 * half);
  } else {
    const u2v d = *reinterpret_cast<const u2v*>(static_cast<const uint16_t*>(Ad) + at * 8 + 4 * half);
    r[0] = d[0];
    r[1] = d[1];
  }
  return r;
}
template <int TY, int RS>
__device__ __forceinline__ f4v down_factor(const u4v& ad, const float (&h)[4], f4v v) {
  if constexpr (TY == DT_F32) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint32_t w = ad[r];
      v = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w), h[r], v, 0, 0, 0);
    }
    return v;
  } else {
    uint16_t w[4], hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = ad[0], y = ad[i >> 1];
      w[i] = RS == RS_INT4 ? round_bits<TY>(static_cast<float>(static_cast<int>((x >> (4 * i)) & 15u) - 8))
                              : static_cast<uint16_t>((y >> (16 * (i & 1))) & 0xFFFFu);
      hi[i] = round_bits<TY>(h[i]);
      lo[i] = round_bits<TY>(h[i] - (TY == DT_F16 ? f16_bits_to_f32(hi[i]) : bf16_bits_to_f32(hi[i])));
    }
    return mfma16k16<TY>(w, lo, mfma16k16<TY>(w, hi, v));
  }
}

// ---------------------------------------------------------------- route --
// Scores of 16 columns over this workgroup's part of the depth, in fp32
// MFMAs (the router runs in FP32; the matrix is small and the MFMAs hide
// behind its loads).
template <int XT, int MT>
__device__ void score_block(const FewArgs& a, int cb, int split, float* red) {
  using XE = typename Elem<XT>::T;
  const int wave = wave_id(), lane = threadIdx.x & 63, l = lane & 15, q = lane >> 4;
  const int n32 = a.d / 32, part = split * NW + wave, parts = a.nsplit * NW;
  const int u0 = static_cast<int>(static_cast<long>(n32) * part / parts);
  const int u1 = static_cast<int>(static_cast<long>(n32) * (part + 1) / parts);
  const XE* xp[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
    xp[m] = static_cast<const XE*>(a.X) + static_cast<long>(min(16 * m + l, a.T - 1)) * a.d + 8 * q;
  // column cb*16 + l, depth 8 q .. of each 32
  const float* wp = a.Wr + (static_cast<long>(q >> 1) * a.NCp + cb * 16 + l) * 16 + 8 * (q & 1);
  const long wstep = 2L * a.NCp * 16;
  struct Slot {
    Raw<XT> x[MT];
    f8 w;
  };
  f4v acc[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) acc[m] = f4v{0.f, 0.f, 0.f, 0.f};
  stream_units<3, Slot>(
      u1 - u0,
      [&](int i, Slot& s) {
        const long u = u0 + i;
        s.w = load_frag<DT_F32>(wp + u * wstep);
#pragma unroll
        for (int m = 0; m < MT; ++m) s.x[m] = load_raw<XT>(xp[m] + u * 32);
      },
      [&](const Slot& s) {
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m] = mfma16<DT_F32>(raw_to_frag<XT, DT_F32>(s.x[m]), s.w, acc[m]);
      });
#pragma unroll
  for (int m = 0; m < MT; ++m) *reinterpret_cast<f4v*>(red + (wave * MT + m) * 256 + lane * 4) = acc[m];
}

// Sum over NWV wavefronts of element (row, column) of a block of NS * 16
// columns, each wavefront's part held as [NS][MT] MFMA accumulators.
template <int NWV, int NS, int MT>
__device__ __forceinline__ float block_sum(const float* red, int row, int col) {
  const int r = row & 15;
  const int at = ((col >> 4) * MT + (row >> 4)) * 256 + (16 * (r >> 2) + (col & 15)) * 4 + (r & 3);
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < NWV; ++w) s += red[w * NS * MT * 256 + at];
  return s;
}

// u = x A for the 32 factor columns of block nb of group g, by half a
// workgroup (8 wavefronts; both halves call it together, real: whether this
// half has a block).  Two blocks per workgroup: 256 experts' blocks and the
// scores' workgroups are all resident at once (a workgroup each left some for
// a second round, 13.8 us the launch).
//
// 4-bit factors: a 64-deep unit of the block is 256 words, word 64 q' + 32 h +
// c for depths 64 u + 32 h + 8 q' .. and column c.  Lane 16 q + l takes words
// 4 (16 q + l) .. + 3 in one load: columns 4 (l % 8) + i at half h = l / 8,
// so the 16 columns of an MFMA are 8 real ones at both halves of the depth,
// and its 16 rows 8 tokens at both: the quarters of the product whose halves
// agree are kept, two MFMAs for one, but a fourth of the weights' loads (4-byte
// loads of each half's 16 columns took 6.4 us of a 256-expert layer's launch),
// and a load of activations takes 8 whole cache lines (a pass
// with rows of 16 tokens at one half each: 33.3 us, now 31.6, at T = 1, 124.4
// and 124.1 at T = 32).  The next 8 tokens take the halves in the other order,
// so the two quarters they keep are the ones that the first 8 leave.
template <int XT, int TY, bool INT4, int T8>
__device__ void u_block(const FewArgs& a, int g, int nb, bool real, float* red) {
  using XE = typename Elem<XT>::T;
  using B = typename Frag<TY>::T;
  const int wave = wave_id() % UW, lane = threadIdx.x & 63, l = lane & 15, q = lane >> 4;
  const int n64 = real ? a.d / 64 : 0, tid = threadIdx.x % (UW * 64);
  const int u0 = n64 * wave / UW, u1 = n64 * (wave + 1) / UW;
  const int cols = a.K * a.Pin * 16;  // column (j * Pin + p) * 16 + rho of the group
  if constexpr (INT4) {
    const int h = l >> 3;
    const uint32_t* wp =
        static_cast<const uint32_t*>(a.At) + g * a.at_gs + static_cast<long>(nb) * (a.d / 16) * 64 + 4 * lane;
    const uint16_t* sp =
        a.At_s + g * a.at_sgs + (static_cast<long>(nb) * (a.d / 32) + h) * 32 + 4 * (l & 7);
    constexpr int MT = (T8 + 1) / 2;  // tiles of 16 tokens
    const bool first = (q >> 1) == h;  // the lane's quarter belongs to the first 8 tokens of a tile
    const XE* xh[T8];
#pragma unroll
    for (int m = 0; m < T8; ++m)
      xh[m] = static_cast<const XE*>(a.X) + static_cast<long>(min(8 * m + (l & 7), a.T - 1)) * a.d +
              32 * (h ^ (m & 1)) + 8 * q;
    f4v acc[4][MT];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[i][m] = f4v{0.f, 0.f, 0.f, 0.f};
    struct Slot {
      Raw<XT> x[T8];
      u4v w;
      u2v s;
    };
    const B ones = q4_ones<TY>();
    stream_units<MT == 1 ? 4 : 2, Slot>(
        u1 - u0,
        [&](int i, Slot& s) {
          const long u = u0 + i;
          s.w = *reinterpret_cast<const u4v*>(wp + u * 256);
          s.s = load_scales<4>(sp + u * 64);
#pragma unroll
          for (int m = 0; m < T8; ++m) s.x[m] = load_raw<XT>(xh[m] + u * 64);
        },
        [&](const Slot& s) {
          B x[T8];
          f4v off[T8];
#pragma unroll
          for (int m = 0; m < T8; ++m) {
            x[m] = raw_to_frag<XT, TY>(s.x[m]);
            const f4v sum = mfma16<TY>(x[m], ones, f4v{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int r = 0; r < 4; ++r) off[m][r] = -kQ4Offset * sum[r];
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t word = s.w[i];
            const B b = q4_frag_plain<TY>(word);
            const float sc = scale_at(s.s, i);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              f4v p = mfma16<TY>(x[2 * m], b, off[2 * m]);
              if constexpr (T8 > 1) {
                const f4v p1 = mfma16<TY>(x[2 * m + 1], b, off[2 * m + 1]);
#pragma unroll
                for (int r = 0; r < 4; ++r) p[r] = first ? p[r] : p1[r];
              }
#pragma unroll
              for (int r = 0; r < 4; ++r) acc[i][m][r] += sc * p[r];
            }
          }
        });
    // the other half's quarter sits at the other q / 2 and the other l / 8
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        f4v v;
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = acc[i][m][r] + __shfl_xor(acc[i][m][r], 40);
        if (q < 2)
          *reinterpret_cast<f4v*>(red + ((wave * 4 + i) * MT + m) * 128 + (16 * h + 8 * q + (l & 7)) * 4) = v;
      }
    __syncthreads();
    for (int v = tid; v < (real ? a.T * 32 : 0); v += UW * 64) {
      const int row = v >> 5, col = v & 31, r = row & 7;
      if (nb * 32 + col >= cols) continue;
      const int at =
          ((col & 3) * MT + (row >> 4)) * 128 + (2 * (row & 8) + 8 * (r >> 2) + (col >> 2)) * 4 + (r & 3);
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < UW; ++w) s += red[w * 4 * MT * 128 + at];
      a.U[(static_cast<long>(row) * a.G + g) * cols + nb * 32 + col] = s * Q4Type<TY>::undo;
    }
  } else {
    constexpr int es = TY == DT_F32 ? 4 : 2;
    // fragment 4 u + q of the block, lane half h, columns 16 c + l: depth 64 u + 32 h + 8 q ..
    constexpr int MT = (T8 + 1) / 2;  // tiles of 16 tokens
    const XE* xp[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
      xp[m] = static_cast<const XE*>(a.X) + static_cast<long>(min(16 * m + l, a.T - 1)) * a.d + 8 * q;
    const char* wp =
        static_cast<const char*>(a.At) + (g * a.at_gs + ((static_cast<long>(nb) * (a.d / 16) + q) * 64 + l) * 8) * es;
    f4v acc[2][MT];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[c][m] = f4v{0.f, 0.f, 0.f, 0.f};
    struct Slot {
      Raw<XT> x[2][MT];
      B w[2][2];
    };
    stream_units<TY == DT_F32 ? 1 : 2, Slot>(
        u1 - u0,
        [&](int i, Slot& s) {
          const long u = u0 + i;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int m = 0; m < MT; ++m) s.x[h][m] = load_raw<XT>(xp[m] + u * 64 + 32 * h);
#pragma unroll
            for (int c = 0; c < 2; ++c) s.w[h][c] = load_frag<TY>(wp + (u * 2048 + 256 * h + 128 * c) * es);
          }
        },
        [&](const Slot& s) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              const B x = raw_to_frag<XT, TY>(s.x[h][m]);
#pragma unroll
              for (int c = 0; c < 2; ++c) acc[c][m] = mfma16<TY>(x, s.w[h][c], acc[c][m]);
            }
        });
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int m = 0; m < MT; ++m)
        *reinterpret_cast<f4v*>(red + ((wave * 2 + c) * MT + m) * 256 + lane * 4) = acc[c][m];
    __syncthreads();
    for (int v = tid; v < (real ? a.T * 32 : 0); v += UW * 64) {
      const int row = v >> 5, col = v & 31;
      if (nb * 32 + col >= cols) continue;
      a.U[(static_cast<long>(row) * a.G + g) * cols + nb * 32 + col] = block_sum<UW, 2, MT>(red, row, col);
    }
  }
}

// LDS of the selecting workgroup.
struct SelectLds {
  int idx[FEW_MAX_T * MAX_SLOTS], gid[FEW_MAX_T * MAX_KG];
  float pg[FEW_MAX_T * MAX_KG];
  uint32_t mask[2][1024];  // tokens of each group and of each expert
  int pos[2][1024];        // non-empty bins before each; then entries before each
  int wsum[2][NW];
  int last;
};

// i / n for i n < 2^32, over = ceil(2^32 / n), or 0 for n = 1.
__device__ __forceinline__ int div_small(int i, uint32_t over) {
  return over ? static_cast<int>(__umulhi(static_cast<uint32_t>(i), over)) : i;
}

// Scores of tokens t0 .. t0 + nt - 1 into sc [nt][NC], biases included: the
// parts other workgroups stored, several elements' loads in flight at once.
__device__ __forceinline__ void gather_scores(const FewArgs& a, int t0, int nt, int NC, float* sc) {
  const long stride = static_cast<long>(a.T) * a.NCp;
  const int total = nt * NC;
#pragma unroll 1
  for (int e0 = threadIdx.x; e0 < total; e0 += 4 * NT) {
    float part[4][4], bias[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = min(e0 + j * NT, total - 1);
      const int tk = div_small(e, a.over_nc), c = e - tk * NC;
      const float* p = a.L + static_cast<long>(t0 + tk) * a.NCp + c;
#pragma unroll
      for (int s = 0; s < 4; ++s)
        part[j][s] = s < a.nsplit ? __hip_atomic_load(p + s * stride, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.f;
      bias[j] = a.bias[c];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (e0 + j * NT < total) sc[e0 + j * NT] = ((part[j][0] + part[j][1]) + (part[j][2] + part[j][3])) + bias[j];
  }
}

// Top-k of up to 16 candidates by each row of 16 lanes (four jobs a
// wavefront): the row's lane r ends up with selection r's exp(score - the
// first's) and index, every lane with the sum of the k, added in order.
__device__ __forceinline__ void row_topk(const float* sv, int n, int k, int lane, float& mye, int& myi, float& sum) {
  const int c = lane & 15, shift = lane & 16;
  float v = c < n ? sv[c] : -INFINITY;
  v = (v == v) ? v : -INFINITY;
  bool left = c < n;
  float top = 0.f;
  sum = 0.f;
  mye = 0.f;
  myi = -1;
  auto turn = [](float x, auto ctrl) {  // the larger of x and the row's x that many lanes on
    return fmaxf(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value, 0xf, 0xf,
                                                               false)));
  };
  using std::integral_constant;
#pragma unroll 1
  for (int r = 0; r < k; ++r) {
    float best = left ? v : -INFINITY;
    best = turn(best, integral_constant<int, 0x128>{});  // row_ror:8, 4, 2, 1
    best = turn(best, integral_constant<int, 0x124>{});
    best = turn(best, integral_constant<int, 0x122>{});
    best = turn(best, integral_constant<int, 0x121>{});
    const unsigned long long m = __ballot(left && v == best);
    const uint32_t mine = (lane < 32 ? static_cast<uint32_t>(m) : static_cast<uint32_t>(m >> 32)) >> shift;
    const int at = __ffs(static_cast<int>(mine & 0xFFFFu)) - 1;
    if (c == at) left = false;
    if (r == 0) top = best;
    const float e = expf(best - top);
    sum += e;
    if (c == r) {
      mye = e;
      myi = at;
    }
  }
}

// Selection for tokens t0 .. t0 + nt - 1 by one workgroup, a job per token for
// the groups and then per (token, chosen group) for the experts: larger score
// first, ties to the lower index; gates are the softmax over the chosen groups
// times the softmax over the chosen experts of each.  Up to 16 candidates are
// a row of lanes each: four wavefronts share the issue of a SIMD, so what
// counts is instructions (T = 32, 16 groups of 16: 9.1 us with a wavefront a
// job, 3.1 with a row).
__device__ __forceinline__ void select_tokens(const FewArgs& a, int t0, int nt, int NC, const float* sc, SelectLds& s) {
  const int wave = wave_id(), lane = threadIdx.x & 63;
#pragma unroll 1
  for (int level = 0; level < (a.K > 1 ? 2 : 1); ++level) {
    const int n = level ? a.K : a.G, k = level ? a.ke : a.kg, jobs = level ? nt * a.kg : nt;
    const int per = n <= 16 ? 4 : 1;  // jobs a wavefront takes at a time
#pragma unroll 1
    for (int i0 = wave * per; i0 < jobs; i0 += NW * per) {
      const int i = n <= 16 ? min(i0 + (lane >> 4), jobs - 1) : i0;
      const int r = n <= 16 ? lane & 15 : lane;  // the lane's selection
      const int tok = level ? div_small(i, a.over_kg) : i;
      const int tr = t0 * a.kg + i;  // level 1: token * kg + rank
      const float* from = sc + tok * NC + (level ? a.G + s.gid[tr] * a.K : 0);
      float e, sum = 0.f;
      int j;
      if (n <= 16) {
        row_topk(from, n, k, lane, e, j, sum);
        if (i0 + (lane >> 4) >= jobs) continue;
      } else {
        float v;
        wave_topk(from, n, k, lane, v, j);
        e = lane < k ? expf(v - lane_value(v, 0)) : 0.f;
#pragma unroll 1
        for (int x = 0; x < k; ++x) sum += lane_value(e, x);
      }
      const float p = e / sum;
      if (r >= k) continue;
      int at, id = j;
      float w = p;
      if (level) {
        at = tr * a.ke + r;  // (t * kg + rank) * ke + b
        id += s.gid[tr] * a.K;
        w *= s.pg[tr];
      } else {
        at = (t0 + i) * a.kg + r;
        s.gid[at] = j;
        s.pg[at] = p;
        a.gidx[at] = j;
      }
      if (level || a.K == 1) {
        s.idx[at] = id;
        a.idx[at] = id;
        a.w[at] = w;
      }
    }
    __syncthreads();
  }
}

// The tokens of each group and of each expert.
__device__ __forceinline__ void make_masks(const FewArgs& a, SelectLds& s) {
  const int tid = threadIdx.x;
  s.mask[0][tid] = 0;
  s.mask[1][tid] = 0;
  __syncthreads();
  if (tid < a.T * a.kg) atomicOr(&s.mask[0][s.gid[tid]], 1u << div_small(tid, a.over_kg));
  if (tid < a.T * a.k) atomicOr(&s.mask[1][s.idx[tid]], 1u << div_small(tid, a.over_k));
  __syncthreads();
}

// The caller's lists, from the masks: an entry's place in its bin's list is
// the entries of lower bins and those of lower tokens in its own.
__device__ __forceinline__ void caller_lists(const FewArgs& a, SelectLds& s) {
  const int tid = threadIdx.x, wave = wave_id(), lane = tid & 63;
  __syncthreads();  // pos is free
  int upto[2], total[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    upto[x] = __popc(s.mask[x][tid]);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int v = __shfl_up(upto[x], d);
      upto[x] += lane >= d ? v : 0;
    }
    if (lane == 63) s.wsum[x][wave] = upto[x];
  }
  __syncthreads();
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    int before = 0;
    total[x] = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const int c = s.wsum[x][w];
      before += w < wave ? c : 0;
      total[x] += c;
    }
    const int mine = __popc(s.mask[x][tid]), off = before + upto[x] - mine, bins = x ? a.E : a.G;
    s.pos[x][tid] = off;
    int* counts = x ? a.counts : a.gcounts;
    int* offsets = x ? a.offsets : a.goffsets;
    if (counts && tid < bins) counts[tid] = mine;
    if (offsets && tid < bins) offsets[tid] = off;
    if (offsets && tid == 0) offsets[bins] = total[x];
  }
  __syncthreads();
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    int* perm = x ? a.perm : a.gperm;
    if (!perm || tid >= a.T * (x ? a.k : a.kg)) continue;
    const int b = x ? s.idx[tid] : s.gid[tid], t = div_small(tid, x ? a.over_k : a.over_kg);
    perm[s.pos[x][b] + __popc(s.mask[x][b] & ((1u << t) - 1))] = t;
  }
}

// The touched groups and experts with their tokens.
// tab: room for (G + min(E, T*k)) * FEW_MAX_T int16.
__device__ __forceinline__ void make_lists(const FewArgs& a, SelectLds& s, int16_t* tab) {
  const int tid = threadIdx.x, wave = wave_id(), lane = tid & 63;
  const int ng = a.T * a.kg, na = a.T * a.k;
  const bool resid = a.resid != RS_NONE;
  if (a.T == 1) {
    // its groups and experts are distinct and in place already
    if (tid == 0) {
      a.glist[0] = ng;
      a.elist[0] = na;
    }
    if (tid < ng) {
      a.grec[tid] = int4{s.gid[tid], tid * a.ke, a.ke, 1};
      a.grow[tid * FEW_MAX_T] = static_cast<int16_t>(tid);
    }
    if (resid && tid < na) {
      a.elist[1 + tid] = s.idx[tid];
      a.eslot[tid * FEW_MAX_T] = static_cast<int16_t>(tid);
    }
    return;
  }
  // groups and experts side by side: non-empty bins before each
  const unsigned long long m0 = __ballot(s.mask[0][tid] != 0), m1 = __ballot(s.mask[1][tid] != 0);
  if (lane == 0) {
    s.wsum[0][wave] = __popcll(m0);
    s.wsum[1][wave] = __popcll(m1);
  }
  __syncthreads();
  int before0 = 0, before1 = 0, tg = 0, te = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const int c0 = s.wsum[0][w], c1 = s.wsum[1][w];
    before0 += w < wave ? c0 : 0;
    before1 += w < wave ? c1 : 0;
    tg += c0;
    te += c1;
  }
  if (!resid) te = 0;
  s.pos[0][tid] = before0 + __popcll(m0 & ((1ull << lane) - 1));
  s.pos[1][tid] = before1 + __popcll(m1 & ((1ull << lane) - 1));
  if (tid == 0) {
    a.glist[0] = tg;
    a.elist[0] = te;
  }
  // tables of the tokens in each, empty at first
  int16_t* etab = tab + a.G * FEW_MAX_T;
  for (int i = tid; i < tg * (FEW_MAX_T / 2); i += NT) reinterpret_cast<int*>(tab)[i] = -1;
  for (int i = tid; i < te * (FEW_MAX_T / 2); i += NT) reinterpret_cast<int*>(etab)[i] = -1;
  __syncthreads();
  if (tid < ng) tab[s.pos[0][s.gid[tid]] * FEW_MAX_T + div_small(tid, a.over_kg)] = static_cast<int16_t>(tid);
  if (resid && tid < na)
    etab[s.pos[1][s.idx[tid]] * FEW_MAX_T + div_small(tid, a.over_k)] = static_cast<int16_t>(tid);
  __syncthreads();
  for (int i = tid; i < tg * (FEW_MAX_T / 2); i += NT)
    reinterpret_cast<int*>(a.grow)[i] = reinterpret_cast<const int*>(tab)[i];
  for (int i = tid; i < te * (FEW_MAX_T / 2); i += NT)
    reinterpret_cast<int*>(a.eslot)[i] = reinterpret_cast<const int*>(etab)[i];
  if (resid && s.mask[1][tid]) a.elist[1 + s.pos[1][tid]] = tid;
  if (tid < a.G && s.mask[0][tid]) {
    // an expert past the last has all touched ones before it
    const int first = resid ? s.pos[1][tid * a.K] : 0;
    const int end = !resid ? 0 : (tid + 1) * a.K < 1024 ? s.pos[1][(tid + 1) * a.K] : te;
    a.grec[s.pos[0][tid]] = int4{tid, first, end - first, __popc(s.mask[0][tid])};
  }
}

// Tokens whose scores the selection holds in LDS at a time.
__host__ __device__ inline int select_chunk(int T, int NC) {
  const int n = 64 * 1024 / (4 * NC);
  return n < T ? n : T;
}

// grid: the score blocks (16 columns x nsplit depth parts) first, then with
// u_all one workgroup per two blocks of 32 factor columns of every group.
//
// Bound by the chain of its latencies: scores (3 us at T = 1, 6 at 32, where
// the 32 rows' loads and fp32 MFMAs count), their way through memory and the
// ticket (1.5), reading them back (1.2 to 3.8), the selection (2 to 3), the
// lists (0.4 at T = 1, else 1.6).  d = 4096, 16 groups of 16 experts, 4-bit
// factors: 9.6 us at T = 1 with 19 MB read, 15.0 at T = 16, 23 at T = 32,
// where the factors' products are the longer side (they decode 256 experts
// for all rows: 21.8 us by themselves).
template <int XT, int TY, int RS, int T8>
__global__ __launch_bounds__(NT) void few_route_kernel(FewArgs a) {
  constexpr int MT = (T8 + 1) / 2;
  extern __shared__ __attribute__((aligned(16))) float red[];  // partial tiles, then scores; last the lists' tables
  __shared__ SelectLds s;
  const int NC = a.G + (a.K > 1 ? a.G * a.K : 0);
  const int ncb = (NC + 15) / 16, nsb = ncb * a.nsplit;
  if (static_cast<int>(blockIdx.x) >= nsb) {
    if constexpr (RS != RS_NONE) {
      const int nbu = (a.K * a.Pin * 16 + 31) / 32, half = wave_id() / UW;
      const int ub = 2 * (blockIdx.x - nsb) + half;
      u_block<XT, TY, RS == RS_INT4, T8>(a, ub / nbu, ub % nbu, ub < a.G * nbu, red + half * UW * 2 * MT * 256);
    }
    return;
  }
  float* sc = red + NW * MT * 256;
  const int cb = blockIdx.x % ncb, split = blockIdx.x / ncb;
  score_block<XT, MT>(a, cb, split, red);
  __syncthreads();
  const bool alone = nsb == 1;  // up to 16 columns in all: this workgroup holds every score
  // Otherwise scores go to memory past the caches (agent scope), each wavefront
  // waits for its own stores, and the workgroup that counts itself in last
  // selects; nobody waits for another.  The scores are read back past the
  // caches too, so no cache needs writing back or dropping: a release fence
  // here, which writes back the whole second-level cache, took 13 us of a
  // 256-expert layer's launch.
  for (int v = threadIdx.x; v < a.T * 16; v += NT) {
    const int row = v >> 4, col = v & 15;
    const float sum = block_sum<NW, 1, MT>(red, row, col);
    if (!alone)
      __hip_atomic_store(a.L + (static_cast<long>(split) * a.T + row) * a.NCp + cb * 16 + col, sum, __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
    else if (col < NC)
      sc[row * NC + col] = sum + a.bias[col];
  }
  if (!alone) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    // the ticket wraps to zero with the last one, ready for the next pass
    if (threadIdx.x == 0)
      s.last = atomicInc(reinterpret_cast<unsigned*>(a.ticket), nsb - 1) == static_cast<unsigned>(nsb - 1) ? 1 : 0;
    __syncthreads();
    if (!s.last) return;
    asm volatile("" ::: "memory");
  }
  const int chunk = alone ? a.T : select_chunk(a.T, NC);
#pragma unroll 1
  for (int t0 = 0; t0 < a.T; t0 += chunk) {
    const int nt = min(chunk, a.T - t0);
    if (!alone) gather_scores(a, t0, nt, NC, sc);
    __syncthreads();
    select_tokens(a, t0, nt, NC, sc, s);
  }
  if (a.T > 1 || a.wants_lists) make_masks(a, s);
  make_lists(a, s, reinterpret_cast<int16_t*>(red));
  if (a.wants_lists) caller_lists(a, s);
}

// U of the chosen experts only: one workgroup per two blocks of 32 factor
// columns, idle where none of the columns' experts is chosen.
template <int XT, int TY, int RS, int T8>
__global__ __launch_bounds__(NT) void few_u_kernel(FewArgs a) {
  constexpr int MT = (T8 + 1) / 2;
  extern __shared__ __attribute__((aligned(16))) float red[];
  __shared__ int hit[2];
  const int nbu = (a.K * a.Pin * 16 + 31) / 32, half = wave_id() / UW, tid = threadIdx.x % (UW * 64);
  const int ub = 2 * blockIdx.x + half, g = ub / nbu, nb = ub % nbu;
  const int per = 2 / a.Pin;  // experts per block
  if (tid == 0) hit[half] = 0;
  __syncthreads();
  if (ub < a.G * nbu && tid < a.T * a.k) {  // at most 512 slots
    const int e = a.idx[tid] - (g * a.K + nb * per);
    if (e >= 0 && e < per) hit[half] = 1;
  }
  __syncthreads();
  if (!hit[0] && !hit[1]) return;
  u_block<XT, TY, RS == RS_INT4, T8>(a, g, nb, hit[half] != 0, red + half * UW * 2 * MT * 256);
}

// ------------------------------------------------------------------- up --
// grid: (touched group a) x (blocks of FT = 32 / Pin columns of f).  A
// workgroup's 32 weight columns are 16 of the gate and the same 16 of the up
// projection (SwiGLU), or 32 of the one input projection (GELU).
//
// Bound by the weights' bytes where they are many (d = 4096, f = 14336, bf16,
// T = 2: 123 us a launch, about 6 TB/s), by the ramp of one round of workgroups
// where they are few (50 MB, T = 1: 14.1 us, 3.6 TB/s; 4-bit, 14 MB: 8.4 us,
// 1.7 TB/s), and beyond 16 tokens by the experts' jobs behind the stream
// (fine-grained 4-bit layer, T = 32: 16.6 us, of which the stream is 11).
template <int XT, int TY, bool Q4, int RS, int MT, int NWV>
__global__ __launch_bounds__(NWV * 64) void few_up_kernel(FewArgs a) {
  using XE = typename Elem<XT>::T;
  using B = typename Frag<TY>::T;
  constexpr int HT = hidden_type(TY, Q4);
  extern __shared__ __attribute__((aligned(16))) float red[];  // partial tiles, then the weighted h
  __shared__ __attribute__((aligned(16))) float z[2][MT * 16][20];  // 20: rows 16 bytes apart mod 128
  __shared__ int srow[FEW_MAX_T];   // rows t*kg + rank of the group's tokens
  const int Pin = a.Pin, FT = 32 / Pin, nfb = a.f / FT;
  const int ga = blockIdx.x / nfb, fb = blockIdx.x % nfb;
  if (ga >= a.glist[0]) return;
  const int4 rec = a.grec[ga];
  const int g = rec.x, first = rec.y, ne = rec.z, n = rec.w;
  const int wave = wave_id(), lane = threadIdx.x & 63, l = lane & 15, q = lane >> 4;
  const int f0 = fb * FT;
  // the group's tokens (bit t), their rows; the i-th of them is row i of the
  // MFMA tiles, and rows past the last repeat it, which costs no further cache
  // lines: a compute unit takes 2.5 cycles for each, and rows of all tokens are
  // 16 an instruction (T = 32: 119 us a pass with them, 107 without; T = 16,
  // fp16 base, 86.3 / 83.9)
  const int grow = lane < a.T ? a.grow[ga * FEW_MAX_T + lane] : -1;
  const uint32_t members = static_cast<uint32_t>(__ballot(grow >= 0));
  const int place = __popc(members & ((1u << (lane & 31)) - 1));
  if (wave == 0 && grow >= 0) srow[place] = grow;
  const int member = __builtin_amdgcn_ds_permute(4 * (grow >= 0 ? place : 63), lane);  // lane i: the i-th
  // The wavefront's jobs: a touched expert and up to 16 of its tokens, expert
  // first + wave, + NWV, ...  (beyond 16 tokens in the batch the expert's own
  // are drawn together first, and where the group has more than 16 the second
  // jobs of all its experts follow the first ones).  Their operands are few but
  // cold, and behind a stream that fills the memory's queues a load takes
  // microseconds: the first job's are read with the first weights, the next
  // one's while a job runs.
  struct Job {
    int e, slot;
    float wgt;
    u4v b[2][TY == DT_F32 ? 2 : 1], s[2], ad[2];  // 4-bit: words in elements 0
    u2v as;
  } job;
  int je = 0, jslot = -1;  // expert, and the slot of the lane's token
  auto job_find = [&](int j) {
    const int i = first + (MT == 2 && j >= ne ? j - ne : j);
    je = a.elist[1 + i];
    if constexpr (MT == 1) {
      jslot = l < a.T ? a.eslot[i * FEW_MAX_T + l] : -1;
    } else {
      const int slot = lane < a.T ? a.eslot[i * FEW_MAX_T + lane] : -1;
      const uint32_t m = static_cast<uint32_t>(__ballot(slot >= 0));
      // the p-th of the expert's tokens to lane p (lanes without one to lane 63)
      const int to = slot >= 0 ? __popc(m & ((1u << lane) - 1)) : 63;
      const int packed = __builtin_amdgcn_ds_permute(4 * to, slot);
      const int from = (j >= ne ? 16 : 0) + l;
      const int mine = __shfl(packed, from);
      jslot = from < __popc(m) ? mine : -1;
    }
  };
  auto job_load = [&](Job& J) {
    J.slot = jslot;
    J.e = je;
    if (MT > 1 && !__any(jslot >= 0)) return;
    J.wgt = a.w[max(jslot, 0)];
    constexpr int es = TY == DT_F32 ? 4 : 2;
    constexpr bool int4r = RS == RS_INT4;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int p = Pin == 2 ? x : 0, col0 = Pin == 2 ? f0 : f0 + 16 * x;  // 16 columns of projection p
      const long blk = static_cast<long>(je * Pin + p) * (a.f / 32) + (col0 >> 5);
      const long at = blk * 64 + 32 * (q & 1) + (col0 & 16) + l;
      if constexpr (int4r) {
        J.b[x][0][0] = static_cast<const uint32_t*>(a.B1)[at];
        J.s[x] = *reinterpret_cast<const u4v*>(a.B1_s + blk * RPAD + 8 * (q & 1));
      } else {
        const u4v* bp = reinterpret_cast<const u4v*>(static_cast<const char*>(a.B1) + at * 8 * es);
        J.b[x][0] = bp[0];
        if constexpr (TY == DT_F32) J.b[x][1] = bp[1];
      }
      const int c0 = Pin == 2 ? f0 : col0;
      const long ad = ((static_cast<long>(je) * (a.f / 32) + (c0 >> 5)) * 2 + ((c0 >> 4) & 1)) * 64 + l + 32 * (q & 1);
      if (Pin == 1 || x == 0) J.ad[x] = load_down_factor<TY, RS>(a.Ad, ad, q >> 1);
    }
    if constexpr (int4r)
      J.as = *reinterpret_cast<const u2v*>(a.Ad_s + (static_cast<long>(je) * (a.f / 32) + (f0 >> 5)) * RPAD + 4 * q);
  };
  const int jobs = RS != RS_NONE ? (MT == 2 && n > 16 ? 2 * ne : ne) : 0;
  if constexpr (RS != RS_NONE)
    if (wave < jobs) job_find(wave);
  auto between = [&]() {
    if constexpr (RS != RS_NONE)
      if (wave < jobs) job_load(job);
  };
  const int n64 = a.d / 64;
  const int u0 = n64 * wave / NWV, u1 = n64 * (wave + 1) / NWV;
  const XE* xp[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
    xp[m] = static_cast<const XE*>(a.X) + static_cast<long>(__shfl(member, min(16 * m + l, n - 1))) * a.d + 8 * q;
  f4v acc[2][MT];
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[c][m] = f4v{0.f, 0.f, 0.f, 0.f};
  // M tiles of rows
  auto stream = [&](auto tiles) {
    constexpr int M = decltype(tiles)::value;
    if constexpr (Q4) {
      const uint32_t* wp =
          static_cast<const uint32_t*>(a.W1) + g * a.w1_gs + (static_cast<long>(fb) * a.w1_units * 64 + lane) * 4;
      const uint16_t* sp = a.W1_s + g * a.w1_sgs + (static_cast<long>(fb) * a.w1_units * 16 + l) * 4;
      struct Slot {
        Raw<XT> x[2][M];
        u4v w;
        u2v s;
      };
      const B ones = q4_ones<TY>();
      stream_units<M == 1 ? 4 : 2, Slot>(
          u1 - u0,
          [&](int i, Slot& s) {
            const long u = u0 + i;
            s.w = *reinterpret_cast<const u4v*>(wp + u * 256);
            s.s = load_scales<4>(sp + u * 64);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int m = 0; m < M; ++m) s.x[h][m] = load_raw<XT>(xp[m] + u * 64 + 32 * h);
          },
          [&](const Slot& s) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              f4v off[M];
              B x[M];
#pragma unroll
              for (int m = 0; m < M; ++m) {
                x[m] = raw_to_frag<XT, TY>(s.x[h][m]);
                const f4v sum = mfma16<TY>(x[m], ones, f4v{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                for (int i = 0; i < 4; ++i) off[m][i] = -kQ4Offset * sum[i];
              }
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const uint32_t word = s.w[2 * h + c];
                const B b = q4_frag<TY>(word);
                const float sc = scale_at(s.s, 2 * h + c);
#pragma unroll
                for (int m = 0; m < M; ++m) {
                  const f4v p = mfma16<TY>(x[m], b, off[m]);
#pragma unroll
                  for (int i = 0; i < 4; ++i) acc[c][m][i] += sc * p[i];
                }
              }
            }
          },
          between);
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[c][m][i] *= Q4Type<TY>::undo;
    } else {
      constexpr int es = TY == DT_F32 ? 4 : 2;
      const char* wp[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int n32 = Pin == 2 ? (fb & ~1) + c : fb, half = Pin == 2 ? fb & 1 : c;
        wp[c] = static_cast<const char*>(a.W1) +
                (g * a.w1_gs + ((static_cast<long>(n32) * (a.d / 16) + q) * 64 + 16 * half + l) * 8) * es;
      }
      struct Slot {
        Raw<XT> x[2][M];
        B w[2][2];
      };
      stream_units<TY == DT_F32 ? 1 : M == 1 ? 3 : 2, Slot>(
          u1 - u0,
          [&](int i, Slot& s) {
            const long u = u0 + i;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int c = 0; c < 2; ++c) s.w[h][c] = load_frag<TY>(wp[c] + (u * 2048 + 256 * h) * es);
#pragma unroll
              for (int m = 0; m < M; ++m) s.x[h][m] = load_raw<XT>(xp[m] + u * 64 + 32 * h);
            }
          },
          [&](const Slot& s) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int m = 0; m < M; ++m) {
                const B x = raw_to_frag<XT, TY>(s.x[h][m]);
#pragma unroll
                for (int c = 0; c < 2; ++c) acc[c][m] = mfma16<TY>(x, s.w[h][c], acc[c][m]);
              }
          },
          between);
    }
  };
  if constexpr (MT == 2) {
    if (n > 16) stream(std::integral_constant<int, 2>{});
    else stream(std::integral_constant<int, 1>{});
  } else {
    stream(std::integral_constant<int, 1>{});
  }
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int m = 0; m < MT; ++m)
      *reinterpret_cast<f4v*>(red + ((wave * 2 + c) * MT + m) * 256 + lane * 4) = acc[c][m];
  __syncthreads();
  for (int v = threadIdx.x; v < n * 32; v += NWV * 64) {
    const int row = v >> 5, col = v & 31;
    z[col >> 4][row][col & 15] = block_sum<NWV, 2, MT>(red, row, col);
  }
  __syncthreads();  // the partial tiles are read: red is free again
  constexpr int planes = hidden_planes(XT, HT);
  auto store_hidden = [&](int row, int c, float s) {
    const long at = static_cast<long>(row) * planes * a.f + f0 + c;
    if constexpr (HT == DT_F32) {
      static_cast<float*>(a.H)[at] = s;
    } else {
      const uint16_t hi = from_f32<HT>(s);
      static_cast<uint16_t*>(a.H)[at] = hi;
      if constexpr (planes == 2) {
        const float back = HT == DT_F16 ? f16_bits_to_f32(hi) : bf16_bits_to_f32(hi);
        static_cast<uint16_t*>(a.H)[at + a.f] = from_f32<HT>(s - back);
      }
    }
  };
  if constexpr (RS == RS_NONE) {
    // the group's experts are its base: one activation, their gates summed
    for (int v = threadIdx.x; v < n * FT; v += NWV * 64) {
      const int c = v % FT, i = v / FT;
      const int row = srow[i];
      float wgt = 0.f;
      for (int b = 0; b < a.ke; ++b) wgt += a.w[row * a.ke + b];
      const float h = a.act == ACT_SWIGLU ? silu_f(z[0][i][c]) * z[1][i][c] : gelu_tanh_f(z[c >> 4][i][c & 15]);
      store_hidden(row, c, wgt * h);
    }
  } else {
    // Everything transposed: MFMA rows are the 16 columns of f, MFMA columns the
    // job's tokens.  z + B u: depth 32 = the 16 rank columns twice, against the
    // two 16-bit parts of u (4-bit B: codes, the scales in u).  The result's
    // lane holds 4 columns of f of its token, which is the operand form of
    // 16x16x16 MFMAs, so h goes into V = A_down^T h (16 rank columns by tokens)
    // from the registers, again in two parts.  The weighted h go to LDS, one
    // row per (token, expert), to be summed per token.
    float* hw = red;  // [tokens of the group][ke][FT]
    for (int j = wave; j < jobs; j += NWV) {
      const Job J = job;
      const bool on = J.slot >= 0;
      const int t = on ? div_small(J.slot, a.over_k) : 0, i = __popc(members & ((1u << t) - 1));
      // u, then the next job's operands behind it
      float u[2][8];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float* up =
            a.U + (static_cast<long>(t) * a.E + J.e) * Pin * 16 + (Pin == 2 ? x : 0) * 16 + 8 * (q & 1);
        const f4v u0 = *reinterpret_cast<const f4v*>(up), u1 = *reinterpret_cast<const f4v*>(up + 4);
#pragma unroll
        for (int r = 0; r < 8; ++r) u[x][r] = r < 4 ? u0[r] : u1[r - 4];
      }
      if (j + NWV < jobs) {
        job_find(j + NWV);
        job_load(job);
      }
      if (!__any(on)) continue;
      const int part = q >> 1;
      float hv[2][4];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        B bw;
        if constexpr (TY == DT_F32) {
          Raw<DT_F32> r;
          r.v[0] = J.b[x][0];
          r.v[1] = J.b[x][1];
          bw = raw_to_frag<DT_F32, DT_F32>(r);
        } else if constexpr (RS == RS_INT4) {
          const uint32_t word = J.b[x][0][0];
          bw = int4_frag_1scale<TY>(word, 0x3C00);  // the codes themselves
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            const uint32_t w = J.s[x][r >> 1];
            u[x][r] *= f16_bits_to_f32(static_cast<uint16_t>((w >> (16 * (r & 1))) & 0xFFFFu));
          }
        } else {
          bw = __builtin_bit_cast(B, J.b[x][0]);
        }
        B bu = round_frag<TY>(u[x]);
        if constexpr (TY == DT_F32) {
          if (part) bu = zero_frag<TY>();
        } else {
          float rest[8];
#pragma unroll
          for (int r = 0; r < 8; ++r) rest[r] = u[x][r] - static_cast<float>(bu[r]);
          const u4v hi = __builtin_bit_cast(u4v, bu), lo = __builtin_bit_cast(u4v, round_frag<TY>(rest));
          bu = __builtin_bit_cast(B, part ? lo : hi);
        }
        const f4v zz = mfma16<TY>(bw, bu, *reinterpret_cast<const f4v*>(&z[x][i][4 * q]));
#pragma unroll
        for (int r = 0; r < 4; ++r) hv[x][r] = zz[r];
      }
      // a token without the expert keeps nothing of what its lane computed
      f4v v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (Pin == 2 && x == 1) break;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float h = Pin == 2 ? silu_f(hv[0][r]) * hv[1][r] : gelu_tanh_f(hv[x][r]);
          hv[x][r] = on ? J.wgt * h : 0.f;
        }
        if (on) {
          const int row = div_small(J.slot, a.over_ke);
          const int at = i * a.ke + (J.slot - row * a.ke);
          *reinterpret_cast<f4v*>(hw + at * FT + 16 * x + 4 * q) = f4v{hv[x][0], hv[x][1], hv[x][2], hv[x][3]};
        }
        v = down_factor<TY, RS>(J.ad[x], hv[x], v);
      }
      if constexpr (RS == RS_INT4) {
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] *= scale_at(J.as, r);
      }
      if (on) *reinterpret_cast<f4v*>(a.Vp + (static_cast<long>(fb) * a.T * a.k + J.slot) * 16 + 4 * q) = v;
    }
    __syncthreads();
    for (int v = threadIdx.x; v < n * FT; v += NWV * 64) {
      const int c = v % FT, i = v / FT, row = srow[i];
      float s = 0.f;
      for (int b = 0; b < a.ke; ++b) s += hw[(i * a.ke + b) * FT + c];
      store_hidden(row, c, s);
    }
  }
}

// ---------------------------------------------------------------- v sum --
// V = the partials of h A_down summed over the blocks of f: 64 sums per
// workgroup, their partials dealt to 16 wavefronts.  Latency: 4.7 us for 0.8 MB
// (T = 16, 8 experts a token, 96 blocks).
__global__ __launch_bounds__(NT) void few_vsum_kernel(FewArgs a) {
  __shared__ float part[NW][64];
  const int nv = a.T * a.k * 16, nfb = a.f * a.Pin / 32;
  const int wave = wave_id(), lane = threadIdx.x & 63, o = blockIdx.x * 64 + lane;
  float s = 0.f;
  if (o < nv) {
#pragma unroll 8
    for (int b = wave; b < nfb; b += NW) s += a.Vp[static_cast<long>(b) * nv + o];
  }
  part[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && o < nv) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += part[w][lane];
    a.V[o] = v;
  }
}

// ----------------------------------------------------------------- down --
// grid: one workgroup per 16 columns of y.  Its wavefronts take consecutive
// ranges of the touched groups' depths, laid end to end.  One tile of MFMA
// rows: 16 tokens, or 8 where the hidden sums have two parts, which are rows
// of their own (parts in rows 0-7 and 8-15).
//   MT = 1: the batch fits the tile.  Row r is token r in every group, a
// token without the group reads a row of zeros, and the sum over groups is
// the accumulator's own.
//   MT > 1: a group's tokens are gathered into pieces of a tile's rows, most
// often one, and a wavefront adds its sums to its own [T][16] block of LDS
// where a piece ends.  Measured (us a pass, tiles of all tokens in every
// group / pieces; d = 4096, f = 1536, 16 groups): T = 32 fp16 base 134 / 126,
// 4-bit base 107 / 92, T = 9 fp16 70.1 / 71.2.
//
// Bound by the weights' bytes like the up product (d = 4096, f = 14336, bf16,
// T = 2: 60 us a launch, about 6 TB/s; 25 MB, T = 1: 8.8 us, 2.9 TB/s), in
// 4 bits and beyond 8 tokens by the hidden sums' loads, one line a row.
//
// The residual tail V B_down is more depth of the same product: two touched
// experts' 16 rank columns are one 32-deep step, whose rows are the V of the
// tokens that chose the expert (zero for the others).  A 4-bit factor's scale
// varies along the rank columns, i.e. along the depth, so it multiplies V,
// which then splits into two 16-bit parts like the hidden sums.
__host__ __device__ inline int few_groups(const FewArgs& a) { return a.G < a.T * a.kg ? a.G : a.T * a.kg; }

constexpr int kDownPartials = 16;  // partials of V a thread reads at a time
constexpr int kDownBatches = 3;

template <int XT, int TY, bool Q4, int RS, int MT>
__global__ __launch_bounds__(NT) void few_down_kernel(FewArgs a) {
  using B = typename Frag<TY>::T;
  // [NW][256] or [NW][T][16], V and a zero row, partials of V, grow, the pieces and their number
  extern __shared__ __attribute__((aligned(16))) float red[];
  const int n = blockIdx.x, nv = RS != RS_NONE ? a.T * a.k * 16 : 0;
  constexpr bool pieces = MT > 1;
  constexpr int planes = hidden_planes(XT, TY);
  constexpr int ROWS = 16 / planes;  // tokens of a tile
  const int block = pieces ? a.T * 16 : 256;
  float* V = red + NW * block;
  float* vpart = V + nv + 16;
  int16_t* grow = reinterpret_cast<int16_t*>(vpart + (nv && !a.v_sum ? NT : 0));
  const int ng = a.glist[0];
  const int tid = threadIdx.x, wave = wave_id(), lane = tid & 63, l = lane & 15, q = lane >> 4;
  float* own = red + wave * block;
  int* piece = reinterpret_cast<int*>(grow + few_groups(a) * FEW_MAX_T);  // (first token << 16) | group ordinal
  int np = ng;
  if constexpr (pieces) {
    // a group's rows, absent ones behind them
    for (int i = wave; i < ng; i += NW) {
      const int row = lane < a.T ? a.grow[i * FEW_MAX_T + lane] : -1;
      const unsigned long long m = __ballot(row >= 0), below = (1ull << lane) - 1;
      const int at = row >= 0 ? __popcll(m & below) : __popcll(m) + __popcll(~m & below);
      if (at < FEW_MAX_T) grow[i * FEW_MAX_T + at] = static_cast<int16_t>(row);
    }
    if (wave == NW - 1) {
      int before = 0;
      for (int i0 = 0; i0 < ng; i0 += 64) {
        const int i = i0 + lane, count = i < ng ? (a.grec[i].w + ROWS - 1) / ROWS : 0;
        int upto = count;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
          const int v = __shfl_up(upto, d);
          upto += lane >= d ? v : 0;
        }
        for (int p = 0; p < count; ++p) piece[1 + before + upto - count + p] = (p * ROWS << 16) | i;
        before += __shfl(upto, 63);
      }
      if (lane == 0) piece[0] = before;
    }
    for (int i = lane; i < block; i += 64) own[i] = 0.f;
    __syncthreads();
    np = __builtin_amdgcn_readfirstlane(piece[0]);
  } else {
    for (int i = tid; i < ng * (FEW_MAX_T / 2); i += NT)
      reinterpret_cast<int*>(grow)[i] = reinterpret_cast<const int*>(a.grow)[i];
    __syncthreads();
  }
  constexpr int UNIT = Q4 ? 128 : 64, NS = UNIT / 32;
  constexpr bool packed = planes == 2 && MT == 1;
  constexpr int TM = planes == 1 ? MT : MT > 1 ? MT / 2 : 1;  // tiles of tokens
  const int nf = (a.f + UNIT - 1) / UNIT;
  const int units = np * nf;
  const int u0 = static_cast<int>(static_cast<long>(units) * wave / NW);
  const int u1 = static_cast<int>(static_cast<long>(units) * (wave + 1) / NW);
  f4v acc = {0.f, 0.f, 0.f, 0.f};
  // the stream's place: piece (a group where the batch fits the tile), unit inside it, the lane's row
  int at_i = 0, pi = u0 / nf, kb = u0 - pi * nf;
  using HE = typename Elem<TY>::T;
  const HE* hp = nullptr;
  const char* wp = nullptr;
  const uint16_t* sp = nullptr;
  constexpr int es = TY == DT_F32 ? 4 : 2;
  auto enter = [&]() {
    int ga = pi, row;
    const int r = l & (ROWS - 1), plane = l / ROWS;
    if constexpr (pieces) {
      const int p = __builtin_amdgcn_readfirstlane(piece[1 + pi]);
      ga = p & 0xFFFF;
      row = grow[ga * FEW_MAX_T + (p >> 16) + r];
    } else {
      row = r < a.T ? grow[ga * FEW_MAX_T + r] : -1;
    }
    const int g = a.grec[ga].x;
    // a token that did not choose the group, a row past a piece's last: zeros
    hp = static_cast<const HE*>(a.H) + (static_cast<long>(row < 0 ? a.zero_row : row) * planes + plane) * a.f;
    if constexpr (Q4) {
      wp = reinterpret_cast<const char*>(static_cast<const uint32_t*>(a.W2) + g * a.w2_gs +
                                         (static_cast<long>(n) * nf * 64 + lane) * 4);
      sp = a.W2_s + g * a.w2_sgs + (static_cast<long>(n) * nf * 16 + l) * 4;
    } else {
      wp = static_cast<const char*>(a.W2) +
           (g * a.w2_gs + ((static_cast<long>(n >> 1) * (a.f / 16) + q) * 64 + 16 * (n & 1) + l) * 8) * es;
    }
  };
  if (u0 < u1) enter();
  auto seek = [&](int i) {  // i is at_i or at_i + 1
    if (i == at_i) return;
    at_i = i;
    if (++kb == nf) {
      kb = 0;
      ++pi;
      enter();
    }
  };
  // a piece's sums to its tokens' rows of the wavefront's block; cur: piece of the sums
  int cur = pi;
  auto leave = [&]() {
    const int p = __builtin_amdgcn_readfirstlane(piece[1 + cur]);
    const int16_t* rows = grow + (p & 0xFFFF) * FEW_MAX_T + (p >> 16);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      float s = Q4 ? acc[v] * Q4Type<TY == DT_F32 ? DT_F16 : TY>::undo : acc[v];
      if constexpr (planes == 2) s += __shfl_xor(s, 32);
      const int row = rows[(4 * q + v) & (ROWS - 1)];
      if (4 * q + v < ROWS && row >= 0) own[div_small(row, a.over_kg) * 16 + l] += s;
      acc[v] = 0.f;
    }
    __builtin_amdgcn_wave_barrier();  // the next piece's lanes read what these wrote
  };
  auto follow = [&](int at) {
    if constexpr (pieces) {
      if (at != cur) {
        leave();
        cur = at;
      }
    }
  };
  // the residual tail: steps of two touched experts, dealt to the wavefronts;
  // a wavefront's first step is read with its first weights
  const int te = nv ? a.elist[0] : 0, steps = (te + 1) / 2;
  struct Tail {
    u4v w[TY == DT_F32 ? 2 : 1], s;
    int slot[TM];
  } tail;
  int te_id = 0, te_slot[TM];
  auto tail_find = [&](int i) {
    const int ei = 2 * i + (q >> 1);
    te_id = a.elist[1 + min(ei, te - 1)];
#pragma unroll
    for (int m = 0; m < TM; ++m) {
      const int t = packed ? (l & 7) : 16 * m + l;
      const int slot = t < a.T && ei < te ? a.eslot[ei * FEW_MAX_T + t] : -1;
      te_slot[m] = slot < 0 ? a.T * a.k : slot;  // the row of zeros
    }
  };
  auto tail_load = [&](Tail& T) {
    const int e = te_id, g = e / a.K, j = e - g * a.K, n32 = n >> 1, hh = q & 1;
    // rank column 8 hh .. of expert j in the permuted depth order
    const int ks = 4 * (j >> 2) + 2 * (j & 1) + hh;
    const long at = (static_cast<long>(n32) * (a.NV / 16) + ks) * 64 + 16 * (n & 1) + l + 32 * ((j >> 1) & 1);
    if constexpr (RS == RS_INT4) {
      T.w[0][0] = static_cast<const uint32_t*>(a.Bd)[g * a.bd_gs + at];
      T.s = *reinterpret_cast<const u4v*>(a.Bd_s + (static_cast<long>(e) * (a.d / 32) + n32) * RPAD + 8 * hh);
    } else {
      const u4v* p = reinterpret_cast<const u4v*>(static_cast<const char*>(a.Bd) + (g * a.bd_gs + at * 8) * es);
      T.w[0] = p[0];
      if constexpr (TY == DT_F32) T.w[1] = p[1];
    }
#pragma unroll
    for (int m = 0; m < TM; ++m) T.slot[m] = te_slot[m];
  };
  if constexpr (RS != RS_NONE)
    if (wave < steps) tail_find(wave);
  f4v tacc[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) tacc[m] = f4v{0.f, 0.f, 0.f, 0.f};
  auto tail_use = [&](const Tail& tail) {
    B b;
    if constexpr (TY == DT_F32) {
      Raw<DT_F32> r;
      r.v[0] = tail.w[0];
      r.v[1] = tail.w[1];
      b = raw_to_frag<DT_F32, DT_F32>(r);
    } else if constexpr (RS == RS_INT4) {
      const uint32_t word = tail.w[0][0];
      b = int4_frag_1scale<TY>(word, 0x3C00);  // the codes themselves
    } else {
      b = __builtin_bit_cast(B, tail.w[0]);
    }
#pragma unroll
    for (int m = 0; m < TM; ++m) {
      const float* vp = V + tail.slot[m] * 16 + 8 * (q & 1);
      float v[8], rest[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        v[r] = vp[r];
        if constexpr (RS == RS_INT4) {
          const uint32_t w = tail.s[r >> 1];
          v[r] *= f16_bits_to_f32(static_cast<uint16_t>((w >> (16 * (r & 1))) & 0xFFFFu));
        }
      }
      const B hi = round_frag<TY>(v);
      if constexpr (planes == 1) {
        tacc[m] = mfma16<TY>(hi, b, tacc[m]);
      } else {
#pragma unroll
        for (int r = 0; r < 8; ++r) rest[r] = v[r] - static_cast<float>(hi[r]);
        const B lo = round_frag<TY>(rest);
        if constexpr (packed) {
          const u4v x = __builtin_bit_cast(u4v, hi), y = __builtin_bit_cast(u4v, lo);
          tacc[0] = mfma16<TY>(__builtin_bit_cast(B, l < 8 ? x : y), b, tacc[0]);
        } else {
          tacc[m] = mfma16<TY>(hi, b, tacc[m]);
          tacc[TM + m] = mfma16<TY>(lo, b, tacc[TM + m]);
        }
      }
    }
  };
  // once the weights are under way: the first tail step, and V into LDS (from
  // the sum's launch, or summed here in an order set by T, k and f alone)
  auto between = [&]() {
    if constexpr (RS == RS_NONE) return;
    if (wave < steps) tail_load(tail);
    if (tid < 16) V[nv + tid] = 0.f;
    if (a.v_sum) {
      for (int o = tid; o < nv; o += NT) V[o] = a.V[o];
      return;
    }
    const int nfb = a.f * a.Pin / 32, parts = NT / nv, p = tid / nv, o = tid - p * nv;
    float s = 0.f;
#pragma unroll 1
    for (int b0 = p; b0 < nfb; b0 += kDownPartials * parts) {
      float x[kDownPartials];
#pragma unroll
      for (int i = 0; i < kDownPartials; ++i) {
        const int b = b0 + i * parts;
        x[i] = p < parts && b < nfb ? a.Vp[static_cast<long>(b) * nv + o] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kDownPartials; ++i) s += x[i];
    }
    vpart[tid] = s;
    __syncthreads();
    if (tid < nv) {
      float v = 0.f;
      for (int i = 0; i < parts; ++i) v += vpart[i * nv + tid];
      V[tid] = v;
    }
  };
  if constexpr (Q4) {
    struct Slot {
      Raw<TY> x[NS];
      u4v w;
      u2v s;
      int at;
    };
    const B ones = q4_ones<TY>();
    stream_units<2, Slot>(
        u1 - u0,
        [&](int i, Slot& s) {
          seek(i);
          s.at = pi;
          s.w = *reinterpret_cast<const u4v*>(wp + static_cast<long>(kb) * 1024);
          s.s = load_scales<4>(sp + static_cast<long>(kb) * 64);
#pragma unroll
          for (int st = 0; st < NS; ++st) {
            // depths past f repeat the row's last ones (their codes are zero)
            const int k = min(kb * UNIT + 32 * st + 8 * q, a.f - 8);
            s.x[st] = load_raw<TY>(hp + k);
          }
        },
        [&](const Slot& s) {
          follow(s.at);
#pragma unroll
          for (int st = 0; st < NS; ++st) {
            const uint32_t word = s.w[st];
            const B b = q4_frag<TY>(word);
            const float sc = scale_at(s.s, st);
            const B x = raw_to_frag<TY, TY>(s.x[st]);
            const f4v sum = mfma16<TY>(x, ones, f4v{0.f, 0.f, 0.f, 0.f});
            f4v off;
#pragma unroll
            for (int i = 0; i < 4; ++i) off[i] = -kQ4Offset * sum[i];
            const f4v p = mfma16<TY>(x, b, off);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] += sc * p[i];
          }
        },
        between);
    if constexpr (!pieces) {
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] *= Q4Type<TY>::undo;
    }
  } else {
    struct Slot {
      Raw<TY> x[2];
      B w[2];
      int at;
    };
    stream_units<TY == DT_F32 ? 2 : 4, Slot>(
        u1 - u0,
        [&](int i, Slot& s) {
          seek(i);
          s.at = pi;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            s.w[h] = load_frag<TY>(wp + (static_cast<long>(kb) * 2048 + 256 * h) * es);
            s.x[h] = load_raw<TY>(hp + kb * 64 + 32 * h + 8 * q);
          }
        },
        [&](const Slot& s) {
          follow(s.at);
#pragma unroll
          for (int h = 0; h < 2; ++h) acc = mfma16<TY>(raw_to_frag<TY, TY>(s.x[h]), s.w[h], acc);
        },
        between);
  }
  if constexpr (RS != RS_NONE) {
    __syncthreads();  // V is in LDS
    for (int i = wave; i < steps; i += NW) {
      const Tail now = tail;
      if (i + NW < steps) {
        tail_find(i + NW);
        tail_load(tail);
      }
      tail_use(now);
    }
  }
  if constexpr (pieces) {
    if (u0 < u1) leave();
    if constexpr (RS != RS_NONE) {
      if (wave < steps) {
#pragma unroll
        for (int m = 0; m < TM; ++m)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int t = 16 * m + 4 * q + v;
            float s = tacc[m][v];
            if constexpr (planes == 2) s += tacc[TM + m][v];
            if (t < a.T) own[t * 16 + l] += s;
          }
      }
    }
  } else {
    *reinterpret_cast<f4v*>(own + lane * 4) = acc + tacc[0];
  }
  __syncthreads();
  for (int v = tid; v < a.T * 16; v += NT) {
    const int t = v >> 4, c = v & 15;
    float s = 0.f;
    if constexpr (pieces) {
#pragma unroll
      for (int w = 0; w < NW; ++w) s += red[w * block + v];
    } else {
#pragma unroll
      for (int p = planes - 1; p >= 0; --p)  // the rests first
        s += block_sum<NW, 1, 1>(red, t + 8 * p, c);
    }
    static_cast<typename Elem<XT>::T*>(a.Y)[static_cast<long>(t) * a.d + n * 16 + c] = from_f32<XT>(s);
  }
}

// --------------------------------------------------------------- repack --
// One thread per fragment lane: 8 values of one column, the order of pack.h's
// pack_frag with the permuted depth; two sources interleave in 32-column blocks.
template <class TS>
__global__ __launch_bounds__(256) void repack_kernel(const TS* src0, const TS* src1, int n_in, int n_out, TS* dst,
                                                     long per_group) {
  const long id = static_cast<long>(blockIdx.x) * 256 + threadIdx.x;
  if (id >= per_group) return;
  const int g = blockIdx.y, KS = n_in / 16;
  const int lane = id & 63;
  const long fr = id >> 6;
  const int ks = static_cast<int>(fr % KS), nb = static_cast<int>(fr / KS);
  const TS* src = src0;
  int col = nb * 32 + (lane & 31);
  if (src1) {
    if (nb & 1) src = src1;
    col = (nb >> 1) * 32 + (lane & 31);
  }
  src += static_cast<long>(g) * n_in * n_out;
  const int k0 = 64 * (ks >> 2) + 32 * (lane >> 5) + 8 * (ks & 3);
  TS* o = dst + (g * per_group + id) * 8;
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = src[static_cast<long>(k0 + e) * n_out + col];
}

// -------------------------------------------------------------- launches --
template <class K>
hipError_t go(K kernel, unsigned grid, unsigned threads, size_t lds, const FewArgs& a, hipStream_t st) {
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(threads), lds, st, a);
  return hipGetLastError();
}

template <int XT, int TY, int RS, int T8>
hipError_t route_t8(const FewArgs& a, hipStream_t st) {
  constexpr int MT = (T8 + 1) / 2;
  const int NC = a.G + (a.K > 1 ? a.G * a.K : 0);
  const unsigned nsb = (NC + 15) / 16 * a.nsplit, nub = (a.G * ((a.K * a.Pin * 16 + 31) / 32) + 1) / 2;
  const size_t tiles = static_cast<size_t>(NW) * 2 * MT * 256 * sizeof(float);  // of u_block
  const size_t scores =
      sizeof(float) * (static_cast<size_t>(NW) * MT * 256 + static_cast<size_t>(select_chunk(a.T, NC)) * NC);
  const size_t tables =
      sizeof(int16_t) * FEW_MAX_T * (a.G + static_cast<size_t>(a.E < a.T * a.k ? a.E : a.T * a.k));
  size_t lds = RS != RS_NONE && a.u_all ? tiles : 0;
  if (scores > lds) lds = scores;
  if (tables > lds) lds = tables;
  hipError_t e = go(few_route_kernel<XT, TY, RS, T8>, nsb + (RS != RS_NONE && a.u_all ? nub : 0), NT, lds, a, st);
  if constexpr (RS != RS_NONE)
    if (e == hipSuccess && !a.u_all) e = go(few_u_kernel<XT, TY, RS, T8>, nub, NT, tiles, a, st);
  return e;
}
template <int XT, int TY, bool Q4, int RS, int MT>
hipError_t up_mt(const FewArgs& a, hipStream_t st) {
  const unsigned grid = static_cast<unsigned>(a.G < a.T * a.kg ? a.G : a.T * a.kg) * (a.f * a.Pin / 32);
  const size_t lds = sizeof(float) * 2 * MT * 256;  // per wavefront
  const size_t hw = RS == RS_NONE ? 0 : sizeof(float) * a.T * a.ke * (32 / a.Pin);
  auto most = [](size_t x, size_t y) { return x > y ? x : y; };
  // More workgroups than compute units: smaller ones, so that one's expert
  // steps overlap the others' streams and the last round is finer.  Without a
  // residual there are no steps and 8 wavefronts keep the longer stream.
  // Measured (us a pass, 4 / 8 / 16 wavefronts): INT4 layer T = 16 89 / 91 /
  // 106, fp16 layer T = 5 33.0 / 34.2 / 41, flat layer T = 2 236 / 229 / 239.
  constexpr int W = RS == RS_NONE ? 8 : 4;
  if (grid > 256) return go(few_up_kernel<XT, TY, Q4, RS, MT, W>, grid, W * 64, most(W * lds, hw), a, st);
  return go(few_up_kernel<XT, TY, Q4, RS, MT, 16>, grid, 1024, most(16 * lds, hw), a, st);
}

template <int XT, int TY, bool Q4, int RS>
hipError_t down_rs(const FewArgs& a, hipStream_t st) {
  const unsigned grid = a.d / 16;
  const int nv = RS != RS_NONE ? a.T * a.k * 16 : 0;
  if (nv && a.v_sum) {
    hipLaunchKernelGGL(few_vsum_kernel, dim3((nv + 63) / 64), dim3(NT), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  constexpr int planes = hidden_planes(XT, TY);
  const int mt = planes == 1 ? (a.T <= 16 ? 1 : 2) : a.T <= 8 ? 1 : a.T <= 16 ? 2 : 4;
  // pieces: a group's are one more than its full tiles of tokens at most
  const size_t tables = few_groups(a) * FEW_MAX_T * sizeof(int16_t) +
                        (mt > 1 ? sizeof(int) * (1 + few_groups(a) + a.T * a.kg * planes / 16) : 0);
  const size_t lds =
      sizeof(float) * (static_cast<size_t>(NW) * (mt > 1 ? a.T * 16 : 256) + nv + 16 + (nv && !a.v_sum ? NT : 0)) +
      tables;
  if (mt == 1) return go(few_down_kernel<XT, TY, Q4, RS, 1>, grid, NT, lds, a, st);
  if (mt == 2) return go(few_down_kernel<XT, TY, Q4, RS, 2>, grid, NT, lds, a, st);
  if constexpr (planes == 2) return go(few_down_kernel<XT, TY, Q4, RS, 4>, grid, NT, lds, a, st);
  return hipErrorInvalidValue;
}

template <int XT, int TY, bool Q4, int RS>
hipError_t pass(const FewArgs& a, hipStream_t st) {
  // eights of tokens: only 4-bit input factors tell 1 from 2
  constexpr int one = RS == RS_INT4 ? 1 : 2;
  hipError_t e = a.T <= 8    ? route_t8<XT, TY, RS, one>(a, st)
                 : a.T <= 16 ? route_t8<XT, TY, RS, 2>(a, st)
                             : route_t8<XT, TY, RS, 4>(a, st);
  if (e == hipSuccess) e = a.T <= 16 ? up_mt<XT, TY, Q4, RS, 1>(a, st) : up_mt<XT, TY, Q4, RS, 2>(a, st);
  if (e == hipSuccess) e = down_rs<XT, hidden_type(TY, Q4), Q4, RS>(a, st);
  return e;
}

}  // namespace

int few_router_splits(int d) {
  // two 32-deep units per wavefront keep the matrix's loads in flight, with at
  // most 4 parts for the selection to add (one workgroup with the whole depth
  // of a 4096 x 8 router needs no exchange of scores but reads for 7.5 us)
  const int s = d / 32 / (2 * NW);
  return s < 1 ? 1 : s > 4 ? 4 : s;
}

bool few_v_sum(const FewArgs& a) {
  const long nv = static_cast<long>(a.T) * a.k * 16, nfb = a.f * a.Pin / 32;
  if (nv > NT) return true;
  const long parts = NT / nv;
  return (nfb + parts - 1) / parts > kDownPartials * kDownBatches;
}

hipError_t launch_few(int xt, int ty, bool q4, const FewArgs& a, hipStream_t st) {
  const int rs = a.resid == RS_NONE ? 0 : a.resid == RS_INT4 ? 2 : 1;
  switch (xt * 100 + ty * 10 + rs + (q4 ? 5 : 0)) {
    case 0: return pass<DT_F32, DT_F32, false, RS_NONE>(a, st);
    case 1: return pass<DT_F32, DT_F32, false, RS_F32>(a, st);
    case 110: return pass<DT_F16, DT_F16, false, RS_NONE>(a, st);
    case 111: return pass<DT_F16, DT_F16, false, RS_F16>(a, st);
    case 112: return pass<DT_F16, DT_F16, false, RS_INT4>(a, st);
    case 115: return pass<DT_F16, DT_F16, true, RS_NONE>(a, st);
    case 117: return pass<DT_F16, DT_F16, true, RS_INT4>(a, st);
    case 220: return pass<DT_BF16, DT_BF16, false, RS_NONE>(a, st);
    case 222: return pass<DT_BF16, DT_BF16, false, RS_INT4>(a, st);
    case 225: return pass<DT_BF16, DT_BF16, true, RS_NONE>(a, st);
    case 227: return pass<DT_BF16, DT_BF16, true, RS_INT4>(a, st);
    case 210: return pass<DT_BF16, DT_F16, false, RS_NONE>(a, st);
    case 211: return pass<DT_BF16, DT_F16, false, RS_F16>(a, st);
    case 212: return pass<DT_BF16, DT_F16, false, RS_INT4>(a, st);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_repack(int es, const void* src0, const void* src1, int groups, int n_in, int n_out, void* dst,
                         hipStream_t st) {
  const long per_group = static_cast<long>(n_in) * n_out * (src1 ? 2 : 1) / 8;
  const dim3 grid(static_cast<unsigned>((per_group + 255) / 256), groups);
  if (es == 4)
    hipLaunchKernelGGL(repack_kernel<float>, grid, dim3(256), 0, st, static_cast<const float*>(src0),
                       static_cast<const float*>(src1), n_in, n_out, static_cast<float*>(dst), per_group);
  else
    hipLaunchKernelGGL(repack_kernel<uint16_t>, grid, dim3(256), 0, st, static_cast<const uint16_t*>(src0),
                       static_cast<const uint16_t*>(src1), n_in, n_out, static_cast<uint16_t*>(dst), per_group);
  return hipGetLastError();
}

}  // namespace cefn
