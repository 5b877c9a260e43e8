// 4-bit weights with group scales: the storage order shared by the packing
// kernel and the kernels that stream the weights for a few rows, and the
// decode into MFMA operands.
//
// A matrix of n_in rows (the depth k of the product) and n_out columns is cut
// into tiles of 16 C columns (C = 1, 2 or 4) and units of 128 / C rows.  One
// unit of one tile is 1 KiB: lane l of a wavefront owns 16 bytes, four words
// of eight codes each, so a unit is one coalesced 16-byte load per lane
// whatever C.  Word j of lane l holds column 16 c + l % 16 of the tile, rows
// 32 s + 8 (l / 16) .. + 7 of the unit, with c = j % C and s = j / C: the
// operand of one 16x16x32 MFMA.  Tiles with few columns (C = 1) give a
// narrow matrix enough workgroups; wide tiles re-use each fragment of the
// activations C times.
//
// Scales: one fp16 per column and `group` rows.  Per tile they lie in rows
// of [16 columns l][E entries], E = C * max(1, (128 / C) / group): entry
// s * C + c of column l, s the group inside the unit.  A unit whose rows lie inside one
// group shares its scale row with the group's other units.
//
// Codes are stored as q + 8 in 0..15, two to a pair of 16-bit halves: code
// c_2i in the low half and c_2i+1 in the high half of the word rotated right
// by 4 i, both at bit `q4_bit` of their half, which is where the type's
// mantissa wants them: OR-ed under the exponent of 16.0 they read as
// 16 + c exactly (4 mantissa bits).  So a decoded code costs less than one
// VALU instruction: 3 rotates and 4 and-ors for 8 codes.  The product then
// subtracts 24 times the sum of the activations, which enters as the
// accumulator operand of the first MFMA of a group (the sum itself comes
// from an MFMA against ones).  Products of an 11- or 8-bit activation with a
// 5-bit number are exact in FP32, so the only rounding is the FP32
// accumulation; the offset enlarges the summands by 24 / 4.6 against codes
// of mean square 21, i.e. by about five times the FP32 rounding of the sum,
// 2^-22 or so, far below the 2^-12 of an fp16 result.
//
// bf16 activations reach 2^128, where 128 products with 31 would overflow
// FP32 though the result need not: their codes and the ones carry a factor
// 2^-12 (exponents of 16 2^-12 and 2^-12), which the last multiplication
// takes off (`undo`).
#pragma once
#include "common.h"

namespace cefn {

constexpr int Q4_ROWS = 32;  // rows (tokens) one launch takes

template <int TY> struct Q4Type;
template <> struct Q4Type<DT_F16> {
  static constexpr uint32_t mask = 0x03C003C0u, magic = 0x4C004C00u, one = 0x3C003C00u;
  static constexpr float undo = 1.0f;
};
template <> struct Q4Type<DT_BF16> {
  static constexpr uint32_t mask = 0x00780078u, magic = 0x3B803B80u, one = 0x39803980u;
  static constexpr float undo = 4096.0f;
};
__host__ __device__ inline int q4_bit(int ty) { return ty == DT_F16 ? 6 : 3; }

// Word of eight codes (0..15 each, code e at nibble e of `nibbles`).
__host__ __device__ inline uint32_t q4_word(uint32_t nibbles, int bit) {
  uint32_t w = 0;
  for (int e = 0; e < 8; ++e) {
    const uint32_t c = (nibbles >> (4 * e)) & 15u;
    const int pos = bit + 16 * (e & 1) + 4 * (e >> 1);  // rotated right by 4 (e / 2): back at bit
    const uint64_t v = static_cast<uint64_t>(c) << (pos & 31);
    w |= static_cast<uint32_t>(v) | static_cast<uint32_t>(v >> 32);
  }
  return w;
}
// Code e of such a word.
__host__ __device__ inline int q4_code(uint32_t w, int e, int bit) {
  const int pos = (bit + 16 * (e & 1) + 4 * (e >> 1)) & 31;
  const uint32_t r = pos ? (w >> pos) | (w << (32 - pos)) : w;
  return static_cast<int>(r & 15u);
}

// The word as an MFMA operand of type TY, each code c as (16 + c) / undo.
template <int TY>
__device__ __forceinline__ typename Frag<TY>::T q4_frag(uint32_t w) {
  u4v r;
  r[0] = (w & Q4Type<TY>::mask) | Q4Type<TY>::magic;
  r[1] = (__builtin_rotateright32(w, 4) & Q4Type<TY>::mask) | Q4Type<TY>::magic;
  r[2] = (__builtin_rotateright32(w, 8) & Q4Type<TY>::mask) | Q4Type<TY>::magic;
  r[3] = (__builtin_rotateright32(w, 12) & Q4Type<TY>::mask) | Q4Type<TY>::magic;
  return __builtin_bit_cast(typename Frag<TY>::T, r);
}
// The same of a word in the residual factors' order (code e at bits 4 e):
// even and odd codes apart, a byte each, then byte i of both into one pair.
template <int TY>
__device__ __forceinline__ typename Frag<TY>::T q4_frag_plain(uint32_t w) {
  const uint32_t even = w & 0x0F0F0F0Fu, odd = (w >> 4) & 0x0F0F0F0Fu;
  constexpr int bit = TY == DT_F16 ? 6 : 3;
  u4v r;
  r[0] = (__builtin_amdgcn_perm(even, odd, 0x0c000c04u) << bit) | Q4Type<TY>::magic;
  r[1] = (__builtin_amdgcn_perm(even, odd, 0x0c010c05u) << bit) | Q4Type<TY>::magic;
  r[2] = (__builtin_amdgcn_perm(even, odd, 0x0c020c06u) << bit) | Q4Type<TY>::magic;
  r[3] = (__builtin_amdgcn_perm(even, odd, 0x0c030c07u) << bit) | Q4Type<TY>::magic;
  return __builtin_bit_cast(typename Frag<TY>::T, r);
}
// Eight times 1 / undo.
template <int TY>
__device__ __forceinline__ typename Frag<TY>::T q4_ones() {
  const u4v r = {Q4Type<TY>::one, Q4Type<TY>::one, Q4Type<TY>::one, Q4Type<TY>::one};
  return __builtin_bit_cast(typename Frag<TY>::T, r);
}
// E (1, 2 or 4) consecutive fp16 scales and one of them.
typedef uint32_t u2v __attribute__((ext_vector_type(2)));
template <int E>
__device__ __forceinline__ u2v load_scales(const uint16_t* p) {
  u2v r = {0u, 0u};
  if constexpr (E == 4) r = *reinterpret_cast<const u2v*>(p);
  else if constexpr (E == 2) r[0] = *reinterpret_cast<const uint32_t*>(p);
  else r[0] = *p;
  return r;
}
__device__ __forceinline__ float scale_at(const u2v& s, int i) {
  const uint32_t w = i < 2 ? s[0] : s[1];
  return f16_bits_to_f32(static_cast<uint16_t>((w >> (16 * (i & 1))) & 0xFFFFu));
}
constexpr float kQ4Offset = 24.0f;  // 16 + (q + 8) - q

// Shape of one packed matrix.
struct Q4Shape {
  int n_in, n_out, C, group;
  __host__ __device__ int unit() const { return 128 / C; }
  __host__ __device__ long tiles() const { return (n_out + 16 * C - 1) / (16 * C); }
  __host__ __device__ long units() const { return (n_in + 127L) / 128 * C; }  // whole runs of 128 rows
  __host__ __device__ int srow_units() const { return group > unit() ? group / unit() : 1; }  // units per scale row
  __host__ __device__ long srows() const { return (units() + srow_units() - 1) / srow_units(); }
  __host__ __device__ int gpu() const { return group >= unit() ? 1 : unit() / group; }  // groups per unit
  __host__ __device__ int entries() const { return C * gpu(); }
  __host__ __device__ long words() const { return tiles() * units() * 256; }
  __host__ __device__ long scales() const { return tiles() * srows() * 16 * entries(); }
};

// Source of a packed matrix.  Either codes (q int8 [n_in][n_out] in [-8, 7]
// with scale fp16 bits [ceil(n_in / group)][n_out]) or values of dtype
// v_dtype [n_in][n_out], quantised on the way: scale = fp16(amax / 7), code =
// rint(v / scale) clamped to [-8, 7], both in FP32; a zero scale has zero
// codes.  Two value sources v[0], v[1] of n_out / 2 columns each interleave in
// blocks of 16 columns (n_src = 2: the gate and up projections of a SwiGLU layer).
struct Q4Source {
  const int8_t* q;
  const uint16_t* scale;
  const void* v[2];
  int v_dtype, n_src;
};
hipError_t launch_q4_pack(const Q4Shape& s, const Q4Source& src, int ty, uint32_t* words, uint16_t* scales,
                          hipStream_t st);
// Codes (int8 [n_in][n_out]) and scales ([ceil(n_in / group)][n_out]) back out of the packed form.
hipError_t launch_q4_unpack(const Q4Shape& s, int ty, const uint32_t* words, const uint16_t* scales, int8_t* q,
                            uint16_t* scale, hipStream_t st);

}  // namespace cefn
