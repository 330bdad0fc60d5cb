// fp4.cuh -- the 4-bit cache row and its conversion to f16 operands.
//
// A row of the 4-bit cache is 416 bytes: 256 bytes of e2m1 codes (dims 2i and
// 2i + 1 in the low and high half of byte i), 32 e4m3 scales (one for 16 dims)
// and the 64 rope dims in f16.  Latent dim d stands for code[d] * scale[d / 16],
// rope dim r for rope[r], both times the cache's kv_scale, which goes to the
// scores and the output instead.
//
// A code has two significant bits and a scale four, so their product has six
// and lies in [2^-10, 2688]: exact in f16.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

namespace fp4 {

constexpr int kRow = 416;       // bytes of a row
constexpr int kScales = 256;    // where its scales begin
constexpr int kRope = 288;      // where its rope dims begin

#ifdef __CUDACC__
// Eight codes to four f16 pairs, the low half of a byte first.
__device__ __forceinline__ uint4 e2m1x8_to_f16x8(uint32_t codes) {
  uint4 r;
  asm("{\n\t"
      ".reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t"
      "}"
      : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
      : "r"(codes));
  return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint4 scaled(uint32_t codes, uint32_t s) {
  const uint4 v = e2m1x8_to_f16x8(codes);
  return make_uint4(mul_f16x2(v.x, s), mul_f16x2(v.y, s), mul_f16x2(v.z, s), mul_f16x2(v.w, s));
}

// One of two e4m3 scales (the low 16 bits of `scales`), twice, as f16.
__device__ __forceinline__ uint32_t scale_pair(uint32_t scales, int which) {
  uint32_t s;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s) : "h"((uint16_t)scales));
  return __byte_perm(s, 0u, which ? 0x3232 : 0x1010);
}

// 32 codes (16 bytes) with two e4m3 scales (the low 16 bits of `scales`) to 32 f16.
__device__ __forceinline__ void convert(uint4 codes, uint32_t scales, uint4 (&out)[4]) {
  uint32_t s;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s) : "h"((uint16_t)scales));
  const uint32_t lo = __byte_perm(s, 0u, 0x1010), hi = __byte_perm(s, 0u, 0x3232);
  out[0] = scaled(codes.x, lo);
  out[1] = scaled(codes.y, lo);
  out[2] = scaled(codes.z, hi);
  out[3] = scaled(codes.w, hi);
}

// Eight values of a block of 16 as codes, the other eight with the lane next to
// this one (lane ^ 1), which calls this too; `scale`: the block's e4m3 scale.
//   q = x / s_kv,  scale = e4m3(max |q| / 6),  code = e2m1(q / scale),
// quotients rounded to fp32, codes and scale to nearest even, saturating.  A
// block whose scale rounds to zero has zero codes; one with a NaN has a NaN
// scale.
__device__ __forceinline__ uint32_t quantise8(const float (&x)[8], float s_kv, uint32_t* scale) {
  const unsigned pair = 3u << (threadIdx.x & 30u);
  float q[8], top = 0.f;
  bool nan = false;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    q[k] = __fdiv_rn(x[k], s_kv);
    nan |= q[k] != q[k];
    top = fmaxf(top, fabsf(q[k]));
  }
  const uint32_t mine = nan ? 0x7FC00000u : __float_as_uint(top);
  const uint32_t both = max(mine, __shfl_xor_sync(pair, mine, 1));  // of values >= 0, or the NaN
  if (both == 0x7FC00000u) {
    *scale = 0x7Fu;
    return 0u;
  }
  uint16_t s8;
  uint32_t s16;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
      : "=h"(s8)
      : "f"(0.f), "f"(__fdiv_rn(__uint_as_float(both), 6.f)));
  *scale = s8;
  if (s8 == 0) return 0u;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s16) : "h"(s8));
  const float d = __half2float(__ushort_as_half((unsigned short)s16));
#pragma unroll
  for (int k = 0; k < 8; ++k) q[k] = __fdiv_rn(q[k], d);
  uint32_t codes;
  asm("{\n\t"
      ".reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t"
      "}"
      : "=r"(codes)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return codes;
}

// A rope dim: x / s_kv in f16, within +-65504 (a NaN stays one).
__device__ __forceinline__ uint32_t rope_pair(float a, float b, float s_kv) {
  a = __fdiv_rn(a, s_kv);
  b = __fdiv_rn(b, s_kv);
  a = a > 65504.f ? 65504.f : a < -65504.f ? -65504.f : a;
  b = b > 65504.f ? 65504.f : b < -65504.f ? -65504.f : b;
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 16-byte piece `piece` (0..71; eight dims) of a row of 576 at `row`: 64 pieces
// of latent, 8 of rope.
__device__ __forceinline__ void store_piece(uint8_t* row, int piece, const float (&x)[8], float s_kv) {
  if (piece >= 64) {
    *reinterpret_cast<uint4*>(row + kRope + (piece - 64) * 16) =
        make_uint4(rope_pair(x[0], x[1], s_kv), rope_pair(x[2], x[3], s_kv),
                   rope_pair(x[4], x[5], s_kv), rope_pair(x[6], x[7], s_kv));
    return;
  }
  uint32_t scale;
  reinterpret_cast<uint32_t*>(row)[piece] = quantise8(x, s_kv, &scale);
  if ((piece & 1) == 0) row[kScales + (piece >> 1)] = (uint8_t)scale;
}
#endif

}  // namespace fp4
