// rope_epilogue.cu -- the step before the decode with the position rotation
// applied on the way: the rotated 576-wide query rows, and the insert of each
// new token's latent row, its rope dims rotated, into the paged cache.
//
// With (cos, sin) the table's row of the token's position, a pair (x, y) of
// rope dims becomes (x cos - y sin, y cos + x sin).  The pair is dims (2i,
// 2i + 1) (interleaved) or (i, i + 32) (half-split), i < 32.  Products and
// sums are fp32; the result is rounded once, to bf16 or to the e4m3 code of
// x / kv_scale.
//
// Eight threads a row, rows ordered (token, H query rows + the cache row):
// thread `sub` takes the 16-byte pieces sub, sub + 8, ... of the row's 72, so
// every access of the eight is a whole 128-byte line, and its last piece (64 +
// sub) is its share of the rope dims.  All nine loads are issued before the
// first store.  Bound by memory (2304 B in and out a query row).
//
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/mla_decode.h"
#include "fp4.cuh"
#include "internal.h"
#include "kv.h"
#include "ptx.cuh"

namespace {

constexpr int kRows = 32;  // rows per CTA
constexpr int kThreads = 8 * kRows;

struct RopeParams {
  const uint16_t *ql, *qp, *kc, *kp;
  int64_t ql_t, ql_h, qp_t, qp_h, kc_t, kp_t;  // strides in elements
  const int64_t* positions;
  const float* cos_sin;  // [max_pos, 64]: 32 cosines, 32 sines
  int64_t max_pos;
  const int64_t* slots;
  uint16_t* q_out;
  void* cache;
  const float* kv_scale;
  int32_t* status;
  int64_t num_slots;
  uint32_t rows;  // tokens * (heads + 1), or (heads + 8)
  int heads, fp8, interleaved, early;
};

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// The 8 rotated values of rope piece e (dims 8e .. 8e + 7) given as `mine`; the
// other seven pieces are with the other lanes of the row's eight.
__device__ __forceinline__ void rotate(bool interleaved, uint4 mine, const float* cs, int e,
                                       float (&o)[8]) {
  const uint32_t a[4] = {mine.x, mine.y, mine.z, mine.w};
  if (interleaved) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(cs) + e);
    const float4 s = __ldg(reinterpret_cast<const float4*>(cs + 32) + e);
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = lo_f(a[i]), y = hi_f(a[i]);
      o[2 * i] = fmaf(x, cc[i], -(y * ss[i]));
      o[2 * i + 1] = fmaf(y, cc[i], x * ss[i]);
    }
    return;
  }
  uint32_t b[4];  // the other half's piece, e ^ 4
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = __shfl_xor_sync(0xffffffffu, a[i], 4);
  const float sign = e < 4 ? -1.f : 1.f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(cs) + 2 * (e & 3) + h);
    const float4 s = __ldg(reinterpret_cast<const float4*>(cs + 32) + 2 * (e & 3) + h);
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t wa = a[2 * h + (i >> 1)], wb = b[2 * h + (i >> 1)];
      const float x = (i & 1) ? hi_f(wa) : lo_f(wa), y = (i & 1) ? hi_f(wb) : lo_f(wb);
      o[4 * h + i] = fmaf(x, cc[i], sign * (y * ss[i]));
    }
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t e4m3x2(float first, float second) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(second), "f"(first));
  return r;
}

__device__ __noinline__ uint2 divided(float4 a, float4 b, float s) {
  return make_uint2(e4m3x2(__fdiv_rn(a.x, s), __fdiv_rn(a.y, s)) | e4m3x2(__fdiv_rn(a.z, s), __fdiv_rn(a.w, s)) << 16,
                    e4m3x2(__fdiv_rn(b.x, s), __fdiv_rn(b.y, s)) | e4m3x2(__fdiv_rn(b.z, s), __fdiv_rn(b.w, s)) << 16);
}

// The e4m3 codes of the fp32 quotients x / s, without the divisions (72 a
// thread were 2 of the kernel's 5.4 us at 64 tokens x 128 heads).  With inv the
// rounded 1 / s, x inv is off by at most 2^-23 of itself and the rounded
// quotient by 2^-24, so the quotient lies between x inv (1 - 2^-21) and x inv
// (1 + 2^-21); where both have the same code, it has that one too, since
// rounding never swaps two values.  Near a border of two codes it is divided
// out, as with an s whose reciprocal leaves the range (inv = NaN then).  A power
// of two, whose quotients often are ties, needs no margin: x inv is exact.
__device__ __forceinline__ uint2 codes(const float (&x)[8], float s, float inv, float margin) {
  uint32_t lo[4], hi[4];
  bool differ = inv != inv;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float a = x[2 * k] * inv, b = x[2 * k + 1] * inv;
    lo[k] = e4m3x2(a * (1.f - margin), b * (1.f - margin));
    hi[k] = e4m3x2(a * (1.f + margin), b * (1.f + margin));
    differ |= lo[k] != hi[k];
  }
  if (differ) return divided(make_float4(x[0], x[1], x[2], x[3]), make_float4(x[4], x[5], x[6], x[7]), s);
  return make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
}

// The 4-bit insert has a form of its own, in which a cache row counts as eight
// rows of one latent piece a thread: eight pieces with their 128 divisions by one
// thread took 6.7 us for a single token, where the copy of a bf16 row takes 1.8.
template <bool kFp4>
__global__ void __launch_bounds__(kThreads, 4) rope_epilogue_kernel(RopeParams p) {
  constexpr int kCacheRows = kFp4 ? 8 : 1;
  const int sub = (int)(threadIdx.x & 7);
  const uint32_t row = blockIdx.x * kRows + (threadIdx.x >> 3);
  // Only inputs that the caller declares older than the kernel before this
  // one may be read ahead of the dependency wait.
  if (!p.early) ptx::grid_dependency_wait();
  const uint32_t t = row / (uint32_t)(p.heads + kCacheRows);
  const int h = (int)(row - t * (uint32_t)(p.heads + kCacheRows));
  const bool active = row < p.rows, cache_row = h >= p.heads, first = h == p.heads;
  int64_t slot = -1;
  const float* cs = p.cos_sin;
  if (active) {
    if (cache_row) slot = p.slots[t];
    int64_t pos = p.positions[t];
    if (pos < 0 || pos >= p.max_pos) {
      if (first && sub == 0 && slot >= 0 && p.status) atomicOr(p.status, MLA_DEVFLAG_POSITION);
      pos = pos < 0 ? 0 : p.max_pos - 1;
    }
    cs += pos * 64;
  }
  if (p.early) ptx::grid_dependency_wait();
  ptx::launch_dependents();
  uint4 v[9];
  if (active) {
    const uint16_t* latent = cache_row ? p.kc + (int64_t)t * p.kc_t
                                       : p.ql + (int64_t)t * p.ql_t + (int64_t)h * p.ql_h;
    const uint16_t* rope = cache_row ? p.kp + (int64_t)t * p.kp_t
                                     : p.qp + (int64_t)t * p.qp_t + (int64_t)h * p.qp_h;
    v[8] = reinterpret_cast<const uint4*>(rope)[sub];
    if (kFp4 && cache_row) {
      v[0] = reinterpret_cast<const uint4*>(latent)[sub + 8 * (h - p.heads)];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = reinterpret_cast<const uint4*>(latent)[sub + 8 * i];
    }
  }
  float o[8];
  rotate(p.interleaved, v[8], cs, sub, o);  // every lane takes part
  if (!active) return;
  if (cache_row) {
    if (slot < 0) return;  // padding token: no insert
    if (slot >= p.num_slots) {
      if (first && sub == 0 && p.status) atomicOr(p.status, MLA_DEVFLAG_BAD_PAGE);
      return;
    }
    if constexpr (kFp4) {  // pieces 2k and 2k + 1 are with neighbouring lanes
      const float s = *p.kv_scale;
      uint8_t* dst = static_cast<uint8_t*>(p.cache) + slot * fp4::kRow;
      const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
      float x[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[2 * k] = lo_f(w[k]);
        x[2 * k + 1] = hi_f(w[k]);
      }
      fp4::store_piece(dst, sub + 8 * (h - p.heads), x, s);
      if (first) fp4::store_piece(dst, 64 + sub, o, s);
      return;
    }
    if (!kFp4 && p.fp8) {
      const float s = *p.kv_scale;
      const bool near = fabsf(s) >= 0x1p-100f && fabsf(s) <= 0x1p100f;
      const float inv = near ? __frcp_rn(s) : NAN;
      const float margin = (__float_as_uint(s) & 0x7FFFFFu) == 0 ? 0.f : 0x1p-21f;
      uint2* dst = reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.cache) + slot * MLA_D_QK) + sub;
#pragma unroll
      for (int i = 0; i < 9; ++i) {
        float x[8];
        if (i < 8) {
          const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x[2 * k] = lo_f(w[k]);
            x[2 * k + 1] = hi_f(w[k]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = o[k];
        }
        dst[8 * i] = codes(x, s, inv, margin);
      }
      return;
    }
  }
  v[8] = make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]),
                    pack_bf16(o[6], o[7]));
  uint4* dst = reinterpret_cast<uint4*>(cache_row ? static_cast<uint16_t*>(p.cache) + slot * MLA_D_QK
                                                  : p.q_out + ((int64_t)t * p.heads + h) * MLA_D_QK) + sub;
#pragma unroll
  for (int i = 0; i < 9; ++i) dst[8 * i] = v[i];
}

bool misaligned(const void* x, uintptr_t a) { return (reinterpret_cast<uintptr_t>(x) % a) != 0; }

// A stride in elements must keep every row 16-byte aligned; a dimension of one
// has none.
bool take_stride(int64_t given, int64_t count, int64_t* out) {
  *out = count > 1 ? given : 0;
  return *out >= 0 && *out % 8 == 0;
}

}  // namespace

extern "C" int mla_decode_rope_epilogue(
    const void* ql_nope, int64_t ql_stride_t, int64_t ql_stride_h, const void* q_pe,
    int64_t q_pe_stride_t, int64_t q_pe_stride_h, const void* kv_c, int64_t kv_c_stride,
    const void* k_pe, int64_t k_pe_stride, const int64_t* positions, const float* cos_sin,
    int64_t max_positions, int32_t interleaved, const int64_t* slot_mapping, int32_t num_tokens,
    int32_t num_heads, void* q_out, void* kv_cache, int64_t num_pages, int32_t page_size,
    int32_t kv_dtype, const float* kv_scale, int32_t inputs_early, int32_t* status,
    void* stream) {
  if (num_tokens < 0 || num_heads < 1 || num_heads > 128 || page_size < 1 || num_pages < 1 ||
      max_positions < 1)
    return MLA_ERR_INVALID_ARG;
  if (!mla::kv_dtype_known(kv_dtype)) return MLA_ERR_INVALID_ARG;
  if (interleaved < 0 || interleaved > 1 || inputs_early < 0 || inputs_early > 1)
    return MLA_ERR_INVALID_ARG;
  if (num_tokens == 0) return MLA_OK;
  if (!ql_nope || !q_pe || !kv_c || !k_pe || !positions || !cos_sin || !slot_mapping || !q_out ||
      !kv_cache || (kv_dtype != MLA_KV_BF16 && !kv_scale))
    return MLA_ERR_INVALID_ARG;
  if (misaligned(ql_nope, 16) || misaligned(q_pe, 16) || misaligned(kv_c, 16) ||
      misaligned(k_pe, 16) || misaligned(cos_sin, 16) || misaligned(q_out, 16) ||
      misaligned(kv_cache, 16) || misaligned(positions, 8) || misaligned(slot_mapping, 8) ||
      misaligned(kv_scale, 4) || misaligned(status, 4))
    return MLA_ERR_INVALID_ARG;
  RopeParams p;
  if (!take_stride(ql_stride_t, num_tokens, &p.ql_t) || !take_stride(ql_stride_h, num_heads, &p.ql_h) ||
      !take_stride(q_pe_stride_t, num_tokens, &p.qp_t) || !take_stride(q_pe_stride_h, num_heads, &p.qp_h) ||
      !take_stride(kv_c_stride, num_tokens, &p.kc_t) || !take_stride(k_pe_stride, num_tokens, &p.kp_t))
    return MLA_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)num_tokens * (num_heads + (kv_dtype == MLA_KV_FP4_E2M1 ? 8 : 1));
  if (rows > INT32_MAX) return MLA_ERR_UNSUPPORTED;
  p.ql = static_cast<const uint16_t*>(ql_nope);
  p.qp = static_cast<const uint16_t*>(q_pe);
  p.kc = static_cast<const uint16_t*>(kv_c);
  p.kp = static_cast<const uint16_t*>(k_pe);
  p.positions = positions;
  p.cos_sin = cos_sin;
  p.max_pos = max_positions;
  p.slots = slot_mapping;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.cache = kv_cache;
  p.kv_scale = kv_scale;
  p.status = status;
  p.num_slots = num_pages * (int64_t)page_size;
  p.rows = (uint32_t)rows;
  p.heads = num_heads;
  p.fp8 = kv_dtype == MLA_KV_FP8_E4M3;
  p.interleaved = interleaved;
  p.early = inputs_early;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((rows + kRows - 1) / kRows), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kernel = kv_dtype == MLA_KV_FP4_E2M1 ? rope_epilogue_kernel<true> : rope_epilogue_kernel<false>;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) return MLA_ERR_CUDA;
  return MLA_OK;
}
