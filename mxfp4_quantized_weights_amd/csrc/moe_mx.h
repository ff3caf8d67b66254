// Shared by the dense MXFP4 operators (mx_quant.hip, mx_matmul.hip): limits,
// argument checks, and the loads and scales of the quantisers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"
#include "moe_device.h"

namespace moe {

constexpr int64_t kMxMaxDim = 1ll << 24;    // rows, columns, M, N, K
constexpr int64_t kMxMaxElems = 1ll << 38;  // elements of one matrix
constexpr int64_t kMxMaxGrid = 1ll << 20;   // workgroups of a launch (the kernels step over what is left)

inline __host__ __device__ int64_t mx_padded(int64_t n) { return (n + 127) / 128 * 128; }
inline bool mx_dtype_ok(int32_t d) { return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F32; }
inline bool mx_matrix_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && cols >= 0 && rows <= kMxMaxDim && cols <= kMxMaxDim && mx_padded(rows) * mx_padded(cols) <= kMxMaxElems;
}
inline bool mx_aligned(const void* p, uintptr_t a) { return (uintptr_t)p % a == 0; }
inline moe_status_t mx_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// Row and / or column quantisation (each pair of outputs may be null).
hipError_t launch_mx_quant(const void* in, bool bf16, int64_t rows, int64_t cols, int64_t ld, uint8_t* q_row,
                           uint8_t* s_row, uint8_t* q_col, uint8_t* s_col, hipStream_t s);

// Sixteen bytes at any element's address: the hardware takes vector accesses
// that are aligned to no more than their elements.
typedef uint32_t v4u_any __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ uint4 mx_read16(const void* p) {
  const v4u_any v = *(const v4u_any*)p;
  return make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void mx_write16(void* p, const uint4& v) { *(v4u_any*)p = v4u_any{v.x, v.y, v.z, v.w}; }

// Largest magnitudes, as the bits of an fp32 value (integer maxima: a floating
// maximum would drop a NaN).
__device__ __forceinline__ uint32_t mx_max_u16x2(uint32_t a, uint32_t b) {
  typedef uint16_t v2u16 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(v2u16, a), __builtin_bit_cast(v2u16, b)));
}
__device__ __forceinline__ uint32_t mx_amax_bf16(const uint4& x) {
  const uint32_t m = mx_max_u16x2(mx_max_u16x2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                                  mx_max_u16x2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
  return max(m << 16, m & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t mx_amax_f32(const uint4& x) {
  return max(max(x.x & 0x7FFFFFFFu, x.y & 0x7FFFFFFFu), max(x.z & 0x7FFFFFFFu, x.w & 0x7FFFFFFFu));
}

// E2M1 codes of values in a group with scale byte b (all zero for b = 255).
// The hardware conversions divide by the scale, round to nearest even and
// saturate to +-6, exactly as the definition: equal to the scaled, clamped and
// converted value for every bf16 value at every scale that its group can have,
// subnormals and the scale 2^-127 included, and for 10^8 fp32 values at and
// next to the midpoints (checked once; the tests hold the codes to the
// definition at every midpoint over fp32's range).
__device__ __forceinline__ uint32_t mx_codes_bf16(const uint4& x, uint32_t b) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  const float s = e8m0_value(b);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(v2bf, x.x), s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(v2bf, x.y), s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(v2bf, x.z), s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(v2bf, x.w), s, 3);
  return b == 255u ? 0u : w;
}
// Four codes in the low 16 bits.
__device__ __forceinline__ uint32_t mx_codes_f32(const uint4& x, uint32_t b) {
  const float s = e8m0_value(b);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(x.x), __uint_as_float(x.y), s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(x.z), __uint_as_float(x.w), s, 1);
  return b == 255u ? 0u : w;
}
// The E2M1 values of 8 codes.
__device__ __forceinline__ void mx_values8(uint32_t w, float (&v)[8]) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
  const v2f c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
  v[0] = a[0]; v[1] = a[1]; v[2] = b[0]; v[3] = b[1];
  v[4] = c[0]; v[5] = c[1]; v[6] = d[0]; v[7] = d[1];
}

// Scale byte of a group from the largest magnitude's bits: as e8m0_byte, and
// 255 (the format's NaN) where the group holds an infinity or a NaN.  Taken
// from the bits, since a floating maximum would drop a NaN.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  return amax_bits >= 0x7F800000u ? 255u : e8m0_byte(__uint_as_float(amax_bits));
}

// Maximum over aligned groups of 4 lanes, received by all four.
__device__ __forceinline__ uint32_t mx_group_max4(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0xB1, 0xF, 0xF, false));  // quad_perm [1,0,3,2]
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x4E, 0xF, 0xF, false));  // [2,3,0,1]
}

// The value of the lane across the middle of its half row of 8.
__device__ __forceinline__ uint32_t mx_row_half_mirror(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x141, 0xF, 0xF, false);
}

}  // namespace moe
