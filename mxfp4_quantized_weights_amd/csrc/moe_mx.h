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
// 16-byte accesses of 8 (bf16) or 4 (fp32) elements from column 0 of every row
inline bool mx_vec_ok(const void* p, int64_t ld, int esize) { return mx_aligned(p, 16) && (ld * esize) % 16 == 0; }
inline moe_status_t mx_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// Row and / or column quantisation (each pair of outputs may be null).
hipError_t launch_mx_quant(const void* in, bool bf16, int64_t rows, int64_t cols, int64_t ld, uint8_t* q_row,
                           uint8_t* s_row, uint8_t* q_col, uint8_t* s_col, hipStream_t s);

// Eight elements from element index `at`, `left` of them inside the row (the
// others are zero), as fp32.  VEC: 16-byte loads are aligned.
template <bool BF16, bool VEC>
__device__ __forceinline__ void mx_load8(const void* in, int64_t at, int64_t left, float (&v)[8]) {
  if constexpr (BF16) {
    const uint16_t* p = (const uint16_t*)in + at;
    if (VEC && left >= 8) {
      const uint4 w = *(const uint4*)p;
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < left ? bf16_to_f32(p[i]) : 0.0f;
    }
  } else {
    const float* p = (const float*)in + at;
    if (VEC && left >= 8) {
      const float4 a = *(const float4*)p, b = *(const float4*)(p + 4);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i] : 0.0f;
    }
  }
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

}  // namespace moe
