// MXFP4 quantisation of a matrix along its rows and along its columns, the
// values that MXFP4 codes stand for, and their C ABI (moe_mxfp4_quant,
// moe_mxfp4_dequant).
//
// The format (OCP MX): E2M1 elements, two per byte, one E8M0 scale per 32.  A
// product sums over the axis its operands are grouped along, so a linear
// layer's forward pass needs x and W grouped along their rows, its backward
// pass dy, x and W along the other axis too.  Both groupings come from one
// read of the matrix.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"
#include "moe_device.h"
#include "moe_mx.h"

namespace moe {

// One workgroup quantises a 128-row x 64-column tile; thread t holds 8
// consecutive columns of row (t / 8) + 32 i, i = 0..3, so a row group of 32 is
// 4 neighbouring lanes.  For the column groups the tile goes through LDS as
// fp32 and thread t takes column t % 64, rows 32 (t / 64) .. +32: 16 bytes of
// codes, gathered in LDS so that a column's 64 bytes leave together.
constexpr int kQTileR = 128, kQTileC = 64;
constexpr int kQLd = kQTileC + 1;  // LDS row stride in floats: row writes and column reads hit distinct banks

// Packs 8 values, scaled by inv = 2^(127 - b) (exact), into 8 E2M1 codes.
__device__ __forceinline__ uint32_t mx_pack8(const float (&v)[8], float inv) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) w |= mx_quant(v[i], inv) << (4 * i);
  return w;
}

template <bool BF16, bool VEC, bool ROW, bool COL>
__global__ __launch_bounds__(256) void mx_quant_kernel(const void* __restrict__ in, int64_t rows, int64_t cols,
                                                       int64_t ld, int64_t cp, int64_t rp, int64_t tiles_c,
                                                       int64_t tiles, uint8_t* __restrict__ q_row,
                                                       uint8_t* __restrict__ s_row, uint8_t* __restrict__ q_col,
                                                       uint8_t* __restrict__ s_col) {
  __shared__ float buf[COL ? kQTileR * kQLd : 1];
  __shared__ uint4 codes[COL ? kQTileC * 4 : 1];
  __shared__ uint32_t scales[COL ? kQTileC : 1];
  const int t = threadIdx.x;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t r0 = tile / tiles_c * kQTileR, c0 = tile % tiles_c * kQTileC;
    const int64_t col = c0 + (t & 7) * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int lr = (t >> 3) + 32 * i;
      const int64_t row = r0 + lr;
      float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (row < rows) mx_load8<BF16, VEC>(in, row * ld + col, cols - col, v);
      if constexpr (ROW) {
        uint32_t a = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) a = max(a, __float_as_uint(v[j]) & 0x7FFFFFFFu);
        a = mx_group_max4(a);
        const uint32_t b = mx_scale_byte(a);
        const uint32_t w = b == 255u ? 0u : mx_pack8(v, e8m0_inverse(b));
        if (row < rows && col < cp) {
          *(uint32_t*)(q_row + row * (cp / 2) + col / 2) = w;
          if ((t & 3) == 0) s_row[row * (cp / 32) + col / 32] = (uint8_t)b;
        }
      }
      if constexpr (COL) {
#pragma unroll
        for (int j = 0; j < 8; ++j) buf[lr * kQLd + (t & 7) * 8 + j] = v[j];
      }
    }
    if constexpr (COL) {
      __syncthreads();
      {
        const int c = t & 63, rg = t >> 6;
        const float* p = buf + rg * 32 * kQLd + c;
        uint32_t a = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) a = max(a, __float_as_uint(p[j * kQLd]) & 0x7FFFFFFFu);
        const uint32_t b = mx_scale_byte(a);
        const float inv = e8m0_inverse(b == 255u ? 0u : b);
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = p[(q * 8 + j) * kQLd];
          w[q] = b == 255u ? 0u : mx_pack8(v, inv);
        }
        codes[c * 4 + rg] = make_uint4(w[0], w[1], w[2], w[3]);
        ((uint8_t*)scales)[c * 4 + rg] = (uint8_t)b;
      }
      __syncthreads();
      {
        const int c = t >> 2, rg = t & 3;
        const int64_t gc = c0 + c, gr = r0 + rg * 32;
        if (gc < cols && gr < rp) {
          *(uint4*)(q_col + gc * (rp / 2) + gr / 2) = codes[t];
          if (rg == 0) *(uint32_t*)(s_col + gc * (rp / 32) + r0 / 32) = scales[c];
        }
      }
    }
  }
}

template <bool BF16, bool VEC>
static hipError_t launch_mx_quant_t(dim3 grid, hipStream_t s, const void* in, int64_t rows, int64_t cols, int64_t ld,
                                    int64_t cp, int64_t rp, int64_t tc, int64_t tiles, uint8_t* qr, uint8_t* sr,
                                    uint8_t* qc, uint8_t* sc) {
  if (qr && qc)
    hipLaunchKernelGGL((mx_quant_kernel<BF16, VEC, true, true>), grid, dim3(256), 0, s, in, rows, cols, ld, cp, rp, tc,
                       tiles, qr, sr, qc, sc);
  else if (qr)
    hipLaunchKernelGGL((mx_quant_kernel<BF16, VEC, true, false>), grid, dim3(256), 0, s, in, rows, cols, ld, cp, rp, tc,
                       tiles, qr, sr, qc, sc);
  else
    hipLaunchKernelGGL((mx_quant_kernel<BF16, VEC, false, true>), grid, dim3(256), 0, s, in, rows, cols, ld, cp, rp, tc,
                       tiles, qr, sr, qc, sc);
  return hipGetLastError();
}

hipError_t launch_mx_quant(const void* in, bool bf16, int64_t rows, int64_t cols, int64_t ld, uint8_t* qr, uint8_t* sr,
                           uint8_t* qc, uint8_t* sc, hipStream_t s) {
  const int64_t cp = mx_padded(cols), rp = mx_padded(rows);
  const int64_t tc = cp / kQTileC, tiles = rp / kQTileR * tc;
  const dim3 grid((unsigned)(tiles < kMxMaxGrid ? tiles : kMxMaxGrid));
  const bool vec = mx_vec_ok(in, ld, bf16 ? 2 : 4);
  if (bf16)
    return vec ? launch_mx_quant_t<true, true>(grid, s, in, rows, cols, ld, cp, rp, tc, tiles, qr, sr, qc, sc)
               : launch_mx_quant_t<true, false>(grid, s, in, rows, cols, ld, cp, rp, tc, tiles, qr, sr, qc, sc);
  return vec ? launch_mx_quant_t<false, true>(grid, s, in, rows, cols, ld, cp, rp, tc, tiles, qr, sr, qc, sc)
             : launch_mx_quant_t<false, false>(grid, s, in, rows, cols, ld, cp, rp, tc, tiles, qr, sr, qc, sc);
}

// E2M1 value of the low nibble of c.
__device__ __forceinline__ float e2m1_value(uint32_t c) {
  const uint32_t e = (c >> 1) & 3u, m = c & 1u;
  // exponent field 0: 0 or 0.5; else (1 + m/2) 2^(e-1)
  const uint32_t bits = e ? ((e + 126u) << 23) | (m << 22) : (m ? 0x3F000000u : 0u);
  return __uint_as_float(bits | ((c & 8u) << 28));
}

// 8 codes per thread.  value = E2M1 * 2^(b - 127): one or two significant
// bits and an exponent of at least -128, exact in fp32 and in bf16 (whose
// subnormals reach 2^-133), so the bf16 form is the fp32 value's upper half.
template <bool BF16, bool VEC>
__global__ __launch_bounds__(256) void mx_dequant_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ sc,
                                                         int64_t units, int64_t upr, int64_t cols, int64_t cp,
                                                         void* __restrict__ out, int64_t ld) {
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < units; u += (int64_t)gridDim.x * 256) {
    const int64_t row = u / upr, col = (u - row * upr) * 8;
    const uint32_t w = *(const uint32_t*)(q + row * (cp / 2) + col / 2);
    const uint32_t b = sc[row * (cp / 32) + col / 32];
    const float scale = b == 255u ? __uint_as_float(0x7FC00000u) : e8m0_value(b);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = e2m1_value(w >> (4 * i)) * scale;
    const int64_t at = row * ld + col;
    if constexpr (BF16) {
      uint16_t* p = (uint16_t*)out + at;
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        h[i] = (__float_as_uint(v[2 * i]) >> 16) | (__float_as_uint(v[2 * i + 1]) & 0xFFFF0000u);
      if (VEC && col + 8 <= cols) {
        *(uint4*)p = make_uint4(h[0], h[1], h[2], h[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (col + i < cols) p[i] = (uint16_t)(h[i / 2] >> (16 * (i & 1)));
      }
    } else {
      float* p = (float*)out + at;
      if (VEC && col + 8 <= cols) {
        *(float4*)p = make_float4(v[0], v[1], v[2], v[3]);
        *(float4*)(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (col + i < cols) p[i] = v[i];
      }
    }
  }
}

static hipError_t launch_mx_dequant(const uint8_t* q, const uint8_t* sc, int64_t rows, int64_t cols, bool bf16,
                                    void* out, int64_t ld, hipStream_t s) {
  const int64_t cp = mx_padded(cols), upr = (cols + 7) / 8, units = rows * upr, blocks = (units + 255) / 256;
  const dim3 grid((unsigned)(blocks < kMxMaxGrid ? blocks : kMxMaxGrid));
  const bool vec = mx_vec_ok(out, ld, bf16 ? 2 : 4);
  if (bf16 && vec)
    hipLaunchKernelGGL((mx_dequant_kernel<true, true>), grid, dim3(256), 0, s, q, sc, units, upr, cols, cp, out, ld);
  else if (bf16)
    hipLaunchKernelGGL((mx_dequant_kernel<true, false>), grid, dim3(256), 0, s, q, sc, units, upr, cols, cp, out, ld);
  else if (vec)
    hipLaunchKernelGGL((mx_dequant_kernel<false, true>), grid, dim3(256), 0, s, q, sc, units, upr, cols, cp, out, ld);
  else
    hipLaunchKernelGGL((mx_dequant_kernel<false, false>), grid, dim3(256), 0, s, q, sc, units, upr, cols, cp, out, ld);
  return hipGetLastError();
}

}  // namespace moe

extern "C" {

moe_status_t moe_mxfp4_quant(const void* in, int32_t in_dtype, int32_t rows, int32_t cols, int64_t ld_in, void* q_row,
                             void* s_row, void* q_col, void* s_col, void* stream) {
  if (!moe::mx_dtype_ok(in_dtype)) return MOE_ERR_UNSUPPORTED;
  if (!moe::mx_matrix_ok(rows, cols) || ld_in < cols) return MOE_ERR_SHAPE;
  if (!!q_row != !!s_row || !!q_col != !!s_col || (rows && cols && !q_row && !q_col)) return MOE_ERR_NULL;
  if (rows == 0 || cols == 0) return MOE_OK;
  if (!in) return MOE_ERR_NULL;
  if (!moe::mx_aligned(q_row, 16) || !moe::mx_aligned(s_row, 4) || !moe::mx_aligned(q_col, 16) ||
      !moe::mx_aligned(s_col, 4) || !moe::mx_aligned(in, in_dtype == MOE_DTYPE_BF16 ? 2 : 4))
    return MOE_ERR_ALIGN;
  return moe::mx_status(moe::launch_mx_quant(in, in_dtype == MOE_DTYPE_BF16, rows, cols, ld_in, (uint8_t*)q_row,
                                             (uint8_t*)s_row, (uint8_t*)q_col, (uint8_t*)s_col, (hipStream_t)stream));
}

moe_status_t moe_mxfp4_dequant(const void* q, const void* scales, int32_t rows, int32_t cols, int32_t out_dtype,
                               void* out, int64_t ld_out, void* stream) {
  if (!moe::mx_dtype_ok(out_dtype)) return MOE_ERR_UNSUPPORTED;
  if (!moe::mx_matrix_ok(rows, cols) || ld_out < cols) return MOE_ERR_SHAPE;
  if (rows == 0 || cols == 0) return MOE_OK;
  if (!q || !scales || !out) return MOE_ERR_NULL;
  if (!moe::mx_aligned(q, 16) || !moe::mx_aligned(scales, 4) ||
      !moe::mx_aligned(out, out_dtype == MOE_DTYPE_BF16 ? 2 : 4))
    return MOE_ERR_ALIGN;
  return moe::mx_status(moe::launch_mx_dequant((const uint8_t*)q, (const uint8_t*)scales, rows, cols,
                                               out_dtype == MOE_DTYPE_BF16, out, ld_out, (hipStream_t)stream));
}

}  // extern "C"
