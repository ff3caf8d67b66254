// Dense MXFP4 products on the FP4 matrix cores and their C ABI
// (moe_mxfp4_matmul, moe_mxfp4_linear, moe_mxfp4_linear_bwd).
//
//   out[m, n] (+)= sum_k deq(a)[m, k] deq(b)[n, k]
//
// Both operands are row-major codes [rows, Kp / 2] with scales [rows, Kp / 32],
// grouped along k, as moe_mxfp4_quant writes them.  The matrix instruction
// applies both scales itself and sums in fp32.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"
#include "moe_device.h"
#include "moe_mx.h"

namespace moe {

typedef float v16f __attribute__((ext_vector_type(16)));

struct MxMatmulArgs {
  const uint8_t *a, *as, *b, *bs;
  int64_t M, N, kb;  // kb: 128-wide K blocks
  void* out;
  int64_t ld;
  int32_t accumulate;
};

// 32x32x64 FP4 product with per-lane E8M0 scales (byte OP of sa and sb).
// Lane l holds row l % 32 of both operands, 32 values of the sum; the result
// lane l holds C[8 (i / 4) + 4 (l / 32) + i % 4][l % 32], i = 0..15.
template <int OP>
__device__ __forceinline__ v16f mfma_fp4_32(const uint4& a, const uint4& b, v16f c, uint32_t sa, uint32_t sb) {
  const v8i va = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const v8i vb = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(va, vb, c, 4, 4, OP, (int)sa, OP, (int)sb);
}

// One wave per 32 x 32 output tile.  b is the first operand, so a lane holds
// runs of four columns of one output row.  In a 128-wide K block lanes 0-31
// take the first 64 values and lanes 32-63 the last: the order of the sum is
// free as long as both operands share it.
template <bool BF16>
__global__ __launch_bounds__(256) void mx_matmul_simple_kernel(MxMatmulArgs p, int64_t tiles_n, int64_t tiles) {
  const int lane = threadIdx.x & 63, r = lane & 31, g = lane >> 5;
  for (int64_t tile = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); tile < tiles; tile += (int64_t)gridDim.x * 4) {
    const int64_t m0 = tile / tiles_n * 32, n0 = tile % tiles_n * 32;
    const int64_t m = min(m0 + r, p.M - 1), n = min(n0 + r, p.N - 1);  // rows past the end are read again
    const uint8_t* pa = p.a + m * p.kb * 64 + 32 * g;
    const uint8_t* pb = p.b + n * p.kb * 64 + 32 * g;
    const uint8_t* psa = p.as + m * p.kb * 4;
    const uint8_t* psb = p.bs + n * p.kb * 4;
    v16f c = {};
    for (int64_t k = 0; k < p.kb; ++k) {
      const uint32_t sa = *(const uint32_t*)(psa + k * 4) >> (16 * g), sb = *(const uint32_t*)(psb + k * 4) >> (16 * g);
      const uint4 a0 = *(const uint4*)(pa + k * 64), a1 = *(const uint4*)(pa + k * 64 + 16);
      const uint4 b0 = *(const uint4*)(pb + k * 64), b1 = *(const uint4*)(pb + k * 64 + 16);
      c = mfma_fp4_32<0>(b0, a0, c, sb, sa);
      c = mfma_fp4_32<1>(b1, a1, c, sb, sa);
    }
    if (m0 + r >= p.M) continue;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int64_t col = n0 + 8 * (i / 4) + 4 * g + i % 4;
      if (col >= p.N) continue;
      const int64_t at = (m0 + r) * p.ld + col;
      if constexpr (BF16)
        ((uint16_t*)p.out)[at] = f32_to_bf16(c[i]);
      else
        ((float*)p.out)[at] = p.accumulate ? ((float*)p.out)[at] + c[i] : c[i];
    }
  }
}

static hipError_t launch_mx_matmul(const MxMatmulArgs& p, bool bf16, hipStream_t s) {
  const int64_t tn = (p.N + 31) / 32, tiles = (p.M + 31) / 32 * tn, blocks = (tiles + 3) / 4;
  const dim3 grid((unsigned)(blocks < kMxMaxGrid ? blocks : kMxMaxGrid));
  if (bf16)
    hipLaunchKernelGGL((mx_matmul_simple_kernel<true>), grid, dim3(256), 0, s, p, tn, tiles);
  else
    hipLaunchKernelGGL((mx_matmul_simple_kernel<false>), grid, dim3(256), 0, s, p, tn, tiles);
  return hipGetLastError();
}

}  // namespace moe

namespace {

using moe::mx_aligned;
using moe::mx_padded;

size_t up256(int64_t v) { return (size_t)((v + 255) / 256 * 256); }
// Bytes of the codes and of the scales of a matrix grouped along `cols`.
size_t code_bytes(int64_t rows, int64_t cols) { return up256(rows * (mx_padded(cols) / 2)); }
size_t scale_bytes(int64_t rows, int64_t cols) { return up256(rows * (mx_padded(cols) / 32)); }
int esize(int32_t dtype) { return dtype == MOE_DTYPE_BF16 ? 2 : 4; }

bool product_ok(int64_t M, int64_t N, int64_t K) {
  return moe::mx_matrix_ok(M, K) && moe::mx_matrix_ok(N, K) && moe::mx_matrix_ok(M, N);
}

size_t matmul_bytes(int64_t, int64_t, int64_t) { return 0; }

moe_status_t run_matmul(int64_t M, int64_t N, int64_t K, const void* a, const void* as, const void* b, const void* bs,
                        int32_t out_dtype, void* out, int64_t ld_out, int32_t accumulate, hipStream_t s) {
  const moe::MxMatmulArgs p{(const uint8_t*)a, (const uint8_t*)as, (const uint8_t*)b, (const uint8_t*)bs, M, N,
                            mx_padded(K) / 128, out, ld_out, accumulate};
  return moe::mx_status(moe::launch_mx_matmul(p, out_dtype == MOE_DTYPE_BF16, s));
}

}  // namespace

extern "C" {

size_t moe_mxfp4_matmul_bytes(int32_t M, int32_t N, int32_t K) {
  return product_ok(M, N, K) ? matmul_bytes(M, N, K) : 0;
}

moe_status_t moe_mxfp4_matmul(int32_t M, int32_t N, int32_t K, const void* a, const void* a_scale, const void* b,
                              const void* b_scale, int32_t out_dtype, void* out, int64_t ld_out, int32_t accumulate,
                              void* ws, size_t ws_bytes, void* stream) {
  if (!moe::mx_dtype_ok(out_dtype) || (accumulate && out_dtype != MOE_DTYPE_F32)) return MOE_ERR_UNSUPPORTED;
  if (!product_ok(M, N, K) || ld_out < N) return MOE_ERR_SHAPE;
  if (M == 0 || N == 0) return MOE_OK;
  if (!out || (K > 0 && (!a || !a_scale || !b || !b_scale))) return MOE_ERR_NULL;
  if (!mx_aligned(a, 16) || !mx_aligned(b, 16) || !mx_aligned(a_scale, 4) || !mx_aligned(b_scale, 4) ||
      !mx_aligned(out, esize(out_dtype)))
    return MOE_ERR_ALIGN;
  const size_t need = matmul_bytes(M, N, K);
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  if (need && !ws) return MOE_ERR_NULL;
  if (need && !mx_aligned(ws, 16)) return MOE_ERR_ALIGN;
  return run_matmul(M, N, K, a, a_scale, b, b_scale, out_dtype, out, ld_out, accumulate, (hipStream_t)stream);
}

size_t moe_mxfp4_linear_bytes(int32_t M, int32_t N, int32_t K) {
  return product_ok(M, N, K) ? code_bytes(M, K) + scale_bytes(M, K) + matmul_bytes(M, N, K) : 0;
}

moe_status_t moe_mxfp4_linear(int32_t M, int32_t N, int32_t K, const void* x, int32_t x_dtype, int64_t ld_x,
                              const void* w, const void* w_scale, int32_t out_dtype, void* out, int64_t ld_out,
                              void* ws, size_t ws_bytes, void* stream) {
  if (!moe::mx_dtype_ok(x_dtype) || !moe::mx_dtype_ok(out_dtype)) return MOE_ERR_UNSUPPORTED;
  if (!product_ok(M, N, K) || ld_x < K || ld_out < N) return MOE_ERR_SHAPE;
  if (M == 0 || N == 0) return MOE_OK;
  if (!out || (K > 0 && (!x || !w || !w_scale))) return MOE_ERR_NULL;
  if (!mx_aligned(x, esize(x_dtype)) || !mx_aligned(w, 16) || !mx_aligned(w_scale, 4) ||
      !mx_aligned(out, esize(out_dtype)))
    return MOE_ERR_ALIGN;
  const size_t need = moe_mxfp4_linear_bytes(M, N, K);
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  if (need && !ws) return MOE_ERR_NULL;
  if (need && !mx_aligned(ws, 16)) return MOE_ERR_ALIGN;
  hipStream_t s = (hipStream_t)stream;
  uint8_t* xq = (uint8_t*)ws;
  uint8_t* xs = xq + code_bytes(M, K);
  if (K > 0) {
    const moe_status_t st =
        moe::mx_status(moe::launch_mx_quant(x, x_dtype == MOE_DTYPE_BF16, M, K, ld_x, xq, xs, nullptr, nullptr, s));
    if (st != MOE_OK) return st;
  }
  return run_matmul(M, N, K, xq, xs, w, w_scale, out_dtype, out, ld_out, 0, s);
}

size_t moe_mxfp4_linear_bwd_bytes(int32_t M, int32_t N, int32_t K) {
  if (!product_ok(M, N, K)) return 0;
  const size_t dx = matmul_bytes(M, K, N), dw = matmul_bytes(N, K, M);
  return code_bytes(M, N) + scale_bytes(M, N) + code_bytes(N, M) + scale_bytes(N, M) + (dx > dw ? dx : dw);
}

moe_status_t moe_mxfp4_linear_bwd(int32_t M, int32_t N, int32_t K, const void* dy, int32_t dy_dtype, int64_t ld_dy,
                                  const void* x_col, const void* x_col_scale, const void* w_col,
                                  const void* w_col_scale, int32_t dx_dtype, void* dx, int64_t ld_dx, float* dw,
                                  int64_t ld_dw, int32_t accumulate, void* ws, size_t ws_bytes, void* stream) {
  if (!moe::mx_dtype_ok(dy_dtype) || (dx && !moe::mx_dtype_ok(dx_dtype))) return MOE_ERR_UNSUPPORTED;
  if (!product_ok(M, N, K) || ld_dy < N || (dx && ld_dx < K) || (dw && ld_dw < K)) return MOE_ERR_SHAPE;
  if (K == 0 || (M == 0 && N == 0)) return MOE_OK;
  const bool want_dx = dx && M > 0, want_dw = dw && N > 0;
  if (!want_dx && !want_dw) return M > 0 && N > 0 ? MOE_ERR_NULL : MOE_OK;
  const bool dots = M > 0 && N > 0;  // else the sums are empty
  if (dots && (!dy || (want_dx && (!w_col || !w_col_scale)) || (want_dw && (!x_col || !x_col_scale))))
    return MOE_ERR_NULL;
  if (!mx_aligned(dy, esize(dy_dtype)) || !mx_aligned(x_col, 16) || !mx_aligned(x_col_scale, 4) ||
      !mx_aligned(w_col, 16) || !mx_aligned(w_col_scale, 4) || (dx && !mx_aligned(dx, esize(dx_dtype))) ||
      !mx_aligned(dw, 4))
    return MOE_ERR_ALIGN;
  const size_t need = moe_mxfp4_linear_bwd_bytes(M, N, K);
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  if (need && !ws) return MOE_ERR_NULL;
  if (need && !mx_aligned(ws, 16)) return MOE_ERR_ALIGN;
  hipStream_t s = (hipStream_t)stream;
  uint8_t* qr = (uint8_t*)ws;
  uint8_t* sr = qr + code_bytes(M, N);
  uint8_t* qc = sr + scale_bytes(M, N);
  uint8_t* sc = qc + code_bytes(N, M);
  moe_status_t st = MOE_OK;
  if (dots)
    st = moe::mx_status(moe::launch_mx_quant(dy, dy_dtype == MOE_DTYPE_BF16, M, N, ld_dy, want_dx ? qr : nullptr,
                                             want_dx ? sr : nullptr, want_dw ? qc : nullptr, want_dw ? sc : nullptr, s));
  if (st == MOE_OK && want_dx) st = run_matmul(M, K, N, qr, sr, w_col, w_col_scale, dx_dtype, dx, ld_dx, 0, s);
  if (st == MOE_OK && want_dw)
    st = run_matmul(N, K, M, qc, sc, x_col, x_col_scale, MOE_DTYPE_F32, dw, ld_dw, accumulate, s);
  return st;
}

}  // extern "C"
