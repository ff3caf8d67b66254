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

// Columns, or rows and columns: one workgroup quantises a tile of 128 x 128.  A
// thread loads 16 bytes of each of 8 rows, all of them in flight; a row group of
// 32 values is 4 (bf16) or 8 (fp32) neighbouring lanes.  For the column groups
// the tile goes through LDS as it is, and a thread takes a dword column of it
// (two bf16 columns or one fp32 column) over 32 rows.  Codes of columns are
// gathered in LDS so that a column's 64 bytes leave together.
//
// Bound by memory, on one MI355X: a 2048 x 4096 fp32 matrix both ways 11.8 us (42
// MB: 3.6 TB/s, where a copy of 1 GiB reaches 5.05), 16384 x 4096 bf16 both ways 47
// us (4.3 TB/s), along its rows alone 28.7 (5.9 TB/s, much of it in the last
// level's cache).
//
// The kernels here take their arguments as one struct: each argument of its own
// costs the host 0.1 us of a launch.
struct MxQuantArgs {
  const void* in;
  int64_t rows, cols, ld, cp, rp, tiles_c, tiles;
  uint8_t *q_row, *s_row, *q_col, *s_col;
};
constexpr int kQTileR = 128;
constexpr int quant_threads(bool bf16) { return bf16 ? 256 : 512; }

// Sixteen bytes of a row: 8 bf16 or 4 fp32 values from element `at`, `left` of
// them inside the row (the others are zero).
template <bool BF16>
__device__ __forceinline__ uint4 mx_load16(const void* in, int64_t at, int64_t left) {
  if constexpr (BF16) {
    const uint16_t* p = (const uint16_t*)in + at;
    if (left >= 8) return mx_read16(p);
    uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) u[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
    return make_uint4(u[0], u[1], u[2], u[3]);
  } else {
    const uint32_t* p = (const uint32_t*)in + at;
    if (left >= 4) return mx_read16(p);
    return make_uint4(left > 0 ? p[0] : 0u, left > 1 ? p[1] : 0u, left > 2 ? p[2] : 0u, 0u);
  }
}

// The codes of one 16-byte load and the scale bytes of the 16 lanes around it,
// 4 (bf16) or 2 (fp32) groups along a row.  bf16: eight codes; fp32: even lanes
// get eight, the next lane's too.
template <bool BF16>
__device__ __forceinline__ void mx_row_group(const uint4& x, int lane, uint32_t& w, uint32_t& sw) {
  uint32_t b;  // the group's scale
  if constexpr (BF16) {
    b = mx_scale_byte(mx_group_max4(mx_amax_bf16(x)));
    w = mx_codes_bf16(x, b);
    sw = b << (8 * (lane % 16 / 4));
    sw |= mx_row_half_mirror(sw);
  } else {
    const uint32_t a = mx_group_max4(mx_amax_f32(x));
    b = mx_scale_byte(max(a, mx_row_half_mirror(a)));
    w = mx_codes_f32(x, b);
    w |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, 0xB1, 0xF, 0xF, false) << 16;
    sw = b << (8 * (lane % 16 / 8));
  }
  sw |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)sw, 0x140, 0xF, 0xF, false);  // row_mirror
}

template <bool BF16, bool ROW>
__global__ __launch_bounds__(quant_threads(BF16)) void mx_quant_kernel(MxQuantArgs p) {
  constexpr int TC = 128, THREADS = quant_threads(BF16);
  constexpr int V = BF16 ? 8 : 4;          // values of a load
  constexpr int TPR = TC / V;              // threads of a row: 16 or 32
  constexpr int RPP = THREADS / TPR;       // rows of a pass: 16
  constexpr int PASSES = kQTileR / RPP;    // 8
  constexpr int DC = TC * (BF16 ? 2 : 4) / 4;  // dword columns
  constexpr int LD = DC + 1;  // LDS row stride in dwords: odd, so a column walks the banks
  __shared__ uint32_t buf[kQTileR * LD];
  __shared__ uint4 codes[TC * 4];
  __shared__ uint32_t cscale[TC];
  const void* __restrict__ in = p.in;
  uint8_t* __restrict__ q_row = p.q_row;
  uint8_t* __restrict__ s_row = p.s_row;
  uint8_t* __restrict__ q_col = p.q_col;
  uint8_t* __restrict__ s_col = p.s_col;
  const int64_t rows = p.rows, cols = p.cols, ld = p.ld, cp = p.cp, rp = p.rp, tiles_c = p.tiles_c, tiles = p.tiles;
  const int t = threadIdx.x;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t r0 = tile / tiles_c * kQTileR, c0 = tile % tiles_c * TC;
    const int lc = t % TPR, lr0 = t / TPR;
    const int64_t col = c0 + lc * V;
    uint4 x[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int64_t row = r0 + lr0 + RPP * i;
      x[i] = row < rows ? mx_load16<BF16>(in, row * ld + col, cols - col) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int64_t row = r0 + lr0 + RPP * i;
      if constexpr (ROW) {
        uint32_t w, sw;
        mx_row_group<BF16>(x[i], lc, w, sw);
        if (row < rows) {
          if (BF16 || lc % 2 == 0) *(uint32_t*)(q_row + row * (cp / 2) + col / 2) = w;
          if (lc % 16 == 0) {
            uint8_t* sr = s_row + row * (cp / 32) + col / 32;
            if constexpr (BF16)
              *(uint32_t*)sr = sw;
            else
              *(uint16_t*)sr = (uint16_t)sw;
          }
        }
      }
      uint32_t* to = buf + (lr0 + RPP * i) * LD + lc * 4;
      to[0] = x[i].x; to[1] = x[i].y; to[2] = x[i].z; to[3] = x[i].w;
    }
    __syncthreads();
    {
      // dword column t % DC, rows 32 (t / DC) .. +32
      const int dc = t % DC, rg = t / DC;
      const uint32_t* from = buf + rg * 32 * LD + dc;
      uint32_t v[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = from[j * LD];
      if constexpr (BF16) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) m = mx_max_u16x2(m, v[j] & 0x7FFF7FFFu);
        const uint32_t b0 = mx_scale_byte(m << 16), b1 = mx_scale_byte(m & 0xFFFF0000u);
        uint32_t w0[4], w1[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t lo[4], hi[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t e = v[8 * q + 2 * j], o = v[8 * q + 2 * j + 1];
            lo[j] = __builtin_amdgcn_perm(o, e, 0x05040100);  // the two rows' first columns
            hi[j] = __builtin_amdgcn_perm(o, e, 0x07060302);  // ... second columns
          }
          w0[q] = mx_codes_bf16(make_uint4(lo[0], lo[1], lo[2], lo[3]), b0);
          w1[q] = mx_codes_bf16(make_uint4(hi[0], hi[1], hi[2], hi[3]), b1);
        }
        codes[(2 * dc) * 4 + rg] = make_uint4(w0[0], w0[1], w0[2], w0[3]);
        codes[(2 * dc + 1) * 4 + rg] = make_uint4(w1[0], w1[1], w1[2], w1[3]);
        ((uint8_t*)cscale)[(2 * dc) * 4 + rg] = (uint8_t)b0;
        ((uint8_t*)cscale)[(2 * dc + 1) * 4 + rg] = (uint8_t)b1;
      } else {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) m = max(m, v[j] & 0x7FFFFFFFu);
        const uint32_t b = mx_scale_byte(m);
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          w[q] = mx_codes_f32(make_uint4(v[8 * q], v[8 * q + 1], v[8 * q + 2], v[8 * q + 3]), b);
          w[q] |= mx_codes_f32(make_uint4(v[8 * q + 4], v[8 * q + 5], v[8 * q + 6], v[8 * q + 7]), b) << 16;
        }
        codes[dc * 4 + rg] = make_uint4(w[0], w[1], w[2], w[3]);
        ((uint8_t*)cscale)[dc * 4 + rg] = (uint8_t)b;
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = t; u < TC * 4; u += THREADS) {
      const int c = u >> 2, rg = u & 3;
      const int64_t gc = c0 + c;
      if (gc < cols) {
        *(uint4*)(q_col + gc * (rp / 2) + r0 / 2 + rg * 16) = codes[u];
        if (rg == 0) *(uint32_t*)(s_col + gc * (rp / 32) + r0 / 32) = cscale[c];
      }
    }
  }
}

// Rows only: the matrix as one list of 16-byte loads, padding included, since
// codes and scales lie one behind the other whatever the row.  A thread has P
// loads 256 apart in flight; a row's groups never straddle 16 lanes.
template <bool BF16, int P>
__global__ __launch_bounds__(256) void mx_quant_rows_kernel(MxQuantArgs p) {
  constexpr int V = BF16 ? 8 : 4;
  const int64_t per_row = p.cp / V, total = p.rows * per_row;
  const int t = threadIdx.x;
  for (int64_t base = (int64_t)blockIdx.x * (256 * P); base < total; base += (int64_t)gridDim.x * (256 * P)) {
    const int64_t row0 = base / per_row;
    uint4 x[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      // (per_row is at most 2^22, what is left of the row below it)
      const uint32_t at = (uint32_t)(base - row0 * per_row) + i * 256 + t;
      const uint32_t down = at / (uint32_t)per_row;
      const int64_t row = row0 + down, col = (int64_t)(at - down * (uint32_t)per_row) * V;
      x[i] = row < p.rows ? mx_load16<BF16>(p.in, row * p.ld + col, p.cols - col) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int64_t unit = base + i * 256 + t;
      uint32_t w, sw;
      mx_row_group<BF16>(x[i], t, w, sw);
      if (unit >= total) continue;
      if constexpr (BF16) {
        *(uint32_t*)(p.q_row + unit * 4) = w;
        if (t % 16 == 0) *(uint32_t*)(p.s_row + unit / 4) = sw;
      } else {
        if (t % 2 == 0) *(uint32_t*)(p.q_row + unit * 2) = w;
        if (t % 16 == 0) *(uint16_t*)(p.s_row + unit / 8) = (uint16_t)sw;
      }
    }
  }
}

template <bool BF16>
static hipError_t launch_mx_quant_t(hipStream_t s, const void* in, int64_t rows, int64_t cols, int64_t ld, uint8_t* qr,
                                    uint8_t* sr, uint8_t* qc, uint8_t* sc) {
  const int64_t cp = mx_padded(cols), rp = mx_padded(rows);
  const int64_t tc = cp / 128, tiles = rp / kQTileR * tc;
  const dim3 grid((unsigned)(tiles < kMxMaxGrid ? tiles : kMxMaxGrid));
  const MxQuantArgs args{in, rows, cols, ld, cp, rp, tc, tiles, qr, sr, qc, sc};
  const auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(quant_threads(BF16)), 0, s, args);
    return hipGetLastError();
  };
  if (!qc) {
    const int64_t loads = rows * (cp / (BF16 ? 8 : 4));
    const auto rows_only = [&](auto kernel, int per_block) {
      const int64_t blocks = (loads + per_block - 1) / per_block;
      const dim3 g((unsigned)(blocks < kMxMaxGrid ? blocks : kMxMaxGrid));
      hipLaunchKernelGGL(kernel, g, dim3(256), 0, s, args);
      return hipGetLastError();
    };
    // 1, 2 or 4 loads per thread, us: 64 x 4096 bf16 (2^15 loads) 2.1, 2.5, 3.1;
    // 333 x 4000 (2^17.4) 2.8, 3.0, 3.7; 2048 x 4096 (2^20) 6.0, 5.6, 6.0; 4096 x
    // 4096 9.3, 8.6, 8.9; 16384 x 4096 (2^23) 34.8, 30.9, 28.7 (8: 30.3)
    if (loads < 1 << 18) return rows_only(mx_quant_rows_kernel<BF16, 1>, 256);
    if (loads < 1 << 22) return rows_only(mx_quant_rows_kernel<BF16, 2>, 512);
    return rows_only(mx_quant_rows_kernel<BF16, 4>, 1024);
  }
  return qr ? run(mx_quant_kernel<BF16, true>) : run(mx_quant_kernel<BF16, false>);
}

hipError_t launch_mx_quant(const void* in, bool bf16, int64_t rows, int64_t cols, int64_t ld, uint8_t* qr, uint8_t* sr,
                           uint8_t* qc, uint8_t* sc, hipStream_t s) {
  return bf16 ? launch_mx_quant_t<true>(s, in, rows, cols, ld, qr, sr, qc, sc)
              : launch_mx_quant_t<false>(s, in, rows, cols, ld, qr, sr, qc, sc);
}

// A workgroup takes 64 rows x 128 columns, a thread 8 codes of four rows.
// value = E2M1 * 2^(b - 127): one or two significant bits and an exponent of at
// least -128, exact in fp32 and in bf16 (whose subnormals reach 2^-133), so the
// bf16 form is the fp32 value's upper half.  The hardware conversion gives the
// E2M1 value; the scale is a product of its own, since its smallest results
// are fp32 subnormals.
struct MxDequantArgs {
  const uint8_t *q, *sc;
  int64_t rows, cols, cp, tiles;
  void* out;
  int64_t ld;
};
constexpr int kDqRows = 64;
template <bool BF16>
__global__ __launch_bounds__(256) void mx_dequant_kernel(MxDequantArgs a) {
  const uint8_t* __restrict__ q = a.q;
  const uint8_t* __restrict__ sc = a.sc;
  void* __restrict__ out = a.out;
  const int64_t rows = a.rows, cols = a.cols, cp = a.cp, tiles = a.tiles, ld = a.ld, tiles_c = cp / 128;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t row0 = tile / tiles_c * kDqRows + threadIdx.x / 16, col = tile % tiles_c * 128 + threadIdx.x % 16 * 8;
    const int left = (int)min(cols - col, (int64_t)8);
    if (left <= 0) continue;
    uint32_t w[kDqRows / 16], b[kDqRows / 16];
#pragma unroll
    for (int i = 0; i < kDqRows / 16; ++i) {
      const int64_t row = min(row0 + 16 * i, rows - 1);
      w[i] = *(const uint32_t*)(q + row * (cp / 2) + col / 2);
      b[i] = sc[row * (cp / 32) + col / 32];
    }
#pragma unroll
    for (int i = 0; i < kDqRows / 16; ++i) {
      const int64_t row = row0 + 16 * i;
      if (row >= rows) break;
      const float scale = b[i] == 255u ? __uint_as_float(0x7FC00000u) : e8m0_value(b[i]);
      float v[8];
      mx_values8(w[i], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= scale;
      if constexpr (BF16) {
        uint16_t* p = (uint16_t*)out + row * ld + col;
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          h[j] = __builtin_amdgcn_perm(__float_as_uint(v[2 * j + 1]), __float_as_uint(v[2 * j]), 0x07060302);
        if (left == 8) {
          mx_write16(p, make_uint4(h[0], h[1], h[2], h[3]));
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < left) p[j] = (uint16_t)(h[j / 2] >> (16 * (j & 1)));
        }
      } else {
        float* p = (float*)out + row * ld + col;
        if (left == 8) {
          mx_write16(p, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
          mx_write16(p + 4, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < left) p[j] = v[j];
        }
      }
    }
  }
}

static hipError_t launch_mx_dequant(const uint8_t* q, const uint8_t* sc, int64_t rows, int64_t cols, bool bf16,
                                    void* out, int64_t ld, hipStream_t s) {
  const int64_t cp = mx_padded(cols), tiles = (rows + kDqRows - 1) / kDqRows * (cp / 128);
  const dim3 grid((unsigned)(tiles < kMxMaxGrid ? tiles : kMxMaxGrid));
  const MxDequantArgs args{q, sc, rows, cols, cp, tiles, out, ld};
  if (bf16)
    hipLaunchKernelGGL((mx_dequant_kernel<true>), grid, dim3(256), 0, s, args);
  else
    hipLaunchKernelGGL((mx_dequant_kernel<false>), grid, dim3(256), 0, s, args);
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
