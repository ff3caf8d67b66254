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
  int32_t vec;              // rows of out take 16-byte stores
  uint32_t tiles_m, tiles_n, pieces;
  int64_t piece_kb;         // K blocks of one piece of a split sum
  float* part;              // [pieces][M][N] partial sums
};

// Eight outputs of a row from element `at`, `left` of them inside it.  vec:
// 16-byte accesses are aligned.
template <bool BF16>
__device__ __forceinline__ void mx_store8(void* out, int64_t at, int64_t left, bool vec, bool accumulate,
                                          const float (&v)[8]) {
  if constexpr (BF16) {
    uint16_t* o = (uint16_t*)out + at;
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = f32_to_bf16(v[2 * i]) | (uint32_t)f32_to_bf16(v[2 * i + 1]) << 16;
    if (vec && left >= 8) {
      *(uint4*)o = make_uint4(h[0], h[1], h[2], h[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) o[i] = (uint16_t)(h[i / 2] >> (16 * (i & 1)));
    }
  } else {
    float* o = (float*)out + at;
    if (vec && left >= 8) {
      float4 a = make_float4(0, 0, 0, 0), b = a;
      if (accumulate) {
        a = *(const float4*)o;
        b = *(const float4*)(o + 4);
      }
      *(float4*)o = make_float4(a.x + v[0], a.y + v[1], a.z + v[2], a.w + v[3]);
      *(float4*)(o + 4) = make_float4(b.x + v[4], b.y + v[5], b.z + v[6], b.w + v[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) o[i] = accumulate ? o[i] + v[i] : v[i];
    }
  }
}

// LDS written by some lanes of a wave is read by others of the same wave: a
// wave's LDS operations complete in order, so ordering the compiler's view is
// all that is needed.
__device__ __forceinline__ void mx_wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// 32x32x64 FP4 product with per-lane E8M0 scales (byte OP of sa and sb).
// Lane l holds row l % 32 of both operands, 32 values of the sum; the result
// lane l holds C[8 (i / 4) + 4 (l / 32) + i % 4][l % 32], i = 0..15.
template <int OP>
__device__ __forceinline__ v16f mfma_fp4_32(const uint4& a, const uint4& b, v16f c, uint32_t sa, uint32_t sb) {
  const v8i va = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const v8i vb = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(va, vb, c, 4, 4, OP, (int)sa, OP, (int)sb);
}

// ---------------------------------------------------------------------------
// Tiled product.  A workgroup of 2 x 2 waves computes a (64 MT) x (64 NT) tile
// of out, a wave a (32 MT) x (32 NT) quarter in registers.  K advances in
// stages of 256: 128 bytes of codes per row, one whole cache line.
//
// A stage goes from memory straight to LDS (global_load_lds), two stages in
// LDS in turn.  A row's eight 16-byte pieces are stored rotated (piece c of
// row r in slot c ^ (r / 2) % 8), so that the 16 rows that a fragment read
// touches at a time fall on distinct banks; the rotation is applied to the
// per-lane source addresses, since the direct loads fill LDS in lane order.
//
// Fragments of one 128-wide half stage are multiplied while those of the next
// half are read, across stages too: by the middle of a stage every wave has
// read the whole of it, so one barrier there both publishes the next stage
// and frees this one's buffer for the loads of the stage after the next.
//
// b is the matrix instruction's first operand, so a lane holds runs of four
// columns of one output row.  In a 128-wide half, lanes 0-31 take the first 64
// values and lanes 32-63 the last (the order of the sum is free as long as
// both operands share it): a lane's two scale bytes are then neighbours.
// ---------------------------------------------------------------------------
template <int MT, int NT>
struct MxTile {
  static constexpr int BM = 64 * MT, BN = 64 * NT, ROWS = BM + BN;
  static constexpr int CODES = ROWS * 128;          // a rows, then b rows
  static constexpr int STAGE = CODES + ROWS * 8;    // scales: [half][row] dwords
  static constexpr int LDS = 2 * STAGE;
  static constexpr int CHUNKS = ROWS / 8 / 4;       // 1 KB loads (8 rows) per wave and stage
  static constexpr int SCALES = ROWS / 64 * 2 / 4;  // 256-byte scale loads per wave and stage (of 64 rows, one half)
  static_assert(ROWS % 128 == 0, "every wave issues the same number of loads");
};

#pragma clang diagnostic push
// M0 is reserved by the compiler, which cannot see these writes; nothing else
// in the library uses it (the test suite checks the built code).
#pragma clang diagnostic ignored "-Winline-asm"
// A wave-uniform pointer, stated as such.
__device__ __forceinline__ const uint8_t* mx_uniform(const uint8_t* p) {
  const uint64_t u = (uint64_t)p;
  // the builtin returns a signed int: widened as it is, a low word from 2^31
  // up would overwrite the high one
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)u);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(u >> 32));
  return (const uint8_t*)((uint64_t)hi << 32 | lo);
}
// 16 (4) bytes per lane from base + off to LDS at lds + 16 (4) * lane.
__device__ __forceinline__ void mx_dma16(const uint8_t* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(mx_uniform(base)), "s"(__builtin_amdgcn_readfirstlane(lds))
               : "memory", "m0");
}
__device__ __forceinline__ void mx_dma4(const uint8_t* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(off), "s"(mx_uniform(base)), "s"(__builtin_amdgcn_readfirstlane(lds))
               : "memory", "m0");
}
#pragma clang diagnostic pop

// Everything this wave has loaded and read has arrived, then all waves meet.
__device__ __forceinline__ void mx_wait_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

template <int MT, int NT, bool BF16>
__global__ __launch_bounds__(256, MT * NT >= 8 ? 1 : 2) void mx_tile_kernel(MxMatmulArgs p) {
  using T = MxTile<MT, NT>;
  extern __shared__ __align__(16) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, g = lane >> 5;
  const int wm = wave >> 1, wn = wave & 1;

  // the workgroup's tile and its share of K
  int64_t m0, n0;
  int piece;
  {
    // workgroups go round the 8 XCDs: each XCD gets a contiguous part of the
    // list, in which runs of GM tile rows share their b columns
    const uint32_t total = p.tiles_m * p.tiles_n * p.pieces, bid = blockIdx.x;
    const uint32_t per = total / 8, rest = total % 8, x = bid % 8;
    uint32_t i = x * per + min(x, rest) + bid / 8;
    const uint32_t tiles = p.tiles_m * p.tiles_n;
    piece = (int)(i / tiles);
    i -= piece * tiles;
    constexpr uint32_t GM = 8;
    const uint32_t band = i / (GM * p.tiles_n), first = band * GM;
    const uint32_t height = min(GM, p.tiles_m - first), j = i - band * GM * p.tiles_n;
    m0 = (int64_t)(first + j % height) * T::BM;
    n0 = (int64_t)(j / height) * T::BN;
  }
  const int64_t kb0 = (int64_t)piece * p.piece_kb;
  const int kb = (int)min(p.piece_kb, p.kb - kb0);  // 128-wide halves of this workgroup
  const int stages = (kb + 1) / 2;

  // Source offsets of this wave's loads, from the tile's first row.  Rows past
  // the matrix are read as its last row; their results are not stored.
  const uint8_t* base_a = p.a + (m0 * p.kb + kb0) * 64;
  const uint8_t* base_b = p.b + (n0 * p.kb + kb0) * 64;
  const uint8_t* base_as = p.as + (m0 * p.kb + kb0) * 4;
  const uint8_t* base_bs = p.bs + (n0 * p.kb + kb0) * 4;
  const int rows_a = (int)min((int64_t)T::BM, p.M - m0), rows_b = (int)min((int64_t)T::BN, p.N - n0);
  uint32_t off[T::CHUNKS], soff[T::SCALES];
#pragma unroll
  for (int q = 0; q < T::CHUNKS; ++q) {
    const int row = (wave * T::CHUNKS + q) * 8 + (lane >> 3);
    const uint32_t in = row < T::BM ? min(row, rows_a - 1) : min(row - T::BM, rows_b - 1);
    off[q] = in * (uint32_t)p.kb * 64u + (((lane & 7) ^ ((row >> 1) & 7)) * 16);
  }
#pragma unroll
  for (int q = 0; q < T::SCALES; ++q) {
    const int c = wave * T::SCALES + q, row = c / 2 * 64 + lane;
    const uint32_t in = row < T::BM ? min(row, rows_a - 1) : min(row - T::BM, rows_b - 1);
    soff[q] = in * (uint32_t)p.kb * 4u + (c & 1) * 4;
  }
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)lds);

  // Loads of stage st.  In a last stage of one half the other half's bytes
  // lie past the row: the first half is loaded twice and not used again.
  auto issue = [&](int st) {
    const uint32_t to = lds0 + (st & 1) * T::STAGE;
    const bool single = 2 * st + 1 >= kb;
#pragma unroll
    for (int q = 0; q < T::CHUNKS; ++q) {
      const int c = wave * T::CHUNKS + q;
      const uint8_t* base = (c * 8 < T::BM ? base_a : base_b) + (int64_t)st * 128;
      // a lane's piece lies in the second half where bit 2 of its slot differs
      // from bit 2 of the rotation, which is bit 0 of c
      mx_dma16(base, single ? off[q] - (((lane ^ (c << 2)) & 4) << 4) : off[q], to + c * 1024);
    }
#pragma unroll
    for (int q = 0; q < T::SCALES; ++q) {
      const int c = wave * T::SCALES + q;
      const uint8_t* base = (c / 2 * 64 < T::BM ? base_as : base_bs) + (int64_t)st * 8;
      mx_dma4(base, single && (c & 1) ? soff[q] - 4 : soff[q], to + T::CODES + ((c & 1) * T::ROWS + c / 2 * 64) * 4);
    }
  };

  v16f acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = v16f{};

  // Fragments of a 128-wide half u (both 64-wide steps): all b tiles of the
  // half, the a tiles two ahead.
  struct Frag {
    uint4 v[2];
    uint32_t s;
  };
  Frag fb[NT], nb[NT], fa[MT + 1];
  const int swz = (r >> 1) & 7;
  auto read = [&](Frag& f, int row, int u) {
    const int h = u & 1;
    const uint8_t* buf = lds + ((u >> 1) & 1) * T::STAGE;
    f.v[0] = *(const uint4*)(buf + row * 128 + ((4 * h + 2 * g) ^ swz) * 16);
    f.v[1] = *(const uint4*)(buf + row * 128 + ((4 * h + 2 * g + 1) ^ swz) * 16);
    f.s = *(const uint32_t*)(buf + T::CODES + (h * T::ROWS + row) * 4) >> (16 * g);
  };
  const int row_a = wm * MT * 32 + r, row_b = T::BM + wn * NT * 32 + r;
  // One half.  The next half's b tiles and first a tile are read during the
  // last tile rows (past the last half: whatever LDS holds, not used).  Where
  // that half lies in the next stage (publish), the stage has to have arrived
  // first, for all waves, and this stage's buffer is free from then on.
  constexpr int kLead = MT >= 2 ? 2 : 1;  // tile rows that cover the next half's reads
  auto half = [&](int u, bool publish) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if (i < MT - 1 && i <= MT - kLead) read(fa[i + 1], row_a + (i + 1) * 32, u);
      if (i == MT - kLead) {
        // every a tile of this half is in registers or on the way
        if (publish) {
          mx_wait_barrier();
          const int st = (u >> 1) + 2;
          if (st < stages) issue(st);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) read(nb[j], row_b + j * 32, u + 1);
        read(fa[MT], row_a, u + 1);
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = mfma_fp4_32<0>(fb[j].v[0], fa[i].v[0], acc[i][j], fb[j].s, fa[i].s);
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = mfma_fp4_32<1>(fb[j].v[1], fa[i].v[1], acc[i][j], fb[j].s, fa[i].s);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) fb[j] = nb[j];
    fa[0] = fa[MT];
  };

  if (stages > 0) {
    issue(0);
    mx_wait_barrier();
    if (stages > 1) issue(1);
#pragma unroll
    for (int j = 0; j < NT; ++j) read(fb[j], row_b + j * 32, 0);
    read(fa[0], row_a, 0);
#pragma unroll 1
    for (int u = 0; u < kb; ++u) half(u, u & 1);
  }
  // every wave is done with the stage buffers, which the tile now goes through
  // on its way out; the matrix core's last results are written before they
  // are read
  mx_wait_barrier();
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);

  // A wave turns 32 rows at a time from the lanes' runs of four columns into
  // whole rows: 16-byte unit c of row r lies in place c ^ (r % units), so that
  // neither side's accesses collide.
  constexpr int UNITS = 8 * NT;  // of four fp32 values, per row of a wave's tile
  float4* turn = (float4*)(lds + wave * 32 * UNITS * 16);
  static_assert(4 * 32 * UNITS * 16 <= T::LDS, "the tile rows fit the stage buffers");
  const int64_t n_wave = n0 + wn * NT * 32;
  float* part = p.part + (int64_t)piece * p.M * p.N;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        turn[r * UNITS + ((j * 8 + 2 * q + g) ^ (r & (UNITS - 1)))] =
            make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
    mx_wave_lds_sync();
    const int64_t m_wave = m0 + (wm * MT + i) * 32;
#pragma unroll 2
    for (int t = lane; t < 32 * UNITS / 2; t += 64) {
      const int row = t / (UNITS / 2), c = t % (UNITS / 2) * 2;
      const float4 x = turn[row * UNITS + (c ^ (row & (UNITS - 1)))], y = turn[row * UNITS + ((c + 1) ^ (row & (UNITS - 1)))];
      const int64_t m = m_wave + row, n = n_wave + c * 4;
      if (m < p.M) {
        const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        if (p.pieces > 1)
          mx_store8<false>(part, m * p.N + n, p.N - n, p.N % 4 == 0, false, v);
        else
          mx_store8<BF16>(p.out, m * p.ld + n, p.N - n, p.vec, p.accumulate, v);
      }
    }
    mx_wave_lds_sync();
  }
}

// out (+)= the pieces' sums, added in piece order.
template <bool BF16>
__global__ __launch_bounds__(256) void mx_join_kernel(MxMatmulArgs p) {
  const int64_t groups = (p.N + 7) / 8, total = p.M * groups;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < total; u += (int64_t)gridDim.x * 256) {
    const int64_t m = u / groups, n = (u - m * groups) * 8;
    float v[8] = {};
    const float* src = p.part + m * p.N + n;
    for (int k = 0; k < (int)p.pieces; ++k, src += p.M * p.N) {
      if (p.N % 8 == 0) {
        const float4 a = *(const float4*)src, b = *(const float4*)(src + 4);
        v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
        v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (n + i < p.N) v[i] += src[i];
      }
    }
    mx_store8<BF16>(p.out, m * p.ld + n, p.N - n, p.vec, p.accumulate, v);
  }
}

// The tile and the split of K for a product.
struct MxPlan {
  int mt, nt, pieces;
  int64_t piece_kb;
};
static MxPlan mx_plan(int64_t M, int64_t N, int64_t kb) {
  static const int kTiles[][2] = {{4, 4}, {2, 4}, {2, 2}, {1, 1}};
  MxPlan best{1, 1, 1, kb};
  for (const auto& t : kTiles) {
    const int64_t tiles = ((M + 64 * t[0] - 1) / (64 * t[0])) * ((N + 64 * t[1] - 1) / (64 * t[1]));
    best = {t[0], t[1], 1, kb};
    if (tiles >= 192) break;
  }
  return best;
}

template <int MT, int NT>
static hipError_t launch_mx_tile(const MxMatmulArgs& p, bool bf16, hipStream_t s) {
  const auto run = [&](auto kernel) {
    const hipError_t e =
        hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, MxTile<MT, NT>::LDS);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3(p.tiles_m * p.tiles_n * p.pieces), dim3(256), (MxTile<MT, NT>::LDS), s, p);
    return hipGetLastError();
  };
  return bf16 ? run(mx_tile_kernel<MT, NT, true>) : run(mx_tile_kernel<MT, NT, false>);
}

static hipError_t launch_mx_matmul(MxMatmulArgs p, bool bf16, hipStream_t s) {
  const MxPlan plan = mx_plan(p.M, p.N, p.kb);
  p.pieces = plan.pieces;
  p.piece_kb = plan.piece_kb;
  p.tiles_m = (uint32_t)((p.M + 64 * plan.mt - 1) / (64 * plan.mt));
  p.tiles_n = (uint32_t)((p.N + 64 * plan.nt - 1) / (64 * plan.nt));
  p.vec = mx_vec_ok(p.out, p.ld, bf16 ? 2 : 4);
  hipError_t e = plan.nt == 4 ? (plan.mt == 4 ? launch_mx_tile<4, 4>(p, bf16, s) : launch_mx_tile<2, 4>(p, bf16, s))
                 : plan.nt == 2 ? launch_mx_tile<2, 2>(p, bf16, s)
                                : launch_mx_tile<1, 1>(p, bf16, s);
  if (e != hipSuccess || plan.pieces == 1) return e;
  const int64_t blocks = (p.M * ((p.N + 7) / 8) + 255) / 256;
  const dim3 grid((unsigned)(blocks < kMxMaxGrid ? blocks : kMxMaxGrid));
  if (bf16)
    hipLaunchKernelGGL(mx_join_kernel<true>, grid, dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL(mx_join_kernel<false>, grid, dim3(256), 0, s, p);
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
  moe::MxMatmulArgs p{};
  p.a = (const uint8_t*)a;
  p.as = (const uint8_t*)as;
  p.b = (const uint8_t*)b;
  p.bs = (const uint8_t*)bs;
  p.M = M;
  p.N = N;
  p.kb = mx_padded(K) / 128;
  p.out = out;
  p.ld = ld_out;
  p.accumulate = accumulate;
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
