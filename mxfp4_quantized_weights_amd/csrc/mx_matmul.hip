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

#include <type_traits>

#include "../../include/moe.h"
#include "moe_device.h"
#include "moe_mx.h"

namespace moe {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
// At any element's address (as v4u_any).
typedef uint32_t v2u_any __attribute__((ext_vector_type(2), aligned(2)));
typedef float v4f_any __attribute__((ext_vector_type(4), aligned(2)));

struct MxMatmulArgs {
  const uint8_t *a, *as, *b, *bs;
  int64_t M, N, kb;         // kb: 128-wide K blocks
  const void* x;            // mx_few_kernel: a as values [M, K], row stride ld_x
  int64_t K, ld_x;
  void* out;
  int64_t ld;
  int32_t accumulate;
  uint32_t tiles_m, tiles_n, pieces;
  int64_t piece_kb;         // K blocks of one piece of a split sum
  int64_t piece_bytes;      // between the pieces' outputs
};

// Two fp32 values rounded to bf16 (nearest even; the hardware conversion).
__device__ __forceinline__ uint32_t mx_bf16x2(float a, float b) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  const v2bf h = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, h);
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
__device__ __forceinline__ v16f mfma_fp4_32(const v4u& a, const v4u& b, v16f c, uint32_t sa, uint32_t sb) {
  const v8i va = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const v8i vb = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
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
// The two stages' loads of 8 rows (1 KB) alternate, so that either is an
// immediate away in a read's address.
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
//
// The 256-wide tiles take a compute unit's registers and LDS whole, so nothing
// else could run while one starts or ends: there a workgroup walks over several
// tiles, and the next one's first two stages load while the last one's results
// are written.
//
// What bounds it, on one MI355X: power first.  16384 x 8192 x 4096 in 260 us is
// 4.2 PFLOP/s, with the clock at 1.8 GHz and the matrix cores busy for 58% of
// its cycles; all zeros run at 2.45 GHz, 197 us.  Of a 256-wide tile's 58000
// cycles 33000 are matrix instructions; without loads, results and their
// turning the same loop takes 45000.  The 128-wide tiles, two workgroups to a
// compute unit, are bound by L2: 4096 x 2048 x 4096 in 22.9 us brings in 58 B/ns
// per compute unit, 14.8 TB/s in all.
// ---------------------------------------------------------------------------
template <int MT, int NT>
struct MxTile {
  static constexpr int BM = 64 * MT, BN = 64 * NT, ROWS = BM + BN;
  static constexpr int CODES = ROWS * 128;            // one stage's codes: a rows, then b rows
  static constexpr int GROUP = ROWS * 16;             // scales of two stages: [row][four halves' dwords]
  static constexpr int CHUNKS = ROWS / 8 / 4;         // 1 KB loads (8 rows) per wave and stage
  static constexpr int SCALES = (ROWS / 64 + 3) / 4;  // 1 KB scale loads (64 rows) per wave and two stages
  static constexpr int BUFFERS = 2 * (CODES + GROUP);
  static constexpr bool WALKS = MT >= 4;              // a workgroup computes several tiles, one after the other
  static constexpr int TURN = WALKS ? BUFFERS : 0;    // where the results are turned: 4 KB per wave
  static constexpr int LDS = WALKS ? BUFFERS + 16384 : BUFFERS + 64;  // (scale reads past the last half reach up to 40 bytes over)
  static_assert(MT == NT && BUFFERS >= 16384 && LDS <= 163840, "waves 0, 1 load a's codes, 2, 3 b's; room for the turned rows");
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
// 16 bytes per lane from base + off to LDS at lds + at + 16 * lane.  (The sum is
// formed here: as a value of its own each load's would be kept in a register.)
__device__ __forceinline__ void mx_dma16(const uint8_t* base, uint32_t off, uint32_t lds, int at) {
  uint32_t to;
  asm volatile("s_add_u32 %0, %3, %4\n\ts_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               : "=&s"(to)
               : "v"(off), "s"(mx_uniform(base)), "s"(__builtin_amdgcn_readfirstlane(lds)), "i"(at)
               : "memory", "m0", "scc");
}
// The same for all lanes or none (`lanes` -1 or 0).  Every lane of the wave is
// active here, before and after.
__device__ __forceinline__ void mx_dma16_if(const uint8_t* base, uint32_t off, uint32_t lds, int at, int lanes) {
  uint32_t to;
  asm volatile(
      "s_add_u32 %0, %3, %4\n\ts_mov_b32 exec_lo, %5\n\ts_mov_b32 exec_hi, %5\n\ts_mov_b32 m0, %0\n\ts_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2\n\ts_mov_b64 exec, -1"
      : "=&s"(to)
      : "v"(off), "s"(mx_uniform(base)), "s"(__builtin_amdgcn_readfirstlane(lds)), "i"(at),
        "s"(__builtin_amdgcn_readfirstlane(lanes))
      : "memory", "m0", "scc");
}
#pragma clang diagnostic pop

// From LDS at byte address at + off (off folds into the instruction).
template <typename V>
__device__ __forceinline__ V lds_read(uint32_t at, int off) {
  return *(const __attribute__((address_space(3))) V*)((const __attribute__((address_space(3))) uint8_t*)(uintptr_t)at + off);
}

// Everything this wave has loaded and read has arrived, then all waves meet.
__device__ __forceinline__ void mx_wait_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// A wave's (32 MT) x (32 NT) results, from row m0 and column n0 on, to out
// [M, N] (row stride ld).  Blocks of 32 rows x 128 bytes are turned in 4 KB of
// the wave's own LDS from the lanes' runs of four columns into whole rows:
// 16-byte unit c of row r lies in place c ^ (r % 8), so that neither side's
// accesses collide.  A whole tile leaves in stores of 1 KB, 2 MT NT of bf16 or
// 4 MT NT of fp32 results, that nobody waits for; else (ragged tiles, and sums
// added to out) everything has been written on return.
template <int MT, int NT, bool BF16>
__device__ __forceinline__ void mx_write_tile(const v16f (&acc)[MT][NT], uint8_t* turn, void* out, int64_t ld, bool accumulate,
                                              int64_t m0, int64_t n0, int64_t M, int64_t N) {
  constexpr int E = BF16 ? 2 : 4;                  // bytes of an element
  constexpr int W = NT * 32 * E < 128 ? NT * 32 * E : 128;  // bytes of a block's row
  constexpr int JN = W / E / 32;                   // 32-column tiles of a block
  constexpr int UNITS = W / 16, ROWS = 64 / UNITS, LOADS = 32 / ROWS;  // a load: ROWS rows, 1 KB
  constexpr int BLOCKS = MT * NT / JN;
  static_assert(ROWS % UNITS == 0, "the rotation is the same in every load");
  uint32_t lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));  // the addresses are worked out here, not kept in registers from tile to tile
  const uint32_t r = lane & 31, g = lane >> 5;
  const uint32_t row0 = lane / UNITS, c0 = lane % UNITS;
  const int rows = (int)min((int64_t)32 * MT, M - m0), cols = (int)min((int64_t)32 * NT, N - n0);
  uint8_t* to = (uint8_t*)out + ((m0 + row0) * ld + n0) * E + c0 * 16;  // the lane's units, block by block
  const uint8_t* from = turn + (row0 * UNITS + (c0 ^ (row0 & (UNITS - 1)))) * 16;
  const int64_t step = ROWS * E * ld;
  typedef typename std::conditional<BF16, uint2, float4>::type Run;  // four columns
  auto pack = [&](int b, Run (&v)[JN * 4]) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < JN * 4; ++q) {
      const v16f& a = acc[b * JN / NT][b * JN % NT + q / 4];
      const int e = 4 * (q % 4);
      if constexpr (BF16)
        v[q] = make_uint2(mx_bf16x2(a[e], a[e + 1]), mx_bf16x2(a[e + 2], a[e + 3]));
      else
        v[q] = make_float4(a[e], a[e + 1], a[e + 2], a[e + 3]);
    }
  };
  auto put = [&](const Run (&v)[JN * 4]) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < JN * 4; ++q) {
      if constexpr (BF16)
        *(uint2*)(turn + (r * UNITS + (q ^ (r & (UNITS - 1)))) * 16 + 8 * g) = v[q];
      else
        *(float4*)(turn + (r * UNITS + ((2 * q + g) ^ (r & (UNITS - 1)))) * 16) = v[q];
    }
    mx_wave_lds_sync();
  };
  const bool whole = cols == 32 * NT && rows == 32 * MT && (BF16 || !accumulate);
  Run v[JN * 4];
  pack(0, v);
#pragma unroll
  for (int b = 0; b < BLOCKS; ++b) {
    put(v);
    v4u x[LOADS];
#pragma unroll
    for (int t = 0; t < LOADS; ++t) x[t] = *(const v4u*)(from + t * 1024);
    if (b + 1 < BLOCKS) pack(b + 1, v);  // while the rows are read
    uint8_t* o = to + b * JN % NT * 32 * E;
    if (whole) {
#pragma unroll
      for (int t = 0; t < LOADS; ++t) __builtin_nontemporal_store(x[t], (v4u_any*)(o + t * step));
    } else {
      const int left = cols - b * JN % NT * 32 - (int)c0 * (16 / E);  // columns from the lane's first on
#pragma unroll 1
      for (int t = 0; t < LOADS; ++t, o += step) {
        if (b * JN / NT * 32 + (int)row0 + t * ROWS >= rows || left <= 0) continue;
        const uint8_t* y = from + t * 1024;
        if (left >= 16 / E) {
          v4f w = *(const v4f*)y;
          if (!BF16 && accumulate) {
            w += *(const v4f_any*)o;
          }
          *(v4f_any*)o = w;
        } else {
#pragma unroll 1
          for (int e = 0; e < left; ++e) {
            if constexpr (BF16)
              ((uint16_t*)o)[e] = ((const uint16_t*)y)[e];
            else
              ((float*)o)[e] = (accumulate ? ((float*)o)[e] : 0.0f) + ((const float*)y)[e];
          }
        }
      }
    }
    if ((b + 1) * JN % NT == 0) to += LOADS * step;
    mx_wave_lds_sync();
    __builtin_amdgcn_sched_barrier(0);
  }
  if (!whole) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

template <int V>
using Int = std::integral_constant<int, V>;
// f(Int<0>) .. f(Int<N - 1>)
template <int N, typename F>
__device__ __forceinline__ void mx_for(F&& f) {
  if constexpr (N > 0) {
    mx_for<N - 1>(f);
    f(Int<N - 1>{});
  }
}

template <int MT, int NT, bool BF16>
__global__ __launch_bounds__(256, MT * NT >= 8 ? 1 : 2) void mx_tile_kernel(MxMatmulArgs p) {
  using T = MxTile<MT, NT>;
  extern __shared__ __align__(16) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, g = lane >> 5;
  const int wm = wave >> 1, wn = wave & 1;

  // The workgroup's tiles and their pieces of K.  Workgroups go round the 8
  // XCDs: each XCD gets a contiguous part of the list of (piece, tile) items,
  // in which runs of GM tile rows share their b columns.
  const uint32_t tiles = p.tiles_m * p.tiles_n, total = tiles * p.pieces;
  const uint32_t xcd = blockIdx.x % 8, share = total / 8, rest = total % 8;
  const uint32_t last_item = (xcd + 1) * share + min(xcd + 1, rest);
  const uint32_t stride = gridDim.x / 8 + (xcd < gridDim.x % 8);  // workgroups on this XCD
  uint32_t item = xcd * share + min(xcd, rest) + blockIdx.x / 8;
  int64_t m0, n0;
  int piece, kb, stages;
  const uint8_t *codes, *scales;
  auto locate = [&]() __attribute__((always_inline)) {
    piece = (int)(item / tiles);
    const uint32_t i = item - piece * tiles;
    constexpr uint32_t GM = 4;
    const uint32_t band = i / (GM * p.tiles_n), first = band * GM;
    const uint32_t height = min(GM, p.tiles_m - first), j = i - band * GM * p.tiles_n;
    m0 = (int64_t)(first + j % height) * T::BM;
    n0 = (int64_t)(j / height) * T::BN;
    const int64_t kb0 = (int64_t)piece * p.piece_kb;
    kb = __builtin_amdgcn_readfirstlane((int)min(p.piece_kb, p.kb - kb0));  // 128-wide halves of this item
    stages = (kb + 1) / 2;
    codes = mx_uniform(wave < 2 ? p.a + (m0 * p.kb + kb0) * 64 : p.b + (n0 * p.kb + kb0) * 64);
    scales = mx_uniform(min(wave * T::SCALES, T::ROWS / 64 - 1) * 64 < T::BM ? p.as + (m0 * p.kb + kb0) * 4
                                                                             : p.bs + (n0 * p.kb + kb0) * 4);
  };
  // Source offsets of this wave's loads, from the tile's first row.  Rows past
  // the matrix are read as its last row; their results are not stored.
  uint32_t off[T::CHUNKS], soff[T::SCALES];
  auto offsets = [&]() __attribute__((always_inline)) {
    int at = lane;
    asm volatile("" : "+v"(at));  // as in mx_write_tile
    const int rows_a = (int)min((int64_t)T::BM, p.M - m0), rows_b = (int)min((int64_t)T::BN, p.N - n0);
#pragma unroll
    for (int q = 0; q < T::CHUNKS; ++q) {
      const int row = (wave * T::CHUNKS + q) * 8 + (at >> 3);
      const uint32_t in = row < T::BM ? min(row, rows_a - 1) : min(row - T::BM, rows_b - 1);
      off[q] = in * (uint32_t)p.kb * 64u + (((at & 7) ^ ((row >> 1) & 7)) * 16);
    }
#pragma unroll
    for (int q = 0; q < T::SCALES; ++q) {
      const int row = min(wave * T::SCALES + q, T::ROWS / 64 - 1) * 64 + at;
      const uint32_t in = row < T::BM ? min(row, rows_a - 1) : min(row - T::BM, rows_b - 1);
      soff[q] = in * (uint32_t)p.kb * 4u;
    }
  };
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)lds);

  // Load x of stage st (par = st % 2).  In a last stage of one half the other
  // half's bytes lie past the row: the first half is loaded twice, and the
  // second not used.  A lane's piece lies in the second half where bit 2 of
  // its slot differs from bit 2 of the rotation, which is bit 0 of the chunk:
  // back0 and back1 take it back there.  IF: only where `lanes` is -1.
  auto issue1 = [&](auto masked, int st, auto par_, auto x_, uint32_t back0, uint32_t back1, int lanes)
                    __attribute__((always_inline)) {
    constexpr int x = decltype(x_)::value, par = decltype(par_)::value;
    const auto load = [&](const uint8_t* base, uint32_t from, uint32_t to, auto at) __attribute__((always_inline)) {
      if constexpr (decltype(masked)::value)
        mx_dma16_if(base, from, to, decltype(at)::value, lanes);
      else
        mx_dma16(base, from, to, decltype(at)::value);
    };
    if constexpr (x < T::CHUNKS) {
      load(codes + (int64_t)st * 128, off[x] - (x & 1 ? back1 : back0), lds0 + wave * (T::CHUNKS * 2048),
           Int<x * 2048 + par * 1024>{});
    } else if constexpr (!par) {
      // scales come for four halves at a time, the last four of the row where
      // fewer are left
      const int c = min(wave * T::SCALES + x - T::CHUNKS, T::ROWS / 64 - 1);
      load(scales + (int64_t)min(2 * st, kb - 4) * 4, soff[x - T::CHUNKS],
           lds0 + 2 * T::CODES + ((st >> 1) & 1) * T::GROUP + c * 1024, Int<0>{});
    }
  };
  auto issue = [&](int st, auto par, auto loads) __attribute__((always_inline)) {
    const bool single = 2 * st + 1 >= kb;
    const uint32_t back0 = single ? (lane & 4) << 4 : 0, back1 = single ? (~lane & 4) << 4 : 0;
    mx_for<decltype(loads)::value>([&](auto x) __attribute__((always_inline)) {
      issue1(std::false_type{}, st, par, x, back0, back1, -1);
    });
  };

  v16f acc[MT][NT];
  // Fragments of a 128-wide half (two 64-wide steps).
  struct Frag {
    v4u v[2];
    uint32_t s;
  };
  Frag fb[2][NT], fa[MT + 1];
  // Addresses of the lane's first a and b row: codes by (half of a stage,
  // step), stage buffer 0.
  const int row_a = wm * MT * 32 + r, row_b = T::BM + wn * NT * 32 + r, swz = (r >> 1) & 7;
  uint32_t ca[2][2], cx[2][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int o = ((4 * (i >> 1) + 2 * g + (i & 1)) ^ swz) * 16;
    ca[i >> 1][i & 1] = lds0 + row_a / 8 * 2048 + row_a % 8 * 128 + o;
    cx[i >> 1][i & 1] = lds0 + row_b / 8 * 2048 + row_b % 8 * 128 + o;
    asm("" : "+v"(ca[i >> 1][i & 1]), "+v"(cx[i >> 1][i & 1]));  // kept, not worked out anew for every read
  }
  uint32_t scale_a = row_a * 16 + 2 * g, scale_b = row_b * 16 + 2 * g;
  asm("" : "+v"(scale_a), "+v"(scale_b));
  auto group_at = [&](int q) __attribute__((always_inline)) -> uint32_t {  // offset of group q's first half in LDS
    return lds0 + 2 * T::CODES + (q & 1) * T::GROUP + (4 * q - min(4 * q, kb - 4)) * 4;
  };
  // part 0, 1: the steps' codes; 2: the scales.  k: half within its group of four.
  auto read_a = [&](Frag& f, int i, int k, uint32_t sc, int part) __attribute__((always_inline)) {
    if (part < 2)
      f.v[part] = lds_read<v4u>(ca[k & 1][part], (k >> 1) * 1024 + i * 8192);
    else
      f.s = lds_read<uint16_t>(sc + scale_a, i * 512 + k * 4);
  };
  auto read_b = [&](Frag& f, int j, int k, uint32_t sc, int part) __attribute__((always_inline)) {
    if (part < 2)
      f.v[part] = lds_read<v4u>(cx[k & 1][part], (k >> 1) * 1024 + j * 8192);
    else
      f.s = lds_read<uint16_t>(sc + scale_b, j * 512 + k * 4);
  };
  // at least so many stores lie between a tile's first loads and its first wait
  constexpr int kStores = T::WALKS ? (BF16 ? MT * NT * 2 : 63) : 0;
  constexpr int kMfma = 2 * MT * NT;
  // The instruction before which stages change hands.  The second half's a
  // tiles 1 .. MT-1 are read before it: what is read after it, other waves' loads
  // may already be writing over.
  constexpr int kPub = MT == 1 ? 0 : MT == 2 ? 4 : (MT - 2) * NT * 2;
  constexpr int kSlots = kMfma - kPub;
  constexpr int kReadSlots = kSlots * 3 / 4;  // the reads, a little ahead of their use
  // The loads of a stage: kOdd of them in the half that frees its buffer, the
  // others over most of the next.  Of the large tiles the second half takes
  // half: a load's 64 addresses keep the compute unit's one address path busy
  // for half a matrix instruction, and four waves share it (16384 x 8192 x
  // 4096: all in the first half 299 us, split 289).
  constexpr int kLoads = T::CHUNKS + T::SCALES;
  constexpr int kOdd = MT >= 4 ? kLoads / 2 : kLoads, kEvenSlots = kMfma * 3 / 4;
  // Half k of group q.  FIRST: of the first group of a tile on a walk, whose
  // first two stages are under way as a whole, the last tile's stores behind
  // them.  LAST: of a group some of whose halves or loads may lie past the end.  Such halves are multiplied with scales of
  // 2^-127 on both sides, whose products vanish in fp32.
  auto half = [&](auto last, auto first, int q, auto k_, uint32_t sc, uint32_t sc_next, Frag (&cb)[NT], Frag (&nb)[NT]) __attribute__((always_inline)) {
    constexpr bool LAST = decltype(last)::value, FIRST = decltype(first)::value;
    constexpr int k = decltype(k_)::value;
    const uint32_t live = 4 * q + k < kb ? 0xFFFF : 0;
    uint32_t sb[NT], sa = 0;
    constexpr Int<k == 0 || k == 3> par;  // the stage being loaded
    const int st = 2 * q + (k == 0 ? 1 : k == 3 ? 3 : 2);
    const bool more = st < stages, single = 2 * st + 1 >= kb;
    uint32_t back0 = 0, back1 = 0;
#pragma unroll
    for (int n = 0; n < kMfma; ++n) {
      const int i = n / (2 * NT), t = n % (2 * NT), j = t % NT;
      if (n == kPub && (k & 1)) {
        if (FIRST && k == 1)
          asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kStores) : "memory");
        else
          mx_wait_barrier();
      }
      if (LAST && ((k & 1) ? n == kPub : (kOdd < kLoads && n == 0))) {
        back0 = single ? (lane & 4) << 4 : 0;
        back1 = single ? (~lane & 4) << 4 : 0;
      }
      __builtin_amdgcn_sched_barrier(0);
      if (t == 0) sa = LAST ? fa[i].s & live : fa[i].s;
      if (i == 0 && t < NT) sb[j] = LAST ? cb[j].s & live : cb[j].s;
      if (t < NT)
        acc[i][j] = mfma_fp4_32<0>(cb[j].v[0], fa[i].v[0], acc[i][j], sb[j], sa);
      else
        acc[i][j] = mfma_fp4_32<1>(cb[j].v[1], fa[i].v[1], acc[i][j], sb[j], sa);
      __builtin_amdgcn_sched_barrier(0);
      // a tiles 1 .. MT-1: all before kPub
      constexpr int kA = 3 * (MT - 1), kSlotsA = kPub > 0 ? kPub - 1 : 1;
      static_assert(kA == 0 || (kA - 1) * kSlotsA / kA < kPub, "read before the stage's buffer is given away");
#pragma unroll
      for (int x = 0; x < kA; ++x)
        if (x * kSlotsA / (kA > 0 ? kA : 1) == n) read_a(fa[1 + x / 3], 1 + x / 3, k, sc, 2 - x % 3);
      // the next half, from kPub on
      constexpr int kN = 3 * (NT + 1);
#pragma unroll
      for (int x = 0; x < kN; ++x)
        if (kPub + x * kReadSlots / kN == n) {
          if (x < 3)
            read_a(fa[MT], 0, (k + 1) & 3, k == 3 ? sc_next : sc, 2 - x % 3);
          else
            read_b(nb[x / 3 - 1], x / 3 - 1, (k + 1) & 3, k == 3 ? sc_next : sc, 2 - x % 3);
        }
      mx_for<kLoads>([&](auto x) __attribute__((always_inline)) {
        constexpr bool now = x < kOdd;  // in the half that frees the buffer
        if (now ? (k & 1) && kPub + x * kSlots / kOdd == n
                : !(k & 1) && !(FIRST && k == 0) && (x - kOdd) * kEvenSlots / (kLoads - kOdd + now) == n)
          issue1(last, st, par, x, back0, back1, more ? -1 : 0);
      });
    }
    __builtin_amdgcn_sched_barrier(0);
    fa[0] = fa[MT];
  };

  // Workgroups that walk start apart: else all write their results at the same
  // time, and all wait for memory with idle matrix cores (16384 x 8192 x 4096:
  // 271 us together, 260 spread over 18000 cycles, 264 over 46000; 16384 x 4096
  // x 2048: 84, 79, 89).
  if (T::WALKS && total > gridDim.x)
    for (uint32_t i = 0; i < blockIdx.x / 8; ++i) __builtin_amdgcn_s_sleep(9);  // 576 cycles
  locate();
  offsets();
  issue(0, Int<0>{}, Int<kLoads>{});
  if (stages > 1) issue(1, Int<1>{}, Int<T::WALKS ? kLoads : kOdd>{});
  // stage 0 has arrived; of stage 1's loads any may still be under way
  if (stages > 1 && !T::WALKS)
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(T::CHUNKS) : "memory");
  else
    mx_wait_barrier();
#pragma unroll 1
  for (;;) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = v16f{};
    uint32_t sc = group_at(0);
#pragma unroll
    for (int x = 0; x < 3; ++x) {
#pragma unroll
      for (int j = 0; j < NT; ++j) read_b(fb[0][j], j, 0, sc, x);
      read_a(fa[0], 0, 0, sc, x);
    }
    int q = 0;
    auto group = [&](auto last, auto first) __attribute__((always_inline)) {
      const uint32_t sc_next = group_at(q + 1);
      half(last, first, q, Int<0>{}, sc, sc_next, fb[0], fb[1]);
      half(last, first, q, Int<1>{}, sc, sc_next, fb[1], fb[0]);
      half(last, first, q, Int<2>{}, sc, sc_next, fb[0], fb[1]);
      half(last, first, q, Int<3>{}, sc, sc_next, fb[1], fb[0]);
      sc = sc_next;
      ++q;
    };
    if constexpr (T::WALKS) group(std::true_type{}, std::true_type{});
    // a group loads up to the stage of halves 4 q + 6 and 4 q + 7
#pragma unroll 1
    while (4 * q + 8 <= kb) group(std::false_type{}, std::false_type{});
#pragma unroll 1
    while (4 * q < kb) group(std::true_type{}, std::false_type{});
    // every wave is done with the stage buffers; the matrix core's last results
    // are written before they are read
    __builtin_amdgcn_sched_barrier(0);
    mx_wait_barrier();
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    const int64_t mw = m0 + wm * MT * 32, nw = n0 + wn * NT * 32;
    uint8_t* const out = (uint8_t*)p.out + piece * p.piece_bytes;
    bool again = false;
    if constexpr (T::WALKS) {
      item += stride;
      again = item < last_item;
      if (again) {
        locate();
        offsets();
        issue(0, Int<0>{}, Int<kLoads>{});
        if (stages > 1) issue(1, Int<1>{}, Int<kLoads>{});
      }
    }
    mx_write_tile<MT, NT, BF16>(acc, lds + T::TURN + wave * 4096, out, p.ld, p.accumulate, mw, nw, p.M, p.N);
    if (!again) break;
    offsets();  // (not kept while the results are on their way out)
    // stage 0 of the next tile; its other loads and the stores may still be under
    // way (it has a stage 1: these tiles' sums are not split, and K has at least
    // four blocks)
    constexpr int kLate = T::CHUNKS + kStores < 63 ? T::CHUNKS + kStores : 63;
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kLate) : "memory");
  }
}

// Sums of KB < 4 128-wide blocks, too short for the stages above: a 64 x 64
// tile per wave, all of its operands straight from memory at once.
template <int KB, bool BF16>
__global__ __launch_bounds__(256) void mx_short_kernel(MxMatmulArgs p, int64_t tiles_n, int64_t tiles) {
  __shared__ __align__(16) uint8_t turn[4][4096];
  constexpr int D = KB ? KB : 1;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 31, g = lane >> 5;
  for (int64_t tile = (int64_t)blockIdx.x * 4 + wave; tile < tiles; tile += (int64_t)gridDim.x * 4) {
    const int64_t m0 = tile / tiles_n * 64, n0 = tile % tiles_n * 64;
    v4u a[D][2][2], b[D][2][2];
    uint32_t sa[D][2], sb[D][2];
#pragma unroll
    for (int k = 0; k < KB; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t m = min(m0 + 32 * i + r, p.M - 1), n = min(n0 + 32 * i + r, p.N - 1);  // rows past the end are read again
        sa[k][i] = *(const uint16_t*)(p.as + (m * KB + k) * 4 + 2 * g);
        sb[k][i] = *(const uint16_t*)(p.bs + (n * KB + k) * 4 + 2 * g);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          a[k][i][h] = *(const v4u*)(p.a + (m * KB + k) * 64 + 32 * g + 16 * h);
          b[k][i][h] = *(const v4u*)(p.b + (n * KB + k) * 64 + 32 * g + 16 * h);
        }
      }
    v16f c[2][2] = {};
#pragma unroll
    for (int k = 0; k < KB; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          c[i][j] = mfma_fp4_32<0>(b[k][j][0], a[k][i][0], c[i][j], sb[k][j], sa[k][i]);
          c[i][j] = mfma_fp4_32<1>(b[k][j][1], a[k][i][1], c[i][j], sb[k][j], sa[k][i]);
        }
    // the matrix core's last results are written before they are read (and no
    // product moves on to where its result is used)
    asm volatile("s_nop 15\n\ts_nop 15" : "+a"(c[0][0]), "+a"(c[0][1]), "+a"(c[1][0]), "+a"(c[1][1])::"memory");
    mx_write_tile<2, 2, BF16>(c, turn[wave], p.out, p.ld, p.accumulate, m0, n0, p.M, p.N);
  }
}

// out (+)= the pieces' sums, added in piece order.
template <bool BF16>
__global__ __launch_bounds__(256) void mx_join_kernel(const float* __restrict__ part, MxMatmulArgs p) {
  const int64_t M = p.M, N = p.N, ld = p.ld;
  const int pieces = (int)p.pieces;
  const int64_t groups = (N + 3) / 4, total = M * groups;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < total; u += (int64_t)gridDim.x * 256) {
    const int64_t m = u / groups, n = (u - m * groups) * 4;
    const int left = (int)min(N - n, (int64_t)4);
    const float* src = part + m * N + n;
    v4f v = {};
    if (left == 4) {
#pragma unroll 8
      for (int k = 0; k < pieces; ++k) v += *(const v4f_any*)(src + (int64_t)k * M * N);
    } else {
      for (int k = 0; k < pieces; ++k)
        for (int i = 0; i < left; ++i) v[i] += src[(int64_t)k * M * N + i];
    }
    if constexpr (BF16) {
      uint16_t* o = (uint16_t*)p.out + m * ld + n;
      const uint32_t h0 = mx_bf16x2(v[0], v[1]), h1 = mx_bf16x2(v[2], v[3]);
      if (left == 4) {
        *(v2u_any*)o = v2u_any{h0, h1};
      } else {
        o[0] = (uint16_t)h0;
        if (left > 1) o[1] = (uint16_t)(h0 >> 16);
        if (left > 2) o[2] = (uint16_t)h1;
      }
    } else {
      float* o = (float*)p.out + m * ld + n;
      if (left == 4) {
        if (p.accumulate) v += *(const v4f_any*)o;
        *(v4f_any*)o = v;
      } else {
        for (int i = 0; i < left; ++i) o[i] = p.accumulate ? o[i] + v[i] : v[i];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Few rows (M <= 16 MB <= 64): the weights stream once past all of them.  A workgroup
// takes 16 columns, its 8 waves every eighth 256-wide pair of K blocks each,
// straight from memory to registers: whole 128-byte lines of 16 rows.  The
// waves' sums meet in LDS and are added in wave order.
//
// In a pair, lane (r, g) holds row r's 64 values from 64 g on, the first 32 of
// them for the first matrix instruction (the order of the sum is free as long
// as both operands share it).
//
// X = 0: a is codes.  1, 2: bf16 or fp32 values, quantised on the way: a lane's
// operand is 32 consecutive values of one row, just one group, so quantising
// takes no exchange between lanes and the single token needs no launch of its
// own for it.
// ---------------------------------------------------------------------------
constexpr int kFewWaves = 8;

// A lane's 32 values of a, and their scale.
struct FewOperand {
  uint4 codes;
  uint32_t scale;
};
template <int X>
struct FewRaw {
  uint4 v[X == 0 ? 1 : X == 1 ? 4 : 8];
};

// 32 values of row m from column `col` on.  WHOLE: they lie inside the row.
template <int X, bool WHOLE>
__device__ __forceinline__ void few_load(FewRaw<X>& f, const MxMatmulArgs& p, int64_t m, int64_t col) {
  if constexpr (X == 0) {
    f.v[0] = *(const uint4*)(p.a + m * p.kb * 64 + col / 2);
  } else {
    constexpr int V = X == 1 ? 8 : 4;  // values of sixteen bytes
    const uint8_t* row = (const uint8_t*)p.x + (m * p.ld_x + col) * (16 / V);
    const int left = (int)min(p.K - col, (int64_t)32);
#pragma unroll
    for (int i = 0; i < 32 / V; ++i) {
      if (WHOLE || left >= V * (i + 1)) {
        f.v[i] = mx_read16(row + 16 * i);
      } else {
        uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (V * i + e < left) {
            if constexpr (X == 1)
              u[e / 2] |= (uint32_t)((const uint16_t*)row)[V * i + e] << (16 * (e & 1));
            else
              u[e] = ((const uint32_t*)row)[V * i + e];
          }
        f.v[i] = make_uint4(u[0], u[1], u[2], u[3]);
      }
    }
  }
}

template <int X>
__device__ __forceinline__ FewOperand few_operand(const FewRaw<X>& f, uint32_t scale) {
  if constexpr (X == 0) {
    return {f.v[0], scale};
  } else if constexpr (X == 1) {
    const uint32_t b = mx_scale_byte(
        max(max(mx_amax_bf16(f.v[0]), mx_amax_bf16(f.v[1])), max(mx_amax_bf16(f.v[2]), mx_amax_bf16(f.v[3]))));
    return {make_uint4(mx_codes_bf16(f.v[0], b), mx_codes_bf16(f.v[1], b), mx_codes_bf16(f.v[2], b),
                       mx_codes_bf16(f.v[3], b)),
            b};
  } else {
    uint32_t m = 0, w[4];
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, mx_amax_f32(f.v[i]));
    const uint32_t b = mx_scale_byte(m);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = mx_codes_f32(f.v[2 * i], b) | mx_codes_f32(f.v[2 * i + 1], b) << 16;
    return {make_uint4(w[0], w[1], w[2], w[3]), b};
  }
}

__device__ __forceinline__ v4f mfma_fp4_16(const uint4& w, uint32_t ws, const FewOperand& x, v4f c) {
  const v8i va = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
  const v8i vb = {(int)x.codes.x, (int)x.codes.y, (int)x.codes.z, (int)x.codes.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(va, vb, c, 4, 4, 0, (int)ws, 0, (int)x.scale);
}

// U pairs k, k + 8, ... of a wave: all loads, then the products.
template <int X, int MB, int U>
__device__ __forceinline__ void few_pairs(const MxMatmulArgs& p, const uint8_t* w, const uint8_t* ws, int64_t k, int r,
                                          int g, v4f (&acc)[MB]) {
  uint4 wv[U][2];
  uint32_t wsc[U], xs[U][MB];
  FewRaw<X> x[U][MB][2];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t q = k + u * kFewWaves;
    wv[u][0] = *(const uint4*)(w + q * 128 + 32 * g);
    wv[u][1] = *(const uint4*)(w + q * 128 + 32 * g + 16);
    wsc[u] = *(const uint16_t*)(ws + q * 8 + 2 * g);
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int64_t m = min((int64_t)(16 * i + r), p.M - 1);
      if constexpr (X == 0) xs[u][i] = *(const uint16_t*)(p.as + m * p.kb * 4 + q * 8 + 2 * g);
#pragma unroll
      for (int h = 0; h < 2; ++h) few_load<X, true>(x[u][i][h], p, m, q * 256 + 64 * g + 32 * h);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        acc[i] = mfma_fp4_16(wv[u][h], wsc[u] >> (8 * h), few_operand<X>(x[u][i][h], X == 0 ? xs[u][i] >> (8 * h) : 0), acc[i]);
}

template <int X, int MB, bool BF16>
__global__ __launch_bounds__(64 * kFewWaves) void mx_few_kernel(MxMatmulArgs p) {
  constexpr int U = X == 0 ? (MB <= 2 ? 4 : 2) : MB == 1 && X == 1 ? 2 : 1;  // pairs in flight per wave
  __shared__ float part[kFewWaves][MB][16][17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int64_t n = min(n0 + r, p.N - 1);  // rows past the end are read again
  const uint8_t* w = p.b + n * p.kb * 64;
  const uint8_t* ws = p.bs + n * p.kb * 4;
  v4f acc[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) acc[i] = v4f{0, 0, 0, 0};
  const int64_t pairs = X == 0 ? p.kb / 2 : p.K / 256;
  int64_t k = wave;
  for (; k + (U - 1) * kFewWaves < pairs; k += U * kFewWaves) few_pairs<X, MB, U>(p, w, ws, k, r, g, acc);
  if constexpr (U >= 4)
    if (k + kFewWaves < pairs) {
      few_pairs<X, MB, 2>(p, w, ws, k, r, g, acc);
      k += 2 * kFewWaves;
    }
  if (U >= 2 && k < pairs) few_pairs<X, MB, 1>(p, w, ws, k, r, g, acc);
  // what is left past the pairs: at most two blocks, the last waves'
  const int64_t block = 2 * pairs + (kFewWaves - 1 - wave);
  if (block < p.kb) {
    const uint4 wv = *(const uint4*)(w + block * 64 + 16 * g);
    const uint32_t wsc = ws[block * 4 + g];
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int64_t m = min((int64_t)(16 * i + r), p.M - 1);
      FewRaw<X> x;
      few_load<X, false>(x, p, m, block * 128 + 32 * g);
      acc[i] = mfma_fp4_16(wv, wsc, few_operand<X>(x, X == 0 ? p.as[(m * p.kb + block) * 4 + g] : 0), acc[i]);
    }
  }
  // the matrix core's last results are written before they are read
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 15" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  // lane: row r of a, columns 4 g .. +4
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) part[wave][i][r][4 * g + j] = acc[i][j];
  __syncthreads();
  for (int t = threadIdx.x; t < MB * 256; t += 64 * kFewWaves) {
    const int m = t >> 4, c = t & 15;
    float v = 0.0f;
#pragma unroll
    for (int q = 0; q < kFewWaves; ++q) v += part[q][m >> 4][m & 15][c];
    if (m < p.M && n0 + c < p.N) {
      const int64_t at = m * p.ld + n0 + c;
      if constexpr (BF16)
        ((uint16_t*)p.out)[at] = f32_to_bf16(v);
      else
        ((float*)p.out)[at] = p.accumulate ? ((float*)p.out)[at] + v : v;
    }
  }
}

// Up to 32 rows go here (2048 x 4096 weights, with the quantisation of x: 7.6
// us at 1 row, 10.6 at 32; in 64-row tiles 10.0 and 12.2), and up to 64 where
// the rows, which every workgroup reads whole, are short: then the tiles' extra
// launch for their split sum costs as much as it saves (us, here / in tiles: 33
// x 8192 x 4096 16.7 / 19.9, 64 x 520 x 3000 11.7 / 12.9, 64 x 4000 x 1000 8.6 /
// 8.9, 48 x 2048 x 4096 12.5 / 12.5; 64 x 2048 x 4096 14.1 / 13.2 in a graph but
// 14 / 17 launched one by one; 64 x 8192 x 4096, whose tiles need no split, 22.0
// / 20.6; 33 x 1024 x 8192 15.4 / 12.4).  Up to 16 rows
// are quantised on the way, unless every workgroup's own pass over x costs more
// than a launch for it (us, on the way / apart: 1 x 2048 x 4096 5.3 / 7.6, 16 x
// 2048 x 4096 7.9 / 8.9, 4 x 8192 x 4096 9.5 / 10.9; but 16 x 8192 x 4096 13.9 /
// 12.7, 4 x 8192 x 8192 16.2 / 15.4).
static bool mx_few_rows(int64_t M, int64_t N, int64_t K) {
  return M <= 32 || (M <= 64 && M * K <= (N <= 4096 ? 64 : 48) * 4096);
}
static bool mx_fused(int64_t M, int64_t N, int64_t K) { return M <= 16 && M * N * K <= 200000000; }

template <int X>
static hipError_t launch_mx_few(const MxMatmulArgs& p, bool bf16, hipStream_t s) {
  const auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)((p.N + 15) / 16)), dim3(64 * kFewWaves), 0, s, p);
    return hipGetLastError();
  };
  if (p.M <= 16) return bf16 ? run(mx_few_kernel<X, 1, true>) : run(mx_few_kernel<X, 1, false>);
  if constexpr (X == 0) {
    if (p.M > 48) return bf16 ? run(mx_few_kernel<X, 4, true>) : run(mx_few_kernel<X, 4, false>);
    if (p.M > 32) return bf16 ? run(mx_few_kernel<X, 3, true>) : run(mx_few_kernel<X, 3, false>);
  }
  return bf16 ? run(mx_few_kernel<X, 2, true>) : run(mx_few_kernel<X, 2, false>);
}

// The tile (64 t x 64 t, t = 4, 2 or 1) and the split of K for a product.
//
// Time in us, fitted to a sweep of 23 products on one MI355X (M 700..16384, N
// 1500..8192, K 512..4096), with c tiles per compute unit and K of kb blocks:
// 256-tiles 3 + 6 and 0.78 kb for every full or partial round of c = 1;
// 128-tiles 2.4 + 1.4 c + max(0.4, 0.26 c) kb; 64-tiles 3 + 0.4 c + max(0.2, 0.13
// c) kb.  The least of the three is the fastest tile or within 3% of it in all
// of them (256 / 128 / 64: 4096 x 4096 x 4096 35.0 / 41.6 / 70.7; 4900 x 4700 x
// 520 41.7 / 28.7 / 33.9; 4900 x 4700 x 4096 69.0 / 66.4 / 106; 2048 x 4096 x 4001
// 25.4 / 21.8 / 36.8; 1024 x 2048 x 4096 23.5 / 13.9 / 12.1; 1024 x 1024 x 1024
// 10.2 / 5.3 / 4.4).
//
// A long sum over few tiles is split into pieces, up to one workgroup per
// compute unit (128 x 2048 x 4096, 64 tiles: 11.3 us whole, 9.8 in 4 pieces;
// 16 x 2048 x 4096, 32 tiles: 10.9 and 7.3 in 8); at 128 tiles the join costs
// what the split gains (256 x 2048 x 4096: 11.6 and 11.9), as it does for sums
// of fewer than 16 halves.
struct MxPlan {
  int t, pieces;
  int64_t piece_kb;
};
static MxPlan mx_plan(int64_t M, int64_t N, int64_t kb) {
  constexpr double kCus = 256;
  MxPlan best{1, 1, kb};
  double best_us = 0;
  int64_t best_tiles = 0;
  for (int t : {4, 2, 1}) {
    const int64_t tiles = ((M + 64 * t - 1) / (64 * t)) * ((N + 64 * t - 1) / (64 * t));
    const double c = (double)tiles / kCus;
    const double us = t == 4   ? 3 + (double)((tiles + 255) / 256) * (6 + 0.78 * (double)kb)
                      : t == 2 ? 2.4 + 1.4 * c + (c * 0.26 > 0.4 ? c * 0.26 : 0.4) * (double)kb
                               : 3 + 0.4 * c + (c * 0.13 > 0.2 ? c * 0.13 : 0.2) * (double)kb;
    if (best_us == 0 || us < best_us) {
      best.t = t;
      best_us = us;
      best_tiles = tiles;
    }
  }
  if (best_tiles <= 64 && best.t < 4 && kb >= 16) {
    int pieces = 1;
    while (pieces < 16 && best_tiles * pieces * 2 <= 256 && kb / (pieces * 2) >= 4) pieces *= 2;
    best.piece_kb = ((kb + pieces - 1) / pieces + 1) / 2 * 2;  // whole stages
    best.pieces = (int)((kb + best.piece_kb - 1) / best.piece_kb);
  }
  return best;
}

template <int MT, int NT>
static hipError_t launch_mx_tile(const MxMatmulArgs& p, bool bf16, hipStream_t s) {
  const uint32_t items = p.tiles_m * p.tiles_n * p.pieces;
  // one workgroup per compute unit that walks, else one per item
  const dim3 grid(MxTile<MT, NT>::WALKS && items > 256 ? 256 : items);
  const auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), (MxTile<MT, NT>::LDS), s, p);
    return hipGetLastError();
  };
  return bf16 ? run(mx_tile_kernel<MT, NT, true>) : run(mx_tile_kernel<MT, NT, false>);
}

static hipError_t launch_mx_matmul(const MxMatmulArgs& p, const MxPlan& plan, bool bf16, float* part, hipStream_t s) {
  if (mx_few_rows(p.M, p.N, p.K)) return launch_mx_few<0>(p, bf16, s);
  if (p.kb < 4) {
    const int64_t tn = (p.N + 63) / 64, tiles = (p.M + 63) / 64 * tn, blocks = (tiles + 3) / 4;
    const dim3 grid((unsigned)(blocks < kMxMaxGrid ? blocks : kMxMaxGrid));
    const auto run = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, p, tn, tiles);
      return hipGetLastError();
    };
    switch (p.kb) {
      case 0: return bf16 ? run(mx_short_kernel<0, true>) : run(mx_short_kernel<0, false>);
      case 1: return bf16 ? run(mx_short_kernel<1, true>) : run(mx_short_kernel<1, false>);
      case 2: return bf16 ? run(mx_short_kernel<2, true>) : run(mx_short_kernel<2, false>);
      default: return bf16 ? run(mx_short_kernel<3, true>) : run(mx_short_kernel<3, false>);
    }
  }
  MxMatmulArgs t = p;
  const bool split = plan.pieces > 1;
  t.pieces = plan.pieces;
  t.piece_kb = plan.piece_kb;
  t.tiles_m = (uint32_t)((p.M + 64 * plan.t - 1) / (64 * plan.t));
  t.tiles_n = (uint32_t)((p.N + 64 * plan.t - 1) / (64 * plan.t));
  if (split) {
    t.out = part;
    t.ld = p.N;
    t.accumulate = 0;
    t.piece_bytes = p.M * p.N * 4;
  }
  const bool tb = bf16 && !split;
  const hipError_t e = plan.t == 4   ? launch_mx_tile<4, 4>(t, tb, s)
                       : plan.t == 2 ? launch_mx_tile<2, 2>(t, tb, s)
                                     : launch_mx_tile<1, 1>(t, tb, s);
  if (e != hipSuccess || !split) return e;
  const int64_t blocks = (p.M * ((p.N + 3) / 4) + 255) / 256;
  const dim3 grid((unsigned)(blocks < kMxMaxGrid ? blocks : kMxMaxGrid));
  MxMatmulArgs j = p;
  j.pieces = plan.pieces;
  if (bf16)
    hipLaunchKernelGGL(mx_join_kernel<true>, grid, dim3(256), 0, s, part, j);
  else
    hipLaunchKernelGGL(mx_join_kernel<false>, grid, dim3(256), 0, s, part, j);
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

// Scratch of a product: the partial sums of a split one.
size_t matmul_bytes(int64_t M, int64_t N, int64_t K) {
  if (M == 0 || N == 0 || moe::mx_few_rows(M, N, K)) return 0;
  const moe::MxPlan plan = moe::mx_plan(M, N, mx_padded(K) / 128);
  return plan.pieces > 1 ? up256(plan.pieces * M * N * 4) : 0;
}

moe::MxMatmulArgs product_args(int64_t M, int64_t N, int64_t K, const void* a, const void* as, const void* b,
                               const void* bs, void* out, int64_t ld_out, int32_t accumulate) {
  moe::MxMatmulArgs p{};
  p.a = (const uint8_t*)a;
  p.as = (const uint8_t*)as;
  p.b = (const uint8_t*)b;
  p.bs = (const uint8_t*)bs;
  p.M = M;
  p.N = N;
  p.K = K;
  p.kb = mx_padded(K) / 128;
  p.out = out;
  p.ld = ld_out;
  p.accumulate = accumulate;
  return p;
}

moe_status_t run_matmul(int64_t M, int64_t N, int64_t K, const void* a, const void* as, const void* b, const void* bs,
                        int32_t out_dtype, void* out, int64_t ld_out, int32_t accumulate, void* part, hipStream_t s) {
  const moe::MxMatmulArgs p = product_args(M, N, K, a, as, b, bs, out, ld_out, accumulate);
  return moe::mx_status(
      moe::launch_mx_matmul(p, moe::mx_plan(M, N, p.kb), out_dtype == MOE_DTYPE_BF16, (float*)part, s));
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
  return run_matmul(M, N, K, a, a_scale, b, b_scale, out_dtype, out, ld_out, accumulate, ws, (hipStream_t)stream);
}

size_t moe_mxfp4_linear_bytes(int32_t M, int32_t N, int32_t K) {
  if (!product_ok(M, N, K) || moe::mx_fused(M, N, K)) return 0;
  return code_bytes(M, K) + scale_bytes(M, K) + matmul_bytes(M, N, K);
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
  if (moe::mx_fused(M, N, K)) {
    moe::MxMatmulArgs p = product_args(M, N, K, nullptr, nullptr, w, w_scale, out, ld_out, 0);
    p.x = x;
    p.ld_x = ld_x;
    const bool bf16 = out_dtype == MOE_DTYPE_BF16;
    return moe::mx_status(x_dtype == MOE_DTYPE_BF16 ? moe::launch_mx_few<1>(p, bf16, s) : moe::launch_mx_few<2>(p, bf16, s));
  }
  uint8_t* xq = (uint8_t*)ws;
  uint8_t* xs = xq + code_bytes(M, K);
  if (K > 0) {
    const moe_status_t st =
        moe::mx_status(moe::launch_mx_quant(x, x_dtype == MOE_DTYPE_BF16, M, K, ld_x, xq, xs, nullptr, nullptr, s));
    if (st != MOE_OK) return st;
  }
  return run_matmul(M, N, K, xq, xs, w, w_scale, out_dtype, out, ld_out, 0, xs + scale_bytes(M, K), s);
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
  void* part = sc + scale_bytes(N, M);  // the two products take turns
  moe_status_t st = MOE_OK;
  if (dots)
    st = moe::mx_status(moe::launch_mx_quant(dy, dy_dtype == MOE_DTYPE_BF16, M, N, ld_dy, want_dx ? qr : nullptr,
                                             want_dx ? sr : nullptr, want_dw ? qc : nullptr, want_dw ? sc : nullptr, s));
  if (st == MOE_OK && want_dx) st = run_matmul(M, K, N, qr, sr, w_col, w_col_scale, dx_dtype, dx, ld_dx, 0, part, s);
  if (st == MOE_OK && want_dw)
    st = run_matmul(N, K, M, qc, sc, x_col, x_col_scale, MOE_DTYPE_F32, dw, ld_dw, accumulate, part, s);
  return st;
}

}  // extern "C"
