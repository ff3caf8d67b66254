// The router's training operators and their C ABI: balance loss, z loss and
// per-expert counts (moe_balance_loss), and the gradient to the router's
// logits (moe_router_bwd).
//
// Tokens t of sequence s (rows seq_offsets[s] .. seq_offsets[s+1]) are valid
// when their mask byte is non-zero and their row holds a logit above -inf.
//   lse_t = log sum_e exp(l_te),  p_te = exp(l_te - lse_t)
//   n_s valid tokens, N = sum n_s, S' sequences with n_s > 0
//   c_se = pairs (t, j) of valid tokens with ids[t, j] = e
//   f_se = E c_se / (k n_s),  P_se = (sum p_te) / n_s
//   balance = (1/S') sum_s sum_e f_se P_se,   z = (1/N) sum lse_t^2
// With f held constant (counts have no gradient),
//   d l_te = p_te (a_se - sum_e' p_te' a_se') + g_z (2/N) lse_t p_te,
//   a_se = g_b E c_se / (S' k n_s^2),
// and through the routing weights w = softmax of the k selected logits
//   d l_te += sum over j with ids[t, j] = e of w_j (dw_j - sum_i w_i dw_i).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/moe.h"
#include "moe_device.h"

namespace moe {

constexpr int kBalWaves = 16;
constexpr int kBalGroups = 16;     // slot groups (waves) of the finishing workgroups
constexpr int kBalMaxExperts = 1024;

struct BalanceArgs {
  const float* logits;
  const int32_t* ids;
  int32_t T, E, k, S, chunk, chunks;  // chunk: tokens of a workgroup
  const uint8_t* mask;
  const int32_t* offsets;  // null: one sequence of all T rows
  float* lse;
  int32_t* counts;         // [S, E]
  int32_t* seq_tokens;     // [S + 2]: n_s, then N and S'
  float* loss;             // [2]
  // partial sums: slot c + s of chunk c and sequence s
  float* psum;             // [chunks + S][E]
  int32_t* pcount;         // [chunks + S][E]
  float* pz;               // [chunks + S]
  int32_t* pn;             // [chunks + S]
  float* seq_loss;         // [S][tiles of 64 experts]
  float* seq_z;            // [S]
  uint32_t* ticket;        // finishing workgroups done
};

__device__ __forceinline__ int seq_offset(const int32_t* offsets, int T, int s) {
  if (!offsets) return s ? T : 0;
  const int o = offsets[s];
  return o < 0 ? 0 : (o > T ? T : o);
}

template <typename V>
__device__ __forceinline__ void device_store(V* p, V v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename V>
__device__ __forceinline__ V device_load(V* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// One expert's f P of a sequence of n valid tokens.
__device__ __forceinline__ float balance_share(int count, float psum, int n, int E, int k) {
  return n > 0 ? ((float)count * (float)E / ((float)k * (float)n)) * (psum / (float)n) : 0.0f;
}

__device__ __forceinline__ void balance_results(const BalanceArgs& p, float loss, float z, int n, int filled) {
  p.loss[0] = filled ? loss / (float)filled : 0.0f;
  p.loss[1] = n ? z / (float)n : 0.0f;
  p.seq_tokens[p.S] = n;
  p.seq_tokens[p.S + 1] = filled;
}

// The first sequence that ends after row t (S if none does): 64 evenly spaced
// ends are compared at a time, one per lane.  Called by whole waves.
__device__ __forceinline__ int seq_of(const int32_t* offsets, int T, int S, int t) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = S;  // the answer lies in [lo, lo + n]
  while (n > 0) {
    const int step = (n + 63) / 64;
    const int i = lo + lane * step + step - 1;  // last sequence of the lane's run
    const bool before = lane * step < n && seq_offset(offsets, T, min(i, lo + n - 1) + 1) <= t;
    const uint64_t m = __ballot(before);
    const int runs = m == ~0ull ? 64 : __builtin_ctzll(~m);  // whole runs that end at or before t
    const int skip = min(runs * step, n);
    lo += skip;
    n = step == 1 ? 0 : min(step - 1, n - skip);
  }
  return lo;
}

// Wave-wide sums and maximum by row operations (quad swaps, mirrors, then the
// rows' last lanes), read back uniformly from lane 63; the order of a sum is
// fixed.  Lanes outside a step's rows add zero.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_or_zero(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ float last_lane(float v) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_or_zero<0xB1, 0xF>(v);   // quad_perm [1,0,3,2]
  v += dpp_or_zero<0x4E, 0xF>(v);   // quad_perm [2,3,0,1]
  v += dpp_or_zero<0x141, 0xF>(v);  // row_half_mirror
  v += dpp_or_zero<0x140, 0xF>(v);  // row_mirror
  v += dpp_or_zero<0x142, 0xA>(v);  // row_bcast:15 into rows 1, 3
  v += dpp_or_zero<0x143, 0xC>(v);  // row_bcast:31 into rows 2, 3
  return last_lane(v);
}
__device__ __forceinline__ int wave_sum(int v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_or_own(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(v), __float_as_int(v), CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp_or_own<0xB1, 0xF>(v));
  v = fmaxf(v, dpp_or_own<0x4E, 0xF>(v));
  v = fmaxf(v, dpp_or_own<0x141, 0xF>(v));
  v = fmaxf(v, dpp_or_own<0x140, 0xF>(v));
  v = fmaxf(v, dpp_or_own<0x142, 0xA>(v));
  v = fmaxf(v, dpp_or_own<0x143, 0xC>(v));
  return last_lane(v);
}

// A token's logits in a wave: lane holds experts lane + 64 i, -inf past the
// last.  Every load is issued (clamped into the row).
template <int VPL>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, float (&v)[VPL]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < VPL; ++i) v[i] = row[min(lane + 64 * i, E - 1)];
}
// exp(v - max), in place, with the row's maximum and sum; false if the row
// holds nothing above -inf.  A NaN counts as something: it has to show.  exp is
// the hardware's exp2 of (v - max) log2 e: off by |v - max| 2^-24 + 2^-23
// relative, and the difference cannot overflow where a scaled logit could.
template <int VPL>
__device__ __forceinline__ bool exp_row(float (&v)[VPL], int E, float& mx, float& sum) {
  const int lane = threadIdx.x & 63;
  bool some = false;
  mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    if (lane + 64 * i >= E) v[i] = -INFINITY;
    some |= !(v[i] == -INFINITY);
    mx = fmaxf(mx, v[i]);
  }
  if (!__any(some)) return false;
  mx = wave_max(mx);
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    v[i] = __builtin_amdgcn_exp2f((v[i] - mx) * 1.4426950408889634f);
    sum += v[i];
  }
  sum = wave_sum(sum);
  return true;
}

// LDS written by some lanes of a wave is read by others of the same wave: a
// wave's LDS operations complete in order, so ordering the compiler's view is
// all that is needed.
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Rows of a wave, all in registers together, by 64-expert columns per lane.
constexpr int bal_rows(int vpl) { return vpl <= 5 ? 4 : vpl <= 8 ? 2 : 1; }
// Tokens of a workgroup: one row set of its waves.
constexpr int bal_chunk(int E) { return kBalWaves * bal_rows((E + 63) / 64); }

// One workgroup per chunk of tokens, one wave per token, U of them in flight:
// the softmax of every row comes first, then the chunk is walked sequence by
// sequence, adding up what is in registers.  Each (chunk, sequence) overlap
// leaves its sums in a slot of its own (c + s: along the rows every new overlap
// raises c or s, so no two share a slot), added up in slot order by
// balance_finish_kernel.  ONE: the only chunk, which writes the results itself.
//
// 16384 tokens of 288 experts in 16 sequences: 11.5 us (19 MB at 1.7 TB/s: a
// workgroup's loads, softmax and sums follow one another, and there is one
// workgroup per compute unit), then 5.8 us to finish, both latency; chunks of
// 32 tokens took 14.9 and 6.6 us.  64 tokens: 6.9 us in the one launch.
template <int VPL, bool ONE>
__global__ __launch_bounds__(64 * kBalWaves) void balance_chunk_kernel(BalanceArgs p) {
  constexpr int U = bal_rows(VPL);
  extern __shared__ float smem[];
  float* red = smem;                                   // [kBalWaves][E]
  int32_t* hist = (int32_t*)(red + kBalWaves * p.E);   // [E]
  __shared__ float red_z[kBalWaves];
  __shared__ int32_t red_n[kBalWaves];
  __shared__ float red_l[kBalWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c = blockIdx.x, tb = c * kBalWaves * U, te = min(p.T, tb + kBalWaves * U);
  if (!ONE && c == 0 && tid == 0) *p.ticket = 0;
  if (ONE)
    for (int i = tid; i < p.S * p.E; i += 64 * kBalWaves) p.counts[i] = 0;
  if (ONE)
    for (int i = tid; i < p.S; i += 64 * kBalWaves) p.seq_tokens[i] = 0;
  // (rows outside every sequence are not valid)
  const int first = min(max(seq_offset(p.offsets, p.T, 0), tb), te);
  const int last = min(max(seq_offset(p.offsets, p.T, p.S), first), te);
  // the sequences from s0 on, 64 at a time: the end of s0 + lane (found before
  // the rows, whose loads it would otherwise wait for)
  int s0 = p.S > 64 && first < last ? seq_of(p.offsets, p.T, p.S, first) : 0;
  int end = seq_offset(p.offsets, p.T, min(s0 + lane, p.S - 1) + 1);
  float v[U][VPL], z[U];
  int id[U];
  bool ok[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int t = tb + wave + u * kBalWaves, in = max(min(t, te - 1), 0);
    ok[u] = t >= first && t < last;
    if (te > tb) {
      load_row<VPL>(p.logits + (int64_t)in * p.E, p.E, v[u]);
      id[u] = lane < p.k ? p.ids[(int64_t)in * p.k + lane] : -1;
      if (p.mask) ok[u] = ok[u] && p.mask[in];
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int t = tb + wave + u * kBalWaves;
    float mx, sum, lse = 0.0f;
    ok[u] = ok[u] && exp_row<VPL>(v[u], p.E, mx, sum);
    if (ok[u]) {
      const float inv = __builtin_amdgcn_rcpf(sum);
      lse = mx + logf(sum);
#pragma unroll
      for (int i = 0; i < VPL; ++i) v[u][i] *= inv;
    }
    z[u] = lse * lse;
    if (lane == 0 && t < te) p.lse[t] = lse;
  }
  float one_loss = 0.0f, one_z = 0.0f;  // ONE, thread 0: sums over the sequences
  int one_n = 0, one_filled = 0;
  int t0 = first;
  while (t0 < last) {
    // the next sequence that ends after row t0
    const uint64_t after = __ballot(s0 + lane < p.S && end > t0);
    if (!after) {
      s0 += 64;
      if (s0 >= p.S) break;
      end = seq_offset(p.offsets, p.T, min(s0 + lane, p.S - 1) + 1);
      continue;
    }
    const int at = __builtin_ctzll(after), s = s0 + at;
    const int t1 = min(__builtin_amdgcn_readlane(end, at), last);
    for (int e = tid; e < p.E; e += 64 * kBalWaves) hist[e] = 0;
    __syncthreads();
    float acc[VPL] = {}, zs = 0.0f;
    int n = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = tb + wave + u * kBalWaves;
      if (ok[u] && t >= t0 && t < t1) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) acc[i] += v[u][i];
        zs += z[u];
        ++n;
        if (id[u] >= 0 && id[u] < p.E) atomicAdd(&hist[id[u]], 1);
      }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + 64 * i < p.E) red[wave * p.E + lane + 64 * i] = acc[i];
    if (lane == 0) {
      red_z[wave] = zs;
      red_n[wave] = n;
    }
    __syncthreads();
    int cnt = 0;
    zs = 0.0f;
#pragma unroll
    for (int w = 0; w < kBalWaves; ++w) {
      zs += red_z[w];
      cnt += red_n[w];
    }
    const int64_t slot = c + s;
    float share = 0.0f;
    for (int e = tid; e < p.E; e += 64 * kBalWaves) {
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kBalWaves; ++w) sum += red[w * p.E + e];
      if constexpr (ONE) {
        p.counts[(int64_t)s * p.E + e] = hist[e];
        share = balance_share(hist[e], sum, cnt, p.E, p.k);  // (E <= 1024: one expert per thread)
      } else {
        p.psum[slot * p.E + e] = sum;
        p.pcount[slot * p.E + e] = hist[e];
      }
    }
    if constexpr (ONE) {
      share = wave_sum(share);
      if (lane == 0) red_l[wave] = share;
      __syncthreads();
      if (tid == 0) {
        for (int w = 0; w < kBalWaves; ++w) one_loss += red_l[w];
        one_z += zs;
        one_n += cnt;
        one_filled += cnt > 0;
        p.seq_tokens[s] = cnt;
      }
    } else if (tid == 0) {
      p.pz[slot] = zs;
      p.pn[slot] = cnt;
    }
    __syncthreads();
    t0 = t1;
  }
  if (ONE && tid == 0) balance_results(p, one_loss, one_z, one_n, one_filled);
}

// Workgroup (s, tile of 64 experts): adds the sequence's slots in a fixed
// order, leaves its counts and its share of the loss; the last workgroup to
// finish adds the shares up, again in a fixed order.  What the workgroups
// exchange goes past the caches of their dies with stores and loads of device
// scope, and a workgroup waits for its own stores before it takes its ticket:
// no cache has to be written back for it.
__global__ __launch_bounds__(64 * kBalGroups) void balance_finish_kernel(BalanceArgs p, int tiles) {
  __shared__ float rp[kBalGroups][64];
  __shared__ int32_t rc[kBalGroups][64];
  __shared__ float rz[kBalGroups], rl[kBalGroups];
  __shared__ int32_t rn[kBalGroups], rf[kBalGroups];
  __shared__ int32_t is_last;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int s = blockIdx.x / tiles, tile = blockIdx.x % tiles;
  const int e = tile * 64 + lane;
  const int lo = seq_offset(p.offsets, p.T, s), hi = seq_offset(p.offsets, p.T, s + 1);
  const int c0 = lo / p.chunk, c1 = lo < hi ? (hi - 1) / p.chunk + 1 : c0;
  float sum = 0.0f;
  int cnt = 0;
  {
    const float* ps = p.psum + min(e, p.E - 1);
    const int32_t* pc = p.pcount + min(e, p.E - 1);
    int c = c0 + wave;
    for (; c + 7 * kBalGroups < c1; c += 8 * kBalGroups) {  // eight slots in flight
      float a[8];
      int32_t b[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] = ps[(int64_t)(c + i * kBalGroups + s) * p.E];
        b[i] = pc[(int64_t)(c + i * kBalGroups + s) * p.E];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum += a[i];
        cnt += b[i];
      }
    }
    for (; c < c1; c += kBalGroups) {
      sum += ps[(int64_t)(c + s) * p.E];
      cnt += pc[(int64_t)(c + s) * p.E];
    }
  }
  float z = 0.0f;
  int n = 0;
  for (int c = c0 + tid; c < c1; c += 64 * kBalGroups) {
    z += p.pz[c + s];
    n += p.pn[c + s];
  }
  z = wave_sum(z);
  n = wave_sum(n);
  rp[wave][lane] = sum;
  rc[wave][lane] = cnt;
  if (lane == 0) {
    rz[wave] = z;
    rn[wave] = n;
  }
  __syncthreads();
  if (wave == 0) {
    sum = z = 0.0f;
    cnt = n = 0;
#pragma unroll
    for (int w = 0; w < kBalGroups; ++w) {
      sum += rp[w][lane];
      cnt += rc[w][lane];
      z += rz[w];
      n += rn[w];
    }
    if (e < p.E) p.counts[(int64_t)s * p.E + e] = cnt;
    const float share = wave_sum(e < p.E ? balance_share(cnt, sum, n, p.E, p.k) : 0.0f);
    if (lane == 0) {
      device_store(&p.seq_loss[(int64_t)s * tiles + tile], share);
      if (tile == 0) {
        device_store(&p.seq_z[s], z);
        device_store(&p.seq_tokens[s], n);
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      const uint32_t done = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      is_last = done == (uint32_t)gridDim.x - 1u;
    }
  }
  __syncthreads();
  if (!is_last) return;
  float l = 0.0f;
  z = 0.0f;
  n = 0;
  int filled = 0;
  for (int i = tid; i < p.S * tiles; i += 64 * kBalGroups) l += device_load(&p.seq_loss[i]);
  for (int i = tid; i < p.S; i += 64 * kBalGroups) {
    z += device_load(&p.seq_z[i]);
    const int ni = device_load(&p.seq_tokens[i]);
    n += ni;
    filled += ni > 0;
  }
  l = wave_sum(l);
  z = wave_sum(z);
  n = wave_sum(n);
  filled = wave_sum(filled);
  if (lane == 0) {
    rl[wave] = l;
    rz[wave] = z;
    rn[wave] = n;
    rf[wave] = filled;
  }
  __syncthreads();
  if (tid == 0) {
    l = z = 0.0f;
    n = filled = 0;
    for (int w = 0; w < kBalGroups; ++w) {
      l += rl[w];
      z += rz[w];
      n += rn[w];
      filled += rf[w];
    }
    balance_results(p, l, z, n, filled);
  }
}

struct RouterBwdArgs {
  const float* logits;
  const int32_t* ids;
  const float* w;
  const float* dw;         // null: no gradient through the routing weights
  int32_t T, E, k, S;
  const uint8_t* mask;
  const int32_t* offsets;
  const float* lse;
  const int32_t* counts;
  const int32_t* seq_tokens;
  const float* d_loss;     // null: no gradient of the losses
  float* d_logits;
};

// One wave per token, everything it needs in flight at once.  The routing
// weights' part is scattered over a row of LDS, one per wave.  16384 tokens of
// 288 experts: 11.4 us, 40 MB at 3.5 TB/s, so near memory's rate; 64 tokens 3.8
// us, a launch's latency.
template <int VPL>
__global__ __launch_bounds__(256) void router_bwd_kernel(RouterBwdArgs p) {
  __shared__ float scatter[4][64 * VPL];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = blockIdx.x * 4 + wave;
  if (t >= p.T) return;
  float v[VPL], d[VPL] = {};
  load_row<VPL>(p.logits + (int64_t)t * p.E, p.E, v);
  int id = -1;
  float w = 0.0f, dw = 0.0f, lse = 0.0f, g0 = 0.0f, g1 = 0.0f;
  if (p.dw && lane < p.k) {
    id = p.ids[(int64_t)t * p.k + lane];
    w = p.w[(int64_t)t * p.k + lane];
    dw = p.dw[(int64_t)t * p.k + lane];
  }
  const bool masked = p.mask && !p.mask[t];
  if (p.d_loss) {
    lse = p.lse[t];
    g0 = p.d_loss[0];
    g1 = p.d_loss[1];
  }
  const int s = p.offsets ? seq_of(p.offsets, p.T, p.S, t) : 0;
  float mx, sum;
  if (!masked && s < p.S && t >= seq_offset(p.offsets, p.T, 0) && exp_row<VPL>(v, p.E, mx, sum)) {
    if (p.d_loss) {
      // p from the row's own maximum and sum: exp(l - lse) loses log E where
      // every logit is the type's lowest value
      const float n = (float)p.seq_tokens[s], N = (float)p.seq_tokens[p.S], filled = (float)p.seq_tokens[p.S + 1];
      const float slope = g0 * (float)p.E / ((float)p.k * filled * n * n);
      const int32_t* counts = p.counts + (int64_t)s * p.E;
      float a[VPL], dot = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) a[i] = (float)counts[min(lane + 64 * i, p.E - 1)];
      const float inv = __builtin_amdgcn_rcpf(sum);
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        v[i] *= inv;
        dot = fmaf(v[i], a[i], dot);
      }
      const float off = fmaf(-slope, wave_sum(dot), g1 * 2.0f * lse / N);
#pragma unroll
      for (int i = 0; i < VPL; ++i) d[i] = v[i] * fmaf(slope, a[i], off);
    }
    if (p.dw) {
      const bool live = id >= 0 && id < p.E;
      w = live ? w : 0.0f;
      const float mean = wave_sum(live ? w * dw : 0.0f);
      float* row = scatter[wave];
#pragma unroll
      for (int i = 0; i < VPL; ++i) row[lane + 64 * i] = 0.0f;
      wave_lds_order();
      if (live) atomicAdd(&row[id], w * (dw - mean));
      wave_lds_order();
#pragma unroll
      for (int i = 0; i < VPL; ++i) d[i] += row[lane + 64 * i];
    }
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (lane + 64 * i < p.E) p.d_logits[(int64_t)t * p.E + lane + 64 * i] = d[i];
}

// Calls f with the number of 64-expert columns a lane holds (as the routing kernels).
template <typename F>
static void with_vpl(int E, F&& f) {
  const int v = (E + 63) / 64;
  if (v <= 1) f(std::integral_constant<int, 1>{});
  else if (v <= 2) f(std::integral_constant<int, 2>{});
  else if (v <= 4) f(std::integral_constant<int, 4>{});
  else if (v <= 5) f(std::integral_constant<int, 5>{});
  else if (v <= 8) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}

static hipError_t launch_balance(const BalanceArgs& p, hipStream_t s) {
  const int tiles = (p.E + 63) / 64;
  const size_t lds = (size_t)(kBalWaves + 1) * p.E * 4;
  const bool one = p.chunks == 1;
  hipError_t err = hipSuccess;
  with_vpl(p.E, [&](auto vpl) {
    constexpr int V = decltype(vpl)::value;
    if (one)
      hipLaunchKernelGGL((balance_chunk_kernel<V, true>), dim3(1), dim3(64 * kBalWaves), lds, s, p);
    else
      hipLaunchKernelGGL((balance_chunk_kernel<V, false>), dim3(p.chunks), dim3(64 * kBalWaves), lds, s, p);
    err = hipGetLastError();
  });
  if (err != hipSuccess || one) return err;
  hipLaunchKernelGGL(balance_finish_kernel, dim3((unsigned)(p.S * tiles)), dim3(64 * kBalGroups), 0, s, p, tiles);
  return hipGetLastError();
}

static hipError_t launch_router_bwd(const RouterBwdArgs& p, hipStream_t s) {
  with_vpl(p.E, [&](auto vpl) {
    hipLaunchKernelGGL(router_bwd_kernel<decltype(vpl)::value>, dim3((p.T + 3) / 4), dim3(256), 0, s, p);
  });
  return hipGetLastError();
}

}  // namespace moe

namespace {

constexpr int64_t kMaxPairs = 1ll << 24;
constexpr int32_t kMaxTopK = 16, kMaxSeqs = 1 << 16;

bool sizes_ok(int32_t T, int32_t E, int32_t k, int32_t S) {
  return T >= 0 && E >= 1 && E <= moe::kBalMaxExperts && k >= 1 && k <= kMaxTopK && k <= E && (int64_t)T * k <= kMaxPairs &&
         S >= 1 && S <= kMaxSeqs;
}
size_t up256(int64_t v) { return (size_t)((v + 255) / 256 * 256); }
bool aligned4(const void* p) { return (uintptr_t)p % 4 == 0; }

}  // namespace

extern "C" {

size_t moe_balance_bytes(int32_t T, int32_t E, int32_t num_seqs) {
  if (!sizes_ok(T, E, 1, num_seqs) || T <= moe::bal_chunk(E)) return 0;  // one workgroup keeps its sums to itself
  const int64_t slots = (T + moe::bal_chunk(E) - 1) / moe::bal_chunk(E) + (int64_t)num_seqs;
  return 2 * up256(slots * E * 4) + 2 * up256(slots * 4) + up256((int64_t)num_seqs * ((E + 63) / 64) * 4) +
         up256((int64_t)num_seqs * 4) + 256;
}

moe_status_t moe_balance_loss(const float* logits, const int32_t* ids, int32_t T, int32_t E, int32_t top_k,
                              const uint8_t* token_mask, const int32_t* seq_offsets, int32_t num_seqs, float* loss,
                              int32_t* counts, int32_t* seq_tokens, float* lse, void* ws, size_t ws_bytes,
                              void* stream) {
  if (!sizes_ok(T, E, top_k, num_seqs) || (!seq_offsets && num_seqs != 1)) return MOE_ERR_SHAPE;
  const size_t need = moe_balance_bytes(T, E, num_seqs);
  if (!loss || !counts || !seq_tokens || (need && !ws) || (T > 0 && (!logits || !ids || !lse))) return MOE_ERR_NULL;
  if (!aligned4(logits) || !aligned4(ids) || !aligned4(seq_offsets) || !aligned4(loss) || !aligned4(counts) ||
      !aligned4(seq_tokens) || !aligned4(lse) || (uintptr_t)ws % 16)
    return MOE_ERR_ALIGN;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  moe::BalanceArgs p{};
  p.logits = logits;
  p.ids = ids;
  p.T = T;
  p.E = E;
  p.k = top_k;
  p.S = num_seqs;
  p.chunk = moe::bal_chunk(E);
  p.chunks = T > 0 ? (T + p.chunk - 1) / p.chunk : 1;  // without tokens: zeros are written all the same
  p.mask = token_mask;
  p.offsets = seq_offsets;
  p.lse = lse;
  p.counts = counts;
  p.seq_tokens = seq_tokens;
  p.loss = loss;
  if (!need) return moe::launch_balance(p, (hipStream_t)stream) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
  const int64_t slots = p.chunks + (int64_t)num_seqs;
  uint8_t* w = (uint8_t*)ws;
  p.psum = (float*)w; w += up256(slots * E * 4);
  p.pcount = (int32_t*)w; w += up256(slots * E * 4);
  p.pz = (float*)w; w += up256(slots * 4);
  p.pn = (int32_t*)w; w += up256(slots * 4);
  p.seq_loss = (float*)w; w += up256((int64_t)num_seqs * ((E + 63) / 64) * 4);
  p.seq_z = (float*)w; w += up256((int64_t)num_seqs * 4);
  p.ticket = (uint32_t*)w;
  return moe::launch_balance(p, (hipStream_t)stream) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status_t moe_router_bwd(const float* logits, const int32_t* ids, const float* weights, const float* d_weights,
                            int32_t T, int32_t E, int32_t top_k, const uint8_t* token_mask,
                            const int32_t* seq_offsets, int32_t num_seqs, const float* lse, const int32_t* counts,
                            const int32_t* seq_tokens, const float* d_loss, float* d_logits, void* stream) {
  if (!sizes_ok(T, E, top_k, num_seqs) || (!seq_offsets && num_seqs != 1)) return MOE_ERR_SHAPE;
  if (T == 0) return MOE_OK;
  if (!logits || !d_logits || (!d_weights && !d_loss)) return MOE_ERR_NULL;
  if (d_weights && (!weights || !ids)) return MOE_ERR_NULL;
  if (d_loss && (!lse || !counts || !seq_tokens)) return MOE_ERR_NULL;
  if (!aligned4(logits) || !aligned4(ids) || !aligned4(weights) || !aligned4(d_weights) || !aligned4(seq_offsets) ||
      !aligned4(lse) || !aligned4(counts) || !aligned4(seq_tokens) || !aligned4(d_loss) || !aligned4(d_logits))
    return MOE_ERR_ALIGN;
  const moe::RouterBwdArgs p{logits, ids, weights, d_weights, T, E, top_k, num_seqs, token_mask, seq_offsets,
                             lse, counts, seq_tokens, d_loss, d_logits};
  return moe::launch_router_bwd(p, (hipStream_t)stream) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // extern "C"
