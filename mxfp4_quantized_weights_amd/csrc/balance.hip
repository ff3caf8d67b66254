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

constexpr int kBalChunk = 64;      // tokens per workgroup
constexpr int kBalWaves = 16;
constexpr int kBalGroups = 16;     // slot groups (waves) of the finishing workgroups
constexpr int kBalMaxExperts = 1024;

struct BalanceArgs {
  const float* logits;
  const int32_t* ids;
  int32_t T, E, k, S, chunks;
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

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}

// One workgroup per chunk of 64 tokens, one wave per token.  The chunk is
// walked sequence by sequence; each (chunk, sequence) overlap leaves its sums
// in a slot of its own (c + s: along the rows every new overlap raises c or s,
// so no two share a slot), added up in slot order by balance_finish_kernel.
template <int VPL>
__global__ __launch_bounds__(64 * kBalWaves) void balance_chunk_kernel(BalanceArgs p) {
  extern __shared__ float smem[];
  float* red = smem;                                   // [kBalWaves][E]
  int32_t* hist = (int32_t*)(red + kBalWaves * p.E);   // [E]
  __shared__ float red_z[kBalWaves];
  __shared__ int32_t red_n[kBalWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c = blockIdx.x, tb = c * kBalChunk, te = min(p.T, tb + kBalChunk);
  if (c == 0 && tid == 0) *p.ticket = 0;
  // rows outside every sequence
  const int first = min(max(seq_offset(p.offsets, p.T, 0), tb), te);
  const int last = min(max(seq_offset(p.offsets, p.T, p.S), first), te);
  for (int t = tb + tid; t < te; t += 64 * kBalWaves)
    if (t < first || t >= last) p.lse[t] = 0.0f;
  int t0 = first;
  while (t0 < last) {
    const int s = p.offsets ? seq_of(p.offsets, p.T, p.S, t0) : 0;
    if (s >= p.S) break;
    const int t1 = max(min(seq_offset(p.offsets, p.T, s + 1), last), t0 + 1);
    for (int e = tid; e < p.E; e += 64 * kBalWaves) hist[e] = 0;
    __syncthreads();
    float acc[VPL] = {}, z = 0.0f;
    int n = 0;
    for (int t = t0 + wave; t < t1; t += kBalWaves) {
      const float* row = p.logits + (int64_t)t * p.E;
      float v[VPL];
#pragma unroll
      for (int i = 0; i < VPL; ++i) v[i] = row[min(lane + 64 * i, p.E - 1)];
      const int id = lane < p.k ? p.ids[(int64_t)t * p.k + lane] : -1;
      const bool masked = p.mask && !p.mask[t];
      float mx = -INFINITY;
      bool some = false;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (lane + 64 * i >= p.E) v[i] = -INFINITY;
        mx = fmaxf(mx, v[i]);
        some |= !(v[i] == -INFINITY);  // a NaN counts: it has to show in the loss
      }
      if (masked || !__any(some)) {
        if (lane == 0) p.lse[t] = 0.0f;
        continue;
      }
      mx = wave_max(mx);
      float ex[VPL], sum = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        ex[i] = expf(v[i] - mx);
        sum += ex[i];
      }
      sum = wave_sum(sum);
      const float lse = mx + logf(sum), inv = 1.0f / sum;
#pragma unroll
      for (int i = 0; i < VPL; ++i) acc[i] += ex[i] * inv;
      z += lse * lse;
      ++n;
      if (lane == 0) p.lse[t] = lse;
      if (id >= 0 && id < p.E) atomicAdd(&hist[id], 1);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + 64 * i < p.E) red[wave * p.E + lane + 64 * i] = acc[i];
    if (lane == 0) {
      red_z[wave] = z;
      red_n[wave] = n;
    }
    __syncthreads();
    const int64_t slot = c + s;
    for (int e = tid; e < p.E; e += 64 * kBalWaves) {
      float sum = 0.0f;
      for (int w = 0; w < kBalWaves; ++w) sum += red[w * p.E + e];
      p.psum[slot * p.E + e] = sum;
      p.pcount[slot * p.E + e] = hist[e];
    }
    if (tid == 0) {
      float sum = 0.0f;
      int cnt = 0;
      for (int w = 0; w < kBalWaves; ++w) {
        sum += red_z[w];
        cnt += red_n[w];
      }
      p.pz[slot] = sum;
      p.pn[slot] = cnt;
    }
    __syncthreads();
    t0 = t1;
  }
}

// Workgroup (s, tile of 64 experts): adds the sequence's slots in a fixed
// order, leaves its counts and its share of the loss; the last workgroup to
// finish adds the shares up, again in a fixed order.
__global__ __launch_bounds__(64 * kBalGroups) void balance_finish_kernel(BalanceArgs p, int tiles) {
  __shared__ float rp[kBalGroups][64];
  __shared__ int32_t rc[kBalGroups][64];
  __shared__ float rz[kBalGroups];
  __shared__ int32_t rn[kBalGroups];
  __shared__ int32_t is_last;
  __shared__ float fz[kBalGroups], fl[kBalGroups];
  __shared__ int32_t fn[kBalGroups], ff[kBalGroups];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int s = blockIdx.x / tiles, tile = blockIdx.x % tiles;
  const int e = tile * 64 + lane;
  const int lo = seq_offset(p.offsets, p.T, s), hi = seq_offset(p.offsets, p.T, s + 1);
  const int c0 = lo / kBalChunk, c1 = lo < hi ? (hi - 1) / kBalChunk + 1 : c0;
  float sum = 0.0f;
  int cnt = 0;
  if (e < p.E) {
#pragma unroll 8
    for (int c = c0 + wave; c < c1; c += kBalGroups) {
      sum += p.psum[(int64_t)(c + s) * p.E + e];
      cnt += p.pcount[(int64_t)(c + s) * p.E + e];
    }
  }
  float z = 0.0f;
  int n = 0;
  for (int c = c0 + tid; c < c1; c += 64 * kBalGroups) {
    z += p.pz[c + s];
    n += p.pn[c + s];
  }
  z = wave_sum(z);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o);
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
    for (int w = 0; w < kBalGroups; ++w) {
      sum += rp[w][lane];
      cnt += rc[w][lane];
      z += rz[w];
      n += rn[w];
    }
    if (e < p.E) p.counts[(int64_t)s * p.E + e] = cnt;
    float share = (n > 0 && e < p.E) ? ((float)cnt * (float)p.E / ((float)p.k * (float)n)) * (sum / (float)n) : 0.0f;
    share = wave_sum(share);
    if (lane == 0) {
      p.seq_loss[(int64_t)s * tiles + tile] = share;
      if (tile == 0) {
        p.seq_z[s] = z;
        p.seq_tokens[s] = n;
      }
      __threadfence();
      const uint32_t done = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
      is_last = done == (uint32_t)gridDim.x - 1u;
    }
  }
  __syncthreads();
  if (!is_last) return;
  __threadfence();
  float l = 0.0f;
  z = 0.0f;
  n = 0;
  int filled = 0;
  for (int i = tid; i < p.S * tiles; i += 64 * kBalGroups)
    l += __hip_atomic_load(&p.seq_loss[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (int i = tid; i < p.S; i += 64 * kBalGroups) {
    z += __hip_atomic_load(&p.seq_z[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const int ni = __hip_atomic_load(&p.seq_tokens[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    n += ni;
    filled += ni > 0;
  }
  l = wave_sum(l);
  z = wave_sum(z);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    n += __shfl_xor(n, o);
    filled += __shfl_xor(filled, o);
  }
  if (lane == 0) {
    fl[wave] = l;
    fz[wave] = z;
    fn[wave] = n;
    ff[wave] = filled;
  }
  __syncthreads();
  if (tid == 0) {
    l = z = 0.0f;
    n = filled = 0;
    for (int w = 0; w < kBalGroups; ++w) {
      l += fl[w];
      z += fz[w];
      n += fn[w];
      filled += ff[w];
    }
    p.loss[0] = filled ? l / (float)filled : 0.0f;
    p.loss[1] = n ? z / (float)n : 0.0f;
    p.seq_tokens[p.S] = n;
    p.seq_tokens[p.S + 1] = filled;
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

// One wave per token.
template <int VPL>
__global__ __launch_bounds__(256) void router_bwd_kernel(RouterBwdArgs p) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= p.T) return;
  const float* row = p.logits + (int64_t)t * p.E;
  float v[VPL], d[VPL] = {};
  bool some = false;
#pragma unroll
  for (int i = 0; i < VPL; ++i) v[i] = row[min(lane + 64 * i, p.E - 1)];
  const int s = p.offsets ? seq_of(p.offsets, p.T, p.S, t) : 0;
  const bool inside = s < p.S && t >= seq_offset(p.offsets, p.T, 0) && !(p.mask && !p.mask[t]);
#pragma unroll
  for (int i = 0; i < VPL; ++i) some |= lane + 64 * i < p.E && !(v[i] == -INFINITY);
  if (inside && __any(some)) {
    if (p.d_loss) {
      const float lse = p.lse[t];
      const float n = (float)p.seq_tokens[s], N = (float)p.seq_tokens[p.S], filled = (float)p.seq_tokens[p.S + 1];
      const float slope = p.d_loss[0] * (float)p.E / ((float)p.k * filled * n * n);
      const float gz = p.d_loss[1] * 2.0f * lse / N;
      // p from the row's own maximum and sum: exp(l - lse) loses log E where
      // every logit is the type's lowest value
      float pr[VPL], a[VPL], mx = -INFINITY, sum = 0.0f, dot = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) mx = fmaxf(mx, lane + 64 * i < p.E ? v[i] : -INFINITY);
      mx = wave_max(mx);
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        pr[i] = lane + 64 * i < p.E ? expf(v[i] - mx) : 0.0f;
        sum += pr[i];
      }
      const float inv = 1.0f / wave_sum(sum);
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = lane + 64 * i;
        pr[i] *= inv;
        a[i] = e < p.E ? slope * (float)p.counts[(int64_t)s * p.E + e] : 0.0f;
        dot += pr[i] * a[i];
      }
      dot = wave_sum(dot);
#pragma unroll
      for (int i = 0; i < VPL; ++i) d[i] = pr[i] * (a[i] - dot + gz);
    }
    if (p.dw) {
      const int id = lane < p.k ? p.ids[(int64_t)t * p.k + lane] : -1;
      const bool live = id >= 0 && id < p.E;
      const float w = live ? p.w[(int64_t)t * p.k + lane] : 0.0f, dw = live ? p.dw[(int64_t)t * p.k + lane] : 0.0f;
      const float mean = wave_sum(w * dw);
      const float through = w * (dw - mean);
      for (int j = 0; j < p.k; ++j) {
        const int ej = __builtin_amdgcn_readlane(id, j);
        const float g = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(through), j));
#pragma unroll
        for (int i = 0; i < VPL; ++i) d[i] += ej == lane + 64 * i ? g : 0.0f;
      }
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
  hipError_t err = hipSuccess;
  with_vpl(p.E, [&](auto vpl) {
    auto kernel = balance_chunk_kernel<decltype(vpl)::value>;
    if (lds > 65536)
      err = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (err == hipSuccess) {
      hipLaunchKernelGGL(kernel, dim3(p.chunks), dim3(64 * kBalWaves), lds, s, p);
      err = hipGetLastError();
    }
  });
  if (err != hipSuccess) return err;
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
  if (!sizes_ok(T, E, 1, num_seqs)) return 0;
  const int64_t slots = (T + moe::kBalChunk - 1) / moe::kBalChunk + (int64_t)num_seqs;
  return 2 * up256(slots * E * 4) + 2 * up256(slots * 4) + up256((int64_t)num_seqs * ((E + 63) / 64) * 4) +
         up256((int64_t)num_seqs * 4) + 256;
}

moe_status_t moe_balance_loss(const float* logits, const int32_t* ids, int32_t T, int32_t E, int32_t top_k,
                              const uint8_t* token_mask, const int32_t* seq_offsets, int32_t num_seqs, float* loss,
                              int32_t* counts, int32_t* seq_tokens, float* lse, void* ws, size_t ws_bytes,
                              void* stream) {
  if (!sizes_ok(T, E, top_k, num_seqs) || (!seq_offsets && num_seqs != 1)) return MOE_ERR_SHAPE;
  if (!loss || !counts || !seq_tokens || !ws || (T > 0 && (!logits || !ids || !lse))) return MOE_ERR_NULL;
  if (!aligned4(logits) || !aligned4(ids) || !aligned4(seq_offsets) || !aligned4(loss) || !aligned4(counts) ||
      !aligned4(seq_tokens) || !aligned4(lse) || (uintptr_t)ws % 16)
    return MOE_ERR_ALIGN;
  if (ws_bytes < moe_balance_bytes(T, E, num_seqs)) return MOE_ERR_WORKSPACE;
  moe::BalanceArgs p{};
  p.logits = logits;
  p.ids = ids;
  p.T = T;
  p.E = E;
  p.k = top_k;
  p.S = num_seqs;
  p.chunks = T > 0 ? (T + moe::kBalChunk - 1) / moe::kBalChunk : 1;  // without tokens: the ticket is still reset
  p.mask = token_mask;
  p.offsets = seq_offsets;
  p.lse = lse;
  p.counts = counts;
  p.seq_tokens = seq_tokens;
  p.loss = loss;
  const int64_t slots = (T + moe::kBalChunk - 1) / moe::kBalChunk + (int64_t)num_seqs;
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
