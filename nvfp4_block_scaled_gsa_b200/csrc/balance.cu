// balance.cu — the router's load-balance loss with its per-expert counts and its gradient.
//
// Over the tokens of sequence s that count (n_s of them), with c[s][e] of their k slots routed to
// expert e, p_t = softmax(logits_t) and S' sequences that hold a token:
//
//   f[s][e] = E c[s][e] / (k n_s)
//   loss    = alpha / S' * sum_s sum_e f[s][e] * (1/n_s) sum_{t in s} p_t[e]
//           = sum_t a_s v_t,   a_s = alpha / (S' n_s),  v_t = sum_e f[s][e] p_t[e]
//   dlogits_t[e] = dloss * a_s * p_t[e] * (f[s][e] - v_t)        (the counts have no gradient)
//
// With the counts known the loss is a sum over tokens of the same v_t that the gradient needs, so
// one pass over the logits gives both; no mean probability per expert is ever formed.  Two launches:
// the counts from the ids (a cluster per sequence, its CTAs' histograms joined through distributed
// shared memory, nothing to zero), and the pass, which loads its first logits while the counts
// are still being made.  Gradient of 40961 x 160: 20.0 us, 2.6 TB/s.  The schedulers issue in 63% of the
// cycles in which an SM is busy (227 warp instructions a token), and what is left is the start, three
// dependent loads, and the tail.  Below that the chain of launches and dependent loads is the bound
// (8192 x 256 with the counts: 12.4 us, 64 x 8: 6.7 us; 40000 x 256 with the counts: 32.8 us).
#include "common.cuh"
#include "launch.h"

namespace nvfp4 {
namespace {

constexpr int kMaxE = 256;
constexpr int kMaxK = 32;
constexpr int kCountThreads = 512;
// CTAs per sequence, up to kClusterSeqs sequences, and one above: 40000 x 256 top-8 in 65 even sequences
// 29.3 us with one CTA each against 33.6 with clusters, in 256 30.4 against 44.4.  One long sequence
// among short ones would want the cluster (65: 52.2 us against 106), but the lengths are not known here.
constexpr int kCountCluster = 8;
constexpr int kClusterSeqs = 64;
constexpr int kThreads = 256;
// CTAs of the pass, at most: the 3 that an SM holds on each of the 148 (more than one round of
// CTAs would pay for the start, three dependent loads, again)
constexpr int kMaxCtas = 148 * 3;
constexpr int kOffsCache = 1024;  // sequence offsets kept in shared memory, at most

__device__ __forceinline__ int clamp_to(int v, int lo, int hi) { return min(max(v, lo), hi); }

// Counts of one sequence by the CTAs of a cluster (or one CTA).
__global__ void __launch_bounds__(kCountThreads) balance_count_kernel(
    const int32_t* __restrict__ ids, int T, int E, int k, const int32_t* __restrict__ seq_offs,
    const uint8_t* __restrict__ mask, int cluster, int32_t* __restrict__ counts,
    int32_t* __restrict__ tokens, uint32_t* __restrict__ ticket, int32_t* __restrict__ dev_status) {
  pdl_trigger();
  __shared__ int hist[kMaxE + 1];  // [E]: the tokens
  const int tid = threadIdx.x;
  const int s = blockIdx.x / cluster, rank = blockIdx.x % cluster;
  for (int e = tid; e <= E; e += kCountThreads) hist[e] = 0;
  if (blockIdx.x == 0 && tid == 0 && ticket != nullptr) *ticket = 0;
  int lo = 0, hi = T;
  bool bad = false;
  if (seq_offs != nullptr) {
    const int a = __ldg(seq_offs + s), b = __ldg(seq_offs + s + 1);
    lo = clamp_to(a, 0, T);
    hi = clamp_to(b, lo, T);
    if (a != lo || b != hi) report(dev_status, NVFP4_DEVERR_BAD_OFFSETS);
  }
  __syncthreads();
  // this CTA's part of the sequence's tokens, and their slots (T * k < 2^30: 32-bit indices)
  const int n = hi - lo, per = (n + cluster - 1) / cluster;
  const int t0 = lo + min(n, per * rank), t1 = lo + min(n, per * (rank + 1));
  int held = 0;
  if (mask == nullptr) {
    held = tid == 0 ? t1 - t0 : 0;
  } else {
    for (int t = t0 + tid; t < t1; t += kCountThreads) held += __ldg(mask + t) != 0;
  }
  held = __reduce_add_sync(0xffffffffu, held);
  if ((tid & 31) == 0 && held) atomicAdd(&hist[E], held);
  constexpr int kAhead = 16;
  const int j1 = t1 * k;
  for (int j = t0 * k + tid; j < j1; j += kCountThreads * kAhead) {
    int id[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int at = j + u * kCountThreads;
      id[u] = -1;
      if (at < j1 && (mask == nullptr || __ldg(mask + static_cast<unsigned>(at) / static_cast<unsigned>(k)) != 0))
        id[u] = __ldg(ids + at);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (id[u] >= E) bad = true;
      else if (id[u] >= 0) atomicAdd(&hist[id[u]], 1);
    }
  }
  if (bad) report(dev_status, NVFP4_DEVERR_BAD_INDEX);
  if (cluster > 1) cluster_sync();
  else __syncthreads();
  for (int e = rank * kCountThreads + tid; e <= E; e += cluster * kCountThreads) {
    int sum = 0;
    if (cluster > 1) {  // kCountCluster CTAs, their words in flight together
      const uint32_t at = smem_u32(&hist[e]);
      int v[kCountCluster];
#pragma unroll
      for (int c = 0; c < kCountCluster; ++c)
        asm volatile("ld.shared::cluster.s32 %0, [%1];"
                     : "=r"(v[c])
                     : "r"(mapa_shared(at, c))
                     : "memory");
#pragma unroll
      for (int c = 0; c < kCountCluster; ++c) sum += v[c];
    } else {
      sum = hist[e];
    }
    if (e < E) counts[(int64_t)s * E + e] = sum;
    else tokens[s] = sum;
  }
  if (cluster > 1) cluster_sync();  // the peers have read this CTA's histogram
}

struct Args {
  const float* logits;
  int64_t ld;
  int T, E, k;
  const int32_t* seq_offs;
  int S;
  const uint8_t* mask;
  float alpha;
  const int32_t* counts;
  const int32_t* tokens;
  const float* dloss;
  float* dlogits;
  int accumulate;
  float* loss;
  double* part;      // [CTAs]
  uint32_t* ticket;  // zero when the CTAs start to finish
  int iters;         // groups of 32 / L tokens per warp
};

// 1 / x by the hardware's approximation, for quotient() to correct.
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// a / b from y = 1 / b, which may be a few steps off: the remainder of a y is exact in one fma, and adding
// its share leaves about half a step.  a = b gives 1 to the bit.
__device__ __forceinline__ float quotient(float a, float b, float y) {
  const float q = a * y;
  return fmaf(fmaf(-q, b, a), y, q);
}

// L lanes per token, 4 * NV logits each; a warp takes 32 / L consecutive tokens at a time.  Many
// logits per lane keep the shuffles of the row sums few (40961 x 160 at 32 lanes of 8: 18.4 us against 17.2
// for the same arithmetic, with a shorter exponential than today's).  VEC: a lane's logits are NV
// 16-byte groups (E % 4 == 0 and rows 16-byte aligned), else words L apart.
template <int L, int NV, bool VEC>
__global__ void __launch_bounds__(kThreads, 3) balance_kernel(const Args A) {
  constexpr int G = 32 / L, kSlots = 4 * NV;
  const int tid = threadIdx.x, lane = tid & 31, l = lane % L, grp = lane / L;
  const int E = A.E;
  auto expert = [&](int i) { return VEC ? 4 * (l + L * (i >> 2)) + (i & 3) : l + L * i; };
  const int64_t warp = (int64_t)blockIdx.x * (kThreads / 32) + (tid >> 5);
  const int64_t t_first = warp * A.iters * G + grp;
  // logits past E, and tokens past T, read as -inf: probability 0
  auto load = [&](int64_t t, float (&v)[kSlots]) {
    const float* row = A.logits + t * A.ld;
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < kSlots; i += 4) {
        float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (t < A.T && expert(i) < E) q = __ldg(reinterpret_cast<const float4*>(row + expert(i)));
        v[i] = q.x;
        v[i + 1] = q.y;
        v[i + 2] = q.z;
        v[i + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kSlots; ++i)
        v[i] = t < A.T && expert(i) < E ? __ldg(row + expert(i)) : -INFINITY;
    }
  };
  auto masked = [&](int64_t t) {
    return A.mask != nullptr && t < A.T && __ldg(A.mask + t) == 0;
  };
  float v[kSlots];
  load(t_first, v);
  bool skip = masked(t_first);
  __shared__ int s_busy, s_offs[kOffsCache], s_counts[kMaxE];
  const int* offs = A.seq_offs;
  if (A.S < kOffsCache) {
    for (int s = tid; s <= A.S; s += kThreads)
      s_offs[s] = A.seq_offs == nullptr ? (s == 0 ? 0 : A.T) : __ldg(A.seq_offs + s);
    offs = s_offs;
  }
  if (tid == 0) s_busy = 0;
  __syncthreads();
  pdl_wait();  // the counts

  // the last sequence that starts at or before t, given offs[lo] <= t < offs[S]
  auto find = [&](int64_t t, int lo) {
    int hi = A.S;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (offs[mid] <= t) lo = mid;
      else hi = mid;
    }
    return lo;
  };
  // The counts of the sequence that the CTA's first token is in (or the first sequence) are read
  // once per CTA: most CTAs lie in one sequence, and thousands of warps reading the same few lines
  // would queue at one slice of L2 (8192 x 256 with the counting: 21.0 us, against 12.7).
  const int64_t t_cta = (int64_t)blockIdx.x * (kThreads / 32) * A.iters * G;
  const int s_cta = t_cta < offs[0] || t_cta >= offs[A.S] ? 0 : find(t_cta, 0);
  int c_cta = 0, busy = 0;
  if (tid < E) c_cta = ld_after(A.counts + (int64_t)s_cta * E + tid);
  const int n_cta = ld_after(A.tokens + s_cta);
  for (int j = tid; j < A.S; j += kThreads) busy += ld_after(A.tokens + j) > 0;
  const float up = A.dloss != nullptr ? __ldg(A.dloss) : 1.0f;
  busy = __reduce_add_sync(0xffffffffu, busy);
  if (lane == 0 && busy) atomicAdd(&s_busy, busy);
  if (tid < E) s_counts[tid] = c_cta;
  __syncthreads();
  const float share = s_busy > 0 ? 1.0f / static_cast<float>(s_busy) : 0.0f;

  // the sequence of the group's current token
  int s = -1, s_end = 0;
  bool inside = false;  // a sequence with tokens
  float f[kSlots], per_token = 0.0f;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) f[i] = 0.0f;
  auto enter = [&](int64_t t) {
    const int lo = max(s, 0);
    if (t >= offs[A.S] || t < offs[lo]) {
      inside = false;
      s_end = t < offs[lo] ? offs[lo] : A.T;
      return;
    }
    s = find(t, lo);
    s_end = offs[s + 1];
    const int n = s == s_cta ? n_cta : ld_after(A.tokens + s);
    inside = n > 0;
    per_token = inside ? A.alpha / static_cast<float>(n) * share : 0.0f;
    const float even = inside ? static_cast<float>(A.k) * static_cast<float>(n) : 1.0f;
    const float per_even = inside ? 1.0f / even : 0.0f;
    int c[kSlots];
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      c[i] = 0;
      if (expert(i) < E)
        c[i] = s == s_cta ? s_counts[expert(i)] : ld_after(A.counts + (int64_t)s * E + expert(i));
    }
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
      f[i] = quotient(static_cast<float>(c[i]) * static_cast<float>(E), even, per_even);
  };

  double sum = 0.0;
  for (int it = 0; it < A.iters; ++it) {
    const int64_t t = t_first + (int64_t)it * G;
    if (t - grp >= A.T) break;  // the whole warp
    float nxt[kSlots];
    bool nxt_skip = false;
    if (it + 1 < A.iters) {
      load(t + G, nxt);
      nxt_skip = masked(t + G);
    }
    if (t < A.T && t >= s_end) enter(t);
    const bool counted = t < A.T && inside && !skip;
    const float coef = per_token;
    float m = v[0];
#pragma unroll
    for (int i = 1; i < kSlots; ++i) m = fmaxf(m, v[i]);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m == -INFINITY) m = 0.0f;  // a row of nothing but -inf: no probabilities
    float z = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      // (2^(x log2 e) by the hardware alone is 2 to 6% faster, but its error grows with |x|: 3.5e-6 at
      // 80 below the maximum)
      v[i] = expf(v[i] - m);
      z += v[i];
      dot += v[i] * f[i];
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) {
      z += __shfl_xor_sync(0xffffffffu, z, o);
      dot += __shfl_xor_sync(0xffffffffu, dot, o);
    }
    // Where every f is 1 (an even load), dot is z to the bit, so vt is 1 and the gradient exactly 0.
    const float y = z == 0.0f ? 0.0f : rcp_approx(z);
    const float inv = quotient(1.0f, z, y), vt = quotient(dot, z, y);
    if (A.loss != nullptr && counted && l == 0)
      sum += static_cast<double>(coef) * static_cast<double>(vt);
    if (A.dlogits != nullptr && t < A.T) {
      float* row = A.dlogits + t * E;
      const float scale = up * coef * inv;
      float d[kSlots];
#pragma unroll
      for (int i = 0; i < kSlots; ++i) d[i] = scale * v[i] * (f[i] - vt);
      if (__any_sync(__activemask(), !counted)) {  // (rare, so a branch and not a select each)
#pragma unroll
        for (int i = 0; i < kSlots; ++i) d[i] = counted ? d[i] : 0.0f;  // whatever the row holds
      }
      if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < kSlots; i += 4) {
          if (expert(i) >= E) continue;
          float4* at = reinterpret_cast<float4*>(row + expert(i));
          float4 o = make_float4(d[i], d[i + 1], d[i + 2], d[i + 3]);
          if (A.accumulate) {
            const float4 was = *at;
            o.x += was.x;
            o.y += was.y;
            o.z += was.z;
            o.w += was.w;
          }
          *at = o;
        }
      } else {
#pragma unroll
        for (int i = 0; i < kSlots; ++i)
          if (expert(i) < E) row[expert(i)] = A.accumulate ? row[expert(i)] + d[i] : d[i];
      }
    }
#pragma unroll
    for (int i = 0; i < kSlots; ++i) v[i] = nxt[i];
    skip = nxt_skip;
  }

  if (A.loss == nullptr) return;
  // one float64 sum per CTA; the CTA that finishes last adds them in order
  __shared__ double s_sum[kThreads / 32];
  __shared__ bool s_last;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_sum[tid >> 5] = sum;
  __syncthreads();
  if (tid == 0) {
    double total = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) total += s_sum[w];
    A.part[blockIdx.x] = total;
    __threadfence();
    s_last = atomicAdd(A.ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  double total = 0.0;
  constexpr int kPer = (kMaxCtas + kThreads - 1) / kThreads;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int c = tid + j * kThreads;
    if (c < static_cast<int>(gridDim.x)) total += ld_after(A.part + c);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (lane == 0) s_sum[tid >> 5] = total;
  __syncthreads();
  if (tid == 0) {
    total = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) total += s_sum[w];
    *A.loss = static_cast<float>(total);
  }
}

// The fewest lanes per token (2, 4, 8 or 16) that hold at most 16 logits each.
int lanes_for(int E) {
  int L = 2;
  while (16 * L < E) L *= 2;
  return L;
}

// iters (token groups per warp) and the grid of the pass
void pass_shape(int T, int E, int& iters, int& ctas) {
  const int G = 32 / lanes_for(E), warps = kThreads / 32;
  const int64_t groups = ((int64_t)T + G - 1) / G;
  const int64_t most = (int64_t)kMaxCtas * warps;
  iters = static_cast<int>((groups + most - 1) / most);
  if (iters < 1) iters = 1;
  const int64_t per_cta = (int64_t)iters * warps;
  ctas = static_cast<int>((groups + per_cta - 1) / per_cta);
  if (ctas < 1) ctas = 1;
}

template <int L, int NV>
nvfp4_status_t launch_pass(Args& a, bool vec, bool early, cudaStream_t s) {
  int ctas;
  pass_shape(a.T, a.E, a.iters, ctas);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = early ? 1 : 0;
  if (vec) cudaLaunchKernelEx(&cfg, balance_kernel<L, NV, true>, static_cast<const Args>(a));
  else cudaLaunchKernelEx(&cfg, balance_kernel<L, NV, false>, static_cast<const Args>(a));
  return check_launch("balance_kernel");
}

nvfp4_status_t pass(Args& a, bool early, cudaStream_t s) {
  const bool vec = a.E % 4 == 0 && a.ld % 4 == 0 && aligned16(a.logits) && aligned16(a.dlogits);
  const int L = lanes_for(a.E), nv = (a.E + 4 * L - 1) / (4 * L);  // nv >= 3 for L > 2
  switch (L) {
    case 2:
      return nv == 1   ? launch_pass<2, 1>(a, vec, early, s)
             : nv == 2 ? launch_pass<2, 2>(a, vec, early, s)
             : nv == 3 ? launch_pass<2, 3>(a, vec, early, s)
                       : launch_pass<2, 4>(a, vec, early, s);
    case 4: return nv == 3 ? launch_pass<4, 3>(a, vec, early, s) : launch_pass<4, 4>(a, vec, early, s);
    case 8: return nv == 3 ? launch_pass<8, 3>(a, vec, early, s) : launch_pass<8, 4>(a, vec, early, s);
    default:
      return nv == 3 ? launch_pass<16, 3>(a, vec, early, s) : launch_pass<16, 4>(a, vec, early, s);
  }
}

constexpr int64_t kPartOffset = 256;  // workspace: the ticket, then a float64 per CTA

nvfp4_status_t check_shape(int T, int E, int k, int64_t ld, int S, const int32_t* seq_offs) {
  if (T < 0 || E < 1 || k < 1 || ld < E || S < 1) return NVFP4_ERR_INVALID_ARG;
  if (E > kMaxE || k > kMaxK || k > E || (int64_t)T * k > (int64_t)1 << 30 || S > (1 << 24))
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (seq_offs == nullptr && S != 1) return NVFP4_ERR_INVALID_ARG;
  return NVFP4_OK;
}

// Whether the gradient's rows lie over any of the logits, which other warps may still have to read.
bool over_logits(const float* logits, int64_t ld, int T, int E, const float* dlogits) {
  return rows_overlap(logits, T, ld * 4, (int64_t)E * 4, dlogits, (int64_t)T * E * 4);
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" size_t moe_balance_loss_workspace_size(int T, int E) {
  if (T < 0 || E < 1 || E > kMaxE) return 0;
  int iters, ctas;
  pass_shape(T, E, iters, ctas);
  return static_cast<size_t>(kPartOffset + (int64_t)ctas * 8);
}

extern "C" nvfp4_status_t moe_balance_loss(const float* logits, int64_t ld, int T, int E, int k,
                                           const int32_t* topk_ids, const int32_t* seq_offs, int S,
                                           const uint8_t* mask, float alpha, int32_t* counts,
                                           int32_t* tokens, float* loss, const float* dloss,
                                           float* dlogits, int accumulate, void* ws,
                                           size_t ws_bytes, int32_t* dev_status,
                                           nvfp4_stream_t stream) {
  nvfp4_status_t st = check_shape(T, E, k, ld, S, seq_offs);
  if (st != NVFP4_OK) return st;
  if (!counts || !tokens || !loss || !ws) return NVFP4_ERR_INVALID_ARG;
  if (T > 0 && (!logits || !topk_ids)) return NVFP4_ERR_INVALID_ARG;
  if (ws_bytes < moe_balance_loss_workspace_size(T, E)) return NVFP4_ERR_WORKSPACE_TOO_SMALL;
  const void* ptrs4[] = {logits, topk_ids, seq_offs, counts, tokens, loss, dloss, dlogits, dev_status};
  for (const void* p : ptrs4)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return NVFP4_ERR_MISALIGNED;
  if (!aligned16(ws)) return NVFP4_ERR_MISALIGNED;
  if (over_logits(logits, ld, T, E, dlogits)) return NVFP4_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(ws);
  uint32_t* ticket = reinterpret_cast<uint32_t*>(base);
  const int cluster = S <= kClusterSeqs ? kCountCluster : 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(S * cluster));
  cfg.blockDim = dim3(kCountThreads);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = static_cast<unsigned>(cluster);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, balance_count_kernel, topk_ids, T, E, k, seq_offs, mask, cluster, counts,
                     tokens, ticket, dev_status);
  st = check_launch("balance_count_kernel");
  if (st != NVFP4_OK) return st;
  Args a{};
  a.logits = logits;
  a.ld = ld;
  a.T = T;
  a.E = E;
  a.k = k;
  a.seq_offs = seq_offs;
  a.S = S;
  a.mask = mask;
  a.alpha = alpha;
  a.counts = counts;
  a.tokens = tokens;
  a.dloss = dloss;
  a.dlogits = dlogits;
  a.accumulate = accumulate;
  a.loss = loss;
  a.part = reinterpret_cast<double*>(base + kPartOffset);
  a.ticket = ticket;
  return pass(a, true, s);
}

extern "C" nvfp4_status_t moe_balance_loss_backward(const float* logits, int64_t ld, int T, int E,
                                                    int k, const int32_t* counts,
                                                    const int32_t* tokens, const int32_t* seq_offs,
                                                    int S, const uint8_t* mask, float alpha,
                                                    const float* dloss, float* dlogits,
                                                    int accumulate, nvfp4_stream_t stream) {
  const nvfp4_status_t st = check_shape(T, E, k, ld, S, seq_offs);
  if (st != NVFP4_OK) return st;
  if (!counts || !tokens) return NVFP4_ERR_INVALID_ARG;
  if (T > 0 && (!logits || !dlogits)) return NVFP4_ERR_INVALID_ARG;
  const void* ptrs4[] = {logits, seq_offs, counts, tokens, dloss, dlogits};
  for (const void* p : ptrs4)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return NVFP4_ERR_MISALIGNED;
  if (over_logits(logits, ld, T, E, dlogits)) return NVFP4_ERR_INVALID_ARG;
  if (T == 0) return NVFP4_OK;
  Args a{};
  a.logits = logits;
  a.ld = ld;
  a.T = T;
  a.E = E;
  a.k = k;
  a.seq_offs = seq_offs;
  a.S = S;
  a.mask = mask;
  a.alpha = alpha;
  a.counts = counts;
  a.tokens = tokens;
  a.dloss = dloss;
  a.dlogits = dlogits;
  a.accumulate = accumulate;
  return pass(a, false, reinterpret_cast<cudaStream_t>(stream));
}
