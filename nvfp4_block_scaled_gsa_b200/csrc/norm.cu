// norm.cu — the norms around a block: the post-norm of its output, its gate, the scaled residual
// sum, and the pre-norm of the next block, with their gradients.
//
//   z = y * rstd(y) * post_gamma;   r' = r + scale * gate * z;   n = r' * rstd(r') * pre_gamma
//   rstd(v) = 1 / sqrt(mean(v^2) + eps)
//
// Forward: one pass; a row stays in registers between its two sums.  n is taken from the
// unrounded r'.
//
// Backward, from dr' and dn (the gradients of r' and n), with u = dn * pre_gamma, rhat = r' * rstd:
//   a  = dr' + rstd(r') * (u - rhat * mean(u * rhat))                 = dr
//   dz = scale * gate * a,   d = dz * post_gamma,   yhat = y * rstd(y)
//   dy = rstd(y) * (d - yhat * mean(d * yhat))
//   dpost_gamma = sum_t dz * yhat,  dpre_gamma = sum_t dn * rhat,  dgate = scale * a * z (summed over
//   whatever the gate was broadcast along)
// The second mean needs a, which needs the first; written out it is a combination of sums that
// do not, with c = scale * gate * post_gamma * yhat:
//   sum(d * yhat) = sum(c * (dr' + rstd u)) - rstd * mean(u * rhat) * sum(c * rhat)
// so a row needs one round of sums, not two.  Rows are brought to shared memory by bulk copies,
// several ahead; a CTA keeps its columns' sums for the gammas (and a channel gate) in registers
// over all its rows, and a second kernel adds the CTAs' sums in order.
//
// Both are bound by memory: 2 values of r and one each of y and n (forward), 3 of r, 2 of y and
// one of n (backward) per element.
#include <atomic>

#include "common.cuh"
#include "launch.h"

namespace nvfp4 {
namespace {

constexpr int kMaxH = 16384;
enum Gate { GATE_NONE = 0, GATE_CHANNEL = 1, GATE_TOKEN = 2, GATE_FULL = 3 };

struct Args {
  const void* r;
  int64_t ld_r;
  const __nv_bfloat16* y;  // NULL: no block output (r' = r)
  int64_t ld_y;
  int64_t T;
  int H;
  const __nv_bfloat16* post_gamma;  // NULL: z = y
  const __nv_bfloat16* gate;
  int gate_kind;
  float scale;
  const __nv_bfloat16* pre_gamma;  // NULL: no n
  float eps;
  float* rstd_post;
  float* rstd_pre;
  // forward
  void* r_out;
  __nv_bfloat16* n_out;
  // backward
  const void* dr_new;  // NULL: zero
  const __nv_bfloat16* dn;  // NULL: zero
  void* dr;
  __nv_bfloat16* dy;
  float* dpost_gamma;
  float* dpre_gamma;
  void* dgate;
  float* part;  // [CTAs][2][H]
  int32_t* status;
};

__device__ __forceinline__ void unpack8(const uint4& q, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// 8 residual values (bf16 or float32) at element i of a row; plain accesses, r_out may be r
template <bool F32>
__device__ __forceinline__ void load8(const void* row, int64_t i, float (&v)[8]) {
  if constexpr (F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(row) + i);
    const float4 a = p[0], b = p[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(row) + i), v);
  }
}
template <bool F32>
__device__ __forceinline__ void store8(void* row, int64_t i, const float (&v)[8]) {
  if constexpr (F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(row) + i);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(row) + i) = pack8(v);
  }
}

// Sum of N values over the CTA, in every thread: within warps by shuffles, then the warps' sums, in
// order of the lanes' tree (the same for every call).  `buf` must not be reused before the next
// barrier.
template <int N>
__device__ __forceinline__ void cta_sums(float (&v)[N], float (*buf)[32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = (blockDim.x + 31) >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
  if (nw == 1) return;
  if (lane == 0)
#pragma unroll
    for (int n = 0; n < N; ++n) buf[n][warp] = v[n];
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = lane < nw ? buf[n][lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
}

// gate values of 8 columns of row t
__device__ __forceinline__ void gate8(const Args& A, int64_t t, int c, float (&g)[8]) {
  if (A.gate_kind == GATE_CHANNEL || A.gate_kind == GATE_FULL) {
    const int64_t at = A.gate_kind == GATE_FULL ? t * A.H + c : c;
    unpack8(__ldg(reinterpret_cast<const uint4*>(A.gate + at)), g);
  } else {
    const float v = A.gate_kind == GATE_TOKEN ? __bfloat162float(A.gate[t]) : 1.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = v;
  }
}

// One row per CTA, C chunks of 8 columns per thread.
template <bool F32, int C>
__global__ void __launch_bounds__(1024) residual_norm_kernel(const Args A) {
  __shared__ float s_sum[2][1][32];
  const int64_t t = blockIdx.x;
  const int H = A.H;
  const char* r_row = static_cast<const char*>(A.r) + t * A.ld_r * (F32 ? 4 : 2);
  float v[C][8];  // r, then r'
  uint4 yq[C];
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int c = (threadIdx.x + j * blockDim.x) * 8;
    yq[j] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
    if (c < H) {
      load8<F32>(r_row, c, v[j]);
      if (A.y != nullptr) yq[j] = __ldg(reinterpret_cast<const uint4*>(A.y + t * A.ld_y + c));
    }
  }
  if (A.y != nullptr) {
    float rstd = 1.0f;
    if (A.post_gamma != nullptr) {
      float ss[1] = {0.0f};
#pragma unroll
      for (int j = 0; j < C; ++j) {
        float y[8];
        unpack8(yq[j], y);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] += y[i] * y[i];
      }
      cta_sums<1>(ss, s_sum[0]);
      rstd = 1.0f / sqrtf(ss[0] / static_cast<float>(H) + A.eps);
      if (threadIdx.x == 0 && A.rstd_post != nullptr) A.rstd_post[t] = rstd;
    }
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = (threadIdx.x + j * blockDim.x) * 8;
      if (c >= H) continue;
      float y[8], g[8];
      unpack8(yq[j], y);
      gate8(A, t, c, g);
      if (A.post_gamma != nullptr) {
        float w[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(A.post_gamma + c)), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = y[i] * rstd * w[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] += A.scale * g[i] * y[i];
      store8<F32>(static_cast<char*>(A.r_out) + t * H * (F32 ? 4 : 2), c, v[j]);
    }
  }
  if (A.pre_gamma == nullptr) return;
  float ss[1] = {0.0f};
#pragma unroll
  for (int j = 0; j < C; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) ss[0] += v[j][i] * v[j][i];
  cta_sums<1>(ss, s_sum[1]);
  const float rstd = 1.0f / sqrtf(ss[0] / static_cast<float>(H) + A.eps);
  if (threadIdx.x == 0 && A.rstd_pre != nullptr) A.rstd_pre[t] = rstd;
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int c = (threadIdx.x + j * blockDim.x) * 8;
    if (c >= H) continue;
    float w[8], o[8];
    unpack8(__ldg(reinterpret_cast<const uint4*>(A.pre_gamma + c)), w);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = v[j][i] * rstd * w[i];
    *reinterpret_cast<uint4*>(A.n_out + t * H + c) = pack8(o);
  }
}

// ------------------------------------------------------------------------------- backward

constexpr int kBwdChunks = 2;   // chunks of 8 columns per thread
constexpr int kBwdStages = 3;   // rows in shared memory, at most

// The rows of one stage: what of dr', dn, r, y and a full gate there is, in this order.
struct RowLayout {
  int dn, r, y, gate, bytes;
};
template <bool F32>
__host__ __device__ inline RowLayout row_layout(const Args& A) {
  RowLayout L;
  const int res = A.H * (F32 ? 4 : 2), half = A.H * 2;
  int o = A.dr_new != nullptr ? res : 0;
  L.dn = o;
  o += A.dn != nullptr ? half : 0;
  L.r = o;
  o += A.dn != nullptr ? res : 0;  // r and y are only needed for rhat, y also for yhat
  L.y = o;
  o += A.y != nullptr ? half : 0;
  L.gate = o;
  o += A.y != nullptr && A.gate_kind == GATE_FULL ? half : 0;
  L.bytes = o;
  return L;
}

// CTA b takes rows b, b + CTAs, ...  MAXT: threads at most (it sets the registers per thread).
template <bool F32, int MAXT>
__global__ void __launch_bounds__(MAXT) residual_norm_backward_kernel(const Args A, int stages) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bar[kBwdStages];
  __shared__ volatile int abort_flag;
  __shared__ float s_sum[2][3][32];
  const int tid = threadIdx.x, H = A.H;
  const RowLayout L = row_layout<F32>(A);
  const int res = F32 ? 4 : 2;
  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < stages; ++i) mbar_init(smem_u32(&bar[i]), 1);
    fence_mbar_init();
  }
  __syncthreads();
  auto fetch = [&](int64_t t, int s) {  // by one thread
    const uint32_t d = smem_u32(smem + s * L.bytes), b = smem_u32(&bar[s]);
    mbar_arrive_expect_tx(b, L.bytes);
    if (A.dr_new != nullptr)
      bulk_load(d, static_cast<const char*>(A.dr_new) + t * H * res, H * res, b);
    if (A.dn != nullptr) {
      bulk_load(d + L.dn, A.dn + t * H, H * 2, b);
      bulk_load(d + L.r, static_cast<const char*>(A.r) + t * A.ld_r * res, H * res, b);
    }
    if (A.y != nullptr) {
      bulk_load(d + L.y, A.y + t * A.ld_y, H * 2, b);
      if (A.gate_kind == GATE_FULL) bulk_load(d + L.gate, A.gate + t * H, H * 2, b);
    }
  };
  const int64_t step = gridDim.x;
  if (tid == 0)
    for (int i = 0; i < stages; ++i)
      if (blockIdx.x + i * step < A.T) fetch(blockIdx.x + i * step, i);

  // this thread's columns of the gammas and a channel gate
  uint4 wpost[kBwdChunks], wpre[kBwdChunks], wgate[kBwdChunks];
#pragma unroll
  for (int j = 0; j < kBwdChunks; ++j) {
    const int c = (tid + j * blockDim.x) * 8;
    wpost[j] = wpre[j] = wgate[j] = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
    if (c < H) {
      if (A.post_gamma != nullptr) wpost[j] = __ldg(reinterpret_cast<const uint4*>(A.post_gamma + c));
      if (A.pre_gamma != nullptr) wpre[j] = __ldg(reinterpret_cast<const uint4*>(A.pre_gamma + c));
      if (A.gate_kind == GATE_CHANNEL) wgate[j] = __ldg(reinterpret_cast<const uint4*>(A.gate + c));
    }
  }
  // sums over rows: of a * yhat (times the gate, unless that is one per channel) and dn * rhat
  float acc_post[kBwdChunks][8], acc_pre[kBwdChunks][8];
#pragma unroll
  for (int j = 0; j < kBwdChunks; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc_post[j][i] = acc_pre[j][i] = 0.0f;
  const float inv_h = 1.0f / static_cast<float>(H);
  const bool has_n = A.dn != nullptr, has_y = A.y != nullptr, post = A.post_gamma != nullptr;

  int it = 0;
  for (int64_t t = blockIdx.x; t < A.T; t += step, ++it) {
    const int s = it % stages;
    const float rs_y = has_y && post ? __ldg(A.rstd_post + t) : 1.0f;
    const float rs_r = has_n ? __ldg(A.rstd_pre + t) : 0.0f;
    const float g_tok = has_y && A.gate_kind == GATE_TOKEN ? __bfloat162float(A.gate[t]) : 1.0f;
    const bool here = mbar_wait_bounded(smem_u32(&bar[s]), (it / stages) & 1, &abort_flag);
    if (!__syncthreads_and(here)) break;  // all threads alike
    const uint8_t* row = smem + s * L.bytes;
    float dr[kBwdChunks][8], rhat[kBwdChunks][8];
    uint4 dnq[kBwdChunks], yq[kBwdChunks], gq[kBwdChunks];
    float sums[3] = {0.0f, 0.0f, 0.0f};  // u * rhat, c * (dr' + rstd u), c * rhat (c without g_tok)
#pragma unroll
    for (int j = 0; j < kBwdChunks; ++j) {
      const int c = (tid + j * blockDim.x) * 8;
      dnq[j] = yq[j] = make_uint4(0u, 0u, 0u, 0u);
      gq[j] = wgate[j];
#pragma unroll
      for (int i = 0; i < 8; ++i) dr[j][i] = rhat[j][i] = 0.0f;
      if (c >= H) continue;
      if (A.dr_new != nullptr) load8<F32>(row, c, dr[j]);
      if (has_y) {
        yq[j] = *reinterpret_cast<const uint4*>(row + L.y + c * 2);
        if (A.gate_kind == GATE_FULL) gq[j] = *reinterpret_cast<const uint4*>(row + L.gate + c * 2);
      }
      float y[8], g[8], w[8], cc[8];
      unpack8(yq[j], y);
      unpack8(gq[j], g);
      unpack8(wpost[j], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) cc[i] = A.scale * g[i] * w[i] * (y[i] * rs_y);
      if (has_n) {
        float rv[8], dn[8], wp[8];
        load8<F32>(row + L.r, c, rv);
        dnq[j] = *reinterpret_cast<const uint4*>(row + L.dn + c * 2);
        unpack8(dnq[j], dn);
        unpack8(wpre[j], wp);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          rhat[j][i] = (rv[i] + g_tok * cc[i]) * rs_r;
          const float u = dn[i] * wp[i];
          dr[j][i] += rs_r * u;
          sums[0] += u * rhat[j][i];
          sums[2] += cc[i] * rhat[j][i];
          acc_pre[j][i] += dn[i] * rhat[j][i];
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sums[1] += cc[i] * dr[j][i];
    }
    cta_sums<3>(sums, s_sum[it & 1]);
    if (blockDim.x <= 32) __syncwarp();
    // every thread has read the stage (the barrier in cta_sums): on to a later row
    if (tid == 0 && t + stages * step < A.T) fetch(t + stages * step, s);
    const float k_r = rs_r * sums[0] * inv_h;         // a = dr' + rstd u - k_r * rhat
    const float s_cy = sums[1] - k_r * sums[2];       // sum of c * a, without g_tok
    const float k_y = post ? g_tok * s_cy * inv_h : 0.0f;  // mean of d * yhat
    if (tid == 0 && A.dgate != nullptr && A.gate_kind == GATE_TOKEN)
      static_cast<float*>(A.dgate)[t] = s_cy;
#pragma unroll
    for (int j = 0; j < kBwdChunks; ++j) {
      const int c = (tid + j * blockDim.x) * 8;
      if (c >= H) continue;
      float a[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = dr[j][i] - k_r * rhat[j][i];
      store8<F32>(static_cast<char*>(A.dr) + t * H * res, c, a);
      if (!has_y) continue;
      float y[8], g[8], w[8], dy[8], dg[8];
      unpack8(yq[j], y);
      unpack8(gq[j], g);
      unpack8(wpost[j], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float yhat = y[i] * rs_y, sg = A.scale * g_tok * g[i];
        dy[i] = rs_y * (sg * w[i] * a[i] - yhat * k_y);
        dg[i] = A.scale * w[i] * yhat * a[i];
        acc_post[j][i] += (A.gate_kind == GATE_CHANNEL ? 1.0f : g_tok * g[i]) * yhat * a[i];
      }
      *reinterpret_cast<uint4*>(A.dy + t * H + c) = pack8(dy);
      if (A.gate_kind == GATE_FULL && A.dgate != nullptr)
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(A.dgate) + t * H + c) = pack8(dg);
    }
  }
  if (abort_flag) {  // let the copies already issued land before the CTA can exit
    if (tid == 0) {
      report(A.status, NVFP4_DEVERR_TIMEOUT);
      volatile int never = 0;
      for (int i = 0; i < stages; ++i)
        if (blockIdx.x + (it + i) * step < A.T)
          mbar_wait_bounded(smem_u32(&bar[(it + i) % stages]), ((it + i) / stages) & 1, &never,
                            NVFP4_WAIT_TIMEOUT_NS / 4);
    }
    return;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (A.part == nullptr) return;
  float* part = A.part + (int64_t)blockIdx.x * 2 * H;
#pragma unroll
  for (int j = 0; j < kBwdChunks; ++j) {
    const int c = (tid + j * blockDim.x) * 8;
    if (c >= H) continue;
    store8<true>(part, c, acc_post[j]);
    store8<true>(part + H, c, acc_pre[j]);
  }
}

// Adds the CTAs' column sums in order (8 interleaved partial sums, then those in order) and makes
// the gradients of them.  32 columns per CTA; blockIdx.y: 0 = post (and channel gate), 1 = pre.
__global__ void __launch_bounds__(256) norm_grads_kernel(const Args A, int parts) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float s[8][33];
  const int col = blockIdx.x * 32 + threadIdx.x, k = threadIdx.y;
  float v = 0.0f;
  if (col < A.H) {
    const float* p = A.part + (int64_t)blockIdx.y * A.H + col;
#pragma unroll 8
    for (int i = k; i < parts; i += 8) v += __ldcg(p + (int64_t)i * 2 * A.H);
  }
  s[k][threadIdx.x] = v;
  __syncthreads();
  if (k != 0 || col >= A.H) return;
  v = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) v += s[i][threadIdx.x];
  if (blockIdx.y == 1) {
    if (A.dpre_gamma != nullptr) A.dpre_gamma[col] = v;
    return;
  }
  const bool channel = A.gate_kind == GATE_CHANNEL;
  const float g = channel ? __bfloat162float(A.gate[col]) : 1.0f;
  const float w = A.post_gamma != nullptr ? __bfloat162float(A.post_gamma[col]) : 1.0f;
  if (A.dpost_gamma != nullptr) A.dpost_gamma[col] = A.scale * g * v;
  if (channel && A.dgate != nullptr) static_cast<float*>(A.dgate)[col] = A.scale * w * v;
}

// ------------------------------------------------------------------------------ host side

constexpr int kSizingSms = 148;

int round32(int v) { return (v + 31) / 32 * 32; }

// threads of the backward kernel, and its CTAs: as many as the SMs hold at 128 registers a thread
int bwd_threads(int H) { return round32((H / 8 + kBwdChunks - 1) / kBwdChunks); }
int bwd_ctas(int64_t T, int H) {
  const int threads = bwd_threads(H);
  const int per_sm = threads >= 512 ? 1 : 512 / threads;
  const int64_t most = (int64_t)kSizingSms * per_sm;
  return static_cast<int>(T < most ? T : most);
}

nvfp4_status_t check_common(const Args& a, int r_dtype) {
  if (a.T < 0 || a.H <= 0 || a.gate_kind < 0 || a.gate_kind > 3 || !(a.eps >= 0.0f) ||
      (r_dtype != 0 && r_dtype != 1))
    return NVFP4_ERR_INVALID_ARG;
  if (a.T > INT32_MAX || a.H % 8 || a.H > kMaxH) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (a.ld_r < a.H || (a.y != nullptr && a.ld_y < a.H)) return NVFP4_ERR_INVALID_ARG;
  if (a.ld_r % 8 || (a.y != nullptr && a.ld_y % 8)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (a.T > 0 && a.y == nullptr && (a.post_gamma != nullptr || a.gate_kind != GATE_NONE))
    return NVFP4_ERR_INVALID_ARG;  // a post-norm or a gate of nothing
  if ((a.gate_kind != GATE_NONE) != (a.gate != nullptr)) return NVFP4_ERR_INVALID_ARG;
  const void* p16[] = {a.r, a.y, a.post_gamma, a.pre_gamma, a.r_out, a.n_out, a.dr_new, a.dn,
                       a.dr, a.dy, a.part};
  for (const void* p : p16)
    if (!aligned16(p)) return NVFP4_ERR_MISALIGNED;
  const uintptr_t gate_mask = a.gate_kind == GATE_TOKEN ? 1u : 15u;
  if (reinterpret_cast<uintptr_t>(a.gate) & gate_mask) return NVFP4_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(a.dgate) & (a.gate_kind == GATE_FULL ? 15u : 3u))
    return NVFP4_ERR_MISALIGNED;
  const void* p4[] = {a.rstd_post, a.rstd_pre, a.dpost_gamma, a.dpre_gamma};
  for (const void* p : p4)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return NVFP4_ERR_MISALIGNED;
  return NVFP4_OK;
}

template <bool F32>
void launch_forward(const Args& a, cudaStream_t s) {
  const int n8 = a.H / 8;
  // Enough rows for every SM several times over: 4 chunks per thread, several CTAs per SM.  Fewer:
  // one chunk (two beyond 8192 columns), so that a row's loads are in flight at once.
  const int chunks = a.T >= 4 * kSizingSms ? 4 : n8 <= 1024 ? 1 : 2;
  const dim3 grid(static_cast<unsigned>(a.T)), block(round32((n8 + chunks - 1) / chunks));
  if (chunks == 4) residual_norm_kernel<F32, 4><<<grid, block, 0, s>>>(a);
  else if (chunks == 2) residual_norm_kernel<F32, 2><<<grid, block, 0, s>>>(a);
  else residual_norm_kernel<F32, 1><<<grid, block, 0, s>>>(a);
}

template <bool F32, int MAXT>
nvfp4_status_t launch_backward(const Args& a, cudaStream_t s) {
  auto* fn = residual_norm_backward_kernel<F32, MAXT>;
  const int threads = bwd_threads(a.H), ctas = bwd_ctas(a.T, a.H);
  const int per_sm = threads >= 512 ? 1 : 512 / threads;
  const int row = row_layout<F32>(a).bytes;
  // the largest row: float32 r and dr', a full gate, kMaxH columns
  constexpr int kMost = kMaxH * 14;
  static_assert(kMost + 2560 <= 228 * 1024, "one row of the widest form");
  // a CTA's share of an SM's 228 KB, less its static shared memory and what the system reserves
  int room = 228 * 1024 / per_sm - 2560;
  room = room < kMost ? room : kMost;
  int stages = room / (row > 0 ? row : 1);
  stages = stages < 1 ? 1 : stages > kBwdStages ? kBwdStages : stages;
  const int smem = stages * row;
  static std::atomic<uint64_t> devices_set{0};
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(devices_set.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost) != cudaSuccess)
      return check_launch("residual_norm_backward_kernel attributes");
    devices_set.fetch_or(bit, std::memory_order_release);
  }
  fn<<<ctas, threads, smem, s>>>(a, stages);
  return check_launch("residual_norm_backward_kernel");
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status_t nvfp4_residual_norm(const void* r, int r_dtype, int64_t ld_r,
                                              const void* y, int64_t ld_y, int64_t T, int H,
                                              const void* post_gamma, const void* gate,
                                              int gate_kind, float scale, const void* pre_gamma,
                                              float eps, void* r_out, void* n_out,
                                              float* rstd_post, float* rstd_pre,
                                              nvfp4_stream_t stream) {
  Args a{};
  a.r = r;
  a.ld_r = ld_r;
  a.y = static_cast<const __nv_bfloat16*>(y);
  a.ld_y = ld_y;
  a.T = T;
  a.H = H;
  a.post_gamma = static_cast<const __nv_bfloat16*>(post_gamma);
  a.gate = static_cast<const __nv_bfloat16*>(gate);
  a.gate_kind = gate_kind;
  a.scale = scale;
  a.pre_gamma = static_cast<const __nv_bfloat16*>(pre_gamma);
  a.eps = eps;
  a.r_out = r_out;
  a.n_out = static_cast<__nv_bfloat16*>(n_out);
  a.rstd_post = rstd_post;
  a.rstd_pre = rstd_pre;
  const nvfp4_status_t st = check_common(a, r_dtype);
  if (st != NVFP4_OK) return st;
  if (T == 0) return NVFP4_OK;
  if (!r || (y && !r_out) || (pre_gamma && !n_out)) return NVFP4_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (r_dtype == 0) launch_forward<true>(a, s);
  else launch_forward<false>(a, s);
  return check_launch("residual_norm_kernel");
}

extern "C" size_t nvfp4_residual_norm_backward_workspace_size(int64_t T, int H) {
  if (T <= 0 || H <= 0 || H > kMaxH || H % 8) return 0;
  return static_cast<size_t>((int64_t)bwd_ctas(T, H) * 2 * H * 4);
}

extern "C" nvfp4_status_t nvfp4_residual_norm_backward(
    const void* dr_new, const void* dn, const void* r, int r_dtype, int64_t ld_r, const void* y,
    int64_t ld_y, int64_t T, int H, const void* post_gamma, const void* gate, int gate_kind,
    float scale, const void* pre_gamma, const float* rstd_post, const float* rstd_pre, void* dr,
    void* dy, float* dpost_gamma, float* dpre_gamma, void* dgate, void* ws, size_t ws_bytes,
    int32_t* dev_status, nvfp4_stream_t stream) {
  Args a{};
  a.r = r;
  a.ld_r = ld_r;
  a.y = static_cast<const __nv_bfloat16*>(y);
  a.ld_y = ld_y;
  a.T = T;
  a.H = H;
  a.post_gamma = static_cast<const __nv_bfloat16*>(post_gamma);
  a.gate = static_cast<const __nv_bfloat16*>(gate);
  a.gate_kind = gate_kind;
  a.scale = scale;
  a.pre_gamma = static_cast<const __nv_bfloat16*>(pre_gamma);
  a.rstd_post = const_cast<float*>(rstd_post);
  a.rstd_pre = const_cast<float*>(rstd_pre);
  a.dr_new = dr_new;
  a.dn = static_cast<const __nv_bfloat16*>(dn);
  a.dr = dr;
  a.dy = static_cast<__nv_bfloat16*>(dy);
  a.dpost_gamma = dpost_gamma;
  a.dpre_gamma = dpre_gamma;
  a.dgate = dgate;
  a.part = static_cast<float*>(ws);
  nvfp4_status_t st = check_common(a, r_dtype);
  if (st != NVFP4_OK) return st;
  if (a.dn && !a.pre_gamma) return NVFP4_ERR_INVALID_ARG;
  if (T > 0) {
    if (!dr_new && !dn) return NVFP4_ERR_INVALID_ARG;  // no gradient comes in
    if (!dr || (y && !dy)) return NVFP4_ERR_INVALID_ARG;
    if (dn && (!r || !rstd_pre)) return NVFP4_ERR_INVALID_ARG;
    if (y && post_gamma && !rstd_post) return NVFP4_ERR_INVALID_ARG;
  }
  if ((dpost_gamma && !post_gamma) || (dpre_gamma && !pre_gamma) || (dgate && !gate))
    return NVFP4_ERR_INVALID_ARG;
  // column sums: of the gammas and a channel gate
  const bool columns = dpost_gamma || dpre_gamma || (dgate && gate_kind == GATE_CHANNEL);
  if (!columns) a.part = nullptr;
  else if (T > 0 &&
           (ws == nullptr || ws_bytes < nvfp4_residual_norm_backward_workspace_size(T, H)))
    return NVFP4_ERR_WORKSPACE_TOO_SMALL;
  a.status = dev_status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int parts = 0;
  if (T > 0) {
    parts = bwd_ctas(T, H);
    const bool few = bwd_threads(H) <= 512;
    if (r_dtype == 0)
      st = few ? launch_backward<true, 512>(a, s) : launch_backward<true, 1024>(a, s);
    else
      st = few ? launch_backward<false, 512>(a, s) : launch_backward<false, 1024>(a, s);
    if (st != NVFP4_OK) return st;
  }
  if (!columns) return NVFP4_OK;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((H + 31) / 32), 2);
  cfg.blockDim = dim3(32, 8);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = T > 0 ? 1 : 0;
  cudaLaunchKernelEx(&cfg, norm_grads_kernel, static_cast<const Args>(a), parts);
  return check_launch("norm_grads_kernel");
}
