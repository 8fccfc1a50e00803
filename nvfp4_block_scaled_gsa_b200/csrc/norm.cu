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
// one of n (backward) per element.  Forward, 8192 x 7168 with a float32 residual: 120 to 125 us, 5.6
// to 5.9 TB/s (86 to 90% of a copy's rate; CTAs that stay and copy their next rows to shared memory
// by themselves took 178); with a bf16 one 110 us (65%), waiting for loads with 28 warps an SM.
// Backward, 8191 x 7168 with the column sums: 167 us with a float32 residual (97%), 139 to 141 us with a
// bf16 one (76%), where the same instructions meet fewer bytes: half of the issue slots are used and the
// rest goes to the one barrier per row, with the registers (128 x 512 threads, half of them column
// sums) allowing one CTA per SM.
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
  float* part;  // [clusters][2][H]
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
// Two float32 values.  (The packed f32x2 instructions were tried for the backward pass and were 6%
// slower at 8191 x 7168.)
struct F2 {
  float x, y;
  __device__ __forceinline__ F2() {}
  __device__ __forceinline__ F2(float lo, float hi) : x(lo), y(hi) {}
  __device__ __forceinline__ explicit F2(float both) : x(both), y(both) {}
  __device__ __forceinline__ float2 get() const { return make_float2(x, y); }
};
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) { return F2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)); }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) { return F2(a.x * b.x, a.y * b.y); }
__device__ __forceinline__ F2 add2(F2 a, F2 b) { return F2(a.x + b.x, a.y + b.y); }
__device__ __forceinline__ void unpack8(const uint4& q, F2 (&v)[4]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = F2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 pack8(const F2 (&v)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = v[i].get();
    const __nv_bfloat162 p = __floats2bfloat162_rn(f.x, f.y);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <bool F32>
__device__ __forceinline__ void load8(const void* p, F2 (&v)[4]) {
  if constexpr (F32) {
    const float4 a = static_cast<const float4*>(p)[0], b = static_cast<const float4*>(p)[1];
    v[0] = F2(a.x, a.y);
    v[1] = F2(a.z, a.w);
    v[2] = F2(b.x, b.y);
    v[3] = F2(b.z, b.w);
  } else {
    unpack8(*static_cast<const uint4*>(p), v);
  }
}
template <bool F32>
__device__ __forceinline__ void store8(void* p, const F2 (&v)[4]) {
  if constexpr (F32) {
    const float2 a = v[0].get(), b = v[1].get(), c = v[2].get(), d = v[3].get();
    static_cast<float4*>(p)[0] = make_float4(a.x, a.y, b.x, b.y);
    static_cast<float4*>(p)[1] = make_float4(c.x, c.y, d.x, d.y);
  } else {
    *static_cast<uint4*>(p) = pack8(v);
  }
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
constexpr int kBwdThreads = 512;
constexpr int kBwdWidth = kBwdThreads * kBwdChunks * 8;  // columns that a CTA can take

// How a row's columns lie on the CTAs of a cluster: `width` each, the last one fewer.  One CTA up to
// 8192 columns, else two (4096 x 16384: 164 us, against 298 with one CTA of 1024 threads, whose 64
// registers spilled).
struct Columns {
  int cluster, width, threads, per_sm;
  explicit Columns(int H) {
    cluster = (H + kBwdWidth - 1) / kBwdWidth;
    width = ((H + cluster - 1) / cluster + 7) / 8 * 8;
    threads = ((width / 8 + kBwdChunks - 1) / kBwdChunks + 31) / 32 * 32;
    // alone on its SM: as many warps for each of the four schedulers
    if (threads > kBwdThreads / 2) threads = (threads + 127) / 128 * 128;
    per_sm = kBwdThreads / threads;  // at 128 registers a thread
  }
};

// A CTA's part of one row in a stage: what of dr', dn, r, y and a full gate there is, in this order.
struct RowLayout {
  int dn, r, y, gate, bytes;
};
template <bool F32>
__host__ __device__ inline RowLayout row_layout(const Args& A, int width) {
  RowLayout L;
  const int res = width * (F32 ? 4 : 2), half = width * 2;
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

// An array that rows are fetched from: this CTA's part of the next row, and where in a stage it goes.
struct Source {
  const char* next;
  int64_t step;
  int at, bytes;
};

// 16 bytes to shared memory of a CTA of the cluster
__device__ __forceinline__ void st_cluster(uint32_t at, float x, float y, float z, float w) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(x), "f"(y), "f"(z), "f"(w)
               : "memory");
}

// Cluster b (CLUSTER: of two CTAs, else one) takes rows b, b + clusters, ...  FULL: the gate has a value
// per element (otherwise it is a factor per row or per column).  ALL: dr', dn and y are all there
// (training's usual call), so that nothing is tested per element.
//
// Per element, with the row's k0 = scale * rstd(y), g_t (a token gate, or 1) and the column's
// w = post_gamma * (a channel gate, or 1):
//   c = k0 y w (its gradient side of the gate left out), r' = r + g_t c, u = rstd dn pre_gamma,
//   a0 = dr' + u; sums of u r', c a0, c r'; then a = a0 - k r', dy = g_t k0 w a - k' y.
template <bool F32, bool CLUSTER, bool FULL, bool ALL>
__global__ void __launch_bounds__(kBwdThreads, 1)
    residual_norm_backward_kernel(const Args A, int stages, int columns) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kSources = FULL ? 5 : 4;
  __shared__ __align__(8) uint64_t bar[kBwdStages];
  __shared__ volatile int abort_flag;
  __shared__ Source s_source[kSources];  // (each read and written by its own thread only)
  __shared__ float s_sum[2][3][32];
  __shared__ float4 s_pair[2][2][CLUSTER ? 16 : 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5, H = A.H;
  const int rank = CLUSTER ? static_cast<int>(cluster_ctarank()) : 0;
  const int col0 = CLUSTER ? rank * columns : 0, width = CLUSTER ? min(columns, H - col0) : H;
  const RowLayout L = row_layout<F32>(A, CLUSTER ? columns : H);
  constexpr int res = F32 ? 4 : 2;
  const int64_t first = CLUSTER ? blockIdx.x / 2 : blockIdx.x, step = CLUSTER ? gridDim.x / 2 : gridDim.x;
  const bool split = CLUSTER || warps > 8;
  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < stages; ++i) mbar_init(smem_u32(&bar[i]), split ? kSources : 1);
    fence_mbar_init();
  }
  // With one CTA per SM each array is fetched by a thread of another warp: with one thread for all of
  // them the row waited for its warp (8191 x 7168 in float32: 173 us, against 166).  With more the
  // others cover it, and the fewer instructions count (8192 x 2048: 46.4 us, against 49.6).
  const int source = lane * warps + warp;
  const bool mine = split && source < kSources;
  if (mine) {
    const void* p = source == 0   ? A.dr_new
                    : source == 1 ? A.dn
                    : source == 2 ? (A.dn != nullptr ? A.r : nullptr)
                    : source == 3 ? A.y
                                  : (A.y != nullptr ? A.gate : nullptr);
    const int64_t ld = source == 2 ? A.ld_r : source == 3 ? A.ld_y : H;
    const int size = source == 0 || source == 2 ? res : 2;
    Source& f = s_source[source];
    f.next = static_cast<const char*>(p) + (first * ld + col0) * size;
    f.step = step * ld * size;
    f.at = source == 0 ? 0 : source == 1 ? L.dn : source == 2 ? L.r : source == 3 ? L.y : L.gate;
    f.bytes = p != nullptr ? width * size : 0;
  }
  if (CLUSTER) cluster_sync();  // the other CTA has started
  else __syncthreads();
  auto fetch = [&](int64_t t, int s) {  // row t: the one behind those fetched before
    const uint32_t d = smem_u32(smem + s * L.bytes), b = smem_u32(&bar[s]);
    if (mine) {
      Source& f = s_source[source];
      mbar_arrive_expect_tx(b, f.bytes);
      if (f.bytes != 0) bulk_load(d + f.at, f.next, f.bytes, b);
      f.next += f.step;
    } else if (!split && tid == 0) {
      mbar_arrive_expect_tx(b, L.bytes);
      if (A.dr_new != nullptr)
        bulk_load(d, static_cast<const char*>(A.dr_new) + t * H * res, H * res, b);
      if (A.dn != nullptr) {
        bulk_load(d + L.dn, A.dn + t * H, H * 2, b);
        bulk_load(d + L.r, static_cast<const char*>(A.r) + t * A.ld_r * res, H * res, b);
      }
      if (A.y != nullptr) {
        bulk_load(d + L.y, A.y + t * A.ld_y, H * 2, b);
        if constexpr (FULL) bulk_load(d + L.gate, A.gate + t * H, H * 2, b);
      }
    }
  };
  for (int i = 0; i < stages; ++i)
    if (first + i * step < A.T) fetch(first + i * step, i);

  // this thread's columns: their factors, and their sums over the rows of a * yhat (times scale
  // and the gate, unless that is one per channel) and of dn * rhat
  F2 w[kBwdChunks][4], acc_post[kBwdChunks][4], acc_pre[kBwdChunks][4];
  uint4 wpre[kBwdChunks];
  int cols[kBwdChunks];  // first column (of the CTA's), or -1
#pragma unroll
  for (int j = 0; j < kBwdChunks; ++j) {
    const int at = (tid + j * blockDim.x) * 8, c = col0 + at;
    cols[j] = at < width ? at : -1;
    wpre[j] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[j][i] = F2(1.0f);
      acc_post[j][i] = acc_pre[j][i] = F2(0.0f);
    }
    if (at >= width) continue;
    if (A.post_gamma != nullptr)
      unpack8(__ldg(reinterpret_cast<const uint4*>(A.post_gamma + c)), w[j]);
    if (A.gate_kind == GATE_CHANNEL) {
      F2 g[4];
      unpack8(__ldg(reinterpret_cast<const uint4*>(A.gate + c)), g);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[j][i] = mul2(w[j][i], g[i]);
    }
    if (A.pre_gamma != nullptr) wpre[j] = __ldg(reinterpret_cast<const uint4*>(A.pre_gamma + c));
  }
  const float inv_h = 1.0f / static_cast<float>(H);
  const bool has_r = ALL || A.dr_new != nullptr, has_n = ALL || A.dn != nullptr;
  const bool has_y = ALL || A.y != nullptr, post = A.post_gamma != nullptr;

  // a row's scalars, read a row ahead
  struct Scalars {
    float rs_y, rs_r, g;
  };
  auto scalars = [&](int64_t t) {
    Scalars v{1.0f, 0.0f, 1.0f};
    if (t < A.T) {
      if (has_y && post) v.rs_y = __ldg(A.rstd_post + t);
      if (has_n) v.rs_r = __ldg(A.rstd_pre + t);
      if (has_y && A.gate_kind == GATE_TOKEN) v.g = __bfloat162float(A.gate[t]);
    }
    return v;
  };
  Scalars next = scalars(first);
  int it = 0, s = 0;
  uint32_t phase = 0;
  bool ok = true;
  char* dr_row = static_cast<char*>(A.dr) + (first * H + col0) * res;
  __nv_bfloat16* dy_row = A.dy + first * H + col0;
  for (int64_t t = first; t < A.T;
       t += step, ++it, dr_row += step * H * res, dy_row += step * H) {
    const float rs_y = next.rs_y, rs_r = next.rs_r, g_t = next.g;
    next = scalars(t + step);
    const float k0 = A.scale * rs_y;
    ok = mbar_wait_bounded(smem_u32(&bar[s]), phase, &abort_flag);
    const uint8_t* row = smem + s * L.bytes;
    F2 a[kBwdChunks][4], rn[kBwdChunks][4];
    uint4 yq[kBwdChunks], gq[kBwdChunks];
    F2 sum2[3] = {F2(0.0f), F2(0.0f), F2(0.0f)};
    const F2 k0_2(k0), g_2(g_t), rs_2(rs_r);
#pragma unroll
    for (int j = 0; j < kBwdChunks; ++j) {
      const int c = cols[j];
      if (c < 0) continue;
      uint4 dnq = make_uint4(0u, 0u, 0u, 0u);
      yq[j] = gq[j] = dnq;
#pragma unroll
      for (int i = 0; i < 4; ++i) a[j][i] = rn[j][i] = F2(0.0f);
      if (has_r) load8<F32>(row + c * res, a[j]);
      if (has_n) {
        load8<F32>(row + L.r + c * res, rn[j]);
        dnq = *reinterpret_cast<const uint4*>(row + L.dn + c * 2);
      }
      if (has_y) {
        yq[j] = *reinterpret_cast<const uint4*>(row + L.y + c * 2);
        if constexpr (FULL) gq[j] = *reinterpret_cast<const uint4*>(row + L.gate + c * 2);
      }
      F2 y[4], dn[4], wp[4], g[4];
      unpack8(yq[j], y);
      unpack8(dnq, dn);
      unpack8(wpre[j], wp);
      if constexpr (FULL) unpack8(gq[j], g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        F2 cc = mul2(mul2(y[i], k0_2), w[j][i]);
        if constexpr (FULL) cc = mul2(cc, g[i]);
        rn[j][i] = fma2(g_2, cc, rn[j][i]);
        const F2 dnr = mul2(dn[i], rs_2), u = mul2(dnr, wp[i]);
        a[j][i] = add2(a[j][i], u);
        sum2[0] = fma2(u, rn[j][i], sum2[0]);
        sum2[1] = fma2(cc, a[j][i], sum2[1]);
        sum2[2] = fma2(cc, rn[j][i], sum2[2]);
        acc_pre[j][i] = fma2(dnr, rn[j][i], acc_pre[j][i]);
      }
    }
    float sums[3];
#pragma unroll
    for (int n = 0; n < 3; ++n) {
      const float2 v = sum2[n].get();
      sums[n] = v.x + v.y;
    }
    // the row's sums, in every thread; the barrier also tells that every thread has read the stage,
    // and whether all found it filled
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int n = 0; n < 3; ++n) sums[n] += __shfl_xor_sync(0xffffffffu, sums[n], o);
    if (CLUSTER) {  // (and every warp's answer to the wait)
      ok = __all_sync(0xffffffffu, ok) != 0;
      if (lane < 2)
        st_cluster(mapa_shared(smem_u32(&s_pair[it & 1][rank][warp]), lane), sums[0], sums[1], sums[2],
                   ok ? 0.0f : 1.0f);
      cluster_sync();
      const float4 v = (lane & 15) < warps ? s_pair[it & 1][lane >> 4][lane & 15]
                                           : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      ok = __all_sync(0xffffffffu, v.w == 0.0f) != 0;
      sums[0] = v.x;
      sums[1] = v.y;
      sums[2] = v.z;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int n = 0; n < 3; ++n) sums[n] += __shfl_xor_sync(0xffffffffu, sums[n], o);
    } else if (blockDim.x > 32) {
      if (lane == 0)
#pragma unroll
        for (int n = 0; n < 3; ++n) s_sum[it & 1][n][tid >> 5] = sums[n];
      ok = __syncthreads_and(ok) != 0;
#pragma unroll
      for (int n = 0; n < 3; ++n)
        sums[n] = lane < static_cast<int>(blockDim.x >> 5) ? s_sum[it & 1][n][lane] : 0.0f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int n = 0; n < 3; ++n) sums[n] += __shfl_xor_sync(0xffffffffu, sums[n], o);
    } else {
      ok = __all_sync(0xffffffffu, ok) != 0;
    }
    if (!ok) break;  // all threads alike
    if (t + stages * step < A.T) fetch(t + stages * step, s);
    // mean(u rhat) rstd per r', and sum(c a) with a = a0 - k_r r'
    const float k_r = sums[0] * inv_h * rs_r * rs_r;
    const float s_ca = sums[1] - k_r * sums[2];
    if (tid == 0 && rank == 0 && A.dgate != nullptr && A.gate_kind == GATE_TOKEN)
      static_cast<float*>(A.dgate)[t] = s_ca;
    // mean(d yhat) yhat rstd(y) = g_t s_ca / H * rstd(y)^2 y
    const F2 k1_2(g_t * k0), k_r2(-k_r), k_y2(post ? -g_t * s_ca * inv_h * rs_y * rs_y : 0.0f);
#pragma unroll
    for (int j = 0; j < kBwdChunks; ++j) {
      const int c = cols[j];
      if (c < 0) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) a[j][i] = fma2(k_r2, rn[j][i], a[j][i]);
      store8<F32>(dr_row + c * res, a[j]);
      if (!has_y) continue;
      F2 y[4], dy[4], g[4], dg[4];
      unpack8(yq[j], y);
      if constexpr (FULL) unpack8(gq[j], g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const F2 b = mul2(a[j][i], k1_2);
        if constexpr (FULL) {
          const F2 bw = mul2(b, w[j][i]);
          dg[i] = mul2(bw, y[i]);
          dy[i] = fma2(bw, g[i], mul2(k_y2, y[i]));
          acc_post[j][i] = fma2(mul2(b, g[i]), y[i], acc_post[j][i]);
        } else {
          dy[i] = fma2(b, w[j][i], mul2(k_y2, y[i]));
          acc_post[j][i] = fma2(b, y[i], acc_post[j][i]);
        }
      }
      *reinterpret_cast<uint4*>(dy_row + c) = pack8(dy);
      if (FULL && A.dgate != nullptr)
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(A.dgate) + t * H + col0 + c) = pack8(dg);
    }
    if (++s == stages) {
      s = 0;
      phase ^= 1;
    }
  }
  if (!ok) {  // let the copies already issued land before the CTA can exit
    if (tid == 0) {
      report(A.status, NVFP4_DEVERR_TIMEOUT);
      volatile int never = 0;
      for (int i = 0; i < stages; ++i)
        if (first + (it + i) * step < A.T)
          mbar_wait_bounded(smem_u32(&bar[(it + i) % stages]), ((it + i) / stages) & 1, &never,
                            NVFP4_WAIT_TIMEOUT_NS / 4);
    }
    return;
  }
  pdl_trigger();
  if (A.part == nullptr) return;
  float* part = A.part + first * 2 * H + col0;
#pragma unroll
  for (int j = 0; j < kBwdChunks; ++j) {
    if (cols[j] < 0) continue;
    store8<true>(part + cols[j], acc_post[j]);
    store8<true>(part + H + cols[j], acc_pre[j]);
  }
}

// Adds the CTAs' column sums in order (8 interleaved partial sums, then those in order) and makes
// the gradients of them.  32 columns per CTA; blockIdx.y: 0 = post (and channel gate), 1 = pre.
__global__ void __launch_bounds__(256) norm_grads_kernel(const Args A, int parts) {
  pdl_wait();
  __shared__ float s[8][33];
  const int col = blockIdx.x * 32 + threadIdx.x, k = threadIdx.y;
  float v = 0.0f;
  if (col < A.H) {
    const float* p = A.part + (int64_t)blockIdx.y * A.H + col;
#pragma unroll 8
    for (int i = k; i < parts; i += 8) v += ld_after(p + (int64_t)i * 2 * A.H);
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
  if (A.dpost_gamma != nullptr) A.dpost_gamma[col] = g * v;
  if (channel && A.dgate != nullptr) static_cast<float*>(A.dgate)[col] = w * v;
}

// ------------------------------------------------------------------------------ host side

constexpr int kSizingSms = 148;

int round32(int v) { return (v + 31) / 32 * 32; }

// clusters of the backward kernel: as many as the SMs hold
int bwd_clusters(int64_t T, int H) {
  const Columns C(H);
  const int64_t most = (int64_t)kSizingSms * C.per_sm / C.cluster;
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

// An array of a call, for the check of outputs that lie over something else: [T][H] in rows `pitch`
// bytes apart, or a plain vector (one row, in no one's place).
struct Span {
  const void* p;
  int64_t rows, pitch, row;  // bytes
  bool vector;
};
Span rows_span(const Args& a, const void* p, int size, int64_t pitch) {
  return {p, a.T, a.T == 1 ? (int64_t)a.H * size : pitch * size, (int64_t)a.H * size, false};
}
Span vector_span(const void* p, int64_t n, int size) { return {p, 1, n * size, n * size, true}; }
// Outputs (dense) apart from one another and from the inputs.  Rows may take the place of the very same
// rows (address, pitch and type): a row is read by the threads that write it, before they do.  Rows
// over other rows would be written by one CTA while another still reads them.
template <int O, int I>
bool outputs_apart(const Span (&outs)[O], const Span (&ins)[I]) {
  for (int i = 0; i < O; ++i) {
    const Span& o = outs[i];
    auto over = [&](const Span& x) {
      return rows_overlap(x.p, x.rows, x.pitch, x.row, o.p, o.rows * o.row);
    };
    for (int j = 0; j < i; ++j)
      if (over(outs[j])) return false;
    for (const Span& in : ins)
      if (over(in) &&
          !(o.p == in.p && !o.vector && !in.vector && o.pitch == in.pitch && o.row == in.row))
        return false;
  }
  return true;
}
Span gate_span(const Args& a) {
  return a.gate_kind == GATE_FULL ? rows_span(a, a.gate, 2, a.H)
                                  : vector_span(a.gate, a.gate_kind == GATE_TOKEN ? a.T : a.H, 2);
}

template <bool F32>
void launch_forward(const Args& a, cudaStream_t s) {
  const int n8 = a.H / 8;
  // Enough rows for every SM several times over: 4 chunks per thread, several CTAs per SM (8192 x
  // 7168 in bf16: 105 us, against 118 with 2 chunks), 2 up to 2048 columns (8192 x 2048: 30.2 us,
  // against 32.7).  Fewer rows: one chunk (two beyond 8192 columns), so that a row's loads are in
  // flight at once.
  const int chunks = a.T >= 4 * kSizingSms ? (n8 <= 256 ? 2 : 4) : n8 <= 1024 ? 1 : 2;
  const dim3 grid(static_cast<unsigned>(a.T)), block(round32((n8 + chunks - 1) / chunks));
  if (chunks == 4) residual_norm_kernel<F32, 4><<<grid, block, 0, s>>>(a);
  else if (chunks == 2) residual_norm_kernel<F32, 2><<<grid, block, 0, s>>>(a);
  else residual_norm_kernel<F32, 1><<<grid, block, 0, s>>>(a);
}

template <bool F32, bool CLUSTER, bool FULL, bool ALL>
nvfp4_status_t launch_backward(const Args& a, const Columns& C, cudaStream_t s) {
  auto* fn = residual_norm_backward_kernel<F32, CLUSTER, FULL, ALL>;
  const int row = row_layout<F32>(a, C.width).bytes;
  // the largest row: float32 r and dr', a full gate, every column that a CTA can take
  constexpr int kMost = 2 * kBwdWidth * 14;
  static_assert(kMost + 2560 <= 228 * 1024, "two rows of the widest form");
  // a CTA's share of an SM's 228 KB, less its static shared memory and what the system reserves
  int room = 228 * 1024 / C.per_sm - 2560;
  room = room < kMost ? room : kMost;
  int stages = room / row;
  stages = stages < 1 ? 1 : stages > kBwdStages ? kBwdStages : stages;
  static std::atomic<uint64_t> devices_set{0};
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(devices_set.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost) != cudaSuccess)
      return check_launch("residual_norm_backward_kernel attributes");
    devices_set.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(bwd_clusters(a.T, a.H) * C.cluster));
  cfg.blockDim = dim3(static_cast<unsigned>(C.threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(stages * row);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = static_cast<unsigned>(C.cluster);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = CLUSTER ? 1 : 0;
  cudaLaunchKernelEx(&cfg, fn, static_cast<const Args>(a), stages, C.width);
  return check_launch("residual_norm_backward_kernel");
}

template <bool F32, bool FULL, bool ALL>
nvfp4_status_t launch_backward(const Args& a, cudaStream_t s) {
  const Columns C(a.H);
  return C.cluster == 1 ? launch_backward<F32, false, FULL, ALL>(a, C, s)
                        : launch_backward<F32, true, FULL, ALL>(a, C, s);
}

template <bool F32>
nvfp4_status_t launch_backward(const Args& a, cudaStream_t s) {
  const bool all = a.dr_new != nullptr && a.dn != nullptr && a.y != nullptr;
  if (a.gate_kind == GATE_FULL)
    return all ? launch_backward<F32, true, true>(a, s) : launch_backward<F32, true, false>(a, s);
  return all ? launch_backward<F32, false, true>(a, s) : launch_backward<F32, false, false>(a, s);
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
  const int res = r_dtype == 0 ? 4 : 2;
  const Span outs[] = {rows_span(a, y ? r_out : nullptr, res, H),
                       rows_span(a, pre_gamma ? n_out : nullptr, 2, H),
                       vector_span(post_gamma ? rstd_post : nullptr, T, 4),
                       vector_span(pre_gamma ? rstd_pre : nullptr, T, 4)};
  const Span ins[] = {rows_span(a, r, res, ld_r), rows_span(a, y, 2, ld_y),
                      vector_span(post_gamma, H, 2), vector_span(pre_gamma, H, 2), gate_span(a)};
  if (!outputs_apart(outs, ins)) return NVFP4_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (r_dtype == 0) launch_forward<true>(a, s);
  else launch_forward<false>(a, s);
  return check_launch("residual_norm_kernel");
}

extern "C" size_t nvfp4_residual_norm_backward_workspace_size(int64_t T, int H) {
  if (T <= 0 || H <= 0 || H > kMaxH || H % 8) return 0;
  return static_cast<size_t>((int64_t)bwd_clusters(T, H) * 2 * H * 4);
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
  if (T > 0) {
    const int res = r_dtype == 0 ? 4 : 2;
    const Span outs[] = {
        rows_span(a, dr, res, H), rows_span(a, y ? dy : nullptr, 2, H), vector_span(dpost_gamma, H, 4),
        vector_span(dpre_gamma, H, 4),
        gate_kind == GATE_FULL ? rows_span(a, dgate, 2, H)
                               : vector_span(dgate, gate_kind == GATE_TOKEN ? T : H, 4),
        vector_span(a.part, columns ? (int64_t)bwd_clusters(T, H) * 2 * H : 0, 4)};
    const Span ins[] = {rows_span(a, dr_new, res, H), rows_span(a, dn, 2, H),
                        rows_span(a, dn ? r : nullptr, res, ld_r), rows_span(a, y, 2, ld_y),
                        vector_span(post_gamma, H, 2), vector_span(pre_gamma, H, 2), gate_span(a),
                        vector_span(post_gamma ? rstd_post : nullptr, T, 4),
                        vector_span(dn ? rstd_pre : nullptr, T, 4)};
    if (!outputs_apart(outs, ins)) return NVFP4_ERR_INVALID_ARG;
  }
  a.status = dev_status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int parts = 0;
  if (T > 0) {
    parts = bwd_clusters(T, H);
    st = r_dtype == 0 ? launch_backward<true>(a, s) : launch_backward<false>(a, s);
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
