// w4a16.cu — products of NVFP4 weights with unquantized activations, for few rows: the dense
// nvfp4_linear_w4a16 and the expert FFN moe_ffn_w4a16.
//
//   out[m][n] = (1/gs) * sum_k x[m][k] * E2M1(code[n][k]) * E4M3(sf[n][k/16])
//
// Bound by reading the weights once (9/16 byte per element).  The weights go from memory to
// registers in the layout the block-scaled GEMMs store them in, are decoded there and enter
// mma.sync (m16n8k16, f16 in, f32 accumulators) as its 16-row operand, the tokens being the
// 8 columns.  tcgen05 takes its operands from shared or tensor memory, so a decoded weight
// would have to be written back before the product; at 8 tokens the product is far from the
// tensor cores' rate and the round trip would be the bound.
//
// Exactness.  E2M1 * E4M3 has at most 6 significant bits and lies in [2^-10, 2688], so the
// decoded weight is exact in f16.  A token's activations are multiplied by one power of two per
// CTA that brings their largest finite magnitude into [2^14, 2^15): a bf16 value is then exact in
// f16 unless it is below 2^-29 of that maximum, where it is off by at most 2^-40 of the maximum
// (less than the float32 sum of K such products is off).  A float32 activation (the FFN's
// intermediate) enters as the sum of two f16 values, off by at most 2^-23 of itself or 2^-39 of
// the maximum.  Infinities and NaNs pass through the conversion and the product as such.
//
// Layout.  A warp owns 32 rows of a 128-row block, rows 8*rg + g + 32*i (g = lane/4, i < 4), and
// per step 256 elements of K, lane q = lane%4 the 64 elements from 64*q: 32 bytes of codes per
// row and one 16-byte line of the scale atom, which holds the scales of exactly those 4 rows and
// 64 elements.  The order of K inside a step is free as long as both operands agree, so a lane's
// own 4 weights of a row are the 4 K positions the MMA wants from it.
#include <cuda_fp16.h>

#include "common.cuh"
#include "launch.h"

namespace nvfp4 {
namespace {

constexpr int kRowWarps = 4;               // 4 x 32 rows = one 128-row scale atom
constexpr int kKWarps = 2;                 // warps that share a row group, over K steps
constexpr int kThreads = 32 * kRowWarps * kKWarps;
constexpr int kWarps = kThreads / 32;
constexpr int kStepK = 256;                // elements of K per warp step
constexpr int kXCache = 4;                 // 256-element pieces of x a warp keeps in registers
constexpr int kXBytes = 64 * 1024;         // shared memory for the staged activations, at most

enum Mode { DENSE = 0, FFN_L1 = 1, FFN_L2 = 2 };

struct Args {
  const uint8_t* codes;   // [E*N][K/2]
  const uint8_t* sf;      // per expert round_up(N, 128) rows of tiled scales
  const float* gs;        // [E]
  int N, K;
  const void* x;          // bf16 [.][ld] (DENSE, FFN_L1) or float [slots][K] (FFN_L2)
  int64_t ld;
  int M;                  // rows of x (DENSE)
  int k;                  // slots per token (FFN_L1)
  const int4* plan;       // {expert, first, count, 0} per busy expert (FFN)
  const int32_t* n_plan;  // number of busy experts
  const int32_t* order;   // slots sorted by expert
  void* out;              // DENSE: [M][N]; FFN_L1: float [slots][N/2]; FFN_L2: float [slots][N]
  int out_f32;            // DENSE
  int splits;             // CTAs of a cluster that share an output block along K
  int chunk_steps;        // K steps of x staged at a time
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8 E2M1 codes -> 4 f16 pairs, exact
__device__ __forceinline__ void decode8(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}
// 2 E4M3 scales -> an f16 pair, exact
__device__ __forceinline__ uint32_t decode_scales(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint4 ldg_once(const void* p) {  // streamed: read by one warp only
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// One warp step of weights: 4 rows x 64 elements per lane.
struct Step {
  uint4 c[4][2];
  uint4 s;
};

// 8 consecutive activations of a lane, as stored
template <Mode MODE>
struct X8 {
  static constexpr int W = MODE == FFN_L2 ? 8 : 4;
  uint32_t raw[W];
  __device__ __forceinline__ void load(const void* row, int64_t k, bool ok) {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      uint4 a = make_uint4(0u, 0u, 0u, 0u);
      // plain loads: the FFN's intermediate was written by the previous kernel
      if (ok) a = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + k * (W / 2) +
                                                  i * 4);
      raw[i] = a.x;
      raw[i + 1] = a.y;
      raw[i + 2] = a.z;
      raw[i + 3] = a.w;
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (MODE == FFN_L2) return __uint_as_float(raw[i]);
    else return __uint_as_float((i & 1) ? raw[i / 2] & 0xFFFF0000u : raw[i / 2] << 16);
  }
  // bits of the largest finite magnitude
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = __float_as_uint(at(i)) & 0x7FFFFFFFu;
      if (b < 0x7F800000u) m = max(m, b);
    }
    return m;
  }
};

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Exponent e with amax * 2^e in [2^14, 2^15), at most 126 (then every value fits f16 anyway);
// 0 for a token without finite nonzero values.
__device__ __forceinline__ int norm_exp(uint32_t amax_bits) {
  const int be = static_cast<int>(amax_bits >> 23);  // 0: zero or subnormal
  if (amax_bits == 0) return 0;
  return min(141 - be, 126);
}
__device__ __forceinline__ float pow2f(int e) {  // e in [-126, 127]
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

template <int NT, Mode MODE>
__global__ void __launch_bounds__(kThreads, NT == 4 ? 1 : 2) w4a16_kernel(const Args A) {
  constexpr int TOK = 8 * NT;
  constexpr int PARTS = MODE == FFN_L2 ? 2 : 1;  // f16 terms an activation is held in
  constexpr int kRedStride = 128 + 4;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t s_amax[TOK];
  __shared__ int s_row[TOK];  // row of x (and, for the FFN, slot) of each token column
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, q = lane & 3;
  const int rg = warp % kRowWarps, wk = warp / kRowWarps;
  const int split = static_cast<int>(blockIdx.x) % A.splits;
  const int rowblk = static_cast<int>(blockIdx.x) / A.splits;

  // which tokens, against which expert
  int e = 0, first = 0, count = A.M;
  if constexpr (MODE != DENSE) {
    pdl_wait();
    pdl_trigger();
    if (static_cast<int>(blockIdx.y) >= *reinterpret_cast<const volatile int32_t*>(A.n_plan)) return;
    const int4 p = A.plan[blockIdx.y];
    e = p.x;
    first = p.y;
    count = p.z;
  }
  const int64_t Npad = (A.N + 127) / 128 * 128;
  const uint8_t* codes = A.codes + (int64_t)e * A.N * (A.K / 2);
  const uint8_t* sf = A.sf + (int64_t)e * Npad * (A.K / 16);
  const float gs = __ldg(A.gs + e);
  const int nsteps = (A.K + kStepK - 1) / kStepK;
  const int st0 = static_cast<int>((int64_t)nsteps * split / A.splits);
  const int st1 = static_cast<int>((int64_t)nsteps * (split + 1) / A.splits);
  const int row0 = rowblk * 128 + 8 * rg + g;  // this lane's first row; the others at +32, +64, +96
  const uint8_t* sline = sf + (int64_t)rowblk * (A.K / 64) * 512 + (8 * rg + g) * 16;

  auto load_step = [&](int s, Step& w) {
    const int kk = s * kStepK + q * 64;
    const bool ok = s < st1 && kk < A.K;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w.c[i][0] = w.c[i][1] = make_uint4(0u, 0u, 0u, 0u);
      if (ok && row0 + 32 * i < A.N) {
        const uint8_t* p = codes + (int64_t)(row0 + 32 * i) * (A.K / 2) + kk / 2;
        w.c[i][0] = ldg_once(p);
        w.c[i][1] = ldg_once(p + 16);
      }
    }
    w.s = make_uint4(0u, 0u, 0u, 0u);
    if (ok) w.s = ldg_once(sline + (int64_t)(kk / 64) * 512);
  };

  // token blocks of TOK: the dense form takes them from the grid, the FFN (an expert rarely has
  // more than one) in a loop
  const int tb_first = MODE == DENSE ? static_cast<int>(blockIdx.y) : 0;
  const int tb_last = MODE == DENSE ? tb_first + 1 : (count + TOK - 1) / TOK;
  for (int tb = tb_first; tb < tb_last; ++tb) {
    const int ntok = min(TOK, count - tb * TOK);
    Step nxt;
    load_step(st0 + wk, nxt);  // in flight while the activations are staged
    if (tid < TOK) {
      s_amax[tid] = 0;
      int r = tb * TOK + tid;
      if constexpr (MODE != DENSE) r = tid < ntok ? __ldg(A.order + first + r) : 0;
      s_row[tid] = r;
    }
    __syncthreads();
    auto x_row = [&](int t) -> const void* {
      const int64_t r = s_row[t];
      if constexpr (MODE == FFN_L2) return static_cast<const float*>(A.x) + r * A.ld;
      else if constexpr (MODE == FFN_L1)
        return static_cast<const __nv_bfloat16*>(A.x) + r / A.k * A.ld;
      else return static_cast<const __nv_bfloat16*>(A.x) + r * A.ld;
    };

    // largest magnitude of each token over this CTA's part of K; pieces of 256 elements, one
    // per warp at a time, the first kXCache of them kept
    const int my_steps = st1 - st0;
    const int pieces = ntok * my_steps;
    X8<MODE> cache[kXCache];
    auto load_piece = [&](int p, X8<MODE>& x) {
      const int t = p / my_steps, kk = (st0 + p % my_steps) * kStepK + lane * 8;
      x.load(x_row(t), kk, kk < A.K);
    };
#pragma unroll
    for (int j = 0; j < kXCache; ++j)
      if (warp + j * kWarps < pieces) load_piece(warp + j * kWarps, cache[j]);
    auto fold = [&](int p, const X8<MODE>& x) {
      uint32_t m = x.amax();
      m = __reduce_max_sync(0xffffffffu, m);
      if (lane == 0) atomicMax(&s_amax[p / my_steps], m);
    };
#pragma unroll
    for (int j = 0; j < kXCache; ++j)
      if (warp + j * kWarps < pieces) fold(warp + j * kWarps, cache[j]);
    for (int p = warp + kXCache * kWarps; p < pieces; p += kWarps) {
      X8<MODE> x;
      load_piece(p, x);
      fold(p, x);
    }
    __syncthreads();

    float acc[2][NT][4];
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[p][n][j] = 0.0f;

    // x of one chunk of steps in shared memory: per token 16-byte groups of 8 elements in the
    // order [step][word][quad lane], rows 64 bytes off a multiple of 128 so that the 8 lanes of
    // a shared-memory phase (2 tokens x 4 quads) touch all banks once
    const int64_t tok_bytes = (int64_t)A.chunk_steps * 512 + 64;
    const int64_t part_bytes = tok_bytes * TOK;
    const bool cached = pieces <= kXCache * kWarps && my_steps <= A.chunk_steps;
    for (int c0 = st0; c0 < st1; c0 += A.chunk_steps) {
      const int c1 = min(st1, c0 + A.chunk_steps);
      if (c0 > st0) __syncthreads();
      const int cs = c1 - c0;
      auto store_piece = [&](int t, int ls, const X8<MODE>& x) {
        const float f = pow2f(norm_exp(s_amax[t]));
        uint32_t h[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = x.at(2 * i) * f, b = x.at(2 * i + 1) * f;
          h[i] = pack_half2(a, b);
          if constexpr (PARTS == 2) {
            const float2 hf = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
            // an infinity or NaN is carried by the first term alone
            l[i] = pack_half2(isfinite(a) ? a - hf.x : 0.0f, isfinite(b) ? b - hf.y : 0.0f);
          }
        }
        uint8_t* d = smem + t * tok_bytes + ((ls * 8 + (lane & 7)) * 4 + (lane >> 3)) * 16;
        *reinterpret_cast<uint4*>(d) = make_uint4(h[0], h[1], h[2], h[3]);
        if constexpr (PARTS == 2)
          *reinterpret_cast<uint4*>(d + part_bytes) = make_uint4(l[0], l[1], l[2], l[3]);
      };
      if (cached) {
#pragma unroll
        for (int j = 0; j < kXCache; ++j) {
          const int p = warp + j * kWarps;
          if (p < pieces) store_piece(p / my_steps, p % my_steps, cache[j]);
        }
      } else {
        for (int p = warp; p < ntok * cs; p += kWarps) {
          const int t = p / cs, kk = (c0 + p % cs) * kStepK + lane * 8;
          X8<MODE> x;
          x.load(x_row(t), kk, kk < A.K);
          store_piece(t, p % cs, x);
        }
      }
      __syncthreads();
      for (int s = c0 + ((wk - (c0 - st0)) & (kKWarps - 1)); s < c1; s += kKWarps) {
        const Step w = nxt;
        load_step(s + kKWarps, nxt);
        uint32_t sc[4][2];
        const uint32_t sw[4] = {w.s.x, w.s.y, w.s.z, w.s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sc[i][0] = decode_scales(sw[i] & 0xFFFFu);
          sc[i][1] = decode_scales(sw[i] >> 16);
        }
        const uint8_t* xs = smem + ((s - c0) * 32 + q) * 16 + g * tok_bytes;
#pragma unroll
        for (int wd = 0; wd < 8; ++wd) {
          uint4 b[PARTS][NT];
#pragma unroll
          for (int pt = 0; pt < PARTS; ++pt)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              b[pt][n] = make_uint4(0u, 0u, 0u, 0u);
              if (n * 8 + g < ntok)
                b[pt][n] = *reinterpret_cast<const uint4*>(xs + pt * part_bytes +
                                                           n * 8 * tok_bytes + wd * 64);
            }
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            uint32_t a[2][4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint4& cv = w.c[2 * p + r][wd >> 2];
              const uint32_t word = (wd & 3) == 0 ? cv.x : (wd & 3) == 1 ? cv.y
                                    : (wd & 3) == 2 ? cv.z : cv.w;
              decode8(word, a[r]);
              // the scale of 16-element group wd / 2, in both halves
              const uint32_t sv = __byte_perm(sc[2 * p + r][wd >> 2], 0u,
                                              (wd & 2) ? 0x3232u : 0x1010u);
#pragma unroll
              for (int j = 0; j < 4; ++j) a[r][j] = mul_f16x2(a[r][j], sv);
            }
#pragma unroll
            for (int pt = 0; pt < PARTS; ++pt)
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                mma_f16(acc[p][n], a[0][0], a[1][0], a[0][1], a[1][1], b[pt][n].x, b[pt][n].y);
                mma_f16(acc[p][n], a[0][2], a[1][2], a[0][3], a[1][3], b[pt][n].z, b[pt][n].w);
              }
          }
        }
      }
    }

    // partial sums of the K warps (and of the cluster's CTAs) -> shared memory, added in order
    __syncthreads();
    float* red = reinterpret_cast<float*>(smem);  // [kKWarps][TOK][kRedStride]
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int t = n * 8 + 2 * q;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        // the token's power of two and the global scale, the one that shrinks the sum first
        const int ne = norm_exp(s_amax[t + c]);
        const float f = pow2f(-ne);
        auto unscale = [&](float v) { return ne > 0 ? v * f / gs : v / gs * f; };
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            red[(wk * TOK + t + c) * kRedStride + 8 * rg + g + 64 * p + 32 * r] =
                unscale(acc[p][n][2 * r + c]);
      }
    }
    if (A.splits > 1) cluster_sync();
    else __syncthreads();
    auto total = [&](int row, int t) {
      float v = 0.0f;
      if (A.splits > 1) {
        for (int c = 0; c < A.splits; ++c) {
#pragma unroll
          for (int w = 0; w < kKWarps; ++w)
            v += ld_cluster_f32(
                mapa_shared(smem_u32(red + (w * TOK + t) * kRedStride + row), c));
        }
      } else {
#pragma unroll
        for (int w = 0; w < kKWarps; ++w) v += red[(w * TOK + t) * kRedStride + row];
      }
      return v;
    };
    const int share = 128 / A.splits, r0 = share * split;
    if constexpr (MODE == FFN_L1) {
      // gate rows 32j + i, up rows 32j + 16 + i -> feature 16j + i
      const int feats = share / 2, I = A.N / 2;
      for (int idx = tid; idx < feats * ntok; idx += kThreads) {
        const int f = idx % feats, t = idx / feats;
        const int row = r0 + (f / 16) * 32 + f % 16;
        const int feat = (rowblk * 128 + r0) / 2 + f;
        const float gate = total(row, t), up = total(row + 16, t);
        const float h = gate * up / (1.0f + expf(-gate));
        if (feat < I) static_cast<float*>(A.out)[(int64_t)s_row[t] * I + feat] = h;
      }
    } else {
      for (int idx = tid; idx < share * ntok; idx += kThreads) {
        const int row = r0 + idx % share, t = idx / share;
        const int n = rowblk * 128 + row;
        const float v = total(row, t);
        if (n < A.N) {
          const int64_t at = (int64_t)s_row[t] * A.N + n;
          if (MODE == FFN_L2 || A.out_f32) static_cast<float*>(A.out)[at] = v;
          else static_cast<__nv_bfloat16*>(A.out)[at] = __float2bfloat16_rn(v);
        }
      }
    }
    // the peers have read this CTA's sums before it leaves or reuses them
    if (A.splits > 1) cluster_sync();
    else __syncthreads();
  }
}

// out[t] = sum over the token's live slots of w * ys[slot], in slot order, FP32 -> bf16.
__global__ void __launch_bounds__(256) combine_slots_kernel(
    const float* __restrict__ ys, const int32_t* __restrict__ ids, const float* __restrict__ w,
    int H, int E, int k, __nv_bfloat16* __restrict__ out) {
  pdl_wait();
  const int t = blockIdx.x;
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * 4;
  if (c >= H) return;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j = 0; j < k; ++j) {
    const int id = ids[t * k + j];
    if (id < 0 || id >= E) continue;
    const float wj = w[t * k + j];
    const float4 y = *reinterpret_cast<const float4*>(ys + ((int64_t)t * k + j) * H + c);
    v[0] += wj * y.x;
    v[1] += wj * y.y;
    v[2] += wj * y.z;
    v[3] += wj * y.w;
  }
  __nv_bfloat162 o[2] = {__floats2bfloat162_rn(v[0], v[1]), __floats2bfloat162_rn(v[2], v[3])};
  *reinterpret_cast<uint2*>(out + (int64_t)t * H + c) = *reinterpret_cast<const uint2*>(o);
}

// CTAs along K for one output block: enough CTAs to give every SM two, while each K warp keeps
// at least one step.
int pick_splits(int64_t blocks, int K, int most) {
  const int steps = (K + kStepK - 1) / kStepK;
  int s = 1;
  while (s < most && blocks * s < 2 * device_sms() && steps / (2 * s) >= kKWarps) s *= 2;
  return s;
}

template <int NT, Mode MODE>
nvfp4_status_t launch(const Args& a, dim3 grid, bool pdl, cudaStream_t s) {
  auto* fn = w4a16_kernel<NT, MODE>;
  constexpr int parts = MODE == FFN_L2 ? 2 : 1;
  const size_t x_bytes = (size_t)(a.chunk_steps * 512 + 64) * 8 * NT * parts;
  const size_t red_bytes = (size_t)kKWarps * 8 * NT * 132 * 4;
  const size_t smem = x_bytes > red_bytes ? x_bytes : red_bytes;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem)) != cudaSuccess)
    return check_launch("w4a16_kernel attributes");
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  int n = 0;
  at[n].id = cudaLaunchAttributeClusterDimension;
  at[n].val.clusterDim.x = static_cast<unsigned>(a.splits);
  at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
  ++n;
  if (pdl) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = at;
  cfg.numAttrs = static_cast<unsigned>(n);
  if (cudaLaunchKernelEx(&cfg, fn, a) != cudaSuccess) return check_launch("w4a16_kernel");
  return check_launch("w4a16_kernel");
}

// K steps of x staged at a time for NT token tiles of `parts` f16 terms.
int pick_chunk(int K, int splits, int NT, int parts) {
  const int steps = (K + kStepK - 1) / kStepK;
  const int mine = (steps + splits - 1) / splits;
  const int fit = kXBytes / (8 * NT * parts * 512);
  return mine < fit ? mine : fit;
}

template <Mode MODE>
nvfp4_status_t launch_nt(int nt, Args a, dim3 grid, bool pdl, cudaStream_t s) {
  a.chunk_steps = pick_chunk(a.K, a.splits, nt, MODE == FFN_L2 ? 2 : 1);
  switch (nt) {
    case 1: return launch<1, MODE>(a, grid, pdl, s);
    case 2: return launch<2, MODE>(a, grid, pdl, s);
    default: return launch<4, MODE>(a, grid, pdl, s);
  }
}

// Byte offsets of the moe_ffn_w4a16 workspace regions (each 256-byte aligned).
struct W4Layout {
  int64_t ids, w, plan, n_plan, order, h, ys, total;
};

W4Layout w4_layout(int T, int H, int I, int E, int k) {
  W4Layout L{};
  const int64_t S = (int64_t)T * k;
  int64_t o = 0;
  auto take = [&](int64_t bytes) {
    const int64_t at = o;
    o = round_up(o + bytes, 256);
    return at;
  };
  L.ids = take(S * 4);
  L.w = take(S * 4);
  L.plan = take((int64_t)E * 16);
  L.n_plan = take(4);
  L.order = take(S * 4);
  L.h = take(S * I * 4);
  L.ys = take(S * H * 4);
  L.total = o;
  return L;
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status_t nvfp4_linear_w4a16(const void* x, int64_t M, int K, int64_t ld,
                                             const uint8_t* w, const uint8_t* sfw,
                                             const float* gs_w, int N, void* out, int out_dtype,
                                             nvfp4_stream_t stream) {
  if (M < 0 || N <= 0 || K <= 0 || ld < K || (out_dtype != 0 && out_dtype != 1))
    return NVFP4_ERR_INVALID_ARG;
  if (K % 64 || ld % 8 || M > (int64_t)65535 * 32 || N > INT32_MAX - 127)
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!w || !sfw || !gs_w) return NVFP4_ERR_INVALID_ARG;
  if (M > 0 && (!x || !out)) return NVFP4_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w) || !aligned16(sfw) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(gs_w) & 3u))
    return NVFP4_ERR_MISALIGNED;
  if (M == 0) return NVFP4_OK;
  const int nt = M <= 8 ? 1 : M <= 16 ? 2 : 4;
  const int64_t rowblks = (N + 127) / 128, tblks = (M + 8 * nt - 1) / (8 * nt);
  Args a{};
  a.codes = w;
  a.sf = sfw;
  a.gs = gs_w;
  a.N = N;
  a.K = K;
  a.x = x;
  a.ld = ld;
  a.M = static_cast<int>(M);
  a.out = out;
  a.out_f32 = out_dtype == 0;
  a.splits = pick_splits(rowblks * tblks, K, 8);
  return launch_nt<DENSE>(nt, a,
                          dim3(static_cast<unsigned>(rowblks * a.splits),
                               static_cast<unsigned>(tblks)),
                          false, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" size_t moe_ffn_w4a16_workspace_size(int T, int H, int I, int E, int k) {
  if (T < 0 || H <= 0 || I <= 0 || E <= 0 || k <= 0) return 0;
  return static_cast<size_t>(w4_layout(T, H, I, E, k).total);
}

extern "C" nvfp4_status_t moe_ffn_w4a16(const void* x_bf16, const float* logits,
                                        const int32_t* topk_ids, const float* topk_w, int T, int H,
                                        int I, int E, int k, const uint8_t* w1,
                                        const uint8_t* sfw1, const float* gs_w1, const uint8_t* w2,
                                        const uint8_t* sfw2, const float* gs_w2, void* out_bf16,
                                        void* ws, size_t ws_bytes, int32_t* dev_status,
                                        nvfp4_stream_t stream) {
  if (T < 0 || E < 1 || E > 256 || k < 1 || k > 32 || k > E || H <= 0 || I <= 0)
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (H % 128 || I % 64) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if ((int64_t)T * k > NVFP4_W4A16_MAX_SLOTS) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return NVFP4_OK;
  if (!x_bf16 || !w1 || !sfw1 || !gs_w1 || !w2 || !sfw2 || !gs_w2 || !out_bf16 || !ws)
    return NVFP4_ERR_INVALID_ARG;
  if (logits == nullptr ? (!topk_ids || !topk_w) : (topk_ids || topk_w))
    return NVFP4_ERR_INVALID_ARG;  // logits, or a given routing: exactly one of them
  const W4Layout L = w4_layout(T, H, I, E, k);
  if (ws_bytes < static_cast<size_t>(L.total)) return NVFP4_ERR_WORKSPACE_TOO_SMALL;
  const void* ptrs16[] = {x_bf16, w1, sfw1, w2, sfw2, out_bf16};
  for (const void* p : ptrs16)
    if (!aligned16(p)) return NVFP4_ERR_MISALIGNED;
  const void* ptrs4[] = {logits, topk_ids, topk_w, gs_w1, gs_w2, dev_status};
  for (const void* p : ptrs4)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return NVFP4_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return NVFP4_ERR_MISALIGNED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(ws);
  const int32_t* ids = topk_ids;
  const float* wts = topk_w;
  if (logits != nullptr) {
    ids = reinterpret_cast<int32_t*>(base + L.ids);
    wts = reinterpret_cast<float*>(base + L.w);
  }
  int4* plan = reinterpret_cast<int4*>(base + L.plan);
  int32_t* n_plan = reinterpret_cast<int32_t*>(base + L.n_plan);
  int32_t* order = reinterpret_cast<int32_t*>(base + L.order);
  float* h = reinterpret_cast<float*>(base + L.h);
  float* ys = reinterpret_cast<float*>(base + L.ys);
  nvfp4_status_t st = slot_plan_launch(logits, T, E, k, const_cast<int32_t*>(ids),
                                       const_cast<float*>(wts), plan, n_plan, order, dev_status, s);
  if (st != NVFP4_OK) return st;
  const int S = T * k, busy = S < E ? S : E;
  // token tiles: what an expert gets on average, doubled
  const int per = 2 * S / E;
  const int nt = per <= 8 ? 1 : per <= 16 ? 2 : 4;
  Args a{};
  a.codes = w1;
  a.sf = sfw1;
  a.gs = gs_w1;
  a.N = 2 * I;
  a.K = H;
  a.x = x_bf16;
  a.ld = H;
  a.k = k;
  a.plan = plan;
  a.n_plan = n_plan;
  a.order = order;
  a.out = h;
  const int blocks1 = 2 * I / 128;
  a.splits = pick_splits((int64_t)blocks1 * busy, H, 4);
  st = launch_nt<FFN_L1>(nt, a, dim3(blocks1 * a.splits, busy), true, s);
  if (st != NVFP4_OK) return st;
  a.codes = w2;
  a.sf = sfw2;
  a.gs = gs_w2;
  a.N = H;
  a.K = I;
  a.x = h;
  a.ld = I;
  a.out = ys;
  const int blocks2 = H / 128;
  a.splits = pick_splits((int64_t)blocks2 * busy, I, 8);
  st = launch_nt<FFN_L2>(nt, a, dim3(blocks2 * a.splits, busy), true, s);
  if (st != NVFP4_OK) return st;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(T, (H / 4 + 255) / 256);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, combine_slots_kernel, static_cast<const float*>(ys), ids, wts, H, E, k,
                     static_cast<__nv_bfloat16*>(out_bf16));
  return check_launch("combine_slots_kernel");
}
