// w4a16.cu — products of NVFP4 weights with unquantized activations, for few rows: the dense
// nvfp4_linear_w4a16 and the expert FFN moe_ffn_w4a16.
//
//   out[m][n] = (1/gs) * sum_k x[m][k] * E2M1(code[n][k]) * E4M3(sf[n][k/16])
//
// Bound by reading the weights once (9/16 byte per element).  TMA brings them to shared memory in
// the layout the block-scaled GEMMs store them in; a warp decodes its rows in registers and
// multiplies with mma.sync (m16n8k16, f16 in, float32 accumulators), the weights being the 16-row
// operand and the tokens the 8 columns.  tcgen05 takes its operands from shared or tensor memory,
// so every decoded weight would have to be written back before the product; at a few tokens the
// product is far from the tensor cores' rate and the round trip would be the bound.
//
// Exactness.  E2M1 * E4M3 has at most 6 significant bits and lies in [2^-10, 2688], so the
// decoded weight is exact in f16.  A row of activations is multiplied by the power of two that
// brings its largest finite magnitude into [2^14, 2^15): a bf16 value is then exact in f16 unless
// it is below 2^-29 of that maximum, where it is off by at most 2^-40 of the maximum (less than
// the float32 sum of K such products is off).  The FFN's float32 intermediate is rounded to f16's
// 11 bits there, 1/8 of the step that the bf16 output is rounded to in the end (a second f16 term
// would double the MMAs, and they would be the bound).  Infinities and NaNs pass through the
// conversion and the product as such.
//
// Layout.  A warp owns 32 rows of a 128-row block, rows 8*rg + g + 32*i (g = lane/4, i < 4), and
// per step 256 elements of K, lane q = lane%4 the 64 elements from 64*q: 32 bytes of codes per
// row and one 16-byte line of a scale atom, which holds the scales of exactly those 4 rows and
// 64 elements.  The order of K inside a step is free as long as both operands agree, so a lane's
// own 4 weights of a row are the 4 K positions the MMA wants from it, and the converted
// activations are stored in that order.
#include <cuda_fp16.h>

#include <atomic>

#include "common.cuh"
#include "launch.h"
#include "topk.cuh"

namespace nvfp4 {
namespace {

constexpr int kRowWarps = 4;               // 4 x 32 rows = one 128-row scale atom
constexpr int kKWarps = 2;                 // warps that share a row group, taking steps in turn
constexpr int kConsumers = kRowWarps * kKWarps;
constexpr int kThreads = 32 * (kConsumers + 1);  // and one warp that issues the copies
constexpr int kStepK = 256;                // elements of K per step
constexpr int kStepX = kStepK * 2;         // bytes of a token's converted activations per step
constexpr int kMaxSplits = 8;              // CTAs of a cluster along K
constexpr int kWTile = 128 * 128;          // codes of a step: 128 rows x 128 bytes
constexpr int kSTile = 4 * 512;            // its scale atoms
// A token's 512 bytes in a stage are 64 bytes off a multiple of 128, so that the 8 lanes of a
// shared-memory phase (2 tokens x 4 quads of 16 bytes) touch every bank once.
constexpr int kXRow = kStepX + 64;
constexpr int kRedStride = 128 + 4;
// XIN: activations that a CTA converts itself, in pieces of one token's step (two per warp, held in
// registers between the two passes).  At 1 x 4096 x 7168 (4 pieces a CTA) 7.4 us against 8.4 us
// with a converting kernel in front; with 28 pieces (1 x 65536 x 7168, 512 CTAs) 58 against 55.
constexpr int kMaxPieces = 2 * kConsumers;

template <int NT, bool XIN>
struct Cfg {
  static constexpr int TOK = 8 * NT;  // token columns
  static constexpr int STAGE = kWTile + kSTile + (XIN ? 0 : (TOK * kXRow + 1023) / 1024 * 1024);
  // two CTAs per SM with up to 16 tokens (so that one's start and end overlap the other's
  // stream), one with 32, whose accumulators need the registers
  static constexpr int CTAS = NT == 4 ? 1 : 2;
  static constexpr int STAGES = NT == 4 ? 6 : 4;
  static constexpr int X_AT = STAGES * STAGE;  // XIN: the activations behind the stages
  static constexpr int SMEM = X_AT + (XIN ? kMaxPieces * kXRow : 0) + 1024;
  static_assert(kKWarps * TOK * kRedStride * 4 <= STAGES * STAGE, "partial sums reuse the stages");
  static_assert(STAGES % kKWarps == 0, "a stage is always the same K warps', or one could wait two phases ahead");
  static_assert(CTAS * (SMEM + 3072) <= 227 * 1024, "shared memory of an SM");
};

enum Mode { DENSE = 0, FFN_L1 = 1, FFN_L2 = 2 };

struct Args {
  const uint8_t* sf;      // per expert round_up(N, 128) rows of tiled scales
  const float* gs;        // [E]
  int N, K;
  const void* x;          // XIN: bf16 activations, rows of ld_bytes
  int64_t ld_bytes;
  const uint8_t* xf;      // else: converted ones, [rows][steps][kStepX bytes]
  const int32_t* exps;    // and [rows] the power of two each row was multiplied by
  int M;                  // rows (DENSE)
  int k;                  // slots per token (FFN)
  const int4* plan;       // {expert, first, count, 0} per busy expert (FFN)
  const int32_t* n_plan;  // number of busy experts
  const int32_t* order;   // slots sorted by expert
  void* out;              // DENSE: [M][N]; FFN_L1: float [slots][N/2]; FFN_L2: float [slots][N]
  int out_f32;            // DENSE
  int splits;             // CTAs of a cluster that share an output block along K
  int32_t* status;
};

// Not volatile: pure functions of their operands, for the compiler to schedule.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same with zero accumulators
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
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
__device__ __forceinline__ uint4 lds16(const uint8_t* p) {
  return *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
// Programmatic dependent launch: wait until the kernels before this one are complete and visible;
// let the next kernel's CTAs start (they wait in turn).
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ------------------------------------------------------------------- converted activations

// Exponent e with amax * 2^e in [2^14, 2^15), at most 126 (then every value fits f16 anyway);
// 0 for a row without finite nonzero values.
__device__ __forceinline__ int norm_exp(uint32_t amax_bits) {
  if (amax_bits == 0) return 0;
  return min(141 - static_cast<int>(amax_bits >> 23), 126);
}
__device__ __forceinline__ float pow2f(int e) {  // e in [-126, 127]
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// What an earlier kernel of a dependent launch wrote is read with these, after pdl_wait(): they are
// ordered behind it, which the compiler does not promise for loads through const __restrict__.
__device__ __forceinline__ uint4 ld_after16(const void* p) {
  uint4 v;
  asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ int32_t ld_after(const int32_t* p) {
  int32_t v;
  asm volatile("ld.global.cg.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// 8 consecutive activations, as stored
template <bool F32>
struct X8 {
  static constexpr int W = F32 ? 8 : 4;
  uint32_t raw[W];
  __device__ __forceinline__ void load(const void* row, int64_t k, bool ok) {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      uint4 a = make_uint4(0u, 0u, 0u, 0u);
      if (ok) a = ld_after16(static_cast<const uint8_t*>(row) + k * (W / 2) + i * 4);
      raw[i] = a.x;
      raw[i + 1] = a.y;
      raw[i + 2] = a.z;
      raw[i + 3] = a.w;
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (F32) return __uint_as_float(raw[i]);
    else return __uint_as_float((i & 1) ? raw[i / 2] & 0xFFFF0000u : raw[i / 2] << 16);
  }
  // float32 bits of the largest finite magnitude
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = __float_as_uint(at(i)) & 0x7FFFFFFFu;
      if (b < 0x7F800000u) m = max(m, b);
    }
    return m;
  }
  // the 8 values times f, as f16
  __device__ __forceinline__ uint4 to_f16(float f) const {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 v = __floats2half2_rn(at(2 * i) * f, at(2 * i + 1) * f);
      h[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    return make_uint4(h[0], h[1], h[2], h[3]);
  }
};

// One CTA converts one row of K activations: the power of two, and the f16 values of every step of
// 256 in the order [word of 8][quad lane] (zeros past K).  `red` holds a word per warp.
constexpr int kPrepCache = 4;  // pieces of 8 a thread keeps between the two passes
template <bool F32>
__device__ __forceinline__ void convert_row(const void* row, int K, uint8_t* out, int32_t* exp_out,
                                            uint32_t* red) {
  const int tid = threadIdx.x, nthr = blockDim.x;
  const int pieces = (K + kStepK - 1) / kStepK * (kStepK / 8);
  X8<F32> c[kPrepCache];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < kPrepCache; ++j) {
    const int64_t k = (int64_t)(tid + j * nthr) * 8;
    c[j].load(row, k, k < K);
  }
#pragma unroll
  for (int j = 0; j < kPrepCache; ++j) m = max(m, c[j].amax());
  for (int p = tid + kPrepCache * nthr; p < pieces; p += nthr) {
    X8<F32> x;
    x.load(row, (int64_t)p * 8, p * (int64_t)8 < K);
    m = max(m, x.amax());
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((tid & 31) == 0) red[tid >> 5] = m;
  __syncthreads();
  m = __reduce_max_sync(0xffffffffu, (tid & 31) < nthr / 32 ? red[tid & 31] : 0u);
  const int e = norm_exp(m);
  const float f = pow2f(e);
  if (tid == 0) *exp_out = e;
  // element 8p: step p / 32, quad lane (p % 32) / 8, word p % 8
  auto put = [&](int p, const X8<F32>& x) {
    *reinterpret_cast<uint4*>(out + (int64_t)(p >> 5) * kStepX +
                              ((p & 7) * 4 + ((p >> 3) & 3)) * 16) = x.to_f16(f);
  };
#pragma unroll
  for (int j = 0; j < kPrepCache; ++j)
    if (tid + j * nthr < pieces) put(tid + j * nthr, c[j]);
  for (int p = tid + kPrepCache * nthr; p < pieces; p += nthr) {
    X8<F32> x;
    x.load(row, (int64_t)p * 8, p * (int64_t)8 < K);
    put(p, x);
  }
}

// One row per CTA.  F32: the FFN's intermediate (after its L1), else the caller's bf16 rows.
template <bool F32>
__global__ void __launch_bounds__(256) convert_kernel(const void* x, int64_t ld_bytes, int K,
                                                      uint8_t* xf, int32_t* exps) {
  __shared__ uint32_t red[32];
  pdl_trigger();
  if constexpr (F32) pdl_wait();
  const int64_t r = blockIdx.x, steps = (K + kStepK - 1) / kStepK;
  convert_row<F32>(static_cast<const uint8_t*>(x) + r * ld_bytes, K, xf + r * steps * kStepX,
                   exps + r, red);
}

// The first kernel of the FFN.  CTA 0 makes the plan: top-k (with logits), slots counted per
// expert, an exclusive scan, and the slots in place.  The order of an expert's slots is whatever
// the atomics give; a slot's result does not depend on it (each is a column of its own).  The
// other CTAs convert one token's activations each.
__global__ void __launch_bounds__(512) plan_kernel(
    const float* __restrict__ logits, int T, int E, int k, int32_t* ids, float* w,
    int4* __restrict__ plan, int32_t* __restrict__ n_plan, int32_t* __restrict__ order,
    const void* __restrict__ x, int H, uint8_t* __restrict__ xf, int32_t* __restrict__ exps,
    int32_t* __restrict__ dev_status) {
  __shared__ int cnt[kMaxE];
  __shared__ int cursor[kMaxE];
  __shared__ uint32_t red[32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  if (blockIdx.x > 0) {
    const int64_t r = blockIdx.x - 1, steps = (H + kStepK - 1) / kStepK;
    convert_row<false>(static_cast<const uint8_t*>(x) + r * H * 2, H, xf + r * steps * kStepX,
                       exps + r, red);
    return;
  }
  if (tid < kMaxE) cnt[tid] = 0;
  if (logits != nullptr)
    for (int t = warp; t < T; t += blockDim.x / 32) topk_token(logits, t, E, k, 1, lane, ids, w);
  __syncthreads();  // also: this CTA's ids are visible to all its threads
  const int S = T * k;
  bool bad = false;
  for (int s = tid; s < S; s += blockDim.x) {
    const int e = ids[s];
    if (e >= E) bad = true;
    else if (e >= 0) atomicAdd(&cnt[e], 1);
  }
  if (bad) report(dev_status, NVFP4_DEVERR_BAD_INDEX);
  __syncthreads();
  if (warp == 0) {  // lane l: experts 8l..8l+7
    int c[kPerLane], sum = 0, busy = 0;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      c[i] = cnt[lane * kPerLane + i];
      sum += c[i];
      busy += c[i] > 0;
    }
    int run = sum, at = busy;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, run, o);
      const int b = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) {
        run += v;
        at += b;
      }
    }
    if (lane == 31) *n_plan = at;
    run -= sum;
    at -= busy;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      cursor[lane * kPerLane + i] = run;
      if (c[i] > 0) plan[at++] = make_int4(lane * kPerLane + i, run, c[i], 0);
      run += c[i];
    }
  }
  __syncthreads();
  for (int s = tid; s < S; s += blockDim.x) {
    const int e = ids[s];
    if (e >= 0 && e < E) order[atomicAdd(&cursor[e], 1)] = s;
  }
}

// ------------------------------------------------------------------------- the product

__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kConsumers) : "memory");
}

// XIN: the CTA converts the activations of its rows and its part of K itself, when they are few;
// otherwise a kernel in front has converted them and they pass through the ring with the weights.
template <int NT, Mode MODE, bool XIN>
__global__ void __launch_bounds__(kThreads, Cfg<NT, XIN>::CTAS)
    w4a16_kernel(const __grid_constant__ CUtensorMap tm, const Args A) {
  static_assert(!XIN || MODE == DENSE, "the FFN's activations are converted in front");
  using C = Cfg<NT, XIN>;
  constexpr int TOK = C::TOK, STAGES = C::STAGES;
  // Accumulators of one step: with one token tile each row pair has two, so that a warp's
  // consecutive MMAs do not wait for one another.
  constexpr int CH = NT == 1 ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t bar_full[STAGES], bar_empty[STAGES];
  __shared__ volatile int abort_flag;
  __shared__ __align__(16) uint8_t zeros[kStepX];  // what columns without a token read
  __shared__ int s_row[TOK], s_exp[TOK];           // output row and power of two of each column
  __shared__ uint32_t s_amax[TOK];                 // XIN
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, q = lane & 3;
  const int split = static_cast<int>(blockIdx.x) % A.splits;
  const int rowblk = static_cast<int>(blockIdx.x) / A.splits;
  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(smem_u32(&bar_full[i]), 1);
      mbar_init(smem_u32(&bar_empty[i]), kRowWarps);
    }
    fence_mbar_init();
  }
  if (tid < kStepX / 16) reinterpret_cast<uint4*>(zeros)[tid] = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();

  // Which tokens, against which expert.  The L2 form's plan is older than the kernel it waits
  // for (the conversion of the intermediate, itself behind the L1), so it is read before that
  // wait and the first weights are already on their way during it.
  int e = 0, first = 0, count = A.M;
  if constexpr (MODE == FFN_L1) pdl_wait();
  if constexpr (MODE != DENSE) {
    pdl_trigger();
    if (static_cast<int>(blockIdx.y) >= ld_after(A.n_plan)) {  // the whole cluster
      pdl_wait();  // no kernel of the chain ends before the ones in front of it
      return;
    }
    const uint4 p = ld_after16(A.plan + blockIdx.y);
    e = static_cast<int>(p.x);
    first = static_cast<int>(p.y);
    count = static_cast<int>(p.z);
  }
  const int atoms_k = A.K / 64;
  const int64_t blk_rows = (A.N + 127) / 128;
  const uint8_t* sf = A.sf + ((int64_t)e * blk_rows + rowblk) * atoms_k * 512;
  const uint32_t gs_bits = __float_as_uint(__ldg(A.gs + e));  // a positive normal number
  const int gs_exp = static_cast<int>(gs_bits >> 23) - 127;
  const float gs_frac = __uint_as_float((gs_bits & 0x7FFFFFu) | 0x3F800000u);
  const int nsteps = (A.K + kStepK - 1) / kStepK;
  const int st0 = static_cast<int>((int64_t)nsteps * split / A.splits);
  const int n_st = static_cast<int>((int64_t)nsteps * (split + 1) / A.splits) - st0;

  // token blocks of TOK: the dense form takes them from the grid, the FFN (an expert rarely has
  // more than one) in a loop
  const int tb_first = MODE == DENSE ? static_cast<int>(blockIdx.y) : 0;
  const int tb_last = MODE == DENSE ? tb_first + 1 : (count + TOK - 1) / TOK;
  uint32_t it0 = 0;  // stages used by earlier token blocks
  for (int tb = tb_first; tb < tb_last; ++tb, it0 += n_st) {
    const int ntok = min(TOK, count - tb * TOK);
    auto out_row = [&](int t) {  // DENSE: the row of x; FFN: the slot
      return MODE == DENSE ? tb * TOK + t : ld_after(A.order + first + tb * TOK + t);
    };
    auto x_row = [&](int r) { return MODE == FFN_L1 ? r / A.k : r; };
    float acc[2][NT][4];
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[p][n][j] = 0.0f;

    if (warp == kConsumers) {
      // =========================== copies ===========================
      const int64_t wrow = (int64_t)e * A.N + rowblk * 128;
      bool ok = true;
      auto wait_empty = [&](int i) {
        const uint32_t it = it0 + i;
        const bool mine =
            mbar_wait_bounded(smem_u32(&bar_empty[it % STAGES]), ((it / STAGES) & 1u) ^ 1u, &abort_flag);
        return __all_sync(0xffffffffu, mine) != 0;
      };
      auto copy_w = [&](int i) {  // codes and scales of step st0 + i
        const uint32_t s = (it0 + i) % STAGES;
        if (lane == 0) {
          const int st = st0 + i, atoms = min(4, atoms_k - st * 4);
          const uint32_t bar = smem_u32(&bar_full[s]), d = smem_u32(smem + s * C::STAGE);
          mbar_arrive_expect_tx(bar, kWTile + atoms * 512 + (XIN ? 0 : ntok * kStepX));
          tma_load_2d(d, &tm, bar, st * 128, static_cast<int>(wrow));
          bulk_load(d + kWTile, sf + (int64_t)st * 4 * 512, atoms * 512, bar);
        }
        __syncwarp();
      };
      const uint8_t* xr = nullptr;
      auto copy_x = [&](int i) {  // lane t: token t
        const uint32_t s = (it0 + i) % STAGES;
        if (!XIN && lane < ntok)
          bulk_load(smem_u32(smem + s * C::STAGE + kWTile + kSTile) + lane * kXRow,
                    xr + (int64_t)(st0 + i) * kStepX, kStepX, smem_u32(&bar_full[s]));
      };
      const int head = min(n_st, STAGES);
      int issued = 0;
      for (; issued < head && ok; ++issued) {
        ok = wait_empty(issued);
        if (!ok) break;
        copy_w(issued);
      }
      // the activations come from the kernel before (and for the L1 and later token blocks this
      // has been waited for already)
      pdl_wait();
      if (!XIN && lane < ntok) xr = A.xf + (int64_t)x_row(out_row(lane)) * nsteps * kStepX;
      for (int i = 0; i < issued; ++i) copy_x(i);
      for (; issued < n_st && ok; ++issued) {
        ok = wait_empty(issued);
        if (!ok) break;
        copy_w(issued);
        copy_x(issued);
      }
      if (!ok) {  // let the copies already issued land before the CTA can exit
        volatile int never = 0;
        for (int i = max(0, issued - STAGES); i < issued; ++i)
          mbar_wait_bounded(smem_u32(&bar_full[(it0 + i) % STAGES]), ((it0 + i) / STAGES) & 1u,
                            &never, NVFP4_WAIT_TIMEOUT_NS / 4);
      }
    } else {
      // =========================== products ===========================
      if (tid < ntok) {
        pdl_wait();
        const int r = out_row(tid);
        s_row[tid] = r;
        if (!XIN) s_exp[tid] = ld_after(A.exps + x_row(r));
      }
      if constexpr (XIN) {
        // pieces (token, step) warp and warp + kConsumers: lane l holds elements 8l .. 8l + 7
        const int pieces = ntok * n_st;
        X8<false> c[kMaxPieces / kConsumers];
#pragma unroll
        for (int j = 0; j < kMaxPieces / kConsumers; ++j) {
          const int p = warp + j * kConsumers, k = (st0 + p % n_st) * kStepK + lane * 8;
          if (p < pieces)
            c[j].load(static_cast<const uint8_t*>(A.x) + (int64_t)(tb * TOK + p / n_st) * A.ld_bytes,
                      k, k < A.K);
        }
        if (tid < TOK) s_amax[tid] = 0;
        consumers_sync();
#pragma unroll
        for (int j = 0; j < kMaxPieces / kConsumers; ++j) {
          const int p = warp + j * kConsumers;
          if (p < pieces) {
            const uint32_t m = __reduce_max_sync(0xffffffffu, c[j].amax());
            if (lane == 0) atomicMax(&s_amax[p / n_st], m);
          }
        }
        consumers_sync();
        if (tid < TOK) s_exp[tid] = norm_exp(s_amax[tid]);
#pragma unroll
        for (int j = 0; j < kMaxPieces / kConsumers; ++j) {
          const int p = warp + j * kConsumers;
          if (p < pieces)
            *reinterpret_cast<uint4*>(smem + C::X_AT + p * kXRow +
                                      ((lane & 7) * 4 + (lane >> 3)) * 16) =
                c[j].to_f16(pow2f(norm_exp(s_amax[p / n_st])));
        }
        consumers_sync();
      }
      const int rg = warp % kRowWarps, wk = warp / kRowWarps;
      // this lane's two 16-byte pieces of a row's 128 bytes (128-byte swizzle: the piece index is
      // xored with the row's index modulo 8, which is g for all of the lane's rows)
      const int row_off = (8 * rg + g) * 128;
      const int piece[2] = {((2 * q) ^ g) * 16, ((2 * q + 1) ^ g) * 16};
      const int scale_off = kWTile + q * 512 + (8 * rg + g) * 16;
      for (int i = wk; i < n_st; i += kKWarps) {
        const uint32_t it = it0 + i, s = it % STAGES;
        const bool mine = mbar_wait_bounded(smem_u32(&bar_full[s]), (it / STAGES) & 1u, &abort_flag);
        if (!__all_sync(0xffffffffu, mine)) break;
        const uint8_t* st = smem + s * C::STAGE;
        const uint8_t* xb[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n)
          xb[n] = (n * 8 + g >= ntok ? zeros
                   : XIN ? smem + C::X_AT + ((n * 8 + g) * n_st + i) * kXRow
                         : st + kWTile + kSTile + (n * 8 + g) * kXRow) +
                  q * 16;
        // One step: 8 words of 8 codes per row.  The sums of a step start from zero and are added
        // to the running sums in plain float32 (the MMA truncates as it accumulates, and over a
        // long K that would drift).
        uint32_t sc[4][2];
        {
          uint4 sv = lds16(st + scale_off);
          // past K the codes are zeros, but the scale bytes are whatever was there
          if ((st0 + i) * kStepK + q * 64 >= A.K) sv = make_uint4(0u, 0u, 0u, 0u);
          const uint32_t sw[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            sc[j][0] = decode_scales(sw[j] & 0xFFFFu);
            sc[j][1] = decode_scales(sw[j] >> 16);
          }
        }
        float tmp[CH][2][NT][4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t w[4][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 v = lds16(st + row_off + j * (32 * 128) + piece[half]);
            w[j][0] = v.x;
            w[j][1] = v.y;
            w[j][2] = v.z;
            w[j][3] = v.w;
          }
#pragma unroll
          for (int wd = 0; wd < 4; ++wd) {
            uint4 b[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) b[n] = lds16(xb[n] + half * 256 + wd * 64);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              uint32_t a[2][4];
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                decode8(w[2 * p + r][wd], a[r]);
                // the scale of 16-element group 2 * half + wd / 2, in both halves
                const uint32_t sv =
                    __byte_perm(sc[2 * p + r][half], 0u, (wd & 2) ? 0x3232u : 0x1010u);
#pragma unroll
                for (int j = 0; j < 4; ++j) a[r][j] = mul_f16x2(a[r][j], sv);
              }
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                auto& t0 = tmp[0][p][n];
                auto& t1 = tmp[CH - 1][p][n];
                if (half == 0 && wd == 0) {
                  mma_f16_first(t0, a[0][0], a[1][0], a[0][1], a[1][1], b[n].x, b[n].y);
                  if constexpr (CH == 2)
                    mma_f16_first(t1, a[0][2], a[1][2], a[0][3], a[1][3], b[n].z, b[n].w);
                  else
                    mma_f16(t1, a[0][2], a[1][2], a[0][3], a[1][3], b[n].z, b[n].w);
                } else {
                  mma_f16(t0, a[0][0], a[1][0], a[0][1], a[1][1], b[n].x, b[n].y);
                  mma_f16(t1, a[0][2], a[1][2], a[0][3], a[1][3], b[n].z, b[n].w);
                }
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bar_empty[s]));
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              acc[p][n][j] += tmp[0][p][n][j];
              if (CH == 2) acc[p][n][j] += tmp[CH - 1][p][n][j];
            }
      }
    }

    // partial sums of the K warps (and of the cluster's CTAs) -> shared memory, added in order
    __syncthreads();
    float* red = reinterpret_cast<float*>(smem);  // [kKWarps][TOK][kRedStride]
    if (warp < kConsumers) {
      const int rg = warp % kRowWarps, wk = warp / kRowWarps;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int t = n * 8 + 2 * q + c;
          if (t >= ntok) continue;
          // undo the row's power of two and the one in the global scale, in two exact steps (the
          // rest of the global scale, in [1, 2), divides the total)
          const int up = -s_exp[t] - gs_exp;  // within [-253, 240]
          const float f0 = pow2f(up / 2), f1 = pow2f(up - up / 2);
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              red[(wk * TOK + t) * kRedStride + 8 * rg + g + 64 * p + 32 * r] =
                  acc[p][n][2 * r + c] * f0 * f1;
            }
        }
    }
    if (A.splits > 1) cluster_sync();
    else __syncthreads();
    auto total = [&](int row, int t) {
      const float* at = red + t * kRedStride + row;
      float v = 0.0f;
      if (A.splits > 1) {
        const uint32_t a = smem_u32(at);
        float part[kMaxSplits][kKWarps];
#pragma unroll
        for (int c = 0; c < kMaxSplits; ++c)
#pragma unroll
          for (int w = 0; w < kKWarps; ++w) {
            part[c][w] = 0.0f;
            if (c < A.splits)
              part[c][w] = ld_cluster_f32(mapa_shared(a + w * TOK * kRedStride * 4, c));
          }
#pragma unroll
        for (int c = 0; c < kMaxSplits; ++c)
#pragma unroll
          for (int w = 0; w < kKWarps; ++w) v += part[c][w];
      } else {
#pragma unroll
        for (int w = 0; w < kKWarps; ++w) v += at[w * TOK * kRedStride];
      }
      return v / gs_frac;
    };
    const int share = 128 / A.splits, r0 = share * split;
    if (!abort_flag) {
      if constexpr (MODE == FFN_L1) {
        // gate rows 32j + i, up rows 32j + 16 + i -> feature 16j + i
        const int feats = share / 2, I = A.N / 2;
        for (int idx = tid; idx < feats * ntok; idx += kThreads) {
          const int f = idx % feats, t = idx / feats;
          const int row = r0 + (f / 16) * 32 + f % 16;
          const float gate = total(row, t), up = total(row + 16, t);
          static_cast<float*>(A.out)[(int64_t)s_row[t] * I + (rowblk * 128 + r0) / 2 + f] =
              gate * up / (1.0f + expf(-gate));
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
    }
    // the peers have read this CTA's sums before it leaves, and its threads before the next
    // token block's copies overwrite them
    if (tb + 1 < tb_last) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    if (A.splits > 1) cluster_sync();
    else __syncthreads();
  }
  if (tid == 0 && abort_flag) report(A.status, NVFP4_DEVERR_TIMEOUT);
}

// out[t] = sum over the token's live slots of w * ys[slot], in slot order, FP32 -> bf16.  Lane j of
// a warp holds slot j's id and weight (k <= 32).
__global__ void __launch_bounds__(256) combine_slots_kernel(const float* ys, const int32_t* ids,
                                                            const float* w, int H, int E, int k,
                                                            __nv_bfloat16* out) {
  pdl_wait();
  const int t = blockIdx.x, lane = threadIdx.x & 31;
  int live = 0;
  float wl = 0.0f;
  if (lane < k) {
    const int id = ld_after(ids + t * k + lane);
    live = id >= 0 && id < E;
    if (live) wl = __int_as_float(ld_after(reinterpret_cast<const int32_t*>(w) + t * k + lane));
  }
  const uint32_t mask = __ballot_sync(0xffffffffu, live);
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * 4;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int kAhead = 8;  // slots whose loads are in flight together
  for (int j0 = 0; j0 < k; j0 += kAhead) {
    uint4 y[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (j0 + j < k && c < H && ((mask >> (j0 + j)) & 1u))
        y[j] = ld_after16(ys + ((int64_t)t * k + j0 + j) * H + c);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const float wj = __shfl_sync(0xffffffffu, wl, (j0 + j) & 31);
      if (j0 + j < k && c < H && ((mask >> (j0 + j)) & 1u)) {
        v[0] += wj * __uint_as_float(y[j].x);
        v[1] += wj * __uint_as_float(y[j].y);
        v[2] += wj * __uint_as_float(y[j].z);
        v[3] += wj * __uint_as_float(y[j].w);
      }
    }
  }
  if (c >= H) return;
  __nv_bfloat162 o[2] = {__floats2bfloat162_rn(v[0], v[1]), __floats2bfloat162_rn(v[2], v[3])};
  *reinterpret_cast<uint2*>(out + (int64_t)t * H + c) = *reinterpret_cast<const uint2*>(o);
}

// ------------------------------------------------------------------------------ host side

// The SM count the K splits are sized for (on another device they are only less well chosen).
constexpr int kSizingSms = 148;

// CTAs along K for one output block: enough CTAs for every SM, while each K warp keeps
// at least one step.
int pick_splits(int64_t blocks, int K, int most) {
  const int steps = (K + kStepK - 1) / kStepK;
  int s = 1;
  while (s < most && blocks * s < kSizingSms && steps / (2 * s) >= kKWarps) s *= 2;
  return s;
}

template <typename... P, typename... V>
nvfp4_status_t launch_after(void (*fn)(P...), dim3 grid, int threads, size_t smem, int cluster,
                            bool early, cudaStream_t s, const char* what, const V&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  int n = 0;
  if (early) {  // behind a kernel of this call: start while that one still runs
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = static_cast<unsigned>(cluster);
    at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = at;
  cfg.numAttrs = static_cast<unsigned>(n);
  cudaLaunchKernelEx(&cfg, fn, P(args)...);
  return check_launch(what);
}

template <int NT, Mode MODE, bool XIN>
nvfp4_status_t launch(const CUtensorMap& tm, const Args& a, dim3 grid, bool early,
                      cudaStream_t s) {
  auto* fn = w4a16_kernel<NT, MODE, XIN>;
  constexpr int smem = Cfg<NT, XIN>::SMEM;
  // the attribute is set once per device (a call costs about as much as a launch)
  static std::atomic<uint64_t> devices_set{0};
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(devices_set.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return check_launch("w4a16_kernel attributes");
    devices_set.fetch_or(bit, std::memory_order_release);
  }
  return launch_after(fn, grid, kThreads, smem, a.splits, early, s, "w4a16_kernel", tm, a);
}

bool weight_map(CUtensorMap* tm, const uint8_t* codes, int64_t rows, int K) {
  if (byte_tensor_map(tm, codes, static_cast<uint64_t>(K / 2), static_cast<uint64_t>(rows)))
    return true;
  set_last_error("cuTensorMapEncodeTiled failed");
  return false;
}

// The product kernel over weights `codes` of `rows` rows, behind the kernel of this call that
// converts its activations.
template <Mode MODE>
nvfp4_status_t launch_nt(int nt, const uint8_t* codes, int64_t rows, const Args& a, dim3 grid,
                         cudaStream_t s) {
  CUtensorMap tm;
  if (!weight_map(&tm, codes, rows, a.K)) return NVFP4_ERR_CUDA;
  switch (nt) {
    case 1: return launch<1, MODE, false>(tm, a, grid, true, s);
    case 2: return launch<2, MODE, false>(tm, a, grid, true, s);
    default: return launch<4, MODE, false>(tm, a, grid, true, s);
  }
}

int64_t converted_bytes(int64_t rows, int K) {
  return rows * ((K + kStepK - 1) / kStepK) * kStepX;
}

// How nvfp4_linear_w4a16 runs a shape, and the byte offsets of its workspace regions (256-byte
// aligned; none when the CTAs convert the activations themselves).
struct LinearW4Plan {
  int nt, splits;
  int64_t rowblks, tblks;
  bool xin;
  int64_t exps, total;
};

LinearW4Plan linear_w4_plan(int64_t M, int N, int K) {
  LinearW4Plan P{};
  P.nt = M <= 8 ? 1 : M <= 16 ? 2 : 4;
  P.rowblks = ((int64_t)N + 127) / 128;
  P.tblks = (M + 8 * P.nt - 1) / (8 * P.nt);
  P.splits = pick_splits(P.rowblks * P.tblks, K, kMaxSplits);
  const int steps = (K + kStepK - 1) / kStepK;
  P.xin = P.nt == 1 && M * ((steps + P.splits - 1) / P.splits) <= kMaxPieces;
  if (!P.xin) {
    P.exps = round_up(converted_bytes(M, K), 256);
    P.total = P.exps + round_up(M * 4, 256);
  }
  return P;
}

// Byte offsets of the moe_ffn_w4a16 workspace regions (each 256-byte aligned).
struct FfnW4Layout {
  int64_t ids, w, plan, n_plan, order, xf, xexp, h, hf, hexp, ys, total;
};

FfnW4Layout ffn_w4_layout(int T, int H, int I, int E, int k) {
  FfnW4Layout L{};
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
  L.xf = take(converted_bytes(T, H));
  L.xexp = take((int64_t)T * 4);
  L.h = take(S * I * 4);
  L.hf = take(converted_bytes(S, I));
  L.hexp = take(S * 4);
  L.ys = take(S * H * 4);
  L.total = o;
  return L;
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" size_t nvfp4_linear_w4a16_workspace_size(int64_t M, int N, int K) {
  if (M <= 0 || N <= 0 || K <= 0) return 0;
  return static_cast<size_t>(linear_w4_plan(M, N, K).total);
}

extern "C" nvfp4_status_t nvfp4_linear_w4a16(const void* x, int64_t M, int K, int64_t ld,
                                             const uint8_t* w, const uint8_t* sfw,
                                             const float* gs_w, int N, void* out, int out_dtype,
                                             void* ws, size_t ws_bytes, int32_t* dev_status,
                                             nvfp4_stream_t stream) {
  if (M < 0 || N <= 0 || K <= 0 || ld < K || (out_dtype != 0 && out_dtype != 1))
    return NVFP4_ERR_INVALID_ARG;
  if (K % 64 || ld % 8 || M > (int64_t)65535 * 32 || N > INT32_MAX - 127)
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!w || !sfw || !gs_w) return NVFP4_ERR_INVALID_ARG;
  if (M > 0 && (!x || !out)) return NVFP4_ERR_INVALID_ARG;
  const LinearW4Plan P = linear_w4_plan(M, N, K);
  if (M > 0 && P.total > 0 && (ws == nullptr || (int64_t)ws_bytes < P.total))
    return NVFP4_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned16(x) || !aligned16(w) || !aligned16(sfw) || !aligned16(out) || !aligned16(ws) ||
      (reinterpret_cast<uintptr_t>(gs_w) & 3u) || (reinterpret_cast<uintptr_t>(dev_status) & 3u))
    return NVFP4_ERR_MISALIGNED;
  if (M == 0) return NVFP4_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(ws);
  Args a{};
  a.sf = sfw;
  a.gs = gs_w;
  a.N = N;
  a.K = K;
  a.x = x;
  a.ld_bytes = ld * 2;
  a.M = static_cast<int>(M);
  a.out = out;
  a.out_f32 = out_dtype == 0;
  a.splits = P.splits;
  a.status = dev_status;
  const dim3 grid(static_cast<unsigned>(P.rowblks * P.splits), static_cast<unsigned>(P.tblks));
  if (P.xin) {
    CUtensorMap tm;
    if (!weight_map(&tm, w, N, K)) return NVFP4_ERR_CUDA;
    return launch<1, DENSE, true>(tm, a, grid, false, s);
  }
  a.xf = base;
  a.exps = reinterpret_cast<const int32_t*>(base + P.exps);
  convert_kernel<false><<<static_cast<unsigned>(M), 256, 0, s>>>(
      x, ld * 2, K, base, reinterpret_cast<int32_t*>(base + P.exps));
  const nvfp4_status_t st = check_launch("convert_kernel");
  if (st != NVFP4_OK) return st;
  return launch_nt<DENSE>(P.nt, w, N, a, grid, s);
}

extern "C" size_t moe_ffn_w4a16_workspace_size(int T, int H, int I, int E, int k) {
  if (T < 0 || H <= 0 || I <= 0 || E <= 0 || k <= 0) return 0;
  return static_cast<size_t>(ffn_w4_layout(T, H, I, E, k).total);
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
  if ((int64_t)E * (H > 2 * I ? H : 2 * (int64_t)I) > INT32_MAX) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return NVFP4_OK;
  if (!x_bf16 || !w1 || !sfw1 || !gs_w1 || !w2 || !sfw2 || !gs_w2 || !out_bf16 || !ws)
    return NVFP4_ERR_INVALID_ARG;
  if (logits == nullptr ? (!topk_ids || !topk_w) : (topk_ids || topk_w))
    return NVFP4_ERR_INVALID_ARG;  // logits, or a given routing: exactly one of them
  const FfnW4Layout L = ffn_w4_layout(T, H, I, E, k);
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
  auto i32 = [&](int64_t off) { return reinterpret_cast<int32_t*>(base + off); };
  auto f32 = [&](int64_t off) { return reinterpret_cast<float*>(base + off); };
  int32_t* ids = logits != nullptr ? i32(L.ids) : const_cast<int32_t*>(topk_ids);
  float* wts = logits != nullptr ? f32(L.w) : const_cast<float*>(topk_w);
  int4* plan = reinterpret_cast<int4*>(base + L.plan);
  plan_kernel<<<1 + T, 512, 0, s>>>(logits, T, E, k, ids, wts, plan, i32(L.n_plan), i32(L.order),
                                    x_bf16, H, base + L.xf, i32(L.xexp), dev_status);
  nvfp4_status_t st = check_launch("plan_kernel");
  if (st != NVFP4_OK) return st;
  const int S = T * k, busy = S < E ? S : E;
  // token tiles: twice what an expert gets on average
  const int per = 2 * S / E;
  const int nt = per <= 8 ? 1 : per <= 16 ? 2 : 4;
  Args a{};
  a.sf = sfw1;
  a.gs = gs_w1;
  a.N = 2 * I;
  a.K = H;
  a.xf = base + L.xf;
  a.exps = i32(L.xexp);
  a.k = k;
  a.plan = plan;
  a.n_plan = i32(L.n_plan);
  a.order = i32(L.order);
  a.out = f32(L.h);
  a.status = dev_status;
  const int blocks1 = 2 * I / 128;
  a.splits = pick_splits((int64_t)blocks1 * busy, H, 4);  // a CTA keeps 32 rows: gate and up
  st = launch_nt<FFN_L1>(nt, w1, (int64_t)E * 2 * I, a, dim3(blocks1 * a.splits, busy), s);
  if (st != NVFP4_OK) return st;
  st = launch_after(
      convert_kernel<true>, dim3(S), 256, 0, 1, true, s, "convert_kernel", f32(L.h), (int64_t)I * 4, I,
      base + L.hf, i32(L.hexp));
  if (st != NVFP4_OK) return st;
  a.sf = sfw2;
  a.gs = gs_w2;
  a.N = H;
  a.K = I;
  a.xf = base + L.hf;
  a.exps = i32(L.hexp);
  a.out = f32(L.ys);
  const int blocks2 = H / 128;
  a.splits = pick_splits((int64_t)blocks2 * busy, I, kMaxSplits);
  st = launch_nt<FFN_L2>(nt, w2, (int64_t)E * H, a, dim3(blocks2 * a.splits, busy), s);
  if (st != NVFP4_OK) return st;
  return launch_after(
      combine_slots_kernel, dim3(T, (H / 4 + 255) / 256), 256, 0, 1, true, s, "combine_slots_kernel",
      f32(L.ys), ids, wts, H, E, k, static_cast<__nv_bfloat16*>(out_bf16));
}
