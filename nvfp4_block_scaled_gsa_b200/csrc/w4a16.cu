// w4a16.cu — products of NVFP4 weights with unquantized activations, for few rows: the dense
// nvfp4_linear_w4a16 and the expert FFN moe_ffn_w4a16.
//
//   out[m][n] = (1/gs) * sum_k x[m][k] * E2M1(code[n][k]) * E4M3(sf[n][k/16])
//
// Bound by reading the weights once (9/16 byte per element): 1 x 151552 x 7168 runs at 5.6 to 6.0
// TB/s (86 to 92% of a copy's rate, with the SM clock), 16 tokens of 256 experts top-8 (H 7168, I
// 2048) in 375 us, 5.4 TB/s; small products by their chain of latencies (1 x 4096 x 7168: 7.3 us,
// against 2.5 at the copy's rate).
//
// TMA brings the weights to shared memory in the layout the block-scaled GEMMs store them in; a
// warp decodes its rows in registers and multiplies with mma.sync (m16n8k16, f16 in, float32
// accumulators), the weights being the 16-row operand and the tokens the 8 columns.  tcgen05 takes
// its operands from shared or tensor memory, so every decoded weight would have to be written back
// before the product; at a few tokens the product is far from the tensor cores' rate and the
// round trip would be the bound.  Per 8 weights of a lane: 4 conversions (2 cycles each on the ALU
// pipe), 4 multiplications by the scale, one MMA (8 cycles), 14 instructions in all; at the
// rate above half of the issue slots are used, and with one CTA per SM instead of two the same
// product runs at 3.3 TB/s.
//
// Exactness.  E2M1 * E4M3 has at most 6 significant bits and lies in [2^-10, 2688], so the
// decoded weight is exact in f16.  A row of activations is multiplied by the power of two that
// brings its largest finite magnitude into [2^14, 2^15): a bf16 value is then exact in f16 unless
// it is below 2^-31 of that maximum, where it is off by at most 2^-39 of the maximum (half an f16
// subnormal step is 2^-25; less than the float32 sum is off that the maximum takes part in).  The
// FFN's float32 intermediate is rounded to f16's 11 bits there, 1/8 of the step that the bf16 output
// is rounded to in the end (a second f16 term would double the MMAs, and they would be the bound).
// Infinities and NaNs pass through the conversion and the product as such.
//
// Layout.  A warp owns 16 or 32 rows of a 128-row block, of which a lane's (g = lane/4) are 32
// apart, and per step 256 elements of K, lane q = lane%4 the 64 elements from 64*q: 32 bytes of
// codes per row, and 4 bytes per row of one 16-byte line of a scale atom, which holds the scales of
// 4 rows 32 apart and 64 elements.  The order of K inside a step is free as long as both operands
// agree, so a lane's own 4 weights of a row are the 4 K positions the MMA wants from it, and the
// converted activations are stored in that order.
#include <cuda_fp16.h>

#include <atomic>

#include "common.cuh"
#include "launch.h"
#include "topk.cuh"

namespace nvfp4 {
namespace {

constexpr int kConsumers = 8;              // warps that multiply
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

// How the 8 warps share a step's 128 rows.  With one token tile (NT = 1) a warp owns 32 rows and two
// warps take the steps in turn: few instructions per weight go to waiting and to the activations
// (16 tokens of 256 experts: 374 us, against 415 with 16 rows a warp).  With two tiles the MMAs
// weigh more and a warp owns 16 rows of every step, which frees the stages sooner and halves the
// accumulators (16 x 65536 x 4096: 47 us, against 54).
template <int NT>
struct Warps {
  static constexpr int KW = NT == 1 ? 2 : 1;  // warps that share rows, taking steps in turn
  static constexpr int P = KW;                // 16-row tiles of a warp
};

template <int NT, bool XIN>
struct Cfg {
  static constexpr int TOK = 8 * NT;  // token columns
  static constexpr int KW = Warps<NT>::KW;
  static constexpr int STAGE = kWTile + kSTile + (XIN ? 0 : (TOK * kXRow + 1023) / 1024 * 1024);
  static constexpr int STAGES = 4;
  static constexpr int X_AT = STAGES * STAGE;  // XIN: the activations behind the stages
  static constexpr int SMEM = X_AT + (XIN ? kMaxPieces * kXRow : 0) + 1024;
  static_assert(KW * TOK * kRedStride * 4 <= STAGES * STAGE, "partial sums reuse the stages");
  static_assert(STAGES % KW == 0, "a stage is always the same warps', or one could wait two phases ahead");
  // two CTAs per SM, so that one's start and end overlap the other's stream (beside the static
  // shared memory, the system takes 1 KB of each)
  static_assert(2 * (SMEM + 2560) <= 228 * 1024, "shared memory of an SM");
};

// A weight tensor and the converted activations it is multiplied with.
struct Operands {
  const uint8_t* sf;      // per expert round_up(N, 128) rows of tiled scales
  const float* gs;        // [E]
  int N, K;
  // FFN: [rows][steps][kStepX bytes], gathered row by row.  Dense: [blocks of 8 * NT rows][steps]
  // [rows][kXRow bytes], so that one copy brings a step of all of a block's rows (16 x 4096 x
  // 7168: 12.4 us with a copy per row).
  const uint8_t* xf;
  const int32_t* exps;    // [rows] the power of two each row was multiplied by
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

// float32 bits of the largest finite magnitude of some values
template <int N>
__device__ __forceinline__ uint32_t amax_of(const float (&v)[N]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
    if (b < 0x7F800000u) m = max(m, b);
  }
  return m;
}
// the values times f, as f16, to `d`
template <int N>
__device__ __forceinline__ void put_f16(uint8_t* d, const float (&v)[N], float f) {
  uint32_t h[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const __half2 p = __floats2half2_rn(v[2 * i] * f, v[2 * i + 1] * f);
    h[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  if constexpr (N == 8) *reinterpret_cast<uint4*>(d) = make_uint4(h[0], h[1], h[2], h[3]);
  else *reinterpret_cast<uint2*>(d) = make_uint2(h[0], h[1]);
}
__device__ __forceinline__ void bf16x8(const uint4& q, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// One CTA converts one row of K activations: the power of two, and the f16 values of every step of
// 256 in the order [word of 8][quad lane] (zeros past K).  load(p, v) gives elements N*p .. N*p +
// N-1, N = 4 or 8; steps are `step_bytes` apart.  `red` holds a word per warp.
template <int N, int kCache, typename Load>  // kCache: pieces a thread keeps between the two passes
__device__ __forceinline__ void convert_row(const Load& load, int K, uint8_t* out,
                                            int64_t step_bytes, int32_t* exp_out, uint32_t* red) {
  const int tid = threadIdx.x, nthr = blockDim.x;
  const int pieces = (K + kStepK - 1) / kStepK * (kStepK / N), live = K / N;
  float c[kCache][N];
  uint32_t m = 0;
  auto get = [&](int p, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.0f;
    if (p < live) load(p, v);
  };
#pragma unroll
  for (int j = 0; j < kCache; ++j) get(tid + j * nthr, c[j]);
#pragma unroll
  for (int j = 0; j < kCache; ++j) m = max(m, amax_of(c[j]));
  for (int p = tid + kCache * nthr; p < live; p += nthr) {
    float v[N];
    get(p, v);
    m = max(m, amax_of(v));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((tid & 31) == 0) red[tid >> 5] = m;
  __syncthreads();
  m = __reduce_max_sync(0xffffffffu, (tid & 31) < nthr / 32 ? red[tid & 31] : 0u);
  const int e = norm_exp(m);
  const float f = pow2f(e);
  if (tid == 0) *exp_out = e;
  // element k: step k / 256, quad lane (k % 256) / 64, word (k % 64) / 8
  auto put = [&](int p, const float (&v)[N]) {
    const int k = p * N;
    put_f16(out + (k >> 8) * step_bytes + (((k >> 3) & 7) * 4 + ((k >> 6) & 3)) * 16 + (k & 7) * 2,
            v, f);
  };
#pragma unroll
  for (int j = 0; j < kCache; ++j)
    if (tid + j * nthr < pieces) put(tid + j * nthr, c[j]);
  for (int p = tid + kCache * nthr; p < pieces; p += nthr) {
    float v[N];
    get(p, v);
    put(p, v);
  }
}
// ... of a bf16 row
__device__ __forceinline__ void convert_bf16_row(const void* row, int K, uint8_t* out,
                                                 int64_t step_bytes, int32_t* exp_out,
                                                 uint32_t* red) {
  convert_row<8, 4>([&](int p, float (&v)[8]) { bf16x8(__ldg(static_cast<const uint4*>(row) + p), v); },
                    K, out, step_bytes, exp_out, red);
}

// The dense form's activations, one row per CTA, in blocks of `tok` rows.
__global__ void __launch_bounds__(256) convert_kernel(const uint8_t* x, int64_t ld_bytes, int K,
                                                      int tok, uint8_t* xf, int32_t* exps) {
  __shared__ uint32_t red[32];
  pdl_trigger();
  const int64_t r = blockIdx.x, steps = (K + kStepK - 1) / kStepK;
  convert_bf16_row(x + r * ld_bytes, K, xf + (r / tok * steps * tok + r % tok) * kXRow,
                   (int64_t)tok * kXRow, exps + r, red);
}

// The first kernel of the FFN.  CTA 0 makes the plan: top-k (with logits), slots counted per
// expert, the experts cut into units of at most `tok` slots, and the slots in place, in ascending
// order within an expert (each warp ranks a contiguous part of them).  The other CTAs convert one
// token's activations each.
constexpr int kPlanThreads = 512;
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(
    const float* __restrict__ logits, int T, int E, int k, int tok, const int32_t* __restrict__ ids,
    float* w, int4* __restrict__ plan, int32_t* __restrict__ n_plan, int32_t* __restrict__ order,
    int32_t* __restrict__ slot_unit, const uint8_t* __restrict__ x, int H,
    uint8_t* __restrict__ xf, int32_t* __restrict__ exps, int32_t* __restrict__ dev_status) {
  constexpr int kWarps = kPlanThreads / 32;
  __shared__ int hist[kWarps][kMaxE];
  __shared__ int first_of[kMaxE], unit_of[kMaxE];
  __shared__ int s_ids[NVFP4_W4A16_MAX_SLOTS];
  __shared__ uint32_t red[32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  if (blockIdx.x > 0) {
    const int64_t r = blockIdx.x - 1, steps = (H + kStepK - 1) / kStepK;
    convert_bf16_row(x + r * H * 2, H, xf + r * steps * kStepX, kStepX, exps + r, red);
    return;
  }
  for (int i = tid; i < kWarps * kMaxE; i += kPlanThreads) (&hist[0][0])[i] = 0;
  const int S = T * k, per = (S + kWarps - 1) / kWarps;
  if (logits != nullptr)
    for (int t = warp; t < T; t += kWarps) topk_token(logits, t, E, k, 1, lane, s_ids, w);
  else
    for (int s = tid; s < S; s += kPlanThreads) s_ids[s] = __ldg(ids + s);
  __syncthreads();
  const int lo = min(S, warp * per), hi = min(S, lo + per);
  bool bad = false;
  for (int s = lo + lane; s < hi; s += 32) {
    const int e = s_ids[s];
    if (e >= E) bad = true;
    else if (e >= 0) atomicAdd(&hist[warp][e], 1);
  }
  if (bad) report(dev_status, NVFP4_DEVERR_BAD_INDEX);
  __syncthreads();
  if (tid < kMaxE) {  // per expert: each warp's first rank, and the count
    int run = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const int c = hist[i][tid];
      hist[i][tid] = run;
      run += c;
    }
    first_of[tid] = run;
  }
  __syncthreads();
  if (warp == 0) {  // lane l: experts 8l..8l+7
    int c[kPerLane], sum = 0, units = 0;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      c[i] = first_of[lane * kPerLane + i];
      sum += c[i];
      units += (c[i] + tok - 1) / tok;
    }
    int run = sum, at = units;
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
    at -= units;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int e = lane * kPerLane + i;
      first_of[e] = run;
      unit_of[e] = at;
      for (int j = 0; j < c[i]; j += tok)
        plan[at++] = make_int4(e, run + j, min(tok, c[i] - j), 0);
      run += c[i];
    }
  }
  __syncthreads();
  for (int base = lo; base < hi; base += 32) {
    const int s = base + lane;
    int e = s < hi ? s_ids[s] : -1;
    if (e >= E) e = -1;
    const unsigned peers = __match_any_sync(0xffffffffu, e);
    const int before = __popc(peers & ((1u << lane) - 1u));
    if (e >= 0) {
      const int rank = hist[warp][e] + before;
      order[first_of[e] + rank] = s;
      slot_unit[s] = unit_of[e] + rank / tok;
    } else if (s < hi) {
      slot_unit[s] = -1;
    }
    __syncwarp();
    if (e >= 0 && before == 0) hist[warp][e] += __popc(peers);
    __syncwarp();
  }
}

// ------------------------------------------------------------------------- the product

// What a lane reads of a stage, and the products of one step: 8 words of 8 codes per row, rows `line`
// + 64 * tile + {0, 32} of the 128.  The sums of a step start from zero and are added to the running
// sums in plain float32 (the MMA truncates as it accumulates, and over a long K that would drift).
template <int NT>
struct Lane {
  static constexpr int P = Warps<NT>::P, KW = Warps<NT>::KW;
  using Acc = float[P][NT][4];
  int line, tile0, wk, q;  // wk: which of the KW warps of these rows this is
  int code_off, piece[2], scale_off;
  __device__ __forceinline__ Lane(int warp, int lane) {
    const int g = lane >> 2, high = warp >> 2;
    line = 8 * (warp & 3) + g;
    tile0 = KW == 1 ? high : 0;
    wk = KW == 1 ? 0 : high;
    q = lane & 3;
    // two 16-byte pieces of a row's 128 bytes (128-byte swizzle: the piece index is xored with the
    // row's index modulo 8, which is g for all of the lane's rows)
    code_off = (line + 64 * tile0) * 128;
    piece[0] = ((2 * q) ^ g) * 16;
    piece[1] = ((2 * q + 1) ^ g) * 16;
    scale_off = kWTile + q * 512 + line * 16 + 8 * tile0;
  }
  __device__ __forceinline__ int row(int p, int r) const { return line + 64 * (tile0 + p) + 32 * r; }
  // left: elements of K from the step's first one on (the last step may hold fewer than 256)
  __device__ __forceinline__ void step(const uint8_t* st, const uint8_t* const (&xb)[NT], int left,
                                       Acc& acc) const {
    // two accumulators where a warp has few, so that consecutive MMAs do not wait for one another
    constexpr int CH = P * NT == 4 ? 1 : 2;
    uint32_t sc[2 * P][2];
    {
      uint4 sv;
      if constexpr (P == 2) {
        sv = lds16(st + scale_off);
      } else {
        const uint2 two = *reinterpret_cast<const uint2*>(st + scale_off);
        sv = make_uint4(two.x, two.y, 0u, 0u);
      }
      // past K the codes are zeros, but the scale bytes are whatever was there
      if (q * 64 >= left) sv = make_uint4(0u, 0u, 0u, 0u);
      const uint32_t sw[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
      for (int j = 0; j < 2 * P; ++j) {
        sc[j][0] = decode_scales(sw[j] & 0xFFFFu);
        sc[j][1] = decode_scales(sw[j] >> 16);
      }
    }
    float tmp[CH][P][NT][4];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t w[2 * P][4];
#pragma unroll
      for (int j = 0; j < 2 * P; ++j) {
        const uint4 v = lds16(st + code_off + j * (32 * 128) + piece[half]);
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
        for (int p = 0; p < P; ++p) {
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
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[p][n][j] += tmp[0][p][n][j];
          if (CH == 2) acc[p][n][j] += tmp[CH - 1][p][n][j];
        }
  }
  static __device__ __forceinline__ void clear(Acc& acc) {
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[p][n][j] = 0.0f;
  }
};

// The global scale (a positive normal number) as 2^exp * frac, and a sum times 2^-row_exp / 2^exp in
// two exact steps; dividing by frac is left.
struct GlobalScale {
  int exp;
  float frac;
  __device__ __forceinline__ explicit GlobalScale(float gs) {
    const uint32_t b = __float_as_uint(gs);
    exp = static_cast<int>(b >> 23) - 127;
    frac = __uint_as_float((b & 0x7FFFFFu) | 0x3F800000u);
  }
  __device__ __forceinline__ void factors(int row_exp, float& f0, float& f1) const {
    const int up = -row_exp - exp;  // within [-253, 240]
    f0 = pow2f(up / 2);
    f1 = pow2f(up - up / 2);
  }
};

// The stage ring: the barriers, and the copies of a step's codes and scales.
template <int STAGES, int KW>
struct Ring {
  uint64_t *full, *empty;
  volatile int* abort_flag;
  __device__ __forceinline__ void init() const {  // by one thread
    *abort_flag = 0;
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), kConsumers / KW);
    }
    fence_mbar_init();
  }
  // whole-warp waits: every lane gets the same answer
  __device__ __forceinline__ bool wait_empty(uint32_t it) const {
    const bool mine =
        mbar_wait_bounded(smem_u32(&empty[it % STAGES]), ((it / STAGES) & 1u) ^ 1u, abort_flag);
    return __all_sync(0xffffffffu, mine) != 0;
  }
  __device__ __forceinline__ bool wait_full(uint32_t it) const {
    const bool mine =
        mbar_wait_bounded(smem_u32(&full[it % STAGES]), (it / STAGES) & 1u, abort_flag);
    return __all_sync(0xffffffffu, mine) != 0;
  }
  __device__ __forceinline__ void release(uint32_t it) const {  // by a warp of the step
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&empty[it % STAGES]));
  }
  // by the copying warp: step st of the 128 rows from `row` on, whose scale atoms start at `sf`;
  // x_bytes of activations follow
  __device__ __forceinline__ void copy_w(uint32_t it, uint8_t* stage, const CUtensorMap* tm, int row,
                                         const uint8_t* sf, int st, int atoms_k, int x_bytes) const {
    if ((threadIdx.x & 31) == 0) {
      const int atoms = min(4, atoms_k - st * 4);
      const uint32_t bar = smem_u32(&full[it % STAGES]), d = smem_u32(stage);
      mbar_arrive_expect_tx(bar, kWTile + atoms * 512 + x_bytes);
      tma_load_2d(d, tm, bar, st * 128, row);
      bulk_load(d + kWTile, sf + (int64_t)st * 4 * 512, atoms * 512, bar);
    }
    __syncwarp();
  }
  // activations of a step: `bytes` to byte `at` of the stage's activations, by one lane
  __device__ __forceinline__ void copy_x(uint32_t it, uint8_t* stage, int at, const uint8_t* x,
                                         int bytes) const {
    bulk_load(smem_u32(stage) + kWTile + kSTile + at, x, bytes, smem_u32(&full[it % STAGES]));
  }
  // By the copying warp behind its last copy: lets the copies already issued land before the stages
  // are used otherwise or the CTA can exit.  Always, since a wait of the other warps may run out when
  // this one has nothing left to wait for (otherwise they have waited for the same copies).
  __device__ __forceinline__ void drain(uint32_t issued) const {
    volatile int never = 0;
    for (uint32_t i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i)
      if (!mbar_wait_bounded(smem_u32(&full[i % STAGES]), (i / STAGES) & 1u, &never,
                             NVFP4_WAIT_TIMEOUT_NS / 4))
        *abort_flag = 1;
  }
};

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  return p + ((1024u - (smem_u32(p) & 1023u)) & 1023u);
}
__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kConsumers) : "memory");
}

// --------------------------------------------------------------- dense, one output block a cluster

struct DenseArgs {
  const void* x;  // XIN: bf16 activations, rows of ld_bytes
  int64_t ld_bytes;
  int M;
  void* out;  // [M][N]
  int out_f32;
  int splits;  // CTAs of a cluster that share an output block along K
  int32_t* status;
};

// For few output blocks: 128 rows of the weight and up to 8 * NT rows of x per cluster, K cut among
// its CTAs, whose sums are joined through distributed shared memory.  XIN: the CTA converts the
// activations of its rows and its part of K itself, when they are few; otherwise a kernel in
// front has converted them and they pass through the ring with the weights.
template <int NT, bool XIN>
__global__ void __launch_bounds__(kThreads, 2)
    dense_kernel(const __grid_constant__ CUtensorMap tm, const Operands W, const DenseArgs A) {
  using C = Cfg<NT, XIN>;
  constexpr int TOK = C::TOK, STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  __shared__ __align__(8) uint64_t bar_full[STAGES], bar_empty[STAGES];
  __shared__ volatile int abort_flag;
  __shared__ __align__(16) uint8_t zeros[kStepX];  // what columns without a token read
  __shared__ int s_exp[TOK];                       // power of two of each column
  __shared__ uint32_t s_amax[TOK];                 // XIN
  const Ring<STAGES, C::KW> ring{bar_full, bar_empty, &abort_flag};
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, q = lane & 3;
  const int split = static_cast<int>(blockIdx.x) % A.splits;
  const int rowblk = static_cast<int>(blockIdx.x) / A.splits;
  const int m0 = static_cast<int>(blockIdx.y) * TOK, ntok = min(TOK, A.M - m0);
  if (tid == 0) ring.init();
  if (tid < kStepX / 16) reinterpret_cast<uint4*>(zeros)[tid] = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
  const int atoms_k = W.K / 64, nsteps = (W.K + kStepK - 1) / kStepK;
  const int st0 = static_cast<int>((int64_t)nsteps * split / A.splits);
  const int n_st = static_cast<int>((int64_t)nsteps * (split + 1) / A.splits) - st0;
  const GlobalScale gs(__ldg(W.gs));
  const Lane<NT> me(warp & 7, lane);
  typename Lane<NT>::Acc acc;
  me.clear(acc);
  if (warp == kConsumers) {
    const uint8_t* sf = W.sf + (int64_t)rowblk * atoms_k * 512;
    auto stage = [&](int i) { return smem + (i % STAGES) * C::STAGE; };
    auto copy_w = [&](int i) {
      ring.copy_w(i, stage(i), &tm, rowblk * 128, sf, st0 + i, atoms_k, XIN ? 0 : ntok * kXRow);
    };
    const uint8_t* xr = W.xf + ((int64_t)blockIdx.y * nsteps + st0) * (TOK * kXRow);
    auto copy_x = [&](int i) {
      if (!XIN && lane == 0)
        ring.copy_x(i, stage(i), 0, xr + (int64_t)i * (TOK * kXRow), ntok * kXRow);
    };
    bool ok = true;
    int issued = 0;
    for (; issued < min(n_st, STAGES); ++issued) copy_w(issued);  // while x is converted
    pdl_wait();
    for (int i = 0; i < issued; ++i) copy_x(i);
    for (; issued < n_st && ok; ++issued) {
      ok = ring.wait_empty(issued);
      if (!ok) break;
      copy_w(issued);
      copy_x(issued);
    }
    ring.drain(issued);
  } else {
    if constexpr (XIN) {
      // pieces (token, step) warp and warp + kConsumers: lane l holds elements 8l .. 8l + 7
      const int pieces = ntok * n_st;
      constexpr int kMine = kMaxPieces / kConsumers;
      float c[kMine][8];
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        const int p = warp + j * kConsumers, k = (st0 + p % n_st) * kStepK + lane * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) c[j][i] = 0.0f;
        if (p < pieces && k < W.K)
          bf16x8(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(A.x) +
                                                      (int64_t)(m0 + p / n_st) * A.ld_bytes + k * 2)),
                 c[j]);
      }
      if (tid < TOK) s_amax[tid] = 0;
      consumers_sync();
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        const int p = warp + j * kConsumers;
        if (p < pieces) {
          const uint32_t m = __reduce_max_sync(0xffffffffu, amax_of(c[j]));
          if (lane == 0) atomicMax(&s_amax[p / n_st], m);
        }
      }
      consumers_sync();
      if (tid < TOK) s_exp[tid] = norm_exp(s_amax[tid]);
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        const int p = warp + j * kConsumers;
        if (p < pieces)
          put_f16(smem + C::X_AT + p * kXRow + ((lane & 7) * 4 + (lane >> 3)) * 16, c[j],
                  pow2f(norm_exp(s_amax[p / n_st])));
      }
      consumers_sync();
    } else if (tid < ntok) {
      pdl_wait();
      s_exp[tid] = ld_after(W.exps + m0 + tid);
    }
    for (int i = me.wk; i < n_st; i += C::KW) {
      if (!ring.wait_full(i)) break;
      const uint8_t* st = smem + (i % STAGES) * C::STAGE;
      const uint8_t* xb[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n)
        xb[n] = (n * 8 + g >= ntok ? zeros
                 : XIN ? smem + C::X_AT + ((n * 8 + g) * n_st + i) * kXRow
                       : st + kWTile + kSTile + (n * 8 + g) * kXRow) +
                q * 16;
      me.step(st, xb, W.K - (st0 + i) * kStepK, acc);
      ring.release(i);
    }
  }

  // partial sums of the warps and of the cluster's CTAs -> shared memory, added in order
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);  // [KW][TOK][kRedStride]
  const bool lost = abort_flag != 0;  // a wait ran out: NaNs, which the cluster's other CTAs pass on
  if (warp < kConsumers) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int t = n * 8 + 2 * q + c;
        if (t >= ntok) continue;
        float f0, f1;
        gs.factors(s_exp[t], f0, f1);
        if (lost) f0 = __int_as_float(0x7FC00000);
#pragma unroll
        for (int p = 0; p < me.P; ++p)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            red[(me.wk * TOK + t) * kRedStride + me.row(p, r)] = acc[p][n][2 * r + c] * f0 * f1;
      }
  }
  if (A.splits > 1) cluster_sync();
  else __syncthreads();
  const int share = 128 / A.splits, r0 = share * split;
  if (!lost) {
    for (int idx = tid; idx < share * ntok; idx += kThreads) {
      const int row = r0 + idx % share, t = idx / share, n = rowblk * 128 + row;
      const float* at = red + t * kRedStride + row;
      float v = 0.0f;
      if (A.splits > 1) {
        const uint32_t a = smem_u32(at);
        float part[kMaxSplits][C::KW];
#pragma unroll
        for (int c = 0; c < kMaxSplits; ++c)
#pragma unroll
          for (int w = 0; w < C::KW; ++w) {
            part[c][w] = 0.0f;
            if (c < A.splits)
              part[c][w] = ld_cluster_f32(mapa_shared(a + w * TOK * kRedStride * 4, c));
          }
#pragma unroll
        for (int c = 0; c < kMaxSplits; ++c)
#pragma unroll
          for (int w = 0; w < C::KW; ++w) v += part[c][w];
      } else {
#pragma unroll
        for (int w = 0; w < C::KW; ++w) v += at[w * TOK * kRedStride];
      }
      v /= gs.frac;
      if (n < W.N) {
        const int64_t o = (int64_t)(m0 + t) * W.N + n;
        if (A.out_f32) static_cast<float*>(A.out)[o] = v;
        else static_cast<__nv_bfloat16*>(A.out)[o] = __float2bfloat16_rn(v);
      }
    }
  }
  if (A.splits > 1) cluster_sync();  // the peers have read this CTA's sums
  if (tid == 0 && lost) report(A.status, NVFP4_DEVERR_TIMEOUT);
}

// ------------------------------------------------------------------------ streamed, in even shares

// For many output blocks: the blocks (a unit of up to 8 * NT tokens against 128 weight rows) follow
// one another, each ceil(K / 256) steps long, and every CTA takes the same number of consecutive
// steps, wherever its share starts and ends.  A CTA's copies run on across blocks.  What a warp
// sums of a block goes to a plane of its own: `part` holds [row][planes][blocks * 128], plane
// KW * piece + wk, a block's pieces counted from the CTA that starts it.  The kernel behind adds
// a block's planes in order.
enum Mode { DENSE = 0, FFN_L1 = 1, FFN_L2 = 2 };
constexpr int kStreamCtas = 2 * 148;  // two per SM, all resident at once

struct Split {
  int blocks;   // of 128 weight rows
  int steps;    // of a block
  int planes;   // of a row, at most
  int kw;       // of them per piece
  int least;    // steps of a CTA
  int units;    // DENSE; the FFN's are counted on the device
  // (the host sees to it that the steps of all blocks fit 31 bits)
  __host__ __device__ int per_cta(int n_units) const {
    const int total = n_units * blocks * steps;
    const int per = static_cast<int>((static_cast<unsigned>(total) + kStreamCtas - 1) / kStreamCtas);
    return per > least ? per : least;
  }
};
// planes that hold something of block b
__device__ __forceinline__ int block_planes(const Split& S, int per, int b) {
  return S.kw * (((b + 1) * S.steps - 1) / per - b * S.steps / per + 1);
}

struct StreamArgs {
  Split split;
  int M;                  // DENSE: rows of x
  int k;                  // FFN: slots per token
  const int4* plan;       // FFN: {expert, first, count, 0} per unit
  const int32_t* n_plan;  // and how many there are
  const int32_t* order;   // slots sorted by expert
  float* part;
  int32_t* status;
};

template <int NT, Mode MODE>
__global__ void __launch_bounds__(kThreads, 2)
    stream_kernel(const __grid_constant__ CUtensorMap tm, const Operands W, const StreamArgs A) {
  using C = Cfg<NT, false>;
  constexpr int TOK = C::TOK, STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  __shared__ __align__(8) uint64_t bar_full[STAGES], bar_empty[STAGES];
  __shared__ volatile int abort_flag;
  __shared__ __align__(16) uint8_t zeros[kStepX];  // what columns without a token read
  const Ring<STAGES, C::KW> ring{bar_full, bar_empty, &abort_flag};
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, q = lane & 3;
  if (tid == 0) ring.init();
  if (tid < kStepX / 16) reinterpret_cast<uint4*>(zeros)[tid] = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
  // The L2 form's plan is older than the kernel it waits for (the one that makes the
  // intermediate, behind the L1, which started after the plan was complete), so it is read before
  // that wait and the first weights are on their way during it.
  if constexpr (MODE == FFN_L1) pdl_wait();
  const Split& S = A.split;
  const int units = MODE == DENSE ? S.units : ld_after(A.n_plan);
  pdl_trigger();
  const int total = units * S.blocks * S.steps, per = S.per_cta(units);
  const int lo = static_cast<int>(min((int64_t)total, (int64_t)per * blockIdx.x));
  const int hi = static_cast<int>(min((int64_t)total, (int64_t)lo + per)), n = hi - lo;
  if (n == 0) {
    pdl_wait();  // no kernel of the chain ends before the ones in front of it
    return;
  }
  const int atoms_k = W.K / 64;

  // a block's unit and weight rows: the dense form goes through the units of one weight block, the
  // FFN through the weight blocks of one unit
  struct Block {
    int rowblk, e, first, count;
  };
  auto block = [&](int b) {
    Block k;
    if constexpr (MODE == DENSE) {
      k.rowblk = b / units;
      k.e = 0;
      k.first = b % units * TOK;
      k.count = min(TOK, A.M - k.first);
    } else {
      k.rowblk = b % S.blocks;
      const uint4 p = ld_after16(A.plan + b / S.blocks);
      k.e = static_cast<int>(p.x);
      k.first = static_cast<int>(p.y);
      k.count = static_cast<int>(p.z);
    }
    return k;
  };
  auto out_row = [&](const Block& k, int t) {  // DENSE: the row of x; FFN: the slot
    return MODE == DENSE ? k.first + t : ld_after(A.order + k.first + t);
  };
  auto x_row = [&](int r) { return MODE == FFN_L1 ? r / A.k : r; };

  if (warp == kConsumers) {
    // =========================== copies ===========================
    auto stage = [&](int i) { return smem + (i % STAGES) * C::STAGE; };
    struct Cursor {
      int b, st;
      Block k;
      const uint8_t *sf, *x;
    };
    auto enter = [&](Cursor& c, bool with_x) {
      c.k = block(c.b);
      c.sf = W.sf + ((int64_t)c.k.e * S.blocks + c.k.rowblk) * atoms_k * 512;
      if (MODE == DENSE) c.x = W.xf + (int64_t)c.k.first * S.steps * kXRow;
      else if (with_x && lane < c.k.count)
        c.x = W.xf + (int64_t)x_row(out_row(c.k, lane)) * S.steps * kStepX;
    };
    auto advance = [&](Cursor& c, bool with_x) {
      if (++c.st == S.steps) {
        c.st = 0;
        if (++c.b * S.steps < hi) enter(c, with_x);
      }
    };
    auto copy_w = [&](int i, const Cursor& c) {
      ring.copy_w(i, stage(i), &tm, c.k.e * W.N + c.k.rowblk * 128, c.sf, c.st, atoms_k,
                  c.k.count * (MODE == DENSE ? kXRow : kStepX));
    };
    auto copy_x = [&](int i, const Cursor& c) {  // DENSE: all rows at once; FFN: lane t's token t
      if constexpr (MODE == DENSE) {
        if (lane == 0)
          ring.copy_x(i, stage(i), 0, c.x + (int64_t)c.st * (TOK * kXRow), c.k.count * kXRow);
      } else if (lane < c.k.count) {
        ring.copy_x(i, stage(i), lane * kXRow, c.x + (int64_t)c.st * kStepX, kStepX);
      }
    };
    Cursor c{lo / S.steps, lo % S.steps, {}, nullptr, nullptr};
    Cursor early = c;
    enter(early, false);
    const int head = min(n, STAGES);
    // while the activations are being made (bringing more than the ring holds into L2 meanwhile
    // made one token's FFN slower: 56 us with 8 steps a CTA against 53.5)
    for (int i = 0; i < head; ++i) {
      copy_w(i, early);
      advance(early, false);
    }
    pdl_wait();
    enter(c, true);
    bool ok = true;
    int i = 0;
    for (; i < n; ++i) {
      if (i >= head) {
        ok = ring.wait_empty(i);
        if (!ok) break;
        copy_w(i, c);
      }
      copy_x(i, c);
      advance(c, true);
    }
    ring.drain(i);
  } else {
    // =========================== products ===========================
    const Lane<NT> me(warp, lane);
    const int64_t n_pad = (int64_t)S.blocks * 128;
    pdl_wait();
    bool ok = true;
    for (int it = 0; it < n && ok;) {
      const int b = (lo + it) / S.steps, s0 = (lo + it) % S.steps, len = min(S.steps - s0, n - it);
      const Block k = block(b);
      const float gs_value = __ldg(W.gs + k.e);
      // this lane's two columns of every token tile
      int row[NT][2], row_exp[NT][2];
#pragma unroll
      for (int t8 = 0; t8 < NT; ++t8)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int t = t8 * 8 + 2 * q + c;
          row[t8][c] = t < k.count ? out_row(k, t) : -1;
          row_exp[t8][c] = row[t8][c] >= 0 ? ld_after(W.exps + x_row(row[t8][c])) : 0;
        }
      typename Lane<NT>::Acc acc;
      me.clear(acc);
      // the stages it + i with (it + i) % KW == wk
      for (int i = (it + me.wk) & (C::KW - 1); i < len; i += C::KW) {
        if (!ring.wait_full(it + i)) {
          ok = false;
          break;
        }
        const uint8_t* st = smem + ((it + i) % STAGES) * C::STAGE;
        const uint8_t* xb[NT];
#pragma unroll
        for (int t8 = 0; t8 < NT; ++t8)
          xb[t8] = (t8 * 8 + g < k.count ? st + kWTile + kSTile + (t8 * 8 + g) * kXRow : zeros) + q * 16;
        me.step(st, xb, W.K - (s0 + i) * kStepK, acc);
        ring.release(it + i);
      }
      it += len;
      const GlobalScale gs(gs_value);
      const int plane = (static_cast<int>(blockIdx.x) - b * S.steps / per) * C::KW + me.wk;
#pragma unroll
      for (int t8 = 0; t8 < NT; ++t8)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (row[t8][c] < 0) continue;
          float f0, f1;
          gs.factors(row_exp[t8][c], f0, f1);
          float* d = A.part + ((int64_t)row[t8][c] * S.planes + plane) * n_pad + k.rowblk * 128;
#pragma unroll
          for (int p = 0; p < me.P; ++p)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              d[me.row(p, r)] = acc[p][t8][2 * r + c] * f0 * f1 / gs.frac;
        }
    }
  }
  __syncthreads();
  if (tid == 0 && abort_flag) report(A.status, NVFP4_DEVERR_TIMEOUT);
}

// Sums over a block's planes, in order, of V groups of 4 consecutive columns; the loads of 8 planes
// are in flight together.
template <int V>
__device__ __forceinline__ void sum_planes(const float* base, const int (&at)[V], int64_t n_pad,
                                           int planes, float (&v)[V][4]) {
  constexpr int kAhead = 8;
#pragma unroll
  for (int g = 0; g < V; ++g)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[g][i] = 0.0f;
  for (int a = 0; a < planes; a += kAhead) {
    uint4 q[kAhead][V];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int g = 0; g < V; ++g)
        if (a + j < planes) q[j][g] = ld_after16(base + (a + j) * n_pad + at[g]);
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int g = 0; g < V; ++g)
        if (a + j < planes) {
          v[g][0] += __uint_as_float(q[j][g].x);
          v[g][1] += __uint_as_float(q[j][g].y);
          v[g][2] += __uint_as_float(q[j][g].z);
          v[g][3] += __uint_as_float(q[j][g].w);
        }
  }
}

// The dense form's output from its planes: 4 columns of a row of x per thread.
__global__ void __launch_bounds__(128) dense_sum_kernel(const float* part, const Split S, int tok,
                                                        int N, void* out, int out_f32) {
  pdl_wait();
  const int m = blockIdx.y, c = (blockIdx.x * blockDim.x + threadIdx.x) * 4;
  if (c >= N) return;
  const int64_t n_pad = (int64_t)S.blocks * 128;
  const int per = S.per_cta(S.units);
  float v[1][4];
  sum_planes<1>(part + (int64_t)m * S.planes * n_pad, {c}, n_pad,
                block_planes(S, per, c / 128 * S.units + m / tok), v);
  const int64_t o = (int64_t)m * N + c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (c + i >= N) break;
    if (out_f32) static_cast<float*>(out)[o + i] = v[0][i];
    else static_cast<__nv_bfloat16*>(out)[o + i] = __float2bfloat16_rn(v[0][i]);
  }
}

// The FFN's intermediate of one slot per CTA: the L1's planes added, h = silu(gate) * up, and its
// conversion for the L2.  Gate rows 32j + i and up rows 32j + 16 + i make feature 16j + i.
__global__ void __launch_bounds__(512) swiglu_kernel(const float* part, const Split S,
                                                     const int32_t* n_plan,
                                                     const int32_t* slot_unit, int I, uint8_t* hf,
                                                     int32_t* exps) {
  __shared__ uint32_t red[32];
  pdl_trigger();
  pdl_wait();
  const int64_t s = blockIdx.x;
  const int unit = ld_after(slot_unit + s);
  if (unit < 0) return;  // dropped
  const int64_t n_pad = (int64_t)S.blocks * 128;
  const int per = S.per_cta(ld_after(n_plan));
  const int64_t steps = (I + kStepK - 1) / kStepK;
  const float* base = part + s * S.planes * n_pad;
  convert_row<4, 1>(
      [&](int p, float (&h)[4]) {
        const int f = p * 4, row = 32 * (f / 16) + f % 16;
        float v[2][4];  // gate, up
        sum_planes<2>(base, {row, row + 16}, n_pad,
                      block_planes(S, per, unit * S.blocks + row / 128), v);
#pragma unroll
        for (int i = 0; i < 4; ++i)  // silu first: gate * up alone may not be finite
          h[i] = v[0][i] / (1.0f + expf(-v[0][i])) * v[1][i];
      },
      I, hf + s * steps * kStepX, kStepX, exps + s, red);
}

// out[t] = sum over the token's live slots, in order, of w * (the L2's planes added).  128 columns of a
// token per CTA: a warp takes every 8th slot, 4 columns a lane.
constexpr int kCombineWarps = 8;
__global__ void __launch_bounds__(32 * kCombineWarps) combine_slots_kernel(
    const float* part, const Split S, const int32_t* n_plan, const int32_t* slot_unit,
    const float* w, int H, int k, __nv_bfloat16* out) {
  __shared__ float4 s_y[kCombineWarps][32];
  pdl_wait();
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.y * 128 + lane * 4;
  const int64_t n_pad = (int64_t)S.blocks * 128;
  const int per = S.per_cta(ld_after(n_plan));
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j0 = 0; j0 < k; j0 += kCombineWarps) {
    const int j = j0 + warp;
    float4 wy = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int unit = j < k ? ld_after(slot_unit + t * k + j) : -1;
    if (unit >= 0) {
      const float wj = ld_after(w + t * k + j);
      float y[1][4];
      sum_planes<1>(part + (t * k + j) * S.planes * n_pad, {c}, n_pad,
                    block_planes(S, per, unit * S.blocks + blockIdx.y), y);
      wy = make_float4(wj * y[0][0], wj * y[0][1], wj * y[0][2], wj * y[0][3]);
    }
    s_y[warp][lane] = wy;
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int i = 0; i < kCombineWarps; ++i) {
        const float4 y = s_y[i][lane];
        v[0] += y.x;
        v[1] += y.y;
        v[2] += y.z;
        v[3] += y.w;
      }
    }
    __syncthreads();
  }
  if (warp != 0) return;
  const __nv_bfloat162 o[2] = {__floats2bfloat162_rn(v[0], v[1]), __floats2bfloat162_rn(v[2], v[3])};
  *reinterpret_cast<uint2*>(out + t * H + c) = *reinterpret_cast<const uint2*>(o);
}

// ------------------------------------------------------------------------------ host side

constexpr int kSizingSms = 148;  // the SM count the K splits are sized for

// CTAs along K for one output block: enough CTAs for every SM, while each keeps at least two steps.
int pick_splits(int64_t blocks, int K, int most) {
  const int steps = (K + kStepK - 1) / kStepK;
  int s = 1;
  while (s < most && blocks * s < kSizingSms && steps / (2 * s) >= 2) s *= 2;
  return s;
}

template <typename... P, typename... V>
nvfp4_status_t launch(void (*fn)(P...), dim3 grid, int threads, size_t smem, int cluster, bool early,
                      cudaStream_t s, const char* what, const V&... args) {
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

// Lets fn use `smem` bytes, once per device (a call costs about as much as a launch).
template <typename Fn>
bool allow_smem(Fn fn, int smem, std::atomic<uint64_t>& devices_set) {
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (devices_set.load(std::memory_order_acquire) & bit) return true;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return false;
  devices_set.fetch_or(bit, std::memory_order_release);
  return true;
}

bool weight_map(CUtensorMap* tm, const uint8_t* codes, int64_t rows, int K) {
  if (byte_tensor_map(tm, codes, static_cast<uint64_t>(K / 2), static_cast<uint64_t>(rows)))
    return true;
  set_last_error("cuTensorMapEncodeTiled failed");
  return false;
}

template <int NT, bool XIN>
nvfp4_status_t launch_dense(const uint8_t* codes, const Operands& w, const DenseArgs& a, dim3 grid,
                            cudaStream_t s) {
  constexpr int smem = Cfg<NT, XIN>::SMEM;
  static std::atomic<uint64_t> devices_set{0};
  if (!allow_smem(dense_kernel<NT, XIN>, smem, devices_set)) return check_launch("dense_kernel");
  CUtensorMap tm;
  if (!weight_map(&tm, codes, w.N, w.K)) return NVFP4_ERR_CUDA;
  return launch(dense_kernel<NT, XIN>, grid, kThreads, smem, a.splits, !XIN, s, "dense_kernel", tm, w,
                a);
}

template <int NT, Mode MODE>
nvfp4_status_t launch_stream(const uint8_t* codes, int64_t rows, const Operands& w,
                             const StreamArgs& a, cudaStream_t s) {
  constexpr int smem = Cfg<NT, false>::SMEM;
  static std::atomic<uint64_t> devices_set{0};
  if (!allow_smem(stream_kernel<NT, MODE>, smem, devices_set)) return check_launch("stream_kernel");
  CUtensorMap tm;
  if (!weight_map(&tm, codes, rows, w.K)) return NVFP4_ERR_CUDA;
  return launch(stream_kernel<NT, MODE>, dim3(kStreamCtas), kThreads, smem, 1, true, s,
                "stream_kernel", tm, w, a);
}
template <Mode MODE>
nvfp4_status_t launch_stream(int nt, const uint8_t* codes, int64_t rows, const Operands& w,
                             const StreamArgs& a, cudaStream_t s) {
  return nt == 1 ? launch_stream<1, MODE>(codes, rows, w, a, s)
                 : launch_stream<2, MODE>(codes, rows, w, a, s);
}

int64_t converted_bytes(int64_t rows, int K) {
  return rows * ((K + kStepK - 1) / kStepK) * kStepX;
}

// Shares of at least `least` steps.
Split make_split(int nt, int N, int K, int64_t least, int units) {
  Split S{};
  S.blocks = static_cast<int>(((int64_t)N + 127) / 128);
  S.steps = (K + kStepK - 1) / kStepK;
  S.least = static_cast<int>(least);
  S.units = units;
  // shares of at least `least` steps that a block of S.steps can lie in
  S.kw = nt == 1 ? Warps<1>::KW : Warps<2>::KW;
  S.planes = S.kw * (S.steps == 1 ? 1 : (S.steps - 2) / S.least + 2);
  return S;
}

// How nvfp4_linear_w4a16 runs a shape, and the byte offsets of its workspace regions (256-byte
// aligned; none when the CTAs convert the activations themselves).
struct LinearW4Plan {
  int nt, splits;
  int64_t rowblks, tblks;
  bool xin, stream;
  Split split;
  int64_t exps, part, total;
};

// The streamed form takes products of at least this many steps per CTA and at most this many rows
// (its planes are float32 [rows][planes][N]).  It has two more kernels around the product: at 12
// steps per CTA (1 x 16384 x 7168) 19.5 us against 18.7 for a cluster per block, at 48 (1 x 65536 x
// 7168) 49.8 against 55.5.
constexpr int kStreamMinSteps = 14;
constexpr int kStreamMaxRows = 64;

LinearW4Plan linear_w4_plan(int64_t M, int N, int K) {
  LinearW4Plan P{};
  P.nt = M <= 8 ? 1 : 2;
  P.rowblks = ((int64_t)N + 127) / 128;
  P.tblks = (M + 8 * P.nt - 1) / (8 * P.nt);
  const int64_t steps = (K + kStepK - 1) / kStepK, total = P.rowblks * P.tblks * steps;
  P.stream = M <= kStreamMaxRows && total >= (int64_t)kStreamMinSteps * kStreamCtas &&
             total <= INT32_MAX;
  if (P.stream) {
    // every CTA's share is known here, so `least` is the share itself
    P.split = make_split(P.nt, N, K, (total + kStreamCtas - 1) / kStreamCtas, static_cast<int>(P.tblks));
  } else {
    P.splits = pick_splits(P.rowblks * P.tblks, K, kMaxSplits);
    P.xin = P.nt == 1 && M * ((steps + P.splits - 1) / P.splits) <= kMaxPieces;
  }
  if (!P.xin) {
    P.exps = round_up(P.tblks * 8 * P.nt * steps * kXRow, 256);
    P.part = P.exps + round_up(M * 4, 256);
    P.total = P.part;
    if (P.stream) P.total += round_up(M * P.split.planes * P.rowblks * 128 * 4, 256);
  }
  return P;
}

// How moe_ffn_w4a16 runs a shape, and the byte offsets of its workspace regions (256-byte aligned).
struct FfnW4Plan {
  int nt;
  Split l1, l2;
  int64_t w, plan, n_plan, order, slot_unit, xf, xexp, hf, hexp, part, total;
};

FfnW4Plan ffn_w4_plan(int T, int H, int I, int E, int k) {
  FfnW4Plan P{};
  const int64_t S = (int64_t)T * k;
  // token tiles: twice what an expert gets on average
  P.nt = 2 * S / E <= 8 ? 1 : 2;
  // With few slots a share may be as short as 4 steps, so that a handful of experts still occupies
  // every CTA; with more, whole blocks (2 pieces at most), which keeps the planes small.
  auto split = [&](int N, int K) {
    const int steps = (K + kStepK - 1) / kStepK;
    return make_split(P.nt, N, K, S <= 64 && steps > 4 ? 4 : steps, 0);
  };
  P.l1 = split(2 * I, H);
  P.l2 = split(H, I);
  int64_t o = 0;
  auto take = [&](int64_t bytes) {
    const int64_t at = o;
    o = round_up(o + bytes, 256);
    return at;
  };
  P.w = take(S * 4);
  P.plan = take(S * 16);
  P.n_plan = take(4);
  P.order = take(S * 4);
  P.slot_unit = take(S * 4);
  P.xf = take(converted_bytes(T, H));
  P.xexp = take((int64_t)T * 4);
  P.hf = take(converted_bytes(S, I));
  P.hexp = take(S * 4);
  // the L1's planes, then the L2's (which writes after the intermediate has been made)
  const int64_t p1 = S * P.l1.planes * P.l1.blocks, p2 = S * P.l2.planes * P.l2.blocks;
  P.part = take((p1 > p2 ? p1 : p2) * 128 * 4);
  P.total = o;
  return P;
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
  if (K % 64 || ld % 8 || M > (int64_t)65535 * 16 || N > INT32_MAX - 127)
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
  // CTAs that have finished write rows of out while others still read x
  if (rows_overlap(x, M, ld * 2, (int64_t)K * 2, out, M * N * (out_dtype == 0 ? 4 : 2)))
    return NVFP4_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(ws);
  int32_t* exps = reinterpret_cast<int32_t*>(base + P.exps);
  if (!P.xin) {
    const nvfp4_status_t st =
        launch(convert_kernel, dim3(static_cast<unsigned>(M)), 256, 0, 1, false, s, "convert_kernel",
               static_cast<const uint8_t*>(x), ld * 2, K, 8 * P.nt, base, exps);
    if (st != NVFP4_OK) return st;
  }
  const Operands op{sfw, gs_w, N, K, base, exps};
  if (P.stream) {
    StreamArgs a{};
    a.split = P.split;
    a.M = static_cast<int>(M);
    a.part = reinterpret_cast<float*>(base + P.part);
    a.status = dev_status;
    const nvfp4_status_t st = launch_stream<DENSE>(P.nt, w, N, op, a, s);
    if (st != NVFP4_OK) return st;
    return launch(dense_sum_kernel, dim3((N / 4 + 128) / 128, static_cast<unsigned>(M)), 128, 0, 1,
                  true, s, "dense_sum_kernel", a.part, P.split, 8 * P.nt, N, out,
                  static_cast<int>(out_dtype == 0));
  }
  const DenseArgs a{x, ld * 2, static_cast<int>(M), out, out_dtype == 0, P.splits, dev_status};
  const dim3 grid(static_cast<unsigned>(P.rowblks * P.splits), static_cast<unsigned>(P.tblks));
  if (P.xin) return launch_dense<1, true>(w, op, a, grid, s);
  return P.nt == 1 ? launch_dense<1, false>(w, op, a, grid, s)
                   : launch_dense<2, false>(w, op, a, grid, s);
}

extern "C" size_t moe_ffn_w4a16_workspace_size(int T, int H, int I, int E, int k) {
  if (T < 0 || H <= 0 || I <= 0 || E <= 0 || k <= 0) return 0;
  return static_cast<size_t>(ffn_w4_plan(T, H, I, E, k).total);
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
  const FfnW4Plan P = ffn_w4_plan(T, H, I, E, k);
  for (const Split& l : {P.l1, P.l2})  // a unit holds a slot at least
    if ((int64_t)T * k * l.blocks * l.steps > INT32_MAX) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (ws_bytes < static_cast<size_t>(P.total)) return NVFP4_ERR_WORKSPACE_TOO_SMALL;
  const void* ptrs16[] = {x_bf16, w1, sfw1, w2, sfw2, out_bf16};
  for (const void* p : ptrs16)
    if (!aligned16(p)) return NVFP4_ERR_MISALIGNED;
  const void* ptrs4[] = {logits, topk_ids, topk_w, gs_w1, gs_w2, dev_status};
  for (const void* p : ptrs4)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return NVFP4_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return NVFP4_ERR_MISALIGNED;
  // CTAs that have finished write rows of out while others still read the weights (x and the ids are
  // read by the first kernel alone: out may be x)
  const int64_t w_bytes = (int64_t)T * k * 4;
  if (rows_overlap(topk_w, 1, w_bytes, w_bytes, out_bf16, (int64_t)T * H * 2))
    return NVFP4_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(ws);
  auto i32 = [&](int64_t off) { return reinterpret_cast<int32_t*>(base + off); };
  float* wts = logits != nullptr ? reinterpret_cast<float*>(base + P.w) : const_cast<float*>(topk_w);
  int4* plan = reinterpret_cast<int4*>(base + P.plan);
  const int S = T * k;
  nvfp4_status_t st =
      launch(plan_kernel, dim3(1 + T), kPlanThreads, 0, 1, false, s, "plan_kernel", logits, T, E, k,
             8 * P.nt, topk_ids, wts, plan, i32(P.n_plan), i32(P.order), i32(P.slot_unit),
             static_cast<const uint8_t*>(x_bf16), H, base + P.xf, i32(P.xexp), dev_status);
  if (st != NVFP4_OK) return st;
  StreamArgs a{};
  a.split = P.l1;
  a.k = k;
  a.plan = plan;
  a.n_plan = i32(P.n_plan);
  a.order = i32(P.order);
  a.part = reinterpret_cast<float*>(base + P.part);
  a.status = dev_status;
  st = launch_stream<FFN_L1>(P.nt, w1, (int64_t)E * 2 * I,
                             Operands{sfw1, gs_w1, 2 * I, H, base + P.xf, i32(P.xexp)}, a, s);
  if (st != NVFP4_OK) return st;
  st = launch(swiglu_kernel, dim3(S), 512, 0, 1, true, s, "swiglu_kernel", a.part, P.l1,
              i32(P.n_plan), i32(P.slot_unit), I, base + P.hf, i32(P.hexp));
  if (st != NVFP4_OK) return st;
  a.split = P.l2;
  st = launch_stream<FFN_L2>(P.nt, w2, (int64_t)E * H,
                             Operands{sfw2, gs_w2, H, I, base + P.hf, i32(P.hexp)}, a, s);
  if (st != NVFP4_OK) return st;
  return launch(combine_slots_kernel, dim3(T, H / 128), 32 * kCombineWarps, 0, 1, true, s,
                "combine_slots_kernel", a.part, P.l2, i32(P.n_plan), i32(P.slot_unit), wts, H, k,
                static_cast<__nv_bfloat16*>(out_bf16));
}
