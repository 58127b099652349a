// mx_gemm16.cuh -- what the two kernels for 16-bit operands share (the
// CTA-pair kernel for large products, the one-CTA split-K kernel for small
// ones, both in mx_gemm16.cu): problem arguments, tile bookkeeping, operand
// descriptors and the epilogue arithmetic.
//
//   D[i, j] = epilogue( sum_k A(i, k) * B(j, k) ),   BF16 or FP16 operands, FP32 sums
//
// Either operand may lie K-major ([rows, k], k contiguous) or MN-major
// ([k, rows], rows contiguous): the weight gradient dW = dY^T X and the input
// gradient dX = dY W read the tensors as the forward pass left them, without
// a transposed copy.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "mx_gemm_common.cuh"
#include "mx_launch.h"

namespace mxk {

// kRaggedM: group g owns rows [off[g], off[g+1]) of A and D, B is [groups, ...];
// kRaggedK: group g owns that range of the reduction, D is [groups, m, n].
enum G16Mode : int { kBatched = 0, kRaggedM = 1, kRaggedK = 2 };

// kEpiPlain: D = acc.  kEpiLinear: z = acc + bias, D = act(z) + residual.
// kEpiPoly: D = alpha * scale * acc + beta * (C + C_lo) + diag * I, with an
// optional low half of D and, for a symmetric D, the mirrored tile.
// Of the pair kernel only: kEpiSum: D = acc in FP32.  kEpiLong: one of the first three
// (args.epi) behind a long sum.
enum G16Epi : int { kEpiPlain = 0, kEpiLinear = 1, kEpiPoly = 2, kEpiSum = 3, kEpiLong = 4 };

// The tensor core's accumulator truncates: a sum of numbers of one sign loses
// about 1e-7 of itself for each 16 terms (6.2e-3 at 2^20 of them, more than half a
// step of BF16).  One accumulator therefore takes at most kSumWhole terms (1e-4, a
// fifth of FP16's half step); a longer sum goes in parts of kSumPart, which are
// added in FP32, rounded (5e-5 whatever its length).
constexpr int kSumWhole = 1 << 14;
constexpr int kSumPart = 1 << 13;

struct G16Args {
  const void* bias;              // [n], operand type (linear)
  const void* res;               // residual or C, rows as D's, pitch res_ld
  const void* res_lo;            // low half of C (poly)
  void* d;                       // out
  void* z;                       // linear: pre-activation; poly: low half of D; null if not wanted
  const int32_t* group_offsets;  // ragged forms
  const float* scale;            // poly: factor per batch entry, raised to scale_pow (null: 1)
  int32_t* status;
  uint64_t wait_ns;
  int64_t d_ld, res_ld;          // elements between rows
  int64_t d_batch, res_batch;    // elements between batch entries
  float alpha, beta, diag;
  int scale_pow;
  int m, n, k;                   // ragged M: m = all rows; ragged K: k = all rows
  int m_tiles, n_tiles;          // of one batch entry (ragged M: n_tiles only)
  int groups;                    // batch entries or groups
  int mode;
  int a_mn, b_mn;                // operand is MN-major
  int a_wide, b_wide;            // MN-major, and one box brings 128 of MN (4-D tensor map)
  int b_per_group;               // B has a z coordinate (batched, ragged M)
  int op_fp16;                   // operands are FP16 (else BF16); also the type of bias, residual, C
  int out_type;                  // MX_BF16 / MX_FP16 / MX_FP32 of D and z
  int epi;                       // kEpiPlain, kEpiLinear or kEpiPoly
  int act;
  int sym;                       // D is symmetric: only tiles on and above the diagonal are computed
  int splits;                    // one-CTA kernel: CTAs of a cluster that share one tile's K
};

// ---------------------------------------------------------------- tiles

// Tiles of a grid of mt x nt: bands of 8 tile rows, down each column of a band
// first, so that the tiles in flight at one time cover a nearly square piece of D
// and share their operands' rows in L2.
constexpr int kBand = 8;

__device__ __forceinline__ void band_decode(int l, int mt, int nt, int& mb, int& nb) {
  const int band = l / (kBand * nt);
  const int m0 = band * kBand;
  const int gm = mt - m0 < kBand ? mt - m0 : kBand;
  const int r = l - m0 * nt;
  nb = r / gm;
  mb = m0 + r - nb * gm;
}

// Tile l of the upper triangle (mb <= nb), column by column: column nb has
// nb + 1 tiles and starts at nb (nb + 1) / 2.
__device__ __forceinline__ void tri_decode(int l, int& mb, int& nb) {
  int c = static_cast<int>((sqrtf(8.0f * static_cast<float>(l) + 1.0f) - 1.0f) * 0.5f);
  while (c * (c + 1) / 2 > l) --c;        // the square root may be off by one either way
  while ((c + 1) * (c + 2) / 2 <= l) ++c;
  nb = c;
  mb = l - c * (c + 1) / 2;
}

__device__ __forceinline__ int g16_tiles_per_entry(const G16Args& a) {
  return a.sym ? a.m_tiles * (a.m_tiles + 1) / 2 : a.m_tiles * a.n_tiles;
}

struct G16Tile {
  int group;
  int row0;      // first row of the tile (ragged M: of all rows)
  int rows_end;  // rows at or beyond this are not the group's
  int mb, nb;
};

// Ragged M: tab[i] is the number of tiles before group i * kTabStep (every
// kTabStep-th group only, for shared memory's sake; the rest is counted from the offsets).
constexpr int kTabStep = 4;

template <int TM>
__device__ __forceinline__ int g16_group_tiles(const G16Args& a, int e) {
  return (__ldg(a.group_offsets + e + 1) - __ldg(a.group_offsets + e) + TM - 1) / TM * a.n_tiles;
}

template <int TM>
__device__ __forceinline__ G16Tile g16_decode(const G16Args& a, const int32_t* tab, int t) {
  G16Tile r;
  if (a.mode == kRaggedM) {
    const int i = last_le(tab, (a.groups - 1) / kTabStep, t);
    int l = t - tab[i];
    r.group = i * kTabStep;
    for (int n; r.group + 1 < a.groups && l >= (n = g16_group_tiles<TM>(a, r.group)); ++r.group) l -= n;
    const int begin = __ldg(a.group_offsets + r.group);
    r.rows_end = __ldg(a.group_offsets + r.group + 1);
    band_decode(l, (r.rows_end - begin + TM - 1) / TM, a.n_tiles, r.mb, r.nb);
    r.row0 = begin + r.mb * TM;
  } else {
    const int per = g16_tiles_per_entry(a);
    r.group = t / per;
    const int l = t - r.group * per;
    if (a.sym)
      tri_decode(l, r.mb, r.nb);
    else
      band_decode(l, a.m_tiles, a.n_tiles, r.mb, r.nb);
    r.row0 = r.mb * TM;
    r.rows_end = a.m;
  }
  return r;
}

// First token and number of tokens of a group (ragged K), else all of K.
__device__ __forceinline__ void g16_k_range(const G16Args& a, int group, int& k0, int& kn) {
  if (a.mode == kRaggedK) {
    k0 = __ldg(a.group_offsets + group);
    kn = __ldg(a.group_offsets + group + 1) - k0;
  } else {
    k0 = 0;
    kn = a.k;
  }
}

// Offsets in order and inside [0, limit]?  (every thread a share of them)
__device__ __forceinline__ int g16_offsets_bad(const G16Args& a, int limit) {
  int bad = 0;
  for (int i = threadIdx.x; i <= a.groups; i += blockDim.x) {
    const int32_t v = __ldg(a.group_offsets + i);
    if (v < 0 || v > limit) bad = 1;
    if (i > 0 && v < __ldg(a.group_offsets + i - 1)) bad = 1;
  }
  return bad;
}

// Fills tab (see g16_decode) and *total, the number of all tiles (one warp).
template <int TM>
__device__ __forceinline__ void g16_prefix(const G16Args& a, int32_t* tab, int bad, uint32_t* total) {
  const int lane = threadIdx.x & 31;
  const int per = ((a.groups + 31) / 32 + kTabStep - 1) / kTabStep * kTabStep;  // groups of a lane
  const int lo = lane * per;
  int sum = 0;
  if (!bad)
    for (int i = lo; i < lo + per && i < a.groups; ++i) sum += g16_group_tiles<TM>(a, i);
  int incl = sum;
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) *total = static_cast<uint32_t>(incl);
  if (bad) return;
  int run = incl - sum;
  for (int i = lo; i < lo + per && i < a.groups; ++i) {
    if (i % kTabStep == 0) tab[i / kTabStep] = run;
    run += g16_group_tiles<TM>(a, i);
  }
}

// ---------------------------------------------------------------- tensor core

// Instruction descriptor for kind::f16 into FP32: both operands of one type;
// bits 15 and 16 mark an MN-major A or B.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int fp16, int a_mn, int b_mn) {
  return (1u << 4)                                    // D format F32
         | (static_cast<uint32_t>(fp16 ? 0 : 1) << 7)   // A format F16 / BF16
         | (static_cast<uint32_t>(fp16 ? 0 : 1) << 10)  // B format
         | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// MN-major operand tile written by TMA with 128-byte swizzling: each K row
// holds 64 elements (128 B), 8-row groups 1024 B apart; the next 64 elements
// along MN lie chunk_bytes further.
__device__ __forceinline__ uint64_t desc_mnmajor_sw128(uint32_t addr, uint32_t chunk_bytes) {
  return smem_desc(addr, chunk_bytes, 1024, kSwizzle128B);
}

// One lane of a converged warp, chosen so that the compiler knows the code it
// guards to be uniform: tcgen05 and TMA operands then stay in uniform registers.
// (Under `lane == 0` every MMA's descriptors went through per-thread registers,
// and the issuing thread, not the tensor cores, bounded the kernel: 8192^3 917 us
// against 751 us, and 707 us with the descriptors advanced instead of rebuilt.)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void tc_mma_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tc_mma_pair_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 4-D tiled TMA load global -> shared, completing on this CTA's `bar`.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int32_t x, int32_t y,
                                            int32_t z, int32_t w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

__device__ __forceinline__ void tc_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tc_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Bounded wait for a phase of a barrier, with the meaning of mbar_wait.  The
// clock is read only once TRIES attempts have failed: reading it after the first,
// as mbar_wait does, delays every wait of a pipeline in step (the producer's for
// a free stage, the MMA issuer's for a full one) by that read (after two: 512 rows
// over 32 experts 0.8 % slower).  An attempt that fails takes up to 4 us, so 32 keep a
// limit to within some 250 us; 2, for waits outside the pipeline, to 16.
template <bool CLUSTER, uint32_t TRIES = 32>
__device__ __forceinline__ bool wait16(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    uint32_t ok;
    if constexpr (CLUSTER)  // success also acquires what other CTAs of the cluster released
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(bar), "r"(parity)
          : "memory");
    else
      ok = mbar_try_wait(bar, parity);
    if (ok) return true;
    if (it % TRIES == 0) {
      if (abort != nullptr && *abort) return false;
      const uint64_t now = global_timer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > limit_ns) return false;
    }
  }
}

// ---------------------------------------------------------------- 16-bit values

__device__ __forceinline__ uint32_t pack16(float lo, float hi, int fp16) {
  if (fp16) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ float2 unpack16(uint32_t w, int fp16) {
  if (fp16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

__device__ __forceinline__ void split8(const uint4 w, int fp16, float (&f)[8]) {
  const float2 a = unpack16(w.x, fp16), b = unpack16(w.y, fp16), c = unpack16(w.z, fp16), d = unpack16(w.w, fp16);
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y; f[4] = c.x; f[5] = c.y; f[6] = d.x; f[7] = d.y;
}

__device__ __forceinline__ void load8(const void* p, int fp16, float (&f)[8]) {
  split8(__ldg(reinterpret_cast<const uint4*>(p)), fp16, f);
}

// ---------------------------------------------------------------- activations

// 2^x and 1/x as the special function unit gives them, results below 2^-126 zero
// (without that, each costs a scaling of small numbers that no activation needs).
__device__ __forceinline__ float exp2_ftz(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_ftz(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

constexpr float kLog2E = 1.4426950408889634f;

// The logistic function: the exponential's infinity for very negative x gives zero.
__device__ __forceinline__ float sigmoid_f32(float x) { return rcp_ftz(1.0f + exp2_ftz(-kLog2E * x)); }

constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// Phi(z) = erfc(-z / sqrt 2) / 2 by the approximation 7.1.26 of Abramowitz and
// Stegun, erfc(x) = t (a1 + t (a2 + ...)) e^(-x^2) with t = 1 / (1 + p x), within
// 1.5e-7.  e: e^(-z^2 / 2).
__device__ __forceinline__ float normal_cdf_f32(float z, float& e) {
  const float t = rcp_ftz(fmaf(0.3275911f * 0.7071067811865476f, fabsf(z), 1.0f));
  float p = fmaf(0.5f * 1.061405429f, t, 0.5f * -1.453152027f);
  p = fmaf(p, t, 0.5f * 1.421413741f);
  p = fmaf(p, t, 0.5f * -0.284496736f);
  p = fmaf(p, t, 0.5f * 0.254829592f);
  e = exp2_ftz(-0.5f * kLog2E * z * z);
  const float half = p * t * e;  // Phi(-|z|)
  return z >= 0.0f ? 1.0f - half : half;
}

// act(z); 0.5 (1 + tanh u) = sigmoid(2 u).  relu keeps a NaN.
__device__ __forceinline__ float act_f32(float z, int act) {
  switch (act) {
    case 1: return z < 0.0f ? 0.0f : z;
    case 2: return z * sigmoid_f32(z);
    case 3: {
      float e;
      return z * normal_cdf_f32(z, e);
    }
    case 4: return z * sigmoid_f32(2.0f * kGeluC * (z + kGeluA * z * z * z));
    default: return z;
  }
}

// act'(z), finite for every finite z.  relu passes on what a NaN z gets.
__device__ __forceinline__ float act_grad_f32(float z, int act) {
  switch (act) {
    case 1: return z <= 0.0f ? 0.0f : 1.0f;
    case 2: {
      const float p = sigmoid_f32(z);
      return p * (1.0f + z * (1.0f - p));
    }
    case 3: {  // Phi(z) + z e^(-z^2 / 2) / sqrt(2 pi): one exponential for both
      float e;
      const float cdf = normal_cdf_f32(z, e);
      return fmaf(z * 0.3989422804014327f, e, cdf);
    }
    case 4: {
      const float p = sigmoid_f32(2.0f * kGeluC * (z + kGeluA * z * z * z));
      const float q = p * (1.0f - p);  // 0 long before z^2 overflows
      return q == 0.0f ? p : p + z * q * 2.0f * kGeluC * (1.0f + 3.0f * kGeluA * z * z);
    }
    default: return 1.0f;
  }
}

// ---------------------------------------------------------------- epilogue

__device__ __forceinline__ float g16_scale(const G16Args& a, int group) {
  if (a.scale == nullptr) return a.alpha;
  const float s = __ldg(a.scale + group);
  return a.scale_pow == 2 ? a.alpha * s * s : a.alpha * s;
}

// The epilogue's arithmetic on C consecutive columns from col0 of one row, in
// place.  `valid`: the row is the group's; columns at or beyond `end` (n, or where
// another CTA's begin) hold values that are never stored.  C's and the residual's
// values come with the call (g16_load_res, zeros where there is none).
//
// First part.  Linear: the pre-activation acc + bias.  Poly: D itself; scale is
// g16_scale of the tile's group.
template <int EPI, int C>
__device__ __forceinline__ void g16_epilogue(const G16Args& a, float (&v)[C], const uint4 (&res)[C / 8],
                                             const uint4 (&low)[C / 8], const float* bias, int group, int64_t row, int col0,
                                             float scale) {
  if constexpr (EPI == kEpiLinear) {
    if (a.bias != nullptr) {
#pragma unroll
      for (int j = 0; j < C; j += 4) {
        const float4 b = *reinterpret_cast<const float4*>(bias + j);
        v[j] += b.x;
        v[j + 1] += b.y;
        v[j + 2] += b.z;
        v[j + 3] += b.w;
      }
    }
  } else if constexpr (EPI == kEpiPoly) {
#pragma unroll
    for (int j = 0; j < C; ++j) v[j] *= scale;
    if (a.res != nullptr) {
      const float beta = a.scale != nullptr && a.scale_pow == 1 ? a.beta * __ldg(a.scale + group) : a.beta;
#pragma unroll
      for (int g = 0; g < C / 8; ++g) {
        float b[8];
        split8(res[g], a.op_fp16, b);
        if (a.res_lo != nullptr) {
          float l[8];
          split8(low[g], a.op_fp16, l);
#pragma unroll
          for (int j = 0; j < 8; ++j) b[j] += l[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[g * 8 + j] = fmaf(beta, b[j], v[g * 8 + j]);
      }
    }
    if (a.diag != 0.0f) {
      const int64_t j = row - col0;
      if (j >= 0 && j < C) {
#pragma unroll
        for (int i = 0; i < C; ++i)
          if (j == i) v[i] += a.diag;
      }
    }
  }
}

// Second part of the linear epilogue: activation and residual.
template <int C>
__device__ __forceinline__ void g16_activate(const G16Args& a, float (&v)[C], const uint4 (&res)[C / 8]) {
  switch (a.act) {  // one loop for each, not a choice for each value
    case 1:
#pragma unroll
      for (int j = 0; j < C; ++j) v[j] = act_f32(v[j], 1);
      break;
    case 2:
#pragma unroll
      for (int j = 0; j < C; ++j) v[j] = act_f32(v[j], 2);
      break;
    case 3:
#pragma unroll
      for (int j = 0; j < C; ++j) v[j] = act_f32(v[j], 3);
      break;
    case 4:
#pragma unroll
      for (int j = 0; j < C; ++j) v[j] = act_f32(v[j], 4);
      break;
    default: break;
  }
  if (a.res != nullptr) {
#pragma unroll
    for (int g = 0; g < C / 8; ++g) {
      float b[8];
      split8(res[g], a.op_fp16, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[g * 8 + j] += b[j];
    }
  }
}

// C columns from col0 of a row of the residual (or C, or its low half).
template <int C>
__device__ __forceinline__ void g16_load_res(const G16Args& a, const void* base, int group, int64_t row, int col0, int end,
                                             bool valid, uint4 (&res)[C / 8]) {
  const uint16_t* p = static_cast<const uint16_t*>(base) + group * a.res_batch + row * a.res_ld + col0;
#pragma unroll
  for (int g = 0; g < C / 8; ++g)
    res[g] = base != nullptr && valid && col0 + g * 8 < end ? __ldg(reinterpret_cast<const uint4*>(p + g * 8))
                                                            : make_uint4(0, 0, 0, 0);
}

// What rounding the values to the output type leaves.
template <int C>
__device__ __forceinline__ void g16_remainder(const G16Args& a, float (&v)[C]) {
  const int h = a.out_type == 1;
#pragma unroll
  for (int j = 0; j < C; j += 2) {
    const float2 r = unpack16(pack16(v[j], v[j + 1], h), h);
    v[j] -= r.x;
    v[j + 1] -= r.y;
  }
}

// C columns of one row to global memory (16-bit), whole groups of 8 columns before
// `end` (rows are padded to a multiple of 8 elements).
template <int C>
__device__ __forceinline__ void g16_store_row(const G16Args& a, void* out, const float (&v)[C], int group, int64_t row,
                                              int col0, int end) {
  uint16_t* to = static_cast<uint16_t*>(out) + group * a.d_batch + row * a.d_ld + col0;
  const int h = a.out_type == 1;
#pragma unroll
  for (int g = 0; g < C / 8; ++g) {
    const float* p = v + g * 8;
    if (col0 + g * 8 < end)
      *reinterpret_cast<uint4*>(to + g * 8) =
          make_uint4(pack16(p[0], p[1], h), pack16(p[2], p[3], h), pack16(p[4], p[5], h), pack16(p[6], p[7], h));
  }
}

// The mirrored half of a symmetric D (16-bit): column col0 + j of this row
// becomes row col0 + j.  Neighbouring lanes trade values, so that each stores two
// rows of one column of a pair: a warp's 32 rows are 64 consecutive bytes there.
// Every lane of the warp calls.  The pair of an odd last row reaches into the row's
// padding (rows are padded to a multiple of 8 elements).
template <int C>
__device__ __forceinline__ void g16_store_mirror(const G16Args& a, const float (&v)[C], int group, int64_t row,
                                                 int col0, int end, bool valid) {
  const int odd = threadIdx.x & 1;
  const bool pair_valid = __shfl_sync(0xFFFFFFFFu, static_cast<int>(valid), threadIdx.x & 30) != 0;
  uint16_t* out = static_cast<uint16_t*>(a.d) + group * a.d_batch + (row - odd);
#pragma unroll
  for (int j = 0; j < C; j += 2) {
    const uint32_t w = pack16(v[j], v[j + 1], a.out_type == 1);
    const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, w, 1);
    // an even lane takes column j of rows row and row + 1, an odd one column j + 1 of row - 1 and row
    const uint32_t two = odd ? __byte_perm(other, w, 0x7632) : __byte_perm(w, other, 0x5410);
    const int col = col0 + j + odd;
    if (pair_valid && col < end) *reinterpret_cast<uint32_t*>(out + col * a.d_ld) = two;
  }
}

}  // namespace mxk
