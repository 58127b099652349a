// mx_ortho.cu -- orthogonalising a batch of matrices by Newton-Schulz products.
//
//   X_0 = G / (|G|_F + eps);   A = X X^T,  B = b A + c A^2,  X <- a X + B X
//
// for matrices with no more rows than columns; a tall one takes A = X^T X and
// X <- a X + X B (the same numbers, transposed) with its operands MN-major, so
// nothing is transposed in memory.  A and B are symmetric: only the tiles on
// and above the diagonal are computed, each stored twice.
//
// Numbers.  The products run on FP16 operands with FP32 sums; every matrix is
// held times a power of two that brings its entries near one (X times 2^sx,
// about sqrt(columns); A and B times 2^12), so that FP16's range is not left and
// its 11 bits are kept.  An iteration multiplies the smallest singular values by
// about a = 3.4, and so the rounding of X in those directions: five steps
// multiply the first rounding by nearly 500.  Therefore X_0 of a 16-bit G is G
// times a power of two, exact but for entries below some 2^-14 of the norm over the root of
// the columns, which fall below FP16's normal range (the rest of 1 / |G|_F is a factor
// of the first step's epilogues), and X is kept as the sum of two FP16 numbers
// while three or more steps follow, the low one entering a X in the
// epilogue.  The products take the high one: B maps into the directions of the
// large singular values, where its rounding is not multiplied.  A, B: one FP16 number.
// While X is small as a whole (eps much larger than G: X_0's norm is |G| / eps) it is held
// times a power of two more, one for each matrix and step, found from a bound of its
// singular values; the epilogues' factors on the device bring them in and out.
//
// Bound by the tensor cores: five steps of 8 x 4096 x 7168 are 17.2 TFLOP and take
// 12.9 ms on a card that has rested (1330 TFLOP/s), 15.3 in loops at its power limit,
// of which the sum of squares and the start are 0.2.  The diagonal tiles' lower
// halves, 6 % of A's and B's, are computed too.  A 256 x 256 matrix takes 106 us, 6 us
// for each of 17 launches.  (Reading an FP32 G of 4 x 7168 x 2048 by 16 bytes instead
// of 4 took the start from 134 to 78 us.)
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>

#include "mx_gemm16.cuh"
#include "mx_launch.h"
#include "mx_ortho.cuh"

namespace mxk {

constexpr int kNormParts = 256; // partial sums of squares per matrix

// Sum of squares of a share of each matrix, in 64 bits: no square of an FP32
// or BF16 number over- or underflows there.
template <typename T>
__global__ void __launch_bounds__(256) ns_square_kernel(const T* __restrict__ g, double* __restrict__ part, int64_t count) {
  __shared__ double sums[8];
  pdl_launch_dependents();
  pdl_wait_prior();
  const T* x = g + blockIdx.y * count;
  double s = 0.0;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  constexpr int V = 16 / sizeof(T);
  if (count % V == 0) {  // every matrix starts on 16 bytes
#pragma unroll 2
    for (int64_t i = t; i < count / V; i += stride) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(x) + i);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) {
          const double v = __uint_as_float(u[j]);
          s = fma(v, v, s);
        } else {
          const float2 f = unpack16(u[j], 0);
          const double v0 = f.x, v1 = f.y;
          s = fma(v0, v0, s);
          s = fma(v1, v1, s);
        }
      }
    }
  } else {
    for (int64_t i = t; i < count; i += stride) {
      const double v = static_cast<float>(x[i]);
      s = fma(v, v, s);
    }
  }
  for (int o = 16; o > 0; o >>= 1) s += __shfl_down_sync(0xFFFFFFFFu, s, o);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 8; ++i) s += sums[i];
    part[blockIdx.y * kNormParts + blockIdx.x] = s;
  }
}

struct NsCoeffs {
  float v[3 * kNsMaxSteps];
  int steps;
};

// X_0 = G 2^(sx - e) as FP16 (and, for an FP32 G, what that leaves), 2^e at most |G|_F, rows
// `pitch` apart.  One warp a row.  And the factors of each step's epilogues,
// [step][matrix]: before step i > 0 what is stored is X 2^(sx - f_i), f_i = 0 unless
// X is small; before the first it is X 2^sx (|G|_F + eps) / 2^e.
//   gram: what XX^T's X still has to be multiplied by, 2^e / (|G|_F + eps), later 2^f_i
//   next: gram / 2^f_(i+1), f = 0 behind the last step
// (both are 2^e / (|G|_F + eps), later 1, for a matrix much larger than eps)
template <typename T>
__global__ void __launch_bounds__(256) ns_start_kernel(const T* __restrict__ g, const double* __restrict__ part, int parts,
                                                       float eps, int log_sx, __half* __restrict__ hi, __half* __restrict__ lo,
                                                       float* __restrict__ gram, float* __restrict__ next,
                                                       const __grid_constant__ NsCoeffs coeffs, int64_t m, int n, int64_t pitch) {
  __shared__ int exponent;
  pdl_launch_dependents();
  pdl_wait_prior();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    double s = 0.0;
    for (int i = lane; i < parts; i += 32) s += part[blockIdx.y * kNormParts + i];
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    const double norm = sqrt(s), f = norm + static_cast<double>(eps);
    const bool usual = norm > 0.0 && isfinite(norm);  // else zeros stay zeros, and what is not finite makes all NaN
    const int e = usual ? ilogb(norm) : 0;
    if (lane == 0) {
      exponent = e;
      if (blockIdx.x == 0) {
        double have = usual ? scalbn(1.0, e) / f : norm == 0.0 ? 1.0 : nan("");
        float bound = usual ? static_cast<float>(norm / f) : 1.0f;
        for (int i = 0; i < coeffs.steps; ++i) {
          bound = ns_next_bound(bound, coeffs.v + 3 * i);
          const int up = bound < kNsSmall && i + 1 < coeffs.steps ? (bound > 0x1p-120f ? ilogbf(bound) : -120) : 0;
          gram[static_cast<int64_t>(i) * gridDim.y + blockIdx.y] = static_cast<float>(have);
          next[static_cast<int64_t>(i) * gridDim.y + blockIdx.y] = static_cast<float>(scalbn(have, -up));
          have = scalbn(1.0, up);
        }
      }
    }
  }
  __syncthreads();
  // 2^(sx - e) in two halves: neither leaves FP32's range
  const int e = log_sx - exponent;
  const float up0 = scalbnf(1.0f, e / 2), up1 = scalbnf(1.0f, e - e / 2);
  const T* x = g + blockIdx.y * m * n;
  __half* xh = hi + blockIdx.y * m * pitch;
  __half* xl = lo == nullptr ? nullptr : lo + blockIdx.y * m * pitch;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + warp; r < m; r += static_cast<int64_t>(gridDim.x) * 8) {
    if (n % 8 == 0) {
#pragma unroll 2
      for (int c = lane * 8; c < n; c += 256) {
        float f[8];
        if constexpr (sizeof(T) == 4) {
          const float4 a = __ldg(reinterpret_cast<const float4*>(x + r * n + c)), b = __ldg(reinterpret_cast<const float4*>(x + r * n + c + 4));
          f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
        } else {
          load8(x + r * n + c, 0, f);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = f[j] * up0 * up1;
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = pack16(f[2 * j], f[2 * j + 1], 1);
        *reinterpret_cast<uint4*>(xh + r * pitch + c) = make_uint4(o[0], o[1], o[2], o[3]);
        if (xl != nullptr) {
          uint32_t l[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 back = unpack16(o[j], 1);
            l[j] = pack16(f[2 * j] - back.x, f[2 * j + 1] - back.y, 1);
          }
          *reinterpret_cast<uint4*>(xl + r * pitch + c) = make_uint4(l[0], l[1], l[2], l[3]);
        }
      }
    } else {
#pragma unroll 4
      for (int c = lane; c < n; c += 32) {
        const float v = static_cast<float>(x[r * n + c]) * up0 * up1;
        const __half h = __float2half_rn(v);
        xh[r * pitch + c] = h;
        if (xl != nullptr) xl[r * pitch + c] = __float2half_rn(v - __half2float(h));
      }
    }
  }
}

// Rows of n values out of rows `pitch` apart.
__global__ void __launch_bounds__(256) ns_pack_kernel(const uint16_t* __restrict__ x, uint16_t* __restrict__ out, int64_t rows,
                                                      int n, int64_t pitch) {
  pdl_launch_dependents();
  pdl_wait_prior();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + warp; r < rows; r += static_cast<int64_t>(gridDim.x) * 8)
    for (int c = lane; c < n; c += 32) out[r * n + c] = x[r * pitch + c];
}

static int64_t pad8(int64_t v) { return (v + 7) / 8 * 8; }
static size_t pad256(size_t v) { return (v + 255) / 256 * 256; }

struct NsPlan {
  int64_t pitch_x, pitch_a, count_x, count_a;  // elements
  bool low;                                    // the low halves of X are kept
  size_t part, gram, next, x[2], xl[2], a, b, bytes;
};

static NsPlan ns_plan(int64_t batch, int64_t m, int64_t n, bool fp32, int steps) {
  NsPlan p = {};
  const int64_t r = m < n ? m : n;
  p.pitch_x = pad8(n);
  p.pitch_a = pad8(r);
  p.count_x = m * p.pitch_x;
  p.count_a = r * p.pitch_a;
  p.low = fp32 || steps > 3;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += pad256(bytes);
    return here;
  };
  p.part = take(static_cast<size_t>(batch) * kNormParts * 8);
  p.gram = take(static_cast<size_t>(batch) * kNsMaxSteps * 4);  // (for any number of steps: a workspace serves them alike)
  p.next = take(static_cast<size_t>(batch) * kNsMaxSteps * 4);
  for (int i = 0; i < 2; ++i) {
    p.x[i] = take(static_cast<size_t>(batch * p.count_x) * 2);
    p.xl[i] = p.low ? take(static_cast<size_t>(batch * p.count_x) * 2) : 0;
  }
  p.a = take(static_cast<size_t>(batch * p.count_a) * 2);
  p.b = take(static_cast<size_t>(batch * p.count_a) * 2);
  p.bytes = at;
  return p;
}

size_t ns_workspace_bytes(int64_t batch, int64_t m, int64_t n, bool fp32, int steps) {
  return ns_plan(batch, m, n, fp32, steps).bytes;
}

template <typename K, typename... Args>
static cudaError_t launch_pdl(K kernel, dim3 grid, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t launch_orthogonalize(const OrthoProblem& q, int num_sms, cudaStream_t stream) {
  const char* forced = std::getenv("MX_ORTHO_CONFIG");  // "general": this path for every size (tests, tuning)
  if (forced == nullptr || std::strcmp(forced, "general") != 0) {
    bool taken = false;
    const cudaError_t e = launch_orthogonalize_small(q, &taken, num_sms, stream);
    if (e != cudaSuccess || taken) return e;
  }
  const NsPlan p = ns_plan(q.batch, q.m, q.n, q.fp32, q.steps);
  uint8_t* ws = static_cast<uint8_t*>(q.workspace);
  double* part = reinterpret_cast<double*>(ws + p.part);
  float* gram = reinterpret_cast<float*>(ws + p.gram);
  float* next = reinterpret_cast<float*>(ws + p.next);
  NsCoeffs coeffs = {};
  coeffs.steps = q.steps;
  for (int i = 0; i < 3 * q.steps; ++i) coeffs.v[i] = q.coeffs[i];
  const bool tall = q.m > q.n;
  const int64_t r = tall ? q.n : q.m, c = tall ? q.m : q.n;
  const int log_sx = static_cast<int>(std::lround(0.5 * std::log2(static_cast<double>(c))));
  const float sx = std::ldexp(1.0f, log_sx), sa = std::ldexp(1.0f, kNsLogSA);

  // enough blocks for the GPU over the whole batch, none without work
  const int64_t count = q.m * q.n;
  int64_t parts = (count + 8191) / 8192;
  const int64_t wanted = (static_cast<int64_t>(num_sms) * 8 + q.batch - 1) / q.batch;
  if (parts > wanted) parts = wanted;
  if (parts > kNormParts) parts = kNormParts;
  const dim3 grid_sq(static_cast<unsigned>(parts), static_cast<unsigned>(q.batch), 1);
  int64_t row_blocks = (q.m + 7) / 8;
  if (row_blocks > wanted) row_blocks = wanted;
  const dim3 grid_st(static_cast<unsigned>(row_blocks), static_cast<unsigned>(q.batch), 1);
  __half* x0 = reinterpret_cast<__half*>(ws + p.x[0]);
  __half* x0l = q.fp32 ? reinterpret_cast<__half*>(ws + p.xl[0]) : nullptr;
  cudaError_t e;
  if (q.fp32) {
    const float* g = static_cast<const float*>(q.g);
    e = launch_pdl(ns_square_kernel<float>, grid_sq, stream, g, part, count);
    if (e != cudaSuccess) return e;
    e = launch_pdl(ns_start_kernel<float>, grid_st, stream, g, static_cast<const double*>(part), static_cast<int>(parts),
                   q.eps, log_sx, x0, x0l, gram, next, coeffs, q.m, static_cast<int>(q.n), p.pitch_x);
  } else {
    const __nv_bfloat16* g = static_cast<const __nv_bfloat16*>(q.g);
    e = launch_pdl(ns_square_kernel<__nv_bfloat16>, grid_sq, stream, g, part, count);
    if (e != cudaSuccess) return e;
    e = launch_pdl(ns_start_kernel<__nv_bfloat16>, grid_st, stream, g, static_cast<const double*>(part),
                   static_cast<int>(parts), q.eps, log_sx, x0, x0l, gram, next, coeffs, q.m, static_cast<int>(q.n), p.pitch_x);
  }
  if (e != cudaSuccess) return e;

  bool low = q.fp32;  // the current X has a low half
  for (int i = 0; i < q.steps; ++i) {
    const float ca = q.coeffs[3 * i], cb = q.coeffs[3 * i + 1], cc = q.coeffs[3 * i + 2];
    const bool last = i == q.steps - 1;
    const bool low_out = i < q.steps - 3;
    // a X in the epilogue where its low half counts, else a on B's diagonal
    const bool add_x = low || low_out;
    void* x = ws + p.x[i & 1];
    void* xl = low ? ws + p.xl[i & 1] : nullptr;

    Gemm16 s = {};
    s.groups = q.batch;
    s.op_fp16 = 1;
    s.out_type = 1;
    s.epi = 2;
    s.status = q.status;

    // A 2^12 = X X^T 2^(12 - 2 sx) gram^2
    Gemm16 ga = s;
    ga.a = ga.b = x;
    ga.a_ld = ga.b_ld = p.pitch_x;
    ga.a_batch = ga.b_batch = p.count_x;
    ga.a_mn = ga.b_mn = tall;
    ga.m = ga.n = r;
    ga.k = c;
    ga.d = ws + p.a;
    ga.d_ld = p.pitch_a;
    ga.d_batch = p.count_a;
    ga.sym = 1;
    ga.alpha = sa / (sx * sx);
    ga.scale = gram + i * q.batch;
    ga.scale_pow = 2;
    e = launch_gemm16(ga, num_sms, stream);
    if (e != cudaSuccess) return e;

    // B 2^12 = b (A 2^12) + c 2^-12 (A 2^12)^2 (+ a 2^12 I)
    Gemm16 gb = s;
    gb.a = gb.b = ws + p.a;
    gb.a_ld = gb.b_ld = p.pitch_a;
    gb.a_batch = gb.b_batch = p.count_a;
    gb.m = gb.n = gb.k = r;
    gb.d = ws + p.b;
    gb.d_ld = p.pitch_a;
    gb.d_batch = p.count_a;
    gb.sym = 1;
    gb.alpha = cc / sa;
    gb.res = ws + p.a;
    gb.res_ld = p.pitch_a;
    gb.res_batch = p.count_a;
    gb.beta = cb;
    gb.diag = add_x ? 0.0f : ca * sa;
    e = launch_gemm16(gb, num_sms, stream);
    if (e != cudaSuccess) return e;

    // X 2^sx = (a (X 2^sx) + 2^-12 (B 2^12) (X 2^sx)) next; the last one without 2^sx, to the output
    Gemm16 gx = s;
    if (tall) {  // X B, B symmetric
      gx.a = x;
      gx.a_ld = p.pitch_x;
      gx.a_batch = p.count_x;
      gx.b = ws + p.b;
      gx.b_ld = p.pitch_a;
      gx.b_batch = p.count_a;
    } else {     // B X, X's columns are D's
      gx.a = ws + p.b;
      gx.a_ld = p.pitch_a;
      gx.a_batch = p.count_a;
      gx.b = x;
      gx.b_ld = p.pitch_x;
      gx.b_batch = p.count_x;
      gx.b_mn = 1;
    }
    gx.m = q.m;
    gx.n = q.n;
    gx.k = r;
    const float unit = last ? 1.0f / sx : 1.0f;
    gx.alpha = unit / sa;
    gx.scale = next + i * q.batch;
    gx.scale_pow = 1;
    if (add_x) {
      gx.res = x;
      gx.res_lo = xl;
      gx.res_ld = p.pitch_x;
      gx.res_batch = p.count_x;
      gx.beta = unit * ca;
    }
    if (last && q.n % 8 == 0) {
      gx.d = q.out;
      gx.d_ld = q.n;
      gx.d_batch = q.m * q.n;
    } else {
      gx.d = ws + p.x[(i + 1) & 1];
      gx.d_ld = p.pitch_x;
      gx.d_batch = p.count_x;
      if (low_out) gx.z = ws + p.xl[(i + 1) & 1];
    }
    if (last) gx.out_type = 0;
    e = launch_gemm16(gx, num_sms, stream);
    if (e != cudaSuccess) return e;
    low = low_out;
  }
  if (q.n % 8 != 0) {  // rows that TMA cannot write
    const int64_t rows = q.batch * q.m;
    int64_t blocks = (rows + 7) / 8;
    if (blocks > num_sms * 8) blocks = num_sms * 8;
    e = launch_pdl(ns_pack_kernel, dim3(static_cast<unsigned>(blocks), 1, 1), stream,
                   reinterpret_cast<const uint16_t*>(ws + p.x[q.steps & 1]), static_cast<uint16_t*>(q.out), rows,
                   static_cast<int>(q.n), p.pitch_x);
  }
  return e;
}

}  // namespace mxk
