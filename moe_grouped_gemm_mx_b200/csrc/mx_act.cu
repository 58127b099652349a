// mx_act.cu -- the element-wise part of mx_linear_act's backward pass:
//
//   dZ = dY * act'(Z)   (one rounding to the operand type)
//   dbias[j] = sum_i dY[i, j] * act'(Z[i, j])   (FP32 products and sums)
//
// One pass over dY and Z: each thread keeps eight columns (16-byte loads and
// stores) over a chunk of rows and leaves their sums; a second small launch
// adds the chunks' sums in order, so the result does not change from call to
// call (with one chunk, up to 1024 rows, the first writes the result).
//
// Bound by its bytes, 6 an element: 65536x4096 takes 262 us with ReLU (6150
// GB/s), 270 with SiLU, 275 with GELU, 279 with its tanh form (5770 GB/s);
// 8192x4096 39 to 43 us, of which 3 are the sums' launch.  The arithmetic is not
// far behind (two special functions and some 20 instructions an element): 48
// registers and two rows in flight a thread; with 64 and four rows GELU took 344 us, with
// 40 registers 286.  A block has 64 columns, 128 bytes of each row; with one
// chunk 16, so that there are blocks for the SMs (333x1000: 8.5 -> 3.1 us).
#include <cuda_runtime.h>
#include <cstdint>

#include "mx_gemm16.cuh"
#include "mx_launch.h"

namespace mxk {

// COLS: columns of a block, COLS / 8 threads of eight.
template <int ACT, int COLS, int FP16>
__global__ void __launch_bounds__(256, 5) act_backward_kernel(const uint16_t* __restrict__ dy,
                                                           const uint16_t* __restrict__ z, uint16_t* __restrict__ dz,
                                                           float* __restrict__ partial, uint16_t* __restrict__ dbias,
                                                           int64_t m, int n, int64_t chunk) {
  constexpr int ROWS = 256 * 8 / COLS;  // rows a block works on at one time
  __shared__ float sums[ROWS][COLS + 1];
  const int tx = threadIdx.x % (COLS / 8), ty = threadIdx.x / (COLS / 8);
  const int col = blockIdx.x * COLS + tx * 8;
  const int64_t r0 = blockIdx.y * chunk;
  const int64_t r1 = r0 + chunk < m ? r0 + chunk : m;
  float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  pdl_launch_dependents();
  pdl_wait_prior();
  if (col < n) {
#pragma unroll 2
    for (int64_t r = r0 + ty; r < r1; r += ROWS) {
      const int64_t at = r * n + col;
      float g[8];
      load8(dy + at, FP16, g);
      if constexpr (ACT != 0) {
        float x[8];
        load8(z + at, FP16, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] *= act_grad_f32(x[j], ACT);
        *reinterpret_cast<uint4*>(dz + at) = make_uint4(pack16(g[0], g[1], FP16), pack16(g[2], g[3], FP16),
                                                        pack16(g[4], g[5], FP16), pack16(g[6], g[7], FP16));
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += g[j];
    }
  }
  if (dbias == nullptr) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) sums[ty][tx * 8 + j] = s[j];
  __syncthreads();
  // a quarter of a warp (COLS 64: all of it alone) adds a column's ROWS sums
  constexpr int PARTS = 256 / COLS < 8 ? 256 / COLS : 8;
  const int c = threadIdx.x / PARTS, part = threadIdx.x % PARTS;
  float t = 0.0f;
  if (c < COLS)
    for (int i = part; i < ROWS; i += PARTS) t += sums[i][c];
#pragma unroll
  for (int o = PARTS / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
  const int to = blockIdx.x * COLS + c;
  if (c < COLS && part == 0 && to < n) {
    if (gridDim.y == 1)
      dbias[to] = static_cast<uint16_t>(pack16(t, 0.0f, FP16) & 0xFFFFu);
    else
      partial[static_cast<int64_t>(blockIdx.y) * n + to] = t;
  }
}

__global__ void __launch_bounds__(256) bias_sum_kernel(const float* __restrict__ partial, uint16_t* __restrict__ dbias,
                                                       int n, int chunks, int fp16) {
  __shared__ float sums[8][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + tx;
  pdl_launch_dependents();
  pdl_wait_prior();
  float s = 0.0f;
  if (col < n)
    for (int i = ty; i < chunks; i += 8) s += partial[static_cast<int64_t>(i) * n + col];
  sums[ty][tx] = s;
  __syncthreads();
  if (ty == 0 && col < n) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += sums[i][tx];
    dbias[col] = static_cast<uint16_t>(pack16(s, 0.0f, fp16) & 0xFFFFu);
  }
}

static cudaLaunchConfig_t pdl_config(dim3 grid, int threads, cudaStream_t stream, cudaLaunchAttribute (&attr)[1]) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// Chunks of rows: one of up to 1024 rows, else enough blocks for the GPU, at
// most 64 sums a column to add.
int64_t act_backward_chunks(int64_t m) {
  if (m <= 1024) return 1;
  const int64_t c = (m + 127) / 128;
  return c < 64 ? c : 64;
}

using ActKernel = void (*)(const uint16_t*, const uint16_t*, uint16_t*, float*, uint16_t*, int64_t, int, int64_t);

template <int COLS, int FP16>
static ActKernel act_kernel(int act) {
  switch (act) {
    case 0: return act_backward_kernel<0, COLS, FP16>;
    case 1: return act_backward_kernel<1, COLS, FP16>;
    case 2: return act_backward_kernel<2, COLS, FP16>;
    case 3: return act_backward_kernel<3, COLS, FP16>;
    default: return act_backward_kernel<4, COLS, FP16>;
  }
}

cudaError_t launch_act_backward(const void* dy, const void* z, void* dz, void* dbias, float* partial, int64_t m,
                                int64_t n, int act, int fp16, cudaStream_t stream) {
  const int64_t chunks = act_backward_chunks(m);
  const int64_t chunk = (m + chunks - 1) / chunks;
  cudaLaunchAttribute attr[1];
  const bool narrow = chunks == 1;
  const int cols = narrow ? 16 : 64;
  cudaLaunchConfig_t cfg = pdl_config(dim3(static_cast<unsigned>((n + cols - 1) / cols),
                                           static_cast<unsigned>((m + chunk - 1) / chunk), 1),
                                      256, stream, attr);
  const uint16_t* y16 = static_cast<const uint16_t*>(dy);
  const uint16_t* z16 = static_cast<const uint16_t*>(z);
  uint16_t* d16 = static_cast<uint16_t*>(dz);
  uint16_t* db = static_cast<uint16_t*>(dbias);
  const ActKernel kernel = narrow ? (fp16 ? act_kernel<16, 1>(act) : act_kernel<16, 0>(act))
                                  : (fp16 ? act_kernel<64, 1>(act) : act_kernel<64, 0>(act));
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, y16, z16, d16, partial, db, m, static_cast<int>(n), chunk);
  if (e != cudaSuccess || !dbias || m <= chunk) return e;
  cfg = pdl_config(dim3(static_cast<unsigned>((n + 31) / 32), 1, 1), 256, stream, attr);
  return cudaLaunchKernelEx(&cfg, bias_sum_kernel, static_cast<const float*>(partial), db,
                            static_cast<int>(n), static_cast<int>((m + chunk - 1) / chunk), fp16);
}

}  // namespace mxk
