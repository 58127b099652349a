// mx_ortho_small.cu -- Newton-Schulz orthogonalisation of matrices with at most
// 128 rows (or columns) in one launch: a cluster of up to 16 CTAs holds a matrix
// on chip from its first read to its last write.
//
// The general path (mx_ortho.cu) launches three products a step; on a matrix of
// 32 x 7168 each is a few microseconds of launch, fill and drain around almost no
// work.  Here, with r the short side and the long side in slices of `slice`
// columns, CTA by CTA:
//   X     FP32 in TMEM (lane = row, times 2^(sx + 12)), so that a X is exact to
//         FP32, and as FP16 (times 2^sx) in shared memory for the products;
//   A     each CTA multiplies its slice's X X^T (K = slice), the partial sums meet in
//         distributed shared memory, each CTA adds some columns (in rank order), and
//         everyone receives all of A 2^12 as FP16;
//   B     = b A + c A^2 in every CTA, as the sum of two FP16 numbers;
//   X     <- a X + B X: TMEM times a while the partial sums are formed, then the
//         product accumulates onto it.
// The chunk of 64 columns of X in shared memory is at the same time a K-major
// operand of X X^T and an MN-major one of B X.  A tall matrix is read and written
// transposed.  One CTA to an SM: the launch asks for all shared memory, since CTAs
// of two clusters that waited for each other's TMEM on two SMs would never finish.
//
// Bound by latency, not by bytes or products (0.14 us): 32 x 7168 takes 37.6 us in 16
// CTAs, 12 for launch, read, norm and result and 5 a step (three products, two
// cluster barriers, two exchanges); the general path takes 102.  (With 256 threads
// and loads of single elements it was 63.)  At 128 registers a thread it spills 36 to 144 bytes.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "mx_gemm16.cuh"
#include "mx_launch.h"
#include "mx_ortho.cuh"

namespace mxk {

constexpr int kNsThreads = 512;  // four warps per TMEM lane quarter
constexpr int kNsGroups = kNsThreads / 128;
constexpr int kNsSmem = 232448;
constexpr int kNsMaxCluster = 16;

struct NsSmallArgs {
  const void* g;
  __nv_bfloat16* out;
  int32_t* status;
  uint64_t wait_ns;
  int m, n;         // of one matrix
  int slice;        // columns of the long side per CTA, a multiple of 64
  int steps;
  int log_sx;
  uint32_t keep;    // steps (a bit each) that take a X of the FP32 X for a matrix much larger than eps
  float eps;
  float coeffs[3 * kNsMaxSteps];
};

__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

__device__ __forceinline__ void st_cluster_b32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_b16(uint32_t addr, uint16_t v) {
  asm volatile("st.shared::cluster.b16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_f64(uint32_t addr, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}

// Byte offset of element (row, k) of a K-major operand of `rows` rows: chunks of
// 64 k, each row 128 bytes, 16-byte pieces swizzled by the row.
__device__ __forceinline__ uint32_t kmajor_at(int rows, int row, int k) {
  return static_cast<uint32_t>((k >> 6) * rows * 128 + row * 128 + ((((k & 63) >> 3) ^ (row & 7)) << 4) + (k & 7) * 2);
}

// 128 bytes from `from` (any address) as 32 words, of which the first `bytes` are
// wanted: nine 16-byte loads and a shift by what `from` lies behind a multiple of 16.
// (Loads of an element each would go to L2 one by one: with all of the SM's memory
// shared there is no L1 to speak of.)  Nothing at or behind `end` is read.
template <int SIZE>
__device__ __forceinline__ void load_line(const uint8_t* from, int bytes, const uint8_t* end, uint32_t (&w)[32]) {
  const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(from) & 15u);
  const uint8_t* base = from - off;
  uint32_t v[36];
#pragma unroll
  for (int b = 0; b < 9; ++b) {
    uint4 q = make_uint4(0, 0, 0, 0);
    if (bytes > 0 && b * 16 < static_cast<int>(off) + bytes) {
      if (base + b * 16 + 16 <= end) {
        q = __ldg(reinterpret_cast<const uint4*>(base + b * 16));
      } else {  // the tensor's last bytes
        uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 16; i += SIZE) {
          if (base + b * 16 + i < end) {
            if constexpr (SIZE == 4)
              u[i / 4] = __ldg(reinterpret_cast<const uint32_t*>(base + b * 16 + i));
            else
              u[i / 4] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(base + b * 16 + i))) << (i & 2) * 8;
          }
        }
        q = make_uint4(u[0], u[1], u[2], u[3]);
      }
    }
    v[4 * b] = q.x;
    v[4 * b + 1] = q.y;
    v[4 * b + 2] = q.z;
    v[4 * b + 3] = q.w;
  }
  const bool by8 = off & 8, by4 = off & 4, by2 = off & 2;
#pragma unroll
  for (int i = 0; i < 34; ++i) v[i] = by8 ? v[i + 2] : v[i];
#pragma unroll
  for (int i = 0; i < 33; ++i) v[i] = by4 ? v[i + 1] : v[i];
#pragma unroll
  for (int i = 0; i < 32; ++i) w[i] = SIZE == 2 && by2 ? __funnelshift_r(v[i], v[i + 1], 16) : v[i];
}

// cs: CTAs of the cluster
template <typename T, int cs>
__global__ void __launch_bounds__(kNsThreads, 1) ns_cluster_kernel(const __grid_constant__ NsSmallArgs args) {
  static_assert(cs >= 1 && cs <= kNsMaxCluster && 16 % cs == 0, "cluster size");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int wgroup = warp >> 2;                   // which chunks of 64 columns
  const int row = (warp & 3) * 32 + lane;         // TMEM lane and matrix row
  const int rank = static_cast<int>(cluster_ctarank());
  const int batch = static_cast<int>(blockIdx.x) / cs;

  const bool tall = args.m > args.n;
  const int r = tall ? args.n : args.m, c = tall ? args.m : args.n;
  const int rp = (r + 15) / 16 * 16;
  const int slice = args.slice, chunks = slice / 64;
  // a warp whose 32 rows lie behind the matrix has no chunks
  const int first = (warp & 3) * 32 < rp ? wgroup : chunks, first16 = (warp & 3) * 32 < rp ? wgroup : rp / 16;
  const int c0 = rank * slice;                    // the slice's first column; those at or beyond c are zeros
  const int w = rp / cs;                          // columns of A this CTA adds up (cs <= 16 divides rp)
  const uint32_t misc = sbase;                                       // see below
  const uint32_t xs = sbase + 1024;                                  // X, FP16
  const uint32_t as = xs + chunks * rp * 128;                        // A
  const uint32_t bs = as + (rp + 63) / 64 * rp * 128;                // B
  const uint32_t recv = bs + (rp + 63) / 64 * rp * 128;              // [source][column][row] partial sums
  // misc: barrier 8, TMEM address 4, pad 4, block sums 16 x 8, cluster sums 16 x 8, factors 3 x 4, failed 4, drain barrier 8, kept steps 4
  const uint32_t bar = misc;
  auto at = [&](uint32_t addr) { return smem + (addr - sbase); };
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(at(misc + 8));
  double* block_sums = reinterpret_cast<double*>(at(misc + 16));
  const uint32_t cluster_sums = misc + 144;
  volatile float* factors = reinterpret_cast<volatile float*>(at(misc + 272));
  const uint32_t failed = misc + 284, drain_bar = misc + 288;
  volatile uint32_t* kept = reinterpret_cast<volatile uint32_t*>(at(misc + 296));

  if (tid == 0) {
    mbar_init(bar, 1);
    mbar_init(drain_bar, 1);
    fence_mbar_init();
    *reinterpret_cast<volatile uint32_t*>(at(failed)) = 0;
  }
  pdl_launch_dependents();
  pdl_wait_prior();
  if (warp == 0) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  cluster_sync();  // every CTA of the cluster runs before its shared memory is written
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t t_row = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  const uint32_t t_a = slice;                     // TMEM column of A's partial sum and of A^2
  // A wait that runs out (ok is the warp's) ends the warp's work: no wait, product or
  // result after it, only the barriers that others are waiting at.  All learn of it
  // at the next step's first cluster barrier and leave the steps there together.
  // (Warp 0 issues all products, each after its own wait for the one before.)
  uint32_t parity = 0;
  bool ok = true;
  auto wait_mma = [&]() {
    if (!ok) return;
    ok = __all_sync(0xFFFFFFFFu, wait16<false>(bar, parity, nullptr, args.wait_ns));
    parity ^= 1u;
    tc_fence_after();
  };

  // ---- read: raw values to TMEM, their squares summed in 64 bits over the cluster
  const T* g = static_cast<const T*>(args.g) + static_cast<int64_t>(batch) * args.m * args.n;
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  const bool aligned = c % (16 / static_cast<int>(sizeof(T))) == 0;  // every row starts on 16 bytes
  for (int j = first; j < chunks; j += kNsGroups) {
    // each lane its own row: a warp's loads fall into 32 lines, but every byte of them
    // is wanted, and the cluster reads a matrix once
    const int col = c0 + j * 64;
    uint32_t v[64];
    if (!tall) {
      const int there = row < r && col < c ? (c - col < 64 ? c - col : 64) : 0;  // columns of the chunk
      const uint8_t* p = reinterpret_cast<const uint8_t*>(g + static_cast<int64_t>(row) * c + col);
      const uint8_t* end = reinterpret_cast<const uint8_t*>(static_cast<const T*>(args.g) +
                                                            static_cast<int64_t>(gridDim.x / cs) * args.m * args.n);
#pragma unroll
      for (int h = 0; h < (sizeof(T) == 4 ? 2 : 1); ++h) {
        constexpr int N = 128 / sizeof(T);
        const int n = there - h * N < 0 ? 0 : there - h * N < N ? there - h * N : N;
        uint32_t w32[32];
        if (aligned) {
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const uint4 u = q * (N / 8) < n ? __ldg(reinterpret_cast<const uint4*>(p + h * 128) + q) : make_uint4(0, 0, 0, 0);
            w32[4 * q] = u.x;
            w32[4 * q + 1] = u.y;
            w32[4 * q + 2] = u.z;
            w32[4 * q + 3] = u.w;
          }
        } else {
          load_line<sizeof(T)>(p + h * 128, n * static_cast<int>(sizeof(T)), end, w32);
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          if constexpr (sizeof(T) == 4) {
            v[h * 32 + i] = i < n ? w32[i] : 0u;
          } else {
            v[2 * i] = 2 * i < n ? w32[i] << 16 : 0u;
            v[2 * i + 1] = 2 * i + 1 < n ? w32[i] & 0xFFFF0000u : 0u;
          }
        }
      }
    } else {
      const T* p = g + static_cast<int64_t>(col) * r + row;
#pragma unroll
      for (int i = 0; i < 64; ++i) {
        const float x = row < r && col + i < c ? static_cast<float>(p[static_cast<int64_t>(i) * r]) : 0.0f;
        v[i] = __float_as_uint(x);
      }
    }
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t half[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        half[i] = v[h * 32 + i];
        const double x = __uint_as_float(half[i]);
        s[i & 3] = fma(x, x, s[i & 3]);
      }
      tc_st_32x32b_x32(t_row + j * 64 + h * 32, half);
    }
  }
  tc_wait_st();
  double own = (s[0] + s[1]) + (s[2] + s[3]);
  for (int o = 16; o > 0; o >>= 1) own += __shfl_down_sync(0xFFFFFFFFu, own, o);
  if (lane == 0) block_sums[warp] = own;
  __syncthreads();
  if (tid < cs) {
    double t = 0.0;
    for (int i = 0; i < kNsThreads / 32; ++i) t += block_sums[i];
    st_cluster_f64(map_to_rank(cluster_sums, tid) + rank * 8, t);
  }
  cluster_sync();
  if (tid == 0) {  // (one thread: the FP64 unit is narrow)
    double sum = 0.0;
    for (int i = 0; i < cs; ++i) sum += reinterpret_cast<const double*>(at(cluster_sums))[i];
    const double f = sqrt(sum) + static_cast<double>(args.eps);
    const bool usual = f > 0.0 && isfinite(f);  // else: zeros stay zeros, anything else becomes NaN
    const int e = usual ? ilogb(f) : 0;
    // 2^(sx - e) in two halves: neither leaves FP32's range
    const int shift = args.log_sx - e;
    factors[0] = scalbnf(1.0f, shift / 2);
    factors[1] = scalbnf(1.0f, shift - shift / 2);
    factors[2] = (usual ? static_cast<float>(scalbn(1.0, e) / f) : f == 0.0 ? 1.0f : nanf("")) * (1 << kNsLogSA);
    uint32_t keep = args.keep;
    float bound = usual ? static_cast<float>(sqrt(sum) / f) : 1.0f;
    if (bound < kNsSmall)  // (a larger one is at most a sixteenth of what `keep` was made for)
      for (int i = 0; i < args.steps; ++i) {
        if (bound < kNsSmall) keep |= 1u << i;
        bound = ns_next_bound(bound, args.coeffs + 3 * i);
      }
    *kept = keep;
  }
  __syncthreads();
  const float up0 = factors[0], up1 = factors[1], up2 = factors[2];
  const uint32_t keep = *kept;
  const float sa = static_cast<float>(1 << kNsLogSA), inv_sa = 1.0f / sa;

  // FP16 copy of a chunk of X for the products (rows of zeros up to rp); v: X 2^(sx + 12)
  auto put_x = [&](int j, int h, const uint32_t (&v)[32]) {
    if (row >= rp) return;
    const uint32_t line = xs + j * rp * 128 + row * 128;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = pack16(__uint_as_float(v[q * 8 + 2 * i]) * inv_sa, __uint_as_float(v[q * 8 + 2 * i + 1]) * inv_sa, 1);
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(line + (((h * 4 + q) ^ (row & 7)) << 4)), "r"(o[0]),
                   "r"(o[1]), "r"(o[2]), "r"(o[3])
                   : "memory");
    }
  };
  // 64 columns of X's TMEM row, both halves on their way at once
  auto load_x = [&](int j, uint32_t (&lo)[32], uint32_t (&hi)[32]) {
    __syncwarp();  // TMEM loads and stores are the whole warp's
    tc_ld_32x32b_x32(t_row + j * 64, lo);
    tc_ld_32x32b_x32(t_row + j * 64 + 32, hi);
    tc_wait_ld();
  };
  for (int j = first; j < chunks; j += kNsGroups) {
    uint32_t v[2][32];
    load_x(j, v[0], v[1]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[h][i] = __float_as_uint(__uint_as_float(v[h][i]) * up0 * up1 * up2);
      tc_st_32x32b_x32(t_row + j * 64 + h * 32, v[h]);
      put_x(j, h, v[h]);
      __syncwarp();
    }
  }
  tc_wait_st();
  const float a_scale = sa / scalbnf(1.0f, 2 * args.log_sx);

  const uint32_t idesc_r = idesc_f16(128, rp, 1, 0, 0);
#pragma unroll 1
  for (int step = 0; step < args.steps; ++step) {
    const float ca = args.coeffs[3 * step], cb = args.coeffs[3 * step + 1], cc = args.coeffs[3 * step + 2];
    // ---- this slice's part of X X^T.  The 128 rows of the first operand reach
    // past X's rp rows into what lies behind: accumulator rows that nobody reads.
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (warp == 0 && ok && elect_one()) {
      tc_fence_after();
      const int live = c - c0 < slice ? (c - c0 > 0 ? (c - c0 + 63) / 64 : 1) : chunks;  // the others are zeros
      uint64_t d = desc_kmajor_sw128(xs);
      for (int j = 0; j < live; ++j, d += rp * 8) {  // descriptors count 16 bytes
        tc_mma_f16(tmem + t_a, d, d, idesc_r, j != 0 ? 1u : 0u);
        tc_mma_f16(tmem + t_a, d + 2, d + 2, idesc_r, 1);
        tc_mma_f16(tmem + t_a, d + 4, d + 4, idesc_r, 1);
        tc_mma_f16(tmem + t_a, d + 6, d + 6, idesc_r, 1);
      }
      tc_commit(bar);
    }
    __syncwarp();
    // ---- meanwhile a X in TMEM.  The last two steps take (a I + B) X of the FP16 X
    // instead, as the general form does: nothing multiplies X's rounding any more,
    // and a X of one X with B X of another would only add the difference (but not while
    // X is small, when a X is all that counts and FP16 has few bits of it).
    const bool add_x = keep >> step & 1;
    for (int j = add_x && ok ? first : chunks; j < chunks; j += kNsGroups) {
      uint32_t v[2][32];
      load_x(j, v[0], v[1]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[h][i] = __float_as_uint(ca * __uint_as_float(v[h][i]));
        tc_st_32x32b_x32(t_row + j * 64 + h * 32, v[h]);
      }
    }
    tc_wait_st();
    wait_mma();
    if (!ok && lane < cs) st_cluster_b32(map_to_rank(failed, lane), 1u);
    // ---- partial sums to the CTAs that add them
    for (int b = ok ? first16 : rp / 16; b < rp / 16; b += kNsGroups) {
      uint32_t v[16];
      __syncwarp();
      tc_ld_32x32b_x16(t_row + t_a + b * 16, v);
      tc_wait_ld();
      if (row < rp) {
        int owner = b * 16 / w, q = b * 16 - owner * w;
        uint32_t to = map_to_rank(recv, owner) + static_cast<uint32_t>(((rank * w + q) * 128 + row) * 4);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          st_cluster_b32(to, v[i]);
          to += 512;
          if (++q == w && i < 15) {
            q = 0;
            to = map_to_rank(recv, ++owner) + static_cast<uint32_t>((rank * w * 128 + row) * 4);
          }
        }
      }
    }
    cluster_sync();
    // (nobody writes here before all have passed the next barrier: the cluster agrees)
    if (*reinterpret_cast<volatile uint32_t*>(at(failed)) != 0) {
      ok = false;
      break;
    }
    // ---- added in rank order, and A 2^12 as FP16 to everyone.  Entry (row, col) is
    // stored as (col, row): the rows of a warp are then consecutive.
    if (row < rp) {
      for (int q = wgroup; q < w; q += kNsGroups) {
        const float* p = reinterpret_cast<const float*>(at(recv)) + q * 128 + row;
        float part[cs], t = 0.0f;
#pragma unroll
        for (int i = 0; i < cs; ++i) part[i] = p[i * w * 128];
#pragma unroll
        for (int i = 0; i < cs; ++i) t += part[i];
        const uint16_t v = static_cast<uint16_t>(pack16(t * a_scale, 0.0f, 1) & 0xFFFFu);
        const uint32_t to = as + kmajor_at(rp, rank * w + q, row);
#pragma unroll
        for (int i = 0; i < cs; ++i) st_cluster_b16(map_to_rank(to, i), v);
      }
    }
    fence_proxy_async_all();
    cluster_sync();
    fence_proxy_async_all();
    tc_fence_before();
    __syncthreads();
    // ---- A^2
    if (warp == 0 && elect_one()) {
      tc_fence_after();
      for (int k = 0; k < rp / 16; ++k) {
        const uint64_t d = desc_kmajor_sw128(as + (k >> 2) * rp * 128 + (k & 3) * 32);
        tc_mma_f16(tmem + t_a, d, d, idesc_r, k != 0 ? 1u : 0u);
      }
      tc_commit(bar);
    }
    __syncwarp();
    wait_mma();
    // ---- B 2^12 = b (A 2^12) + c 2^-12 (A 2^12)^2 (+ a 2^12 I), and what its rounding
    // leaves in A's place (A^2 is done, each entry of A is read by the lane that
    // writes there): near the fixed point a and B cancel to a fifth, and B's rounding
    // was half the method's error
    for (int b = ok ? first16 : rp / 16; b < rp / 16; b += kNsGroups) {
      uint32_t v[16];
      __syncwarp();
      tc_ld_32x32b_x16(t_row + t_a + b * 16, v);
      tc_wait_ld();
      if (row < rp) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t where = kmajor_at(rp, row, b * 16 + q * 8);
          const uint4 a4 = *reinterpret_cast<const uint4*>(at(as + where));
          const uint32_t u[4] = {a4.x, a4.y, a4.z, a4.w};
          uint32_t o[4], l[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 af = unpack16(u[i], 1);
            const int col = b * 16 + q * 8 + 2 * i;
            const float d0 = !add_x && col == row ? ca * sa : 0.0f, d1 = !add_x && col + 1 == row ? ca * sa : 0.0f;
            const float b0 = fmaf(cb, af.x, fmaf(__uint_as_float(v[q * 8 + 2 * i]), cc * inv_sa, d0));
            const float b1 = fmaf(cb, af.y, fmaf(__uint_as_float(v[q * 8 + 2 * i + 1]), cc * inv_sa, d1));
            o[i] = pack16(b0, b1, 1);
            const float2 h = unpack16(o[i], 1);
            l[i] = pack16(b0 - h.x, b1 - h.y, 1);
          }
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(bs + where), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                       : "memory");
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(as + where), "r"(l[0]), "r"(l[1]), "r"(l[2]), "r"(l[3])
                       : "memory");
        }
      }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    // ---- a X + B X, up to 256 columns an instruction
    if (warp == 0 && ok && elect_one()) {
      tc_fence_after();
      for (int n0 = 0; n0 < slice; n0 += 256) {
        const uint32_t idesc = idesc_f16(128, slice - n0 < 256 ? slice - n0 : 256, 1, 0, 1);
        for (int k = 0; k < rp / 16; ++k) {
          const uint64_t x = desc_mnmajor_sw128(xs + (n0 / 64) * rp * 128 + k * 2048, rp * 128);
          const uint32_t at_k = (k >> 2) * rp * 128 + (k & 3) * 32;
          tc_mma_f16(tmem + n0, desc_kmajor_sw128(bs + at_k), x, idesc, add_x || k != 0 ? 1u : 0u);
          tc_mma_f16(tmem + n0, desc_kmajor_sw128(as + at_k), x, idesc, 1);
        }
      }
      tc_commit(bar);
    }
    __syncwarp();
    wait_mma();
    if (step + 1 < args.steps) {
      for (int j = ok ? first : chunks; j < chunks; j += kNsGroups) {
        uint32_t v[2][32];
        load_x(j, v[0], v[1]);
        put_x(j, 0, v[0]);
        put_x(j, 1, v[1]);
      }
    }
  }

  // ---- out
  const float last = inv_sa * scalbnf(1.0f, -args.log_sx);
  __nv_bfloat16* out = args.out + static_cast<int64_t>(batch) * args.m * args.n;
  for (int j = ok ? first : chunks; j < chunks; j += kNsGroups) {
    const int col = c0 + j * 64;
    uint32_t v[2][32], o[32];  // o: pairs of columns
    load_x(j, v[0], v[1]);
#pragma unroll
    for (int i = 0; i < 32; ++i)
      o[i] = pack16(__uint_as_float(v[i / 16][i % 16 * 2]) * last, __uint_as_float(v[i / 16][i % 16 * 2 + 1]) * last, 0);
    if (row < r) {
      uint16_t* p = reinterpret_cast<uint16_t*>(out) + (tall ? static_cast<int64_t>(col) * r + row : static_cast<int64_t>(row) * c + col);
      if (tall) {
#pragma unroll
        for (int k = 0; k < 64; ++k)
          if (col + k < c) p[static_cast<int64_t>(k) * r] = static_cast<uint16_t>(o[k / 2] >> (k & 1) * 16);
      } else if (c % 8 == 0) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (col + q * 8 < c) reinterpret_cast<uint4*>(p)[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
      } else {  // pairs on 4 bytes: of a row that starts between them from its second value on
        const int there = c - col < 64 ? c - col : 64, odd = reinterpret_cast<uintptr_t>(p) & 2 ? 1 : 0;
        if (odd && there > 0) p[0] = static_cast<uint16_t>(o[0]);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const uint32_t pair = odd ? (i < 31 ? __funnelshift_r(o[i], o[i + 1], 16) : o[i] >> 16) : o[i];
          const int at2 = 2 * i + odd;
          if (at2 + 1 < there)
            *reinterpret_cast<uint32_t*>(p + at2) = pair;
          else if (at2 < there)
            p[at2] = static_cast<uint16_t>(pair);
        }
      }
    }
  }
  if (!ok && lane == 0) report(args.status, 0x4);
  // products still under way end before their operands and accumulators are given up
  if (warp == 0 && !ok && elect_one()) {
    tc_commit(drain_bar);
    wait16<false>(drain_bar, 0, nullptr, 100000000ull);
  }
  __syncwarp();
  // no CTA leaves while another may still write into its shared memory
  tc_fence_before();
  cluster_sync();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ======================================================================= host

constexpr int kNsDevices = 64;

using NsKernel = void (*)(NsSmallArgs);

template <typename T>
static NsKernel ns_kernel(int cs) {
  switch (cs) {
    case 1: return ns_cluster_kernel<T, 1>;
    case 2: return ns_cluster_kernel<T, 2>;
    case 4: return ns_cluster_kernel<T, 4>;
    case 8: return ns_cluster_kernel<T, 8>;
    default: return ns_cluster_kernel<T, 16>;
  }
}

// Clusters of `cs` CTAs that the GPU holds at once (0: none).
template <typename T>
static int ns_clusters(int cs) {
  static std::atomic<int> known[kNsDevices][kNsMaxCluster + 1];  // 0 unknown, else the number + 1
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= kNsDevices) return 0;
  int v = known[dev][cs].load(std::memory_order_acquire);
  if (v == 0) {
    int n = 0;
    const NsKernel kernel = ns_kernel<T>(cs);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>(cs), 1, 1);
    cfg.blockDim = dim3(kNsThreads, 1, 1);
    cfg.dynamicSmemBytes = kNsSmem;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cs);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNsSmem) != cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    v = n + 1;
    known[dev][cs].store(v, std::memory_order_release);
  }
  return v - 1;
}

static int ns_slice(int64_t c, int cs) { return static_cast<int>(((c + cs - 1) / cs + 63) / 64 * 64); }

// Does a slice's X, A and partial sums fit TMEM's 512 columns, and everything shared memory?
static bool ns_fits(int r, int slice, int cs) {
  const int rp = (r + 15) / 16 * 16;
  if (slice + rp > 512) return false;
  const int operands = 1024 + slice / 64 * rp * 128 + 2 * ((rp + 63) / 64) * rp * 128;
  // behind B there are the partial sums, and room for the (128 - rp) rows that the
  // products' 128-row operands read past B's end
  const int behind = rp * 512 > (128 - rp) * 128 ? rp * 512 : (128 - rp) * 128;
  return 1024 + operands + behind <= kNsSmem;
}

template <typename T>
static cudaError_t ns_small(const OrthoProblem& q, bool* taken, int num_sms, cudaStream_t stream) {
  *taken = false;
  const int64_t r = q.m < q.n ? q.m : q.n, c = q.m < q.n ? q.n : q.m;
  if (r > 128 || c > kNsMaxCluster * 448) return cudaSuccess;
  // the smallest cluster that holds the matrix; larger ones, down to 128 columns a
  // CTA, while the whole batch fits the GPU at once
  int cs = 0;
  for (int s = 1; s <= kNsMaxCluster; s *= 2) {
    if (!ns_fits(static_cast<int>(r), ns_slice(c, s), s)) continue;
    const int held = ns_clusters<T>(s);
    if (held == 0) break;
    if (cs != 0 && (q.batch > held || ns_slice(c, s / 2) <= 128)) break;
    cs = s;
  }
  if (cs == 0) return cudaSuccess;
  *taken = true;
  NsSmallArgs a = {};
  a.g = q.g;
  a.out = static_cast<__nv_bfloat16*>(q.out);
  a.status = q.status;
  a.wait_ns = wait_limit_ns();
  a.m = static_cast<int>(q.m);
  a.n = static_cast<int>(q.n);
  a.slice = ns_slice(c, cs);
  a.steps = q.steps;
  a.log_sx = static_cast<int>(std::lround(0.5 * std::log2(static_cast<double>(c))));
  a.eps = q.eps;
  for (int i = 0; i < 3 * q.steps; ++i) a.coeffs[i] = q.coeffs[i];
  float bound = 1.0f;
  for (int i = 0; i < q.steps; ++i) {
    if (i == 0 || i + 2 < q.steps || bound < kNsSmall) a.keep |= 1u << i;
    bound = ns_next_bound(bound, q.coeffs + 3 * i);
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(static_cast<unsigned>(q.batch * cs), 1, 1);
  cfg.blockDim = dim3(kNsThreads, 1, 1);
  cfg.dynamicSmemBytes = kNsSmem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cs);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, ns_kernel<T>(cs), a);
}

cudaError_t launch_orthogonalize_small(const OrthoProblem& q, bool* taken, int num_sms, cudaStream_t stream) {
  return q.fp32 ? ns_small<float>(q, taken, num_sms, stream) : ns_small<__nv_bfloat16>(q, taken, num_sms, stream);
}

}  // namespace mxk
