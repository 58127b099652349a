// mx_api.cu -- the extern "C" boundary declared in include/mx.h: argument
// validation, then one kernel launch per call on the caller's stream.  No
// memory is allocated per call; the only device memory the library owns is the
// 4-byte internal status word below.
#include <cuda_runtime.h>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/mx.h"

#include "mx_launch.h"

namespace {

constexpr int64_t kMaxGroups = 1024;
constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

__device__ int32_t g_internal_status = 0;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int num_sms() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  static int cached_dev = -1, cached = 0;
  if (dev != cached_dev) {
    int v = 0;
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    cached = v;
    cached_dev = dev;
  }
  return cached;
}

int32_t* internal_status_ptr() {
  void* p = nullptr;
  if (cudaGetSymbolAddress(&p, g_internal_status) != cudaSuccess) return nullptr;
  return static_cast<int32_t*>(p);
}

mx_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MX_OK : MX_ERR_CUDA; }

constexpr uint64_t kDefaultWaitNs = 2000000000ull;  // 2 s
std::atomic<uint64_t> g_wait_ns{kDefaultWaitNs};

}  // namespace

uint64_t mxk::wait_limit_ns() { return g_wait_ns.load(std::memory_order_relaxed); }

extern "C" {

const char* mx_status_string(int status) {
  switch (status) {
    case MX_OK: return "MX_OK";
    case MX_ERR_INVALID_ARGUMENT: return "MX_ERR_INVALID_ARGUMENT";
    case MX_ERR_UNSUPPORTED_SHAPE: return "MX_ERR_UNSUPPORTED_SHAPE";
    case MX_ERR_MISALIGNED: return "MX_ERR_MISALIGNED";
    case MX_ERR_CUDA: return "MX_ERR_CUDA";
    default: return "MX_ERR_UNKNOWN";
  }
}

size_t mx_scale_bytes(int64_t rows, int64_t k) {
  if (rows <= 0 || k <= 0) return 0;
  const int64_t kb = (k + 31) / 32;
  return static_cast<size_t>(((rows + 127) / 128) * 128 * ((kb + 3) / 4) * 4);
}

// Host-side checks of one quantisation job; MX_OK with *empty set for a no-op.
static mx_status check_quant_job(const void* x, int64_t groups, int64_t rows, int64_t k, const void* q,
                                 const void* sf, bool* empty) {
  *empty = false;
  if (groups < 0 || rows < 0 || k < 0) return MX_ERR_INVALID_ARGUMENT;
  if (k % 32 != 0) return MX_ERR_UNSUPPORTED_SHAPE;
  if (groups == 0 || rows == 0 || k == 0) {
    *empty = true;
    return MX_OK;
  }
  if (!x || !q || !sf) return MX_ERR_INVALID_ARGUMENT;
  if (!aligned16(x) || !aligned16(q) || !aligned16(sf)) return MX_ERR_MISALIGNED;
  if (rows > kMaxDim || groups * rows > kMaxDim || groups * rows * (k / 32) >= (int64_t(1) << 31))
    return MX_ERR_UNSUPPORTED_SHAPE;
  return MX_OK;
}

static mx_status quantize_impl(const void* x, int64_t groups, int64_t rows, int64_t k, void* q, void* sf,
                               mx_stream_t stream) {
  bool empty = false;
  mx_status st = check_quant_job(x, groups, rows, k, q, sf, &empty);
  if (st != MX_OK || empty) return st;
  const int sms = num_sms();
  if (sms <= 0) return MX_ERR_CUDA;
  mxk::QuantSpec spec{x, q, sf, groups, rows, k, static_cast<int64_t>(mx_scale_bytes(rows, k))};
  return from_cuda(mxk::launch_quant_batch(&spec, 1, sms, reinterpret_cast<cudaStream_t>(stream), nullptr));
}

mx_status mx_quantize_bf16_to_e4m3(const void* x_bf16, int64_t rows, int64_t k, void* q_e4m3, void* sf_ue8m0,
                                   mx_stream_t stream) {
  return quantize_impl(x_bf16, 1, rows, k, q_e4m3, sf_ue8m0, stream);
}

mx_status mx_quantize_bf16_to_e4m3_grouped(const void* x_bf16, int64_t groups, int64_t rows, int64_t k,
                                           void* q_e4m3, void* sf_ue8m0, mx_stream_t stream) {
  return quantize_impl(x_bf16, groups, rows, k, q_e4m3, sf_ue8m0, stream);
}

static mx_status quantize_multi(const mx_quant_job* jobs, int32_t count, mx_stream_t stream, bool lean) {
  if (count < 0 || (count > 0 && !jobs)) return MX_ERR_INVALID_ARGUMENT;
  // validate everything before launching anything
  int nonempty = 0;
  for (int32_t i = 0; i < count; ++i) {
    bool empty = false;
    mx_status st = check_quant_job(jobs[i].x_bf16, jobs[i].groups, jobs[i].rows, jobs[i].k, jobs[i].q_e4m3,
                                   jobs[i].sf_ue8m0, &empty);
    if (st != MX_OK) return st;
    nonempty += empty ? 0 : 1;
  }
  if (nonempty == 0) return MX_OK;
  const int sms = num_sms();
  if (sms <= 0) return MX_ERR_CUDA;
  mxk::QuantSpec specs[mxk::kMaxQuantJobs];
  int n = 0;
  for (int32_t i = 0; i < count; ++i) {
    const mx_quant_job& j = jobs[i];
    if (j.groups == 0 || j.rows == 0 || j.k == 0) continue;
    specs[n++] = mxk::QuantSpec{j.x_bf16, j.q_e4m3, j.sf_ue8m0, j.groups, j.rows, j.k,
                                static_cast<int64_t>(mx_scale_bytes(j.rows, j.k))};
    if (n == mxk::kMaxQuantJobs) {
      cudaError_t e = mxk::launch_quant_batch(specs, n, sms, reinterpret_cast<cudaStream_t>(stream), nullptr, lean);
      if (e != cudaSuccess) return MX_ERR_CUDA;
      n = 0;
    }
  }
  if (n > 0) {
    cudaError_t e = mxk::launch_quant_batch(specs, n, sms, reinterpret_cast<cudaStream_t>(stream), nullptr, lean);
    if (e != cudaSuccess) return MX_ERR_CUDA;
  }
  return MX_OK;
}

mx_status mx_quantize_bf16_to_e4m3_multi(const mx_quant_job* jobs, int32_t count, mx_stream_t stream) {
  return quantize_multi(jobs, count, stream, false);
}

mx_status mx_quantize_bf16_to_e4m3_multi_lean(const mx_quant_job* jobs, int32_t count, mx_stream_t stream) {
  return quantize_multi(jobs, count, stream, true);
}

mx_status mx_quantize_bf16_to_e4m3_transposed(const void* x_bf16, int64_t groups, int64_t rows, int64_t cols,
                                              void* q_e4m3, void* sf_ue8m0, mx_stream_t stream) {
  if (groups < 0 || rows < 0 || cols < 0) return MX_ERR_INVALID_ARGUMENT;
  if (rows % 32 != 0 || cols % 8 != 0) return MX_ERR_UNSUPPORTED_SHAPE;
  if (groups == 0 || rows == 0 || cols == 0) return MX_OK;
  if (!x_bf16 || !q_e4m3 || !sf_ue8m0) return MX_ERR_INVALID_ARGUMENT;
  if (!aligned16(x_bf16) || !aligned16(q_e4m3) || !aligned16(sf_ue8m0)) return MX_ERR_MISALIGNED;
  if (rows > kMaxDim || cols > kMaxDim || groups * rows * cols / 32 >= (int64_t(1) << 40))
    return MX_ERR_UNSUPPORTED_SHAPE;
  return from_cuda(mxk::launch_quant_transposed(x_bf16, groups, rows, cols, q_e4m3, sf_ue8m0,
                                                static_cast<int64_t>(mx_scale_bytes(cols, rows)),
                                                internal_status_ptr(), num_sms(),
                                                reinterpret_cast<cudaStream_t>(stream)));
}

static mx_status check_gemm_common(const void* qa, const void* sfa, const void* qb, const void* sfb, void* d,
                                   int64_t m, int64_t n, int64_t k, int64_t groups) {
  if (m < 0 || n < 0 || k < 0 || groups < 0) return MX_ERR_INVALID_ARGUMENT;
  if (k == 0 || k % 128 != 0 || n % 16 != 0) return MX_ERR_UNSUPPORTED_SHAPE;
  if (m > kMaxDim || n > kMaxDim || k > kMaxDim || groups > kMaxGroups) return MX_ERR_UNSUPPORTED_SHAPE;
  if (!qa || !sfa || !qb || !sfb || !d) return MX_ERR_INVALID_ARGUMENT;
  if (!aligned16(qa) || !aligned16(sfa) || !aligned16(qb) || !aligned16(sfb) || !aligned16(d))
    return MX_ERR_MISALIGNED;
  return MX_OK;
}

mx_status mx_gemm(const void* qa, const void* sfa, const void* qb, const void* sfb, void* d_bf16, int64_t m,
                  int64_t n, int64_t k, int32_t* dev_status, mx_stream_t stream) {
  if (m < 0 || n < 0 || k < 0) return MX_ERR_INVALID_ARGUMENT;
  if (m == 0 || n == 0) {
    if (k % 128 != 0 || k == 0 || n % 16 != 0) return MX_ERR_UNSUPPORTED_SHAPE;
    return MX_OK;
  }
  mx_status st = check_gemm_common(qa, sfa, qb, sfb, d_bf16, m, n, k, 1);
  if (st != MX_OK) return st;
  const int sms = num_sms();
  if (sms <= 0) return MX_ERR_CUDA;
  int32_t* status = dev_status ? dev_status : internal_status_ptr();
  if (!status) return MX_ERR_CUDA;
  mxk::GemmProblem p{qa, sfa, qb, sfb, d_bf16, nullptr, nullptr, status, m, n, k, 1, 0};
  return from_cuda(mxk::launch_gemm(p, sms, reinterpret_cast<cudaStream_t>(stream), nullptr));
}

mx_status mx_gemm_batch(const mx_gemm_problem* problems, int32_t count, int32_t* dev_status, mx_stream_t stream) {
  static_assert(MX_GEMM_BATCH_MAX == mxk::kMaxBatch, "batch limit");
  if (!problems || count < 1 || count > MX_GEMM_BATCH_MAX) return MX_ERR_INVALID_ARGUMENT;
  mxk::GemmProblem ps[MX_GEMM_BATCH_MAX];
  int32_t* status = nullptr;
  int n_live = 0;
  for (int32_t i = 0; i < count; ++i) {  // every problem checked before anything is launched
    const mx_gemm_problem& q = problems[i];
    if (q.m < 0 || q.n < 0 || q.k < 0) return MX_ERR_INVALID_ARGUMENT;
    if (q.m == 0 || q.n == 0) {
      if (q.k % 128 != 0 || q.k == 0 || q.n % 16 != 0) return MX_ERR_UNSUPPORTED_SHAPE;
      continue;
    }
    mx_status st = check_gemm_common(q.qa, q.sfa, q.qb, q.sfb, q.d_bf16, q.m, q.n, q.k, 1);
    if (st != MX_OK) return st;
    ++n_live;
  }
  if (n_live == 0) return MX_OK;
  const int sms = num_sms();
  if (sms <= 0) return MX_ERR_CUDA;
  status = dev_status ? dev_status : internal_status_ptr();
  if (!status) return MX_ERR_CUDA;
  int n = 0;
  for (int32_t i = 0; i < count; ++i) {
    const mx_gemm_problem& q = problems[i];
    if (q.m == 0 || q.n == 0) continue;
    ps[n++] = mxk::GemmProblem{q.qa, q.sfa, q.qb, q.sfb, q.d_bf16, nullptr, nullptr, status, q.m, q.n, q.k, 1, 0};
  }
  return from_cuda(mxk::launch_gemm_batch(ps, n, sms, reinterpret_cast<cudaStream_t>(stream), nullptr));
}

mx_status mx_grouped_gemm_contiguous(const void* qa, const void* sfa, const void* qb, const void* sfb,
                                     const int32_t* group_offsets, int32_t groups, int64_t m_total, int64_t n,
                                     int64_t k, void* d_bf16, int32_t* dev_status, mx_stream_t stream) {
  if (groups < 0 || m_total < 0 || n < 0 || k < 0) return MX_ERR_INVALID_ARGUMENT;
  if (k == 0 || k % 128 != 0 || n % 16 != 0) return MX_ERR_UNSUPPORTED_SHAPE;
  if (groups == 0 || m_total == 0 || n == 0) return MX_OK;
  if (!group_offsets) return MX_ERR_INVALID_ARGUMENT;
  mx_status st = check_gemm_common(qa, sfa, qb, sfb, d_bf16, m_total, n, k, groups);
  if (st != MX_OK) return st;
  if (reinterpret_cast<uintptr_t>(group_offsets) & 3u) return MX_ERR_MISALIGNED;
  const int sms = num_sms();
  if (sms <= 0) return MX_ERR_CUDA;
  int32_t* status = dev_status ? dev_status : internal_status_ptr();
  if (!status) return MX_ERR_CUDA;
  mxk::GemmProblem p{qa, sfa, qb, sfb, d_bf16, group_offsets, nullptr, status, m_total, n, k, groups, 1};
  return from_cuda(mxk::launch_gemm(p, sms, reinterpret_cast<cudaStream_t>(stream), nullptr));
}

mx_status mx_grouped_gemm_masked(const void* qa, const void* sfa, const void* qb, const void* sfb,
                                 const int32_t* masked_m, int32_t groups, int64_t max_m, int64_t n, int64_t k,
                                 void* d_bf16, int32_t* dev_status, mx_stream_t stream) {
  if (groups < 0 || max_m < 0 || n < 0 || k < 0) return MX_ERR_INVALID_ARGUMENT;
  if (k == 0 || k % 128 != 0 || n % 16 != 0) return MX_ERR_UNSUPPORTED_SHAPE;
  if (groups == 0 || max_m == 0 || n == 0) return MX_OK;
  if (!masked_m) return MX_ERR_INVALID_ARGUMENT;
  if (groups * max_m > kMaxDim) return MX_ERR_UNSUPPORTED_SHAPE;
  mx_status st = check_gemm_common(qa, sfa, qb, sfb, d_bf16, max_m, n, k, groups);
  if (st != MX_OK) return st;
  if (reinterpret_cast<uintptr_t>(masked_m) & 3u) return MX_ERR_MISALIGNED;
  const int sms = num_sms();
  if (sms <= 0) return MX_ERR_CUDA;
  int32_t* status = dev_status ? dev_status : internal_status_ptr();
  if (!status) return MX_ERR_CUDA;
  mxk::GemmProblem p{qa, sfa, qb, sfb, d_bf16, nullptr, masked_m, status, max_m, n, k, groups, 2};
  return from_cuda(mxk::launch_gemm(p, sms, reinterpret_cast<cudaStream_t>(stream), nullptr));
}

mx_status mx_grouped_gemm_kgrouped(const void* qa, const void* sfa, const void* qb, const void* sfb,
                                   const int32_t* group_offsets, int32_t groups, int64_t m, int64_t n,
                                   int64_t k_total, void* d_bf16, int32_t* dev_status, mx_stream_t stream) {
  if (groups < 0 || m < 0 || n < 0 || k_total < 0) return MX_ERR_INVALID_ARGUMENT;
  if (k_total == 0 || k_total % 128 != 0 || n % 16 != 0) return MX_ERR_UNSUPPORTED_SHAPE;
  if (groups == 0 || m == 0 || n == 0) return MX_OK;
  if (!group_offsets) return MX_ERR_INVALID_ARGUMENT;
  if (groups * m > kMaxDim) return MX_ERR_UNSUPPORTED_SHAPE;
  mx_status st = check_gemm_common(qa, sfa, qb, sfb, d_bf16, m, n, k_total, groups);
  if (st != MX_OK) return st;
  if (reinterpret_cast<uintptr_t>(group_offsets) & 3u) return MX_ERR_MISALIGNED;
  const int sms = num_sms();
  if (sms <= 0) return MX_ERR_CUDA;
  int32_t* status = dev_status ? dev_status : internal_status_ptr();
  if (!status) return MX_ERR_CUDA;
  mxk::GemmProblem p{qa, sfa, qb, sfb, d_bf16, group_offsets, nullptr, status, m, n, k_total, groups, 3};
  return from_cuda(mxk::launch_gemm(p, sms, reinterpret_cast<cudaStream_t>(stream), nullptr));
}

// ---------------------------------------------------------------- tile-wise FP32-scaled FP8

static mx_status tw_quantize(const void* x, int64_t rows, int64_t k, void* q, float* s, bool blocks,
                             mx_stream_t stream) {
  if (rows < 0 || k < 0) return MX_ERR_INVALID_ARGUMENT;
  if (k % 128 != 0) return MX_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0 || k == 0) return MX_OK;
  if (!x || !q || !s) return MX_ERR_INVALID_ARGUMENT;
  if (!aligned16(x) || !aligned16(q) || (reinterpret_cast<uintptr_t>(s) & 3u)) return MX_ERR_MISALIGNED;
  if (rows > kMaxDim || k > kMaxDim) return MX_ERR_UNSUPPORTED_SHAPE;
  // the 1 x 128 kernel numbers its (8 rows x 128 columns) items in 32 bits
  if ((rows + 7) / 8 * (k / 128) > 0xFFFFFFF0LL) return MX_ERR_UNSUPPORTED_SHAPE;
  return from_cuda(mxk::launch_tw_quant(x, rows, k, q, s, blocks, reinterpret_cast<cudaStream_t>(stream)));
}

mx_status mx_quantize_bf16_to_e4m3_tile1x128(const void* x_bf16, int64_t rows, int64_t k, void* q_e4m3,
                                             float* scales, mx_stream_t stream) {
  return tw_quantize(x_bf16, rows, k, q_e4m3, scales, false, stream);
}

mx_status mx_quantize_bf16_to_e4m3_block128x128(const void* x_bf16, int64_t rows, int64_t k, void* q_e4m3,
                                                float* scales, mx_stream_t stream) {
  return tw_quantize(x_bf16, rows, k, q_e4m3, scales, true, stream);
}

static mx_status tw_gemm(const void* qa, const float* sa, const void* qb, const float* sb,
                         const int32_t* group_offsets, int32_t groups, int64_t m, int64_t n, int64_t k, void* d,
                         int32_t* dev_status, int mode, mx_stream_t stream) {
  if (groups < 0 || m < 0 || n < 0 || k < 0) return MX_ERR_INVALID_ARGUMENT;
  if (k == 0 || k % 128 != 0 || n % 16 != 0) return MX_ERR_UNSUPPORTED_SHAPE;
  if (groups == 0 || m == 0 || n == 0) return MX_OK;
  if (!qa || !sa || !qb || !sb || !d || (mode == 1 && !group_offsets)) return MX_ERR_INVALID_ARGUMENT;
  if (!aligned16(qa) || !aligned16(qb) || !aligned16(d) || (reinterpret_cast<uintptr_t>(sa) & 3u) ||
      (reinterpret_cast<uintptr_t>(sb) & 3u) || (reinterpret_cast<uintptr_t>(group_offsets) & 3u))
    return MX_ERR_MISALIGNED;
  if (m > kMaxDim || n > kMaxDim || k > kMaxDim || groups > kMaxGroups) return MX_ERR_UNSUPPORTED_SHAPE;
  const int sms = num_sms();
  if (sms <= 0) return MX_ERR_CUDA;
  int32_t* status = dev_status ? dev_status : internal_status_ptr();
  if (!status) return MX_ERR_CUDA;
  mxk::TwProblem p{qa, sa, qb, sb, d, group_offsets, status, m, n, k, groups, mode};
  return from_cuda(mxk::launch_gemm_tw(p, sms, reinterpret_cast<cudaStream_t>(stream)));
}

mx_status mx_gemm_tilewise(const void* qa, const float* sa, const void* qb, const float* sb, void* d_bf16,
                           int64_t m, int64_t n, int64_t k, int32_t* dev_status, mx_stream_t stream) {
  return tw_gemm(qa, sa, qb, sb, nullptr, 1, m, n, k, d_bf16, dev_status, 0, stream);
}

mx_status mx_grouped_gemm_contiguous_tilewise(const void* qa, const float* sa, const void* qb, const float* sb,
                                              const int32_t* group_offsets, int32_t groups, int64_t m_total,
                                              int64_t n, int64_t k, void* d_bf16, int32_t* dev_status,
                                              mx_stream_t stream) {
  return tw_gemm(qa, sa, qb, sb, group_offsets, groups, m_total, n, k, d_bf16, dev_status, 1, stream);
}

// ---------------------------------------------------------------- fused SwiGLU + MXFP8 (expert MLP, first half)

static mx_status check_swiglu(const void* qh, const void* sfh, int64_t i_dim) {
  if (i_dim <= 0) return MX_ERR_INVALID_ARGUMENT;
  if (i_dim % 128 != 0 || 2 * i_dim > kMaxDim) return MX_ERR_UNSUPPORTED_SHAPE;
  if (!qh || !sfh) return MX_ERR_INVALID_ARGUMENT;
  if (!aligned16(qh) || !aligned16(sfh)) return MX_ERR_MISALIGNED;
  return MX_OK;
}

mx_status mx_gemm_swiglu_quant(const void* qa, const void* sfa, const void* qb, const void* sfb, void* qh,
                               void* sfh, int64_t m, int64_t i_dim, int64_t k, int32_t* dev_status,
                               mx_stream_t stream) {
  if (m < 0 || i_dim < 0 || k < 0) return MX_ERR_INVALID_ARGUMENT;
  if (k == 0 || k % 128 != 0) return MX_ERR_UNSUPPORTED_SHAPE;
  if (m == 0) return i_dim % 128 == 0 ? MX_OK : MX_ERR_UNSUPPORTED_SHAPE;
  mx_status st = check_swiglu(qh, sfh, i_dim);
  if (st != MX_OK) return st;
  st = check_gemm_common(qa, sfa, qb, sfb, qh, m, 2 * i_dim, k, 1);
  if (st != MX_OK) return st;
  const int sms = num_sms();
  if (sms <= 0) return MX_ERR_CUDA;
  int32_t* status = dev_status ? dev_status : internal_status_ptr();
  if (!status) return MX_ERR_CUDA;
  mxk::GemmProblem p{qa, sfa, qb, sfb, qh, nullptr, nullptr, status, m, 2 * i_dim, k, 1, 0};
  p.i_dim = i_dim;
  p.sf_out = sfh;
  return from_cuda(mxk::launch_gemm(p, sms, reinterpret_cast<cudaStream_t>(stream), nullptr));
}

mx_status mx_grouped_gemm_contiguous_swiglu_quant(const void* qa, const void* sfa, const void* qb, const void* sfb,
                                                  const int32_t* group_offsets, int32_t groups, int64_t m_total,
                                                  int64_t i_dim, int64_t k, void* qh, void* sfh,
                                                  int32_t* dev_status, mx_stream_t stream) {
  if (groups < 0 || m_total < 0 || i_dim < 0 || k < 0) return MX_ERR_INVALID_ARGUMENT;
  if (k == 0 || k % 128 != 0 || i_dim % 128 != 0) return MX_ERR_UNSUPPORTED_SHAPE;
  if (groups == 0 || m_total == 0 || i_dim == 0) return MX_OK;
  if (!group_offsets) return MX_ERR_INVALID_ARGUMENT;
  mx_status st = check_swiglu(qh, sfh, i_dim);
  if (st != MX_OK) return st;
  st = check_gemm_common(qa, sfa, qb, sfb, qh, m_total, 2 * i_dim, k, groups);
  if (st != MX_OK) return st;
  if (reinterpret_cast<uintptr_t>(group_offsets) & 3u) return MX_ERR_MISALIGNED;
  const int sms = num_sms();
  if (sms <= 0) return MX_ERR_CUDA;
  int32_t* status = dev_status ? dev_status : internal_status_ptr();
  if (!status) return MX_ERR_CUDA;
  mxk::GemmProblem p{qa, sfa, qb, sfb, qh, group_offsets, nullptr, status, m_total, 2 * i_dim, k, groups, 1};
  p.i_dim = i_dim;
  p.sf_out = sfh;
  return from_cuda(mxk::launch_gemm(p, sms, reinterpret_cast<cudaStream_t>(stream), nullptr));
}

mx_status mx_grouped_gemm_masked_swiglu_quant(const void* qa, const void* sfa, const void* qb, const void* sfb,
                                              const int32_t* masked_m, int32_t groups, int64_t max_m, int64_t i_dim,
                                              int64_t k, void* qh, void* sfh, int32_t* dev_status,
                                              mx_stream_t stream) {
  if (groups < 0 || max_m < 0 || i_dim < 0 || k < 0) return MX_ERR_INVALID_ARGUMENT;
  if (k == 0 || k % 128 != 0 || i_dim % 128 != 0) return MX_ERR_UNSUPPORTED_SHAPE;
  if (groups == 0 || max_m == 0 || i_dim == 0) return MX_OK;
  if (!masked_m) return MX_ERR_INVALID_ARGUMENT;
  if (groups * max_m > kMaxDim) return MX_ERR_UNSUPPORTED_SHAPE;
  mx_status st = check_swiglu(qh, sfh, i_dim);
  if (st != MX_OK) return st;
  st = check_gemm_common(qa, sfa, qb, sfb, qh, max_m, 2 * i_dim, k, groups);
  if (st != MX_OK) return st;
  if (reinterpret_cast<uintptr_t>(masked_m) & 3u) return MX_ERR_MISALIGNED;
  const int sms = num_sms();
  if (sms <= 0) return MX_ERR_CUDA;
  int32_t* status = dev_status ? dev_status : internal_status_ptr();
  if (!status) return MX_ERR_CUDA;
  mxk::GemmProblem p{qa, sfa, qb, sfb, qh, nullptr, masked_m, status, max_m, 2 * i_dim, k, groups, 2};
  p.i_dim = i_dim;
  p.sf_out = sfh;
  return from_cuda(mxk::launch_gemm(p, sms, reinterpret_cast<cudaStream_t>(stream), nullptr));
}

int64_t mx_moe_max_rows(int64_t n, int32_t experts, int32_t pad) {
  if (n < 0 || experts <= 0 || pad <= 0) return 0;
  const int64_t rows = n + static_cast<int64_t>(experts) * (pad - 1);
  return (rows + 127) / 128 * 128;
}

mx_status mx_moe_route(const int32_t* ids, int64_t n, int32_t experts, int32_t pad, int32_t* counts,
                       int32_t* offsets, int32_t* row, int32_t* dropped, mx_stream_t stream) {
  if (n < 0 || experts < 1 || experts > kMaxGroups || pad < 1 || pad > 128) return MX_ERR_INVALID_ARGUMENT;
  if (n > kMaxDim - 1024) return MX_ERR_UNSUPPORTED_SHAPE;
  if (!counts || !offsets || (n > 0 && (!ids || !row))) return MX_ERR_INVALID_ARGUMENT;
  if ((reinterpret_cast<uintptr_t>(ids) | reinterpret_cast<uintptr_t>(counts) | reinterpret_cast<uintptr_t>(offsets) |
       reinterpret_cast<uintptr_t>(row) | reinterpret_cast<uintptr_t>(dropped)) & 3u)
    return MX_ERR_MISALIGNED;
  return from_cuda(mxk::launch_moe_route(ids, n, experts, pad, counts, offsets, row, dropped,
                                         static_cast<cudaStream_t>(stream)));
}

static mx_status check_place(const void* src, int64_t n_src, int64_t k, const int32_t* row, int32_t fan,
                             const int32_t* counts, const int32_t* offsets, int32_t experts, int32_t pad,
                             int64_t m_rows, const void* q, const void* sf, bool tiled) {
  if (n_src < 0 || k < 0 || m_rows < 0 || fan < 1 || fan > 64 || pad < 1 || pad > 128 || experts < 0 ||
      experts > kMaxGroups)
    return MX_ERR_INVALID_ARGUMENT;
  if (k % 128 != 0 || (tiled && m_rows % 128 != 0)) return MX_ERR_UNSUPPORTED_SHAPE;
  if (k > kMaxDim || m_rows > kMaxDim || n_src > kMaxDim || n_src * static_cast<int64_t>(fan) > kMaxDim)
    return MX_ERR_UNSUPPORTED_SHAPE;
  if (pad > 1 && experts > 0 && (!counts || !offsets)) return MX_ERR_INVALID_ARGUMENT;
  if (k == 0 || (n_src == 0 && (pad == 1 || experts == 0))) return MX_OK;
  if (!q || !sf || (n_src > 0 && (!src || !row))) return MX_ERR_INVALID_ARGUMENT;
  if (!aligned16(src) || !aligned16(q) || !aligned16(sf)) return MX_ERR_MISALIGNED;
  return MX_OK;
}

mx_status mx_moe_dispatch_quant(const void* x_bf16, int64_t tokens, int64_t k, const int32_t* row, int32_t topk,
                                const int32_t* counts, const int32_t* offsets, int32_t experts, int32_t pad,
                                int64_t m_rows, void* q_e4m3, void* sf, int32_t sf_row_major,
                                int32_t* dev_status, mx_stream_t stream) {
  mx_status st = check_place(x_bf16, tokens, k, row, topk, counts, offsets, experts, pad, m_rows, q_e4m3, sf,
                             sf_row_major == 0);
  if (st != MX_OK) return st;
  if (k == 0 || (tokens == 0 && (pad == 1 || experts == 0))) return MX_OK;
  mxk::MoePlace p = {};
  p.src = x_bf16;
  p.row = row;
  p.counts = counts;
  p.offsets = offsets;
  p.q = q_e4m3;
  p.sf = sf;
  p.status = dev_status ? dev_status : internal_status_ptr();
  p.n_src = tokens;
  p.m_rows = m_rows;
  p.k = k;
  p.fan = topk;
  p.experts = experts;
  p.pad = pad;
  p.sf_row_major = sf_row_major != 0;
  p.quantize = true;
  return from_cuda(mxk::launch_moe_place(p, static_cast<cudaStream_t>(stream)));
}

mx_status mx_moe_scatter_rows(const void* q_src, const void* sf_src, int64_t n_src, int64_t k,
                              const int32_t* dst_row, const int32_t* counts, const int32_t* offsets,
                              int32_t experts, int32_t pad, int64_t m_rows, void* q_dst, void* sf_dst,
                              int32_t* dev_status, mx_stream_t stream) {
  mx_status st = check_place(q_src, n_src, k, dst_row, 1, counts, offsets, experts, pad, m_rows, q_dst, sf_dst, true);
  if (st != MX_OK) return st;
  if (k == 0 || (n_src == 0 && (pad == 1 || experts == 0))) return MX_OK;
  if (n_src > 0 && !sf_src) return MX_ERR_INVALID_ARGUMENT;
  mxk::MoePlace p = {};
  p.src = q_src;
  p.src_sf = sf_src;
  p.row = dst_row;
  p.counts = counts;
  p.offsets = offsets;
  p.q = q_dst;
  p.sf = sf_dst;
  p.status = dev_status ? dev_status : internal_status_ptr();
  p.n_src = n_src;
  p.m_rows = m_rows;
  p.k = k;
  p.fan = 1;
  p.experts = experts;
  p.pad = pad;
  p.sf_row_major = 0;
  p.quantize = false;
  return from_cuda(mxk::launch_moe_place(p, static_cast<cudaStream_t>(stream)));
}

mx_status mx_gather_rows(const void* src, int64_t src_rows, int64_t row_bytes, const int32_t* idx, int64_t n,
                         void* dst, int32_t* dev_status, mx_stream_t stream) {
  if (src_rows < 0 || row_bytes < 0 || n < 0) return MX_ERR_INVALID_ARGUMENT;
  if (row_bytes % 16 != 0) return MX_ERR_UNSUPPORTED_SHAPE;
  if (n > kMaxDim || src_rows > kMaxDim) return MX_ERR_UNSUPPORTED_SHAPE;
  if (n == 0 || row_bytes == 0) return MX_OK;
  if (!idx || !dst || (src_rows > 0 && !src)) return MX_ERR_INVALID_ARGUMENT;
  if (!aligned16(src) || !aligned16(dst)) return MX_ERR_MISALIGNED;
  int32_t* status = dev_status ? dev_status : internal_status_ptr();
  return from_cuda(mxk::launch_moe_gather(src, src_rows, row_bytes, idx, n, dst, status,
                                          static_cast<cudaStream_t>(stream)));
}

mx_status mx_moe_combine(const void* y_bf16, int64_t y_rows, int64_t n_cols, const int32_t* row, const float* w,
                         int64_t tokens, int32_t topk, void* out_bf16, int32_t* dev_status, mx_stream_t stream) {
  if (y_rows < 0 || n_cols < 0 || tokens < 0 || topk < 1 || topk > 64) return MX_ERR_INVALID_ARGUMENT;
  if (n_cols % 8 != 0) return MX_ERR_UNSUPPORTED_SHAPE;
  if (tokens > kMaxDim || y_rows > kMaxDim || tokens * static_cast<int64_t>(topk) > kMaxDim)
    return MX_ERR_UNSUPPORTED_SHAPE;
  if (tokens == 0 || n_cols == 0) return MX_OK;
  if (!row || !w || !out_bf16 || (y_rows > 0 && !y_bf16)) return MX_ERR_INVALID_ARGUMENT;
  if (!aligned16(y_bf16) || !aligned16(out_bf16) || (reinterpret_cast<uintptr_t>(w) & 3u) ||
      (reinterpret_cast<uintptr_t>(row) & 3u))
    return MX_ERR_MISALIGNED;
  int32_t* status = dev_status ? dev_status : internal_status_ptr();
  return from_cuda(mxk::launch_moe_combine(y_bf16, nullptr, nullptr, 0, y_rows, n_cols, row, w, tokens, topk,
                                           out_bf16, status, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ expert parallelism over peer memory

mx_status mx_moe_peer_plan(const int32_t* ids, const int32_t* row_send, int64_t n, const int32_t* count_table,
                           int32_t ranks, int32_t rank, int32_t experts, int32_t pad, int32_t* dst_rank,
                           int32_t* dst_row, int32_t* counts_local, int32_t* offsets_local, int32_t* dev_status,
                           mx_stream_t stream) {
  if (n < 0 || ranks < 1 || ranks > kMaxGroups || rank < 0 || rank >= ranks || experts < 1 ||
      experts > kMaxGroups || pad < 1 || pad > 128 || experts % ranks != 0)
    return MX_ERR_INVALID_ARGUMENT;
  // every entry of every rank plus each expert's padding: the largest row
  // index and padded offset the plan can produce must fit in int32
  if (n * static_cast<int64_t>(ranks) + static_cast<int64_t>(experts) * (pad - 1) > kMaxDim)
    return MX_ERR_UNSUPPORTED_SHAPE;
  if (!count_table || !counts_local || !offsets_local || (n > 0 && (!ids || !row_send || !dst_rank || !dst_row)))
    return MX_ERR_INVALID_ARGUMENT;
  if ((reinterpret_cast<uintptr_t>(ids) | reinterpret_cast<uintptr_t>(row_send) |
       reinterpret_cast<uintptr_t>(count_table) | reinterpret_cast<uintptr_t>(dst_rank) |
       reinterpret_cast<uintptr_t>(dst_row) | reinterpret_cast<uintptr_t>(counts_local) |
       reinterpret_cast<uintptr_t>(offsets_local)) & 3u)
    return MX_ERR_MISALIGNED;
  const int sms = num_sms();
  if (sms <= 0) return MX_ERR_CUDA;
  int32_t* status = dev_status ? dev_status : internal_status_ptr();
  if (!status) return MX_ERR_CUDA;
  return from_cuda(mxk::launch_moe_peer_plan(ids, row_send, n, count_table, ranks, rank, experts, pad, dst_rank,
                                             dst_row, counts_local, offsets_local, status, sms,
                                             static_cast<cudaStream_t>(stream)));
}

mx_status mx_moe_dispatch_quant_peer(const void* x_bf16, int64_t tokens, int64_t k, const int32_t* dst_rank,
                                     const int32_t* dst_row, int32_t topk, void* const* q_peers,
                                     void* const* sf_peers, int32_t ranks, int64_t m_rows, void* q_local,
                                     void* sf_local, const int32_t* counts_local, const int32_t* offsets_local,
                                     int32_t experts_local, int32_t pad, int32_t* dev_status, mx_stream_t stream) {
  if (ranks < 1 || ranks > kMaxGroups) return MX_ERR_INVALID_ARGUMENT;
  mx_status st = check_place(x_bf16, tokens, k, dst_row, topk, counts_local, offsets_local, experts_local, pad,
                             m_rows, q_local, sf_local, true);
  if (st != MX_OK) return st;
  if (k == 0 || (tokens == 0 && (pad == 1 || experts_local == 0))) return MX_OK;
  if (tokens > 0 && (!dst_rank || !q_peers || !sf_peers)) return MX_ERR_INVALID_ARGUMENT;
  if ((reinterpret_cast<uintptr_t>(q_peers) | reinterpret_cast<uintptr_t>(sf_peers)) & 7u ||
      (reinterpret_cast<uintptr_t>(dst_rank) & 3u))
    return MX_ERR_MISALIGNED;
  mxk::MoePlace p = {};
  p.src = x_bf16;
  p.row = dst_row;
  p.counts = counts_local;
  p.offsets = offsets_local;
  p.q = q_local;
  p.sf = sf_local;
  p.status = dev_status ? dev_status : internal_status_ptr();
  p.n_src = tokens;
  p.m_rows = m_rows;
  p.k = k;
  p.fan = topk;
  p.experts = experts_local;
  p.pad = pad;
  p.sf_row_major = 0;
  p.quantize = true;
  p.q_peers = q_peers;
  p.sf_peers = sf_peers;
  p.row_rank = dst_rank;
  p.ranks = ranks;
  return from_cuda(mxk::launch_moe_place(p, static_cast<cudaStream_t>(stream)));
}

mx_status mx_moe_combine_peer(const void* const* y_peers, int32_t ranks, int64_t y_rows, int64_t n_cols,
                              const int32_t* src_rank, const int32_t* src_row, const float* w, int64_t tokens,
                              int32_t topk, void* out_bf16, int32_t* dev_status, mx_stream_t stream) {
  if (ranks < 1 || ranks > kMaxGroups || y_rows < 0 || n_cols < 0 || tokens < 0 || topk < 1 || topk > 64)
    return MX_ERR_INVALID_ARGUMENT;
  if (n_cols % 8 != 0) return MX_ERR_UNSUPPORTED_SHAPE;
  if (tokens > kMaxDim || y_rows > kMaxDim || tokens * static_cast<int64_t>(topk) > kMaxDim)
    return MX_ERR_UNSUPPORTED_SHAPE;
  if (tokens == 0 || n_cols == 0) return MX_OK;
  if (!y_peers || !src_rank || !src_row || !w || !out_bf16) return MX_ERR_INVALID_ARGUMENT;
  if (!aligned16(out_bf16) || (reinterpret_cast<uintptr_t>(y_peers) & 7u) ||
      ((reinterpret_cast<uintptr_t>(w) | reinterpret_cast<uintptr_t>(src_rank) |
        reinterpret_cast<uintptr_t>(src_row)) & 3u))
    return MX_ERR_MISALIGNED;
  int32_t* status = dev_status ? dev_status : internal_status_ptr();
  return from_cuda(mxk::launch_moe_combine(nullptr, y_peers, src_rank, ranks, y_rows, n_cols, src_row, w, tokens,
                                           topk, out_bf16, status, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ 16-bit products

// Row and tile numbers of the 16-bit kernels are 32-bit, with room for a tile
// behind the last row.
constexpr int64_t kMaxDim16 = (int64_t(1) << 31) - 1024;
// What one tile sums over: 2^27 take about a second on a pair of SMs, and a wait
// for an accumulator may take two (mx_set_wait_limit_ns).
constexpr int64_t kMaxSum16 = int64_t(1) << 27;

static bool dtype16(int32_t t) { return t == MX_BF16 || t == MX_FP16; }

static bool misaligned16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned16(p)) return true;
  return false;
}

// Device and status word of a call that launches.
static mx_status launch_context(int32_t* dev_status, int* sms, int32_t** status) {
  *sms = num_sms();
  if (*sms <= 0) return MX_ERR_CUDA;
  *status = dev_status ? dev_status : internal_status_ptr();
  return *status ? MX_OK : MX_ERR_CUDA;
}

static mx_status zero_bytes(void* p, int64_t bytes, mx_stream_t stream) {
  return from_cuda(cudaMemsetAsync(p, 0, static_cast<size_t>(bytes), static_cast<cudaStream_t>(stream)));
}

// A dense product of row-major tensors: D [m, n] = A B^T with A [m, k] (a_mn: [k, m]), B [n, k] (b_mn: [k, n]).
static mxk::Gemm16 dense16(const void* a, int a_mn, const void* b, int b_mn, void* d, int64_t m, int64_t n, int64_t k,
                           int32_t dtype, int32_t* status) {
  mxk::Gemm16 g = {};
  g.a = a;
  g.a_mn = a_mn;
  g.a_ld = a_mn ? m : k;
  g.a_batch = m * k;
  g.b = b;
  g.b_mn = b_mn;
  g.b_ld = b_mn ? n : k;
  g.b_batch = n * k;
  g.d = d;
  g.d_ld = n;
  g.d_batch = m * n;
  g.m = m;
  g.n = n;
  g.k = k;
  g.groups = 1;
  g.op_fp16 = dtype == MX_FP16;
  g.out_type = dtype;
  g.status = status;
  return g;
}

static mx_status check_linear(int64_t m, int64_t n, int64_t k, int32_t dtype, int32_t act) {
  if (m < 0 || n < 0 || k < 0 || !dtype16(dtype) || act < MX_ACT_NONE || act > MX_ACT_GELU_TANH)
    return MX_ERR_INVALID_ARGUMENT;
  if (k == 0 || k % 8 != 0 || n % 8 != 0 || m > kMaxDim16 || n > kMaxDim16 || k > kMaxSum16)
    return MX_ERR_UNSUPPORTED_SHAPE;
  return MX_OK;
}

mx_status mx_linear_act(const void* x, const void* w, const void* bias, const void* residual, void* z, void* y,
                        int64_t m, int64_t n, int64_t k, int32_t dtype, int32_t act, int32_t* dev_status,
                        mx_stream_t stream) {
  mx_status st = check_linear(m, n, k, dtype, act);
  if (st != MX_OK || m == 0 || n == 0) return st;
  if (!x || !w || !y) return MX_ERR_INVALID_ARGUMENT;
  if (misaligned16({x, w, bias, residual, z, y})) return MX_ERR_MISALIGNED;
  int sms;
  int32_t* status;
  st = launch_context(dev_status, &sms, &status);
  if (st != MX_OK) return st;
  mxk::Gemm16 g = dense16(x, 0, w, 0, y, m, n, k, dtype, status);
  g.epi = bias || residual || z || act != MX_ACT_NONE ? 1 : 0;
  g.bias = bias;
  g.res = residual;
  g.res_ld = n;
  g.res_batch = m * n;
  g.z = z;
  g.act = act;
  return from_cuda(mxk::launch_gemm16(g, sms, static_cast<cudaStream_t>(stream)));
}

size_t mx_linear_act_backward_workspace_bytes(int64_t m, int64_t n) {
  if (m <= 0 || n <= 0) return 0;
  const int64_t chunks = mxk::act_backward_chunks(m);
  return chunks == 1 ? 0 : static_cast<size_t>(chunks * n) * sizeof(float);
}

mx_status mx_linear_act_backward(const void* dy, const void* z, const void* x, const void* w, void* dz, void* dx,
                                 void* dw, void* dbias, int64_t m, int64_t n, int64_t k, int32_t dtype, int32_t act,
                                 void* workspace, size_t workspace_bytes, int32_t* dev_status, mx_stream_t stream) {
  mx_status st = check_linear(m, n, k, dtype, act);
  if (st != MX_OK) return st;
  if ((dx && n > kMaxSum16) || (dw && m > kMaxSum16)) return MX_ERR_UNSUPPORTED_SHAPE;
  if (misaligned16({dy, z, x, w, dz, dx, dw, dbias, workspace})) return MX_ERR_MISALIGNED;
  if (m == 0 || n == 0) {  // empty sums
    if (m > 0 && dx) return zero_bytes(dx, m * k * 2, stream);
    if (n > 0 && dw) st = zero_bytes(dw, n * k * 2, stream);
    if (st == MX_OK && n > 0 && dbias) st = zero_bytes(dbias, n * 2, stream);
    return st;
  }
  if (!dy || (dx && !w) || (dw && !x) || (act != MX_ACT_NONE && (!z || !dz))) return MX_ERR_INVALID_ARGUMENT;
  const size_t needed = dbias ? mx_linear_act_backward_workspace_bytes(m, n) : 0;
  if (needed > 0 && (!workspace || workspace_bytes < needed)) return MX_ERR_INVALID_ARGUMENT;
  if (!dx && !dw && !dbias) return MX_OK;
  int sms;
  int32_t* status;
  st = launch_context(dev_status, &sms, &status);
  if (st != MX_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (act != MX_ACT_NONE || dbias)
    e = mxk::launch_act_backward(dy, z, dz, dbias, static_cast<float*>(workspace), m, n, act, dtype == MX_FP16, s);
  const void* g = act != MX_ACT_NONE ? dz : dy;
  const mxk::Gemm16 gx = dense16(g, 0, w, 1, dx, m, k, n, dtype, status);
  const mxk::Gemm16 gw = dense16(g, 1, x, 1, dw, n, k, m, dtype, status);
  if (e == cudaSuccess && dx && dw) {
    e = mxk::launch_gemm16_two(gx, gw, sms, s);
  } else {
    if (e == cudaSuccess && dx) e = mxk::launch_gemm16(gx, sms, s);
    if (e == cudaSuccess && dw) e = mxk::launch_gemm16(gw, sms, s);
  }
  return from_cuda(e);
}

static mx_status check_ragged(const void* a, const void* b, const int32_t* group_offsets, int32_t groups,
                              int64_t m_total, int64_t n, int64_t k, int64_t summed, int32_t dtype, const void* d,
                              bool* empty) {
  *empty = false;
  if (groups < 0 || m_total < 0 || n < 0 || k < 0 || !dtype16(dtype)) return MX_ERR_INVALID_ARGUMENT;
  if (n == 0 || k == 0 || n % 8 != 0 || k % 8 != 0 || n > kMaxDim16 || k > kMaxDim16 || m_total > kMaxDim16 ||
      groups > kMaxGroups || summed > kMaxSum16)
    return MX_ERR_UNSUPPORTED_SHAPE;
  if (groups == 0 || m_total == 0) {
    *empty = true;
    return MX_OK;
  }
  if (!a || !b || !d || !group_offsets) return MX_ERR_INVALID_ARGUMENT;
  if (misaligned16({a, b, d}) || (reinterpret_cast<uintptr_t>(group_offsets) & 3u)) return MX_ERR_MISALIGNED;
  return MX_OK;
}

mx_status mx_grouped_gemm_ragged(const void* a, const void* b, const int32_t* group_offsets, int32_t groups,
                                 int64_t m_total, int64_t n, int64_t k, int32_t dtype, void* d, int32_t* dev_status,
                                 mx_stream_t stream) {
  bool empty;
  mx_status st = check_ragged(a, b, group_offsets, groups, m_total, n, k, k, dtype, d, &empty);
  if (st != MX_OK || empty) return st;
  int sms;
  int32_t* status;
  st = launch_context(dev_status, &sms, &status);
  if (st != MX_OK) return st;
  mxk::Gemm16 g = dense16(a, 0, b, 0, d, m_total, n, k, dtype, status);
  g.mode = 1;
  g.groups = groups;
  g.group_offsets = group_offsets;
  return from_cuda(mxk::launch_gemm16(g, sms, static_cast<cudaStream_t>(stream)));
}

mx_status mx_grouped_gemm_ragged_dgrad(const void* dd, const void* b, const int32_t* group_offsets, int32_t groups,
                                       int64_t m_total, int64_t n, int64_t k, int32_t dtype, void* da,
                                       int32_t* dev_status, mx_stream_t stream) {
  bool empty;
  mx_status st = check_ragged(dd, b, group_offsets, groups, m_total, n, k, n, dtype, da, &empty);
  if (st != MX_OK || empty) return st;
  int sms;
  int32_t* status;
  st = launch_context(dev_status, &sms, &status);
  if (st != MX_OK) return st;
  mxk::Gemm16 g = dense16(dd, 0, b, 1, da, m_total, k, n, dtype, status);
  g.mode = 1;
  g.groups = groups;
  g.group_offsets = group_offsets;
  return from_cuda(mxk::launch_gemm16(g, sms, static_cast<cudaStream_t>(stream)));
}

mx_status mx_grouped_gemm_ragged_wgrad(const void* dd, const void* a, const int32_t* group_offsets, int32_t groups,
                                       int64_t m_total, int64_t n, int64_t k, int32_t dtype, int32_t out_dtype,
                                       void* db, int32_t* dev_status, mx_stream_t stream) {
  if (out_dtype != dtype && out_dtype != MX_FP32) return MX_ERR_INVALID_ARGUMENT;
  bool empty;
  mx_status st = check_ragged(dd, a, group_offsets, groups, m_total, n, k, m_total, dtype, db, &empty);
  if (st != MX_OK) return st;
  if (empty) {
    if (groups == 0) return MX_OK;
    if (!db) return MX_ERR_INVALID_ARGUMENT;
    if (!aligned16(db)) return MX_ERR_MISALIGNED;
    return zero_bytes(db, groups * n * k * (out_dtype == MX_FP32 ? 4 : 2), stream);
  }
  int sms;
  int32_t* status;
  st = launch_context(dev_status, &sms, &status);
  if (st != MX_OK) return st;
  mxk::Gemm16 g = dense16(dd, 1, a, 1, db, n, k, m_total, dtype, status);
  g.mode = 2;
  g.groups = groups;
  g.group_offsets = group_offsets;
  g.out_type = out_dtype;
  return from_cuda(mxk::launch_gemm16(g, sms, static_cast<cudaStream_t>(stream)));
}

// Do the steps keep every matrix inside FP16's range?  The singular values lie
// in [0, u]; their next bound is the largest |a s + b s^3 + c s^5| there, and the
// entries of A, B and a I + B are at most the largest |s^2|, |b s^2 + c s^4| and
// |a + b s^2 + c s^4| (of symmetric matrices no entry exceeds the norm).
static bool ns_coefficients_fit(const float* coeffs, int steps) {
  double u = 1.0;
  for (int i = 0; i < steps; ++i) {
    const double a = coeffs[3 * i], b = coeffs[3 * i + 1], c = coeffs[3 * i + 2];
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return false;
    double largest = 0.0, poly = 0.0;
    auto look = [&](double t) {  // t = s^2
      if (!(t >= 0.0 && t <= u * u)) return;
      const double q = b * t + c * t * t;
      largest = std::fmax(largest, std::fabs((a + q) * std::sqrt(t)));
      poly = std::fmax(poly, std::fmax(std::fabs(q), std::fabs(a + q)));
    };
    look(0.0);
    look(u * u);
    if (c != 0.0) {
      look(-b / (2.0 * c));                       // extremum of b t + c t^2
      const double disc = 9.0 * b * b - 20.0 * a * c;  // of the odd quintic: 5 c t^2 + 3 b t + a = 0
      if (disc >= 0.0) {
        look((-3.0 * b + std::sqrt(disc)) / (10.0 * c));
        look((-3.0 * b - std::sqrt(disc)) / (10.0 * c));
      }
    } else if (b != 0.0) {
      look(-a / (3.0 * b));
    }
    if (poly > 15.5) return false;
    u = 1.01 * largest;  // room for the roundings
    if (!(u <= 3.9)) return false;
    if (u == 0.0) u = 1e-3;
  }
  return true;
}

size_t mx_orthogonalize_workspace_bytes(int64_t batch, int64_t m, int64_t n, int32_t g_dtype, int32_t steps) {
  if (batch <= 0 || m <= 0 || n <= 0 || steps <= 0 || batch > 65535 || m > (int64_t(1) << 20) || n > (int64_t(1) << 20))
    return 0;
  return mxk::ns_workspace_bytes(batch, m, n, g_dtype == MX_FP32, steps);
}

mx_status mx_orthogonalize(const void* g, int32_t g_dtype, void* out_bf16, int64_t batch, int64_t m, int64_t n,
                           int32_t steps, const float* coeffs, float eps, void* workspace, size_t workspace_bytes,
                           int32_t* dev_status, mx_stream_t stream) {
  if (batch < 0 || m < 0 || n < 0 || (g_dtype != MX_BF16 && g_dtype != MX_FP32) || steps < 1 || steps > 16 || !coeffs ||
      !(eps >= 0.0f) || !std::isfinite(eps) || !ns_coefficients_fit(coeffs, steps))
    return MX_ERR_INVALID_ARGUMENT;
  if (batch > 65535 || m > (int64_t(1) << 20) || n > (int64_t(1) << 20)) return MX_ERR_UNSUPPORTED_SHAPE;
  if (batch == 0 || m == 0 || n == 0) return MX_OK;
  if (!g || !out_bf16 || !workspace) return MX_ERR_INVALID_ARGUMENT;
  if (misaligned16({g, out_bf16}) || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return MX_ERR_MISALIGNED;
  if (workspace_bytes < mxk::ns_workspace_bytes(batch, m, n, g_dtype == MX_FP32, steps)) return MX_ERR_INVALID_ARGUMENT;
  int sms;
  int32_t* status;
  mx_status st = launch_context(dev_status, &sms, &status);
  if (st != MX_OK) return st;
  mxk::OrthoProblem q{g, out_bf16, workspace, status, coeffs, batch, m, n, steps, eps, g_dtype == MX_FP32};
  return from_cuda(mxk::launch_orthogonalize(q, sms, static_cast<cudaStream_t>(stream)));
}

mx_status mx_set_wait_limit_ns(uint64_t ns) {
  g_wait_ns.store(ns == 0 ? kDefaultWaitNs : ns, std::memory_order_relaxed);
  return MX_OK;
}

uint64_t mx_wait_limit_ns(void) { return g_wait_ns.load(std::memory_order_relaxed); }

mx_status mx_read_internal_status(int32_t* host_out, int clear) {
  if (!host_out) return MX_ERR_INVALID_ARGUMENT;
  if (cudaDeviceSynchronize() != cudaSuccess) return MX_ERR_CUDA;
  if (cudaMemcpyFromSymbol(host_out, g_internal_status, sizeof(int32_t)) != cudaSuccess) return MX_ERR_CUDA;
  if (clear) {
    const int32_t zero = 0;
    if (cudaMemcpyToSymbol(g_internal_status, &zero, sizeof(int32_t)) != cudaSuccess) return MX_ERR_CUDA;
  }
  return MX_OK;
}

}  // extern "C"
