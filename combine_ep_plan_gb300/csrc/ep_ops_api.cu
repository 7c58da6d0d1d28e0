// ep_ops_api.cu — the C ABI of the operators around the plan: argument checks
// and launches.  Host code, and the status word that products without a
// handle report to, with the kernel that takes errors out of it.
#include <climits>
#include <cstdint>
#include <mutex>

#include "ep_experts.h"
#include "ep_internal.cuh"

namespace {

// The errors recorded on a device, and the one that is being reported.
__device__ unsigned g_ops_status[2];

struct TakeDev {
  unsigned* status;
  unsigned* taken;
};

// Takes the error to report, and only it, out of the status word.  One atomic:
// bits that products on other streams set meanwhile stay for the next report.
__global__ void ep_take_status_kernel(TakeDev d) {
  ep::pdl_wait();
  const unsigned seen = *static_cast<volatile unsigned*>(d.status);
  const unsigned report = seen & ep::kStTimeout ? ep::kStTimeout : seen & ep::kStCapacity;
  *d.taken = report != 0 ? atomicAnd(d.status, ~report) & report : 0u;
}

constexpr unsigned long long kDefaultWaitNs = 2000000000ull;
unsigned long long g_wait_ns = kDefaultWaitNs;
int g_suppress = 0;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

ep_status_t cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return EP_OK;
  if (e == cudaErrorMemoryAllocation) return EP_ERR_OOM;
  return EP_ERR_CUDA;
}

bool float_type(ep_dtype_t t) { return t == EP_DTYPE_BF16 || t == EP_DTYPE_F32; }
size_t size_of(ep_dtype_t t) { return t == EP_DTYPE_F32 ? 4 : 2; }
cudaStream_t cu(ep_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

bool route_shape(int64_t T, int E, int K, int64_t ld, int score, int flags, float scale) {
  if (T < 0 || T > INT32_MAX || E < 1 || E > EP_MAX_EXPERTS || K < 1 || K > EP_MAX_TOPK || K > E || ld < E) return false;
  if (score != EP_SCORE_SOFTMAX && score != EP_SCORE_SIGMOID) return false;
  return (flags & ~EP_ROUTE_RENORMALIZE) == 0 && scale == scale;
}

// The device address of the library's status word, or NULL.
unsigned* ops_status() {
  void* p = nullptr;
  return cudaGetSymbolAddress(&p, g_ops_status) == cudaSuccess ? static_cast<unsigned*>(p) : nullptr;
}

ep_status_t check_matmul(const int8_t* a, const float* a_scales, int64_t a_rows, const int8_t* w, const float* w_scales,
                         int E, int64_t N, int64_t K, const int32_t* offsets, const int32_t* rows, ep_dtype_t out_dtype,
                         void* out, int64_t out_rows) {
  if (E < 1 || E > EP_MAX_EXPERTS || N < 1 || N > EP_MAX_MATMUL_DIM || K < 16 || K > EP_MAX_MATMUL_DIM || K % 16 != 0)
    return EP_ERR_INVALID;
  if (a_rows < 0 || a_rows >= INT32_MAX || out_rows < 0 || out_rows >= INT32_MAX) return EP_ERR_INVALID;
  if (!float_type(out_dtype) || !w || !w_scales || (E > 1 && !offsets)) return EP_ERR_INVALID;
  if (!rows && out_rows > a_rows) return EP_ERR_INVALID;
  if (!aligned(w, 16) || !aligned(w_scales, 4) || !aligned(offsets, 4) || !aligned(rows, 4)) return EP_ERR_INVALID;
  if (out_rows > 0 && (!out || !aligned(out, 16))) return EP_ERR_INVALID;
  if (a_rows > 0 && (!a || !a_scales || !aligned(a, 16) || !aligned(a_scales, 4))) return EP_ERR_INVALID;
  return EP_OK;
}

ep_status_t run_matmul(const int8_t* a, const float* a_scales, int64_t a_rows, const int8_t* w, const float* w_scales,
                       int E, int64_t N, int64_t K, const int32_t* offsets, const int32_t* rows, ep_dtype_t out_dtype,
                       void* out, int64_t out_rows, unsigned* status, cudaStream_t stream) {
  if (out_rows == 0) return EP_OK;
  ep::MatmulDev d;
  d.a = a;
  d.a_scale = a_scales;
  d.w = w;
  d.w_scale = w_scales;
  d.offsets = offsets;
  d.rows = rows;
  d.out = out;
  d.status = status;
  d.a_rows = a_rows;
  d.out_rows = out_rows;
  d.E = E;
  d.N = static_cast<int>(N);
  d.K = static_cast<int>(K);
  d.wait_ns = g_wait_ns;
  d.suppress = g_suppress;
  return cuda_status(ep::launch_matmul(d, out_dtype == EP_DTYPE_BF16, stream));
}

}  // namespace

extern "C" {

ep_status_t ep_route(const void* logits, ep_dtype_t dtype, int64_t T, int E, int64_t ld, int K, ep_score_t score,
                     const float* bias, int G, int TG, int flags, float scale, int64_t* topk_idx, float* topk_weights,
                     ep_stream_t stream) {
  if (!float_type(dtype) || !route_shape(T, E, K, ld, score, flags, scale)) return EP_ERR_INVALID;
  if (G < 1 || G > EP_MAX_GROUPS || E % G != 0 || TG < 1 || TG > G) return EP_ERR_INVALID;
  if (T == 0) return EP_OK;
  if (!logits || !topk_idx || !topk_weights || !aligned(logits, size_of(dtype)) || !aligned(bias, 4) ||
      !aligned(topk_idx, 8) || !aligned(topk_weights, 4))
    return EP_ERR_INVALID;
  ep::RouteDev d;
  d.logits = logits;
  d.bias = bias;
  d.topk_idx = topk_idx;
  d.topk_weights = topk_weights;
  d.T = T;
  d.ld = ld;
  d.E = E;
  d.K = K;
  d.G = G == TG ? 1 : G;  // all groups kept: no groups
  d.TG = G == TG ? 1 : TG;
  const unsigned per = static_cast<unsigned>(E / d.G);
  d.per_magic = per > 1 ? static_cast<unsigned>((0x100000000ull + per - 1) / per) : 0u;
  d.sigmoid = score == EP_SCORE_SIGMOID;
  d.renorm = (flags & EP_ROUTE_RENORMALIZE) != 0;
  d.vec = ld % 4 == 0 && aligned(logits, 4 * size_of(dtype));
  d.vec_bias = aligned(bias, 16);
  d.scale = scale;
  return cuda_status(ep::launch_route(d, dtype == EP_DTYPE_BF16, cu(stream)));
}

ep_status_t ep_route_backward(const void* logits, ep_dtype_t dtype, int64_t T, int E, int64_t ld, int K,
                              ep_score_t score, int flags, float scale, const int64_t* topk_idx,
                              const float* grad_weights, void* grad_logits, ep_stream_t stream) {
  if (!float_type(dtype) || !route_shape(T, E, K, ld, score, flags, scale)) return EP_ERR_INVALID;
  if (T == 0) return EP_OK;
  if (!logits || !topk_idx || !grad_weights || !grad_logits || !aligned(logits, size_of(dtype)) ||
      !aligned(topk_idx, 8) || !aligned(grad_weights, 4) || !aligned(grad_logits, size_of(dtype)))
    return EP_ERR_INVALID;
  ep::RouteBwdDev d;
  d.logits = logits;
  d.topk_idx = topk_idx;
  d.grad_weights = grad_weights;
  d.grad_logits = grad_logits;
  d.T = T;
  d.ld = ld;
  d.E = E;
  d.K = K;
  d.sigmoid = score == EP_SCORE_SIGMOID;
  d.renorm = (flags & EP_ROUTE_RENORMALIZE) != 0;
  d.vec = ld % 4 == 0 && aligned(logits, 4 * size_of(dtype));
  d.vec_out = E % 4 == 0 && aligned(grad_logits, 4 * size_of(dtype));
  d.scale = scale;
  return cuda_status(ep::launch_route_backward(d, dtype == EP_DTYPE_BF16, cu(stream)));
}

ep_status_t ep_quantize_int8(const void* x, ep_dtype_t dtype, int64_t rows, int64_t width, int64_t ld, int gated,
                             const int32_t* num_rows, int8_t* codes, float* scales, ep_stream_t stream) {
  if (!float_type(dtype) || rows < 0 || rows > INT32_MAX || width < 8 || width > EP_MAX_MATMUL_DIM || width % 8 != 0)
    return EP_ERR_INVALID;
  const int64_t per_piece = 16 / static_cast<int64_t>(size_of(dtype));
  if (ld < (gated ? 2 * width : width) || ld % per_piece != 0) return EP_ERR_INVALID;
  if (rows == 0) return EP_OK;
  if (!x || !codes || !scales || !aligned(x, 16) || !aligned(codes, 8) || !aligned(scales, 4) || !aligned(num_rows, 4))
    return EP_ERR_INVALID;
  ep::QuantDev d;
  d.x = x;
  d.num_rows = num_rows;
  d.codes = codes;
  d.scales = scales;
  d.rows = rows;
  d.ld = ld;
  d.F = static_cast<int>(width);
  return cuda_status(ep::launch_quantize(d, dtype == EP_DTYPE_BF16, gated != 0, cu(stream)));
}

ep_status_t ep_matmul_int8(const int8_t* a, const float* a_scales, int64_t a_rows, const int8_t* w,
                           const float* w_scales, int E, int64_t N, int64_t K, const int32_t* offsets,
                           const int32_t* rows, ep_dtype_t out_dtype, void* out, int64_t out_rows,
                           ep_stream_t stream) {
  const ep_status_t st = check_matmul(a, a_scales, a_rows, w, w_scales, E, N, K, offsets, rows, out_dtype, out, out_rows);
  if (st != EP_OK) return st;
  unsigned* status = ops_status();
  if (!status) return EP_ERR_CUDA;
  return run_matmul(a, a_scales, a_rows, w, w_scales, E, N, K, offsets, rows, out_dtype, out, out_rows, status,
                    cu(stream));
}

ep_status_t ep_expert_matmul_int8(ep_handle_t h, const int8_t* a, const float* a_scales, int64_t a_rows, const int8_t* w,
                                  const float* w_scales, int64_t N, int64_t K, int gather, ep_dtype_t out_dtype,
                                  void* out, int64_t out_rows, ep_stream_t stream) {
  if (!h) return EP_ERR_INVALID;
  int E = 0;
  const void *offsets = nullptr, *rows = nullptr;
  int64_t shape[3] = {0, 0, 0};
  int nd = 0;
  ep_status_t st = ep_handle_info(h, nullptr, nullptr, nullptr, &E, nullptr, nullptr);
  if (st == EP_OK) st = ep_handle_get(h, EP_FIELD_EXPERT_OFFSETS, &offsets, shape, &nd);
  if (st == EP_OK && gather) {
    st = ep_handle_get(h, EP_FIELD_EXP_SRC, &rows, shape, &nd);
    if (st == EP_OK && out_rows > shape[0]) return EP_ERR_INVALID;
  }
  if (st != EP_OK) return st;
  st = check_matmul(a, a_scales, a_rows, w, w_scales, E, N, K, static_cast<const int32_t*>(offsets),
                    static_cast<const int32_t*>(rows), out_dtype, out, out_rows);
  if (st != EP_OK) return st;
  return run_matmul(a, a_scales, a_rows, w, w_scales, E, N, K, static_cast<const int32_t*>(offsets),
                    static_cast<const int32_t*>(rows), out_dtype, out, out_rows, ep::handle_status(h), cu(stream));
}

ep_status_t ep_matmul_status(ep_stream_t stream) {
  unsigned* p = ops_status();
  if (!p) return EP_ERR_CUDA;
  cudaError_t e = cudaStreamSynchronize(cu(stream));
  if (e != cudaSuccess) return cuda_status(e);
  static std::mutex one;  // the reported word is one per device
  const std::lock_guard<std::mutex> lock(one);
  unsigned st = 0;
  e = ep::launch_pdl(ep_take_status_kernel, 1, 1, cu(stream), TakeDev{p, p + 1});
  if (e == cudaSuccess) e = cudaMemcpyAsync(&st, p + 1, sizeof st, cudaMemcpyDeviceToHost, cu(stream));
  if (e == cudaSuccess) e = cudaStreamSynchronize(cu(stream));
  if (e != cudaSuccess) return cuda_status(e);
  if (st & ep::kStTimeout) return EP_ERR_TIMEOUT;
  if (st & ep::kStCapacity) return EP_ERR_CAPACITY;
  return EP_OK;
}

void ep_debug_set_matmul_wait(int64_t limit_us, int suppress) {
  g_wait_ns = limit_us > 0 ? static_cast<unsigned long long>(limit_us) * 1000ull : kDefaultWaitNs;
  g_suppress = suppress;
}

}  // extern "C"
