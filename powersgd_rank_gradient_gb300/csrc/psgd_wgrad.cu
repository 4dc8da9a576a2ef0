// The weight gradient of a linear layer from its input's 8-bit checkpoint.
//
//   dW[o, i] = [dW +] sum over rows t of grad[t, o] x[t, i],   x = codes * scales
//
// The checkpoint is restored to the gradient's type in the handle's memory (in
// bf16 exactly: 4 significant bits times a power of two), and the product runs
// on the tensor cores with both operands as they lie, the summed dimension being
// the rows (psgd_gemm.cu).  Products of 16-bit values are exact in fp32 and the sums
// fp32, so a bucket in fp32 gets an fp32 gradient.
#include <algorithm>
#include <new>
#include <type_traits>

#include "psgd_mma.cuh"

struct psgd_wgrad {
  int device = 0, pairs = 0;
  long long outs = 0, ins = 0, most = 0;
  long long op = 0, ip = 0;         // row strides: multiples of 8 elements
  void* x = nullptr;                // most x ip, the checkpoint restored
  void* g = nullptr;                // most x op, a gradient that TMA cannot read in place
  float* slots = nullptr;
  int* error = nullptr;
  size_t bytes = 0;
};

using namespace psgd;
using namespace psgd::ops;

namespace {

constexpr long long kMostRows = 1 << 24;

// Rows of any stride into rows of `to` words: a CTA takes runs of 2048 words of a row, eight words a thread under way.
template <typename W> __global__ void __launch_bounds__(256) k_align(const W* src, long long stride, long long rows, int cols, W* dst, long long to, int runs) {
  after_previous();
  next_may_launch();
  for (long long i = blockIdx.x; i < rows * runs; i += gridDim.x) {
    const long long r = runs == 1 ? i : i / runs;
    const int first = (int)(i - r * runs) * 2048 + threadIdx.x;
    const W* s = src + r * stride;
    W* d = dst + r * to;
    W x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (first + 256 * k < cols) x[k] = s[first + 256 * k];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (first + 256 * k < cols) d[first + 256 * k] = x[k];
  }
}

}  // namespace

cudaError_t psgd::mma::align_rows(const void* src, long long stride, long long rows, long long cols, void* dst, long long to, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  const auto go = [&](auto* w, int by) {
    using W = std::remove_pointer_t<decltype(w)>;
    const long long runs = units(cols / by, 2048);
    return launch_early(k_align<W>, (unsigned)std::min<long long>(rows * runs, 152 * 16), 256, 0, 1, st, (const W*)src, stride / by, rows,
                        (int)(cols / by), (W*)dst, to / by, (int)runs);
  };
  // two elements at a time where all rows begin and end between words of two
  if ((uintptr_t)src % 4 == 0 && stride % 2 == 0 && cols % 2 == 0) return go((uint32_t*)nullptr, 2);
  return go((uint16_t*)nullptr, 1);
}

extern "C" int psgd_wgrad_create(int64_t outs, int64_t ins, int64_t max_rows, int32_t device, psgd_wgrad** out) {
  const std::string who = "psgd_wgrad_create";
  if (!out) return fail(PSGD_EINVAL, who + ": out is NULL");
  *out = nullptr;
  if (outs < 1 || outs > (1 << 20) || ins < 1 || ins > (1 << 20)) return fail(PSGD_EINVAL, who + ": features must be in [1, 2^20]");
  if (max_rows < 0 || max_rows > kMostRows) return fail(PSGD_EINVAL, who + ": max_rows must be in [0, 2^24]");
  if (device < 0 || device >= 64) return fail(PSGD_EINVAL, who + ": device ordinal must be in [0, 63]");
  int count = 0;
  cudaError_t e = cudaGetDeviceCount(&count);
  if (e != cudaSuccess) return cuda_fail("psgd_wgrad_create: cudaGetDeviceCount", e);
  if (device >= count) return fail(PSGD_ECUDA, who + ": no such device");
  psgd_wgrad* h = new (std::nothrow) psgd_wgrad;
  if (!h) return fail(PSGD_ENOMEM, who + ": out of host memory");
  DeviceScope scope(device);
  h->device = device;
  h->outs = outs;
  h->ins = ins;
  h->most = max_rows;
  h->op = units(outs, 8) * 8;
  h->ip = units(ins, 8) * 8;
  e = mma::pairs_of(device, &h->pairs);
  const auto get = [&](auto** p, long long bytes) {
    bytes = std::max(bytes, 16LL);
    if (e == cudaSuccess) e = cudaMalloc((void**)p, bytes);
    if (e == cudaSuccess) h->bytes += bytes;
    else *p = nullptr;
  };
  get(&h->x, max_rows * h->ip * 2);
  get(&h->g, max_rows * h->op * 2);
  get(&h->slots, 2 * h->pairs * mma::kSlotFloats * 4);
  get(&h->error, 4);
  if (e == cudaSuccess) e = cudaMemset(h->error, 0, 4);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    const int rc = cuda_fail(who.c_str(), e);
    psgd_wgrad_destroy(h);
    return rc;
  }
  *out = h;
  return PSGD_OK;
}

extern "C" void psgd_wgrad_destroy(psgd_wgrad* h) {
  if (!h) return;
  {
    DeviceScope scope(h->device);
    cudaFree(h->x);
    cudaFree(h->g);
    cudaFree(h->slots);
    cudaFree(h->error);
  }
  delete h;
}

extern "C" size_t psgd_wgrad_workspace_bytes(const psgd_wgrad* h) { return h ? h->bytes : 0; }

extern "C" int psgd_wgrad_backward(psgd_wgrad* h, const void* grad, psgd_dtype dtype, int64_t grad_stride, int64_t rows,
                                   const void* codes, psgd_code code, const float* scales, void* dweight,
                                   psgd_dtype dweight_dtype, int64_t dweight_stride, int32_t accumulate, void* stream) {
  const std::string who = "psgd_wgrad_backward";
  if (!h) return fail(PSGD_EINVAL, who + ": NULL handle");
  if (dtype != PSGD_F16 && dtype != PSGD_BF16) return fail(PSGD_EINVAL, who + ": the gradient must be float16 or bfloat16");
  if (!dtype_ok(dweight_dtype)) return fail(PSGD_EINVAL, who + ": unknown dtype");
  if (code != PSGD_E4M3 && code != PSGD_E5M2) return fail(PSGD_EINVAL, who + ": unknown 8-bit format");
  if (rows < 0 || rows > h->most) return fail(PSGD_EINVAL, who + ": rows must be in [0, max_rows]");
  if (rows > 0 && (!grad || !codes || !scales)) return fail(PSGD_EINVAL, who + ": NULL operand");
  if (!dweight) return fail(PSGD_EINVAL, who + ": dweight is NULL");
  if (!span_ok(rows, grad_stride) || !span_ok(h->outs, dweight_stride)) return fail(PSGD_EINVAL, who + ": bad row stride");
  if (h->outs > 1 && dweight_stride < h->ins) return fail(PSGD_EINVAL, who + ": dweight's rows overlap");
  const long long wb = extent(h->outs, h->ins, dweight_stride, dweight_dtype);
  if (overlap(dweight, wb, grad, extent(rows, h->outs, grad_stride, dtype)) || overlap(dweight, wb, codes, rows * h->ins) ||
      overlap(dweight, wb, scales, rows * units(h->ins, 128) * 4))
    return fail(PSGD_EINVAL, who + ": dweight overlaps another operand");
  DeviceScope scope(h->device);
  const cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  if (rows > 0) {
    const int rc = psgd_activation_restore(codes, code, scales, rows, h->ins, h->x, dtype, h->ip, h->device, stream);
    if (rc) return rc;
    if (rows == 1 && aligned16(grad)) grad_stride = h->op;  // of one row no stride counts
    if (!mma::in_place(grad, grad_stride, h->outs)) {
      e = mma::align_rows(grad, grad_stride, rows, h->outs, h->g, h->op, st);
      grad = h->g;
      grad_stride = h->op;
    }
  } else {
    grad = h->g;
    grad_stride = h->op;
  }
  mma::Product p{};
  const bool bf16 = dtype == PSGD_BF16;
  if (e == cudaSuccess) e = mma::make_map(&p.a, grad, rows, h->outs, grad_stride, mma::box_rows(true), bf16);
  if (e == cudaSuccess) e = mma::make_map(&p.b, h->x, rows, h->ins, h->ip, mma::box_rows(true), bf16);
  if (e != cudaSuccess) return cuda_fail(who.c_str(), e);
  p.m = (int)h->outs, p.n = (int)h->ins, p.k = (int)rows;
  p.a_m_rows = p.b_m_rows = 1;
  p.bf16 = bf16;
  p.error = h->error;
  p.out = dweight, p.ldo = dweight_stride, p.dtype = dweight_dtype, p.accumulate = accumulate != 0;
  p.slots = h->slots;
  p.chunk = mma::chunk_of(rows, dweight_dtype);
  e = mma::enqueue(mma::kOut, p, h->device, h->pairs, st);
  return e == cudaSuccess ? PSGD_OK : cuda_fail(who.c_str(), e);
}

// Reads and clears a handle's error word.
int psgd::mma::take_error(const char* who, int* error, int device, void* stream) {
  DeviceScope scope(device);
  const cudaStream_t st = (cudaStream_t)stream;
  int bad = 0;
  cudaError_t e = cudaMemcpyAsync(&bad, error, 4, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaMemsetAsync(error, 0, 4, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(who, e);
  return bad ? fail(PSGD_ETIMEOUT, std::string(who) + ": a wait on the GPU gave up; results since the last status are not valid") : PSGD_OK;
}

extern "C" int psgd_wgrad_status(psgd_wgrad* h, void* stream) {
  if (!h) return fail(PSGD_EINVAL, "psgd_wgrad_status: NULL handle");
  return mma::take_error("psgd_wgrad_status", h->error, h->device, stream);
}
