// The weight gradient of a linear layer from its input's 8-bit checkpoint.
//
//   dW[o, i] = [dW +] sum over rows t of grad[t, o] x[t, i],   x = codes * scales
//
// The checkpoint is restored to the gradient's type in the handle's memory (in
// bf16 exactly: 4 significant bits times a power of two), and the product runs
// on the tensor cores with both operands as they lie, the summed dimension being
// the rows (psgd_gemm.cu).  Products of 16-bit values are exact in fp32 and the sums
// fp32, taken out of the tensor cores where they are long, so a bucket in fp32 gets an fp32 gradient.
#include <algorithm>
#include <new>
#include <type_traits>

#include "psgd_mma.cuh"

struct psgd_wgrad {
  int device = 0, pairs = 0;
  long long outs = 0, ins = 0, most = 0;
  long long ip = 0;                 // row stride of x: a multiple of 8 elements
  long long copied = 0, gp = 0;     // columns that g holds, a multiple of 256 or all; its row stride, a multiple of 8
  void* x = nullptr;                // most x ip, the checkpoint restored
  void* g = nullptr;                // most x gp, a piece of a gradient that TMA cannot read in place
  float* slots = nullptr;
  int* error = nullptr;
  size_t bytes = 0;
};

using namespace psgd;
using namespace psgd::ops;

namespace {

constexpr long long kMostRows = 1 << 24;
// Of a gradient that TMA cannot read in place.  Rows of whole 16-byte units seldom need it (16384 x 6400 x 1600 in pieces of
// 32 MB 462 us, whole 323, read in place 226), others mostly do (32768 x 6399 x 256 in two pieces 300 us, whole 274).
constexpr long long kCopyBytes = 32LL << 20, kOddCopyBytes = 512LL << 20;

// Rows of any stride into rows of `to` words: a CTA takes runs of 2048 words of a row, eight words a thread under way (a
// weight gradient from 4961 x 5114 43 us, with four 42, with sixteen 40; from 16384 x 1001 31, 31 and 39).
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
  h->ip = units(ins, 8) * 8;
  // equal pieces of whole tiles
  const long long tiles = units(outs, mma::kTile);
  const long long fit = std::max(1LL, (outs % 8 ? kOddCopyBytes : kCopyBytes) / (std::max<long long>(max_rows, 1) * mma::kTile * 2));
  h->copied = std::min<long long>(outs, units(tiles, units(tiles, fit)) * mma::kTile);
  h->gp = units(h->copied, 8) * 8;
  e = mma::pairs_of(device, &h->pairs);
  const auto get = [&](auto** p, long long bytes) {
    bytes = std::max(bytes, 16LL);
    if (e == cudaSuccess) e = cudaMalloc((void**)p, bytes);
    if (e == cudaSuccess) h->bytes += bytes;
    else *p = nullptr;
  };
  get(&h->x, max_rows * h->ip * 2);
  get(&h->g, max_rows * h->gp * 2);
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
  long long piece = h->outs;  // columns of the gradient that a product takes
  bool copy = false;
  if (rows > 0) {
    const int rc = psgd_activation_restore(codes, code, scales, rows, h->ins, h->x, dtype, h->ip, h->device, stream);
    if (rc) return rc;
    if (rows == 1 && aligned16(grad)) grad_stride = units(h->outs, 8) * 8;  // of one row no stride counts
    copy = !mma::in_place(grad, grad_stride, h->outs);
    if (copy) piece = h->copied;
  } else {  // (a map needs an address, which nothing is read from)
    grad = h->x;
    grad_stride = units(h->outs, 8) * 8;
  }
  mma::Product p{};
  p.bf16 = dtype == PSGD_BF16;
  p.n = (int)h->ins, p.k = (int)rows;
  p.a_m_rows = p.b_m_rows = 1;
  p.error = h->error;
  p.ldo = dweight_stride, p.dtype = dweight_dtype, p.accumulate = accumulate != 0;
  p.slots = h->slots;
  p.chunk = mma::chunk_of(rows, dweight_dtype);
  cudaError_t e = mma::make_map(&p.b, h->x, rows, h->ins, h->ip, mma::box_rows(true), p.bf16);
  for (long long first = 0; first < h->outs && e == cudaSuccess; first += piece) {
    const long long n = std::min(piece, h->outs - first);
    const void* from = (const char*)grad + first * 2;
    if (copy) {
      e = mma::align_rows(from, grad_stride, rows, n, h->g, h->gp, st);
      from = h->g;
    }
    if (e == cudaSuccess) e = mma::make_map(&p.a, from, rows, n, copy ? h->gp : grad_stride, mma::box_rows(true), p.bf16);
    p.m = (int)n;
    p.out = (char*)dweight + first * dweight_stride * dtype_size(dweight_dtype);
    if (e == cudaSuccess) e = mma::enqueue(mma::kOut, p, h->device, h->pairs, st);
  }
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
