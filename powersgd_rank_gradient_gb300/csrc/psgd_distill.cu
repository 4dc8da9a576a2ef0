// Distillation from a teacher's top logits: per-row losses, and the gradient
// of the logits in the same call.
//
//   p_k  = softmax over the row's valid entries of t_k / T      (valid: 0 <= i_k < V)
//   q    = softmax(z / T) over the vocabulary
//   loss = w T^2 sum_k p_k (log p_k - log q[i_k])
//   dz_j = c w T (q_j - sum over k with i_k = j of p_k)
//
// The softmax keeps a running maximum and sum in fp32 per thread, joined over
// the CTA.  A row without a weight (w = 0) or without a valid entry of finite
// mass has loss 0 and gradient 0 whatever its logits hold; they are not read.
#include <algorithm>

#include "psgd_ops.cuh"

namespace psgd {
namespace ops {
namespace {

constexpr int kDistillThreads = 512;
constexpr int kDistillWarps = kDistillThreads / 32;

struct DistillArgs {
  const void* z;
  long long zs;
  const void* t;
  long long ts;
  const void* index;
  long long is;
  const float* weights;
  void* dz;
  long long dzs;
  float* losses;
  long long rows;
  int vocab, k;
  int tdtype, index64;
  float temperature, scale;
};

__device__ __forceinline__ float block_max(float v, float* buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_max(v);
  __syncthreads();
  if (lane == 0) buf[warp] = v;
  __syncthreads();
  v = buf[0];
  for (int w = 1; w < kDistillWarps; ++w) v = fmaxf(v, buf[w]);
  return v;
}
__device__ __forceinline__ float block_sum(float v, float* buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_sum(v);
  __syncthreads();
  if (lane == 0) buf[warp] = v;
  __syncthreads();
  v = 0.f;
  for (int w = 0; w < kDistillWarps; ++w) v += buf[w];
  return v;
}

// One CTA per row; the logits are read twice.
template <typename Z> __global__ void __launch_bounds__(kDistillThreads) k_distill(DistillArgs a) {
  __shared__ float buf[kDistillWarps];
  __shared__ float p[PSGD_DISTILL_MAX_K];
  __shared__ int at[PSGD_DISTILL_MAX_K];
  const int tid = threadIdx.x;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const Z* z = (const Z*)a.z + row * a.zs;
    Z* dz = a.dz ? (Z*)a.dz + row * a.dzs : nullptr;
    const float w = a.weights ? __ldg(a.weights + row) : 1.f;
    const float inv_t = 1.f / a.temperature;
    __syncthreads();
    // the teacher's entries: validity, then their softmax
    float m = -INFINITY;
    bool mass = false;
    for (int k = tid; k < a.k; k += kDistillThreads) {
      const long long i = a.index64 ? __ldg((const long long*)a.index + row * a.is + k)
                                    : (long long)__ldg((const int*)a.index + row * a.is + k);
      const bool valid = i >= 0 && i < a.vocab;
      const float t = valid ? load_any(a.t, a.tdtype, row * a.ts + k) * inv_t : -INFINITY;
      at[k] = valid ? (int)i : -1;
      p[k] = t;
      m = fmaxf(m, t);
      mass |= t != -INFINITY;
    }
    const bool live = __syncthreads_or(mass) && w != 0.f;
    if (!live) {
      if (tid == 0) a.losses[row] = 0.f;
      if (dz)
        for (int j = tid; j < a.vocab; j += kDistillThreads) dz[j] = from_f<Z>(0.f);
      continue;
    }
    m = block_max(m, buf);
    float s = 0.f;
    for (int k = tid; k < a.k; k += kDistillThreads) {
      const float e = at[k] >= 0 ? expf(p[k] - m) : 0.f;
      p[k] = e;
      s += e;
    }
    const float inv_p = 1.f / block_sum(s, buf);
    for (int k = tid; k < a.k; k += kDistillThreads) p[k] *= inv_p;
    // the student's maximum and sum
    const float c = inv_t * 1.4426950408889634f;
    float zm = -INFINITY, zs = 0.f;
    for (int j = tid; j < a.vocab; j += kDistillThreads) {
      const float v = to_f(z[j]);
      if (v > zm) {
        zs *= exp2f((zm - v) * c);
        zm = v;
      }
      zs += exp2f((v - (zm == -INFINITY ? 0.f : zm)) * c);
    }
    const float top = block_max(zm, buf);
    const float base = top == -INFINITY ? 0.f : top;
    zs = block_sum(zs * exp2f((zm - base) * c), buf);
    const float logz = logf(zs);
    float part = 0.f;
    for (int k = tid; k < a.k; k += kDistillThreads)
      if (at[k] >= 0 && !(p[k] == 0.f)) part += p[k] * (logf(p[k]) - ((to_f(z[at[k]]) - base) * inv_t - logz));
    part = block_sum(part, buf);
    if (tid == 0) a.losses[row] = w * (a.temperature * a.temperature) * part;
    if (!dz) continue;
    const float f = w * a.temperature * a.scale, fq = f / zs;
    // dz may be z itself: the targets' logits are read before any is written
    float target[PSGD_DISTILL_MAX_K / kDistillThreads];
#pragma unroll
    for (int n = 0; n < PSGD_DISTILL_MAX_K / kDistillThreads; ++n) {
      const int k = tid + n * kDistillThreads;
      target[n] = 0.f;
      if (k < a.k && at[k] >= 0) {
        float sum = 0.f;
        for (int o = 0; o < a.k; ++o)
          if (at[o] == at[k]) sum += p[o];
        target[n] = exp2f((to_f(z[at[k]]) - base) * c) * fq - sum * f;
      }
    }
    __syncthreads();
    for (int j = tid; j < a.vocab; j += kDistillThreads) dz[j] = from_f<Z>(exp2f((to_f(z[j]) - base) * c) * fq);
    __syncthreads();
#pragma unroll
    for (int n = 0; n < PSGD_DISTILL_MAX_K / kDistillThreads; ++n) {
      const int k = tid + n * kDistillThreads;
      if (k < a.k && at[k] >= 0) dz[at[k]] = from_f<Z>(target[n]);
    }
  }
}

}  // namespace
}  // namespace ops
}  // namespace psgd

using namespace psgd;
using namespace psgd::ops;

extern "C" int psgd_distill(const void* logits, psgd_dtype dtype, int64_t logits_stride, int64_t rows, int64_t vocab,
                            const void* teacher, psgd_dtype teacher_dtype, int64_t teacher_stride, const void* index,
                            int32_t index_bits, int64_t index_stride, int32_t k, float temperature,
                            const float* weights, float grad_scale, float* losses, void* dlogits,
                            int64_t dlogits_stride, void* stream) {
  const char* who = "psgd_distill";
  if (!dtype_ok(dtype) || !dtype_ok(teacher_dtype)) return fail(PSGD_EINVAL, "psgd_distill: unknown dtype");
  if (index_bits != 32 && index_bits != 64) return fail(PSGD_EINVAL, "psgd_distill: index_bits must be 32 or 64");
  if (rows < 0 || rows > 0x7fffffff) return fail(PSGD_EINVAL, "psgd_distill: rows must be in [0, 2^31 - 1]");
  if (vocab < 1 || vocab > (1 << 30)) return fail(PSGD_EINVAL, "psgd_distill: vocab must be in [1, 2^30]");
  if (k < 1 || k > PSGD_DISTILL_MAX_K) return fail(PSGD_EINVAL, "psgd_distill: k must be in [1, PSGD_DISTILL_MAX_K]");
  if (!(temperature > 0.f) || !isfinite(temperature))
    return fail(PSGD_EINVAL, "psgd_distill: temperature must be finite and > 0");
  if (rows == 0) return PSGD_OK;
  if (!logits || !teacher || !index || !losses) return fail(PSGD_EINVAL, "psgd_distill: NULL pointer");
  if (!span_ok(rows, logits_stride) || !span_ok(rows, teacher_stride) || !span_ok(rows, index_stride) ||
      (dlogits && !span_ok(rows, dlogits_stride)))
    return fail(PSGD_EINVAL, "psgd_distill: bad row stride");
  if (dlogits && rows > 1 && dlogits_stride < vocab) return fail(PSGD_EINVAL, "psgd_distill: dlogits: rows overlap");
  const long long zb = extent(rows, vocab, logits_stride, dtype), tb = extent(rows, k, teacher_stride, teacher_dtype);
  const long long ib = ((rows - 1) * index_stride + k) * (index_bits / 8);
  const long long db = dlogits ? extent(rows, vocab, dlogits_stride, dtype) : 0;
  const bool in_place = dlogits == logits && dlogits_stride == logits_stride;
  if ((!in_place && overlap(dlogits, db, logits, zb)) || overlap(dlogits, db, teacher, tb) ||
      overlap(dlogits, db, index, ib) || overlap(dlogits, db, weights, rows * 4) ||
      overlap(dlogits, db, losses, rows * 4) || overlap(losses, rows * 4, logits, zb) ||
      overlap(losses, rows * 4, teacher, tb) || overlap(losses, rows * 4, index, ib) ||
      overlap(losses, rows * 4, weights, rows * 4))
    return fail(PSGD_EINVAL, "psgd_distill: an output overlaps another operand (dlogits may be logits itself)");
  DistillArgs a{logits, logits_stride, teacher, teacher_stride, index, index_stride, weights, dlogits, dlogits_stride,
                losses, rows, (int)vocab, k, (int)teacher_dtype, index_bits == 64, temperature, grad_scale};
  const unsigned grid = (unsigned)rows;
  const cudaStream_t st = (cudaStream_t)stream;
  if (dtype == PSGD_F32) k_distill<float><<<grid, kDistillThreads, 0, st>>>(a);
  else if (dtype == PSGD_F16) k_distill<__half><<<grid, kDistillThreads, 0, st>>>(a);
  else k_distill<__nv_bfloat16><<<grid, kDistillThreads, 0, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? PSGD_OK : cuda_fail(who, e);
}
