// Distillation from a teacher's top logits: per-row losses, and the gradient
// of the logits in the same call.
//
//   p_k  = softmax over the row's valid entries of t_k / T      (valid: 0 <= i_k < V)
//   q    = softmax(z / T) over the vocabulary
//   loss = w T^2 sum_k p_k (log p_k - log q[i_k])
//   dz_j = c w T (q_j - sum over k with i_k = j of p_k)
//
// A row's logits are read once: the CTAs of a cluster hold it in shared memory
// between the softmax's sums and the gradient.  The softmax keeps a running
// maximum and sum in fp32 per thread, joined over the warps and then over the
// cluster.  A row without a weight (w = 0) or without a valid entry of finite
// mass has loss 0 and gradient 0 whatever its logits hold; they are not read.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "psgd_ops.cuh"

namespace cg = cooperative_groups;

namespace psgd {
namespace ops {
namespace {

constexpr int kDistillThreads = 512;
constexpr int kDistillWarps = kDistillThreads / 32;
constexpr int kMaxCluster = 8;           // CTAs of a row
constexpr int kHalfSmem = 104 * 1024;    // of a row in one CTA, two of which fit an SM beside their static arrays
constexpr int kFullSmem = 212 * 1024;    // of a row in one CTA, alone on its SM

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

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Sums or maxima over a CTA of any whole number of warps, returned to all of
// its threads; `buf` holds one float a warp.
__device__ __forceinline__ float block_max(float v, float* buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  v = warp_max(v);
  __syncthreads();
  if (lane == 0) buf[warp] = v;
  __syncthreads();
  return warp_max(lane < warps ? buf[lane] : -INFINITY);
}
__device__ __forceinline__ float block_sum(float v, float* buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  v = warp_sum(v);
  __syncthreads();
  if (lane == 0) buf[warp] = v;
  __syncthreads();
  return warp_sum(lane < warps ? buf[lane] : 0.f);
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

// Everything below works in powers of two: with c = log2(e) / T the softmax is
// 2^((z_j - r) c) over its sum, r the largest logit.  The difference comes
// first: c z_j - c r in one fused operation would leave c r's rounding error in
// the exponent, which is without bound for masks of the type's lowest value.
//
// The teacher's entries of one row: validity (at[k], -1 where not), and their
// softmax p[k].  Returns whether the row counts at all.
__device__ __forceinline__ bool teacher_softmax(const DistillArgs& a, long long row, float w, float* p, int* at,
                                                float* buf) {
  const float inv_t = 1.f / a.temperature;
  float m = -INFINITY;
  bool mass = false;
  for (int k = threadIdx.x; k < a.k; k += blockDim.x) {
    const long long i = a.index64 ? __ldg((const long long*)a.index + row * a.is + k)
                                  : (long long)__ldg((const int*)a.index + row * a.is + k);
    const bool valid = i >= 0 && i < a.vocab;
    const float t = valid ? load_any(a.t, a.tdtype, row * a.ts + k) * inv_t : -INFINITY;
    at[k] = valid ? (int)i : -1;
    p[k] = t;
    m = fmaxf(m, t);
    mass |= t != -INFINITY;
  }
  if (!__syncthreads_or(mass) || w == 0.f) return false;
  m = block_max(m, buf);
  float s = 0.f;
  for (int k = threadIdx.x; k < a.k; k += blockDim.x) {
    const float e = at[k] >= 0 ? expf(p[k] - m) : 0.f;
    p[k] = e;
    s += e;
  }
  const float inv_p = 1.f / block_sum(s, buf);
  for (int k = threadIdx.x; k < a.k; k += blockDim.x) p[k] *= inv_p;
  __syncthreads();
  return true;
}

// p_k's sum over the entries that name the same element as entry k.
__device__ __forceinline__ float mass_at(const float* p, const int* at, int n, int k) {
  float sum = 0.f;
  for (int o = 0; o < n; ++o)
    if (at[o] == at[k]) sum += p[o];
  return sum;
}

// A 16-byte granule of a row as floats.
template <typename Z> __device__ __forceinline__ void unpack(const uint4& u, float* f) {
  const Z* v = reinterpret_cast<const Z*>(&u);
#pragma unroll
  for (int i = 0; i < Vec16<Z>::N; ++i) f[i] = to_f(v[i]);
}

// One cluster per row; CTA r of C holds the row's granules [r n / C, (r + 1) n / C)
// in shared memory, n the number of aligned 16-byte granules that the row
// touches (its first and last may be shared with the neighbouring rows).
// ALIGNED: the gradient's rows start at the same place of a granule as the
// logits' do, so whole granules are stored.
template <typename Z, bool ALIGNED>
__global__ void __launch_bounds__(kDistillThreads, 2) k_distill_chip(DistillArgs a, int ctas) {
  constexpr int NE = Vec16<Z>::N;
  constexpr int U = 4;  // granules in flight per thread
  extern __shared__ uint4 slice[];
  __shared__ float buf[kDistillWarps], bufs[kDistillWarps], bufp[kDistillWarps];
  __shared__ float p[PSGD_DISTILL_MAX_K];
  __shared__ int at[PSGD_DISTILL_MAX_K];
  __shared__ float2 peers[kMaxCluster];
  __shared__ float parts[kMaxCluster];
  const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = threads >> 5;
  const long long row = blockIdx.x / ctas;
  const int rank = blockIdx.x - (int)row * ctas;
  const Z* z = (const Z*)a.z + row * a.zs;
  Z* dz = a.dz ? (Z*)a.dz + row * a.dzs : nullptr;
  const int head = (int)(((uintptr_t)z & 15) / sizeof(Z));  // elements of the first granule before the row
  const int granules = (head + a.vocab + NE - 1) / NE;
  const int g0 = (int)((long long)granules * rank / ctas), g1 = (int)((long long)granules * (rank + 1) / ctas);
  const float w = a.weights ? __ldg(a.weights + row) : 1.f;
  if (ctas > 1) cluster_arrive();  // a peer's shared memory is written once all have started
  const bool live = teacher_softmax(a, row, w, p, at, buf);

  auto store = [&](int g, const float* f) {
    const int j0 = g * NE - head;
    if (ALIGNED && j0 >= 0 && j0 + NE <= a.vocab) {
      store_pack<Z, NE>(dz + j0, f);
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (j0 + i >= 0 && j0 + i < a.vocab) dz[j0 + i] = from_f<Z>(f[i]);
    }
  };

  if (!live) {  // the same for every CTA of the cluster
    if (rank == 0 && tid == 0) a.losses[row] = 0.f;
    if (dz) {
      float zero[NE];
#pragma unroll
      for (int i = 0; i < NE; ++i) zero[i] = 0.f;
      for (int g = g0 + tid; g < g1; g += threads) store(g, zero);
    }
    if (ctas > 1) cluster_wait();
    return;
  }

  const float c = kLog2e / a.temperature;
  float r = -INFINITY, s = 0.f;
  for (int g = g0 + tid; g < g1; g += threads * U) {
    uint4 v[U];
#pragma unroll
    for (int n = 0; n < U; ++n) {
      const int gg = g + n * threads;
      const int j0 = gg * NE - head;
      if (gg < g1 && j0 >= 0 && j0 + NE <= a.vocab) {
        v[n] = *reinterpret_cast<const uint4*>(z + j0);
      } else {
        Z* e = reinterpret_cast<Z*>(&v[n]);
#pragma unroll
        for (int i = 0; i < NE; ++i)
          e[i] = gg < g1 && j0 + i >= 0 && j0 + i < a.vocab ? z[j0 + i] : from_f<Z>(-INFINITY);
      }
    }
    float top = -INFINITY;
#pragma unroll
    for (int n = 0; n < U; ++n) {
      if (g + n * threads < g1) slice[g + n * threads - g0] = v[n];
      float f[NE];
      unpack<Z>(v[n], f);
#pragma unroll
      for (int i = 0; i < NE; ++i) top = fmaxf(top, f[i]);
    }
    if (top > r) {
      s *= exp2_fast((r - top) * c);
      r = top;
    }
    const float base = r == -INFINITY ? 0.f : r;
#pragma unroll
    for (int n = 0; n < U; ++n) {
      float f[NE];
      unpack<Z>(v[n], f);
#pragma unroll
      for (int i = 0; i < NE; ++i) s += exp2_fast((f[i] - base) * c);
    }
  }
  // over the warp, the CTA, the cluster
  auto shifted = [c](float s, float r, float to) { return r == -INFINITY ? s : s * exp2_fast((r - to) * c); };
  float top = warp_max(r);
  s = warp_sum(shifted(s, r, top));
  if (lane == 0) {
    buf[warp] = top;
    bufs[warp] = s;
  }
  __syncthreads();
  r = lane < warps ? buf[lane] : -INFINITY;
  s = lane < warps ? bufs[lane] : 0.f;
  top = warp_max(r);
  s = warp_sum(shifted(s, r, top));
  if (ctas > 1) {
    cg::cluster_group cluster = cg::this_cluster();
    cluster_wait();
    if (tid < ctas) *cluster.map_shared_rank(&peers[rank], tid) = make_float2(top, s);
    cluster.sync();
    r = lane < ctas ? peers[lane].x : -INFINITY;
    s = lane < ctas ? peers[lane].y : 0.f;
    top = warp_max(r);
    s = warp_sum(shifted(s, r, top));
  }
  const float base = top == -INFINITY ? 0.f : top;
  const float log2_s = log2f(s);
  const float f = w * a.temperature * a.scale, fq = f / s;
  // the entries that fall into this CTA's slice: their part of the loss, and their gradients
  const Z* held = reinterpret_cast<const Z*>(slice) + head - (long long)g0 * NE;
  float part = 0.f;
  for (int k = tid; k < a.k; k += threads) {
    const int j = at[k];
    const bool mine = j >= 0 && (j + head) / NE >= g0 && (j + head) / NE < g1;
    if (mine) {
      const float x = (to_f(held[j]) - base) * c;
      if (!(p[k] == 0.f)) part += p[k] * (logf(p[k]) - kLn2 * (x - log2_s));
    }
  }
  part = warp_sum(part);
  if (lane == 0) bufp[warp] = part;
  if (dz) {
    for (int g = g0 + tid; g < g1; g += threads) {
      float q[NE];
      unpack<Z>(slice[g - g0], q);
#pragma unroll
      for (int i = 0; i < NE; ++i) q[i] = exp2_fast((q[i] - base) * c) * fq;
      store(g, q);
    }
  }
  __syncthreads();
  if (dz) {
    for (int k = tid; k < a.k; k += threads) {
      const int j = at[k];
      if (j >= 0 && (j + head) / NE >= g0 && (j + head) / NE < g1)
        dz[j] = from_f<Z>(exp2_fast((to_f(held[j]) - base) * c) * fq - mass_at(p, at, a.k, k) * f);
    }
  }
  part = 0.f;
  if (tid == 0)
    for (int v = 0; v < warps; ++v) part += bufp[v];
  if (ctas > 1) {
    cg::cluster_group cluster = cg::this_cluster();
    if (tid == 0) *cluster.map_shared_rank(&parts[rank], 0) = part;
    cluster.sync();
    if (rank == 0 && tid == 0) {
      part = 0.f;
      for (int v = 0; v < ctas; ++v) part += parts[v];
    }
  }
  if (rank == 0 && tid == 0) a.losses[row] = w * (a.temperature * a.temperature) * part;
}

// Rows larger than a cluster's shared memory: one CTA per row, which reads the
// logits twice.
template <typename Z> __global__ void __launch_bounds__(kDistillThreads) k_distill_long(DistillArgs a) {
  __shared__ float buf[kDistillWarps];
  __shared__ float p[PSGD_DISTILL_MAX_K];
  __shared__ int at[PSGD_DISTILL_MAX_K];
  const int tid = threadIdx.x;
  const long long row = blockIdx.x;
  const Z* z = (const Z*)a.z + row * a.zs;
  Z* dz = a.dz ? (Z*)a.dz + row * a.dzs : nullptr;
  const float w = a.weights ? __ldg(a.weights + row) : 1.f;
  if (!teacher_softmax(a, row, w, p, at, buf)) {
    if (tid == 0) a.losses[row] = 0.f;
    if (dz)
      for (int j = tid; j < a.vocab; j += kDistillThreads) dz[j] = from_f<Z>(0.f);
    return;
  }
  const float c = kLog2e / a.temperature;
  float r = -INFINITY, s = 0.f;
  for (int j = tid; j < a.vocab; j += kDistillThreads) {
    const float v = to_f(z[j]);
    if (v > r) {
      s *= exp2_fast((r - v) * c);
      r = v;
    }
    s += exp2_fast((v - (r == -INFINITY ? 0.f : r)) * c);
  }
  const float top = block_max(r, buf);
  const float base = top == -INFINITY ? 0.f : top;
  s = block_sum(r == -INFINITY ? s : s * exp2_fast((r - base) * c), buf);
  const float log2_s = log2f(s);
  float part = 0.f;
  for (int k = tid; k < a.k; k += kDistillThreads)
    if (at[k] >= 0 && !(p[k] == 0.f))
      part += p[k] * (logf(p[k]) - kLn2 * ((to_f(z[at[k]]) - base) * c - log2_s));
  part = block_sum(part, buf);
  if (tid == 0) a.losses[row] = w * (a.temperature * a.temperature) * part;
  if (!dz) return;
  const float f = w * a.temperature * a.scale, fq = f / s;
  // dz may be z itself: the entries' logits are read before any is written
  float target[PSGD_DISTILL_MAX_K / kDistillThreads];
#pragma unroll
  for (int n = 0; n < PSGD_DISTILL_MAX_K / kDistillThreads; ++n) {
    const int k = tid + n * kDistillThreads;
    target[n] = 0.f;
    if (k < a.k && at[k] >= 0)
      target[n] = exp2_fast((to_f(z[at[k]]) - base) * c) * fq - mass_at(p, at, a.k, k) * f;
  }
  __syncthreads();
  for (int j = tid; j < a.vocab; j += kDistillThreads) dz[j] = from_f<Z>(exp2_fast((to_f(z[j]) - base) * c) * fq);
  __syncthreads();
#pragma unroll
  for (int n = 0; n < PSGD_DISTILL_MAX_K / kDistillThreads; ++n) {
    const int k = tid + n * kDistillThreads;
    if (k < a.k && at[k] >= 0) dz[at[k]] = from_f<Z>(target[n]);
  }
}

// How a row is spread: CTAs of its cluster (0: too long for one), threads.
struct RowPlan {
  int ctas;
  int threads;
  size_t smem;
};

RowPlan plan_row(long long vocab, int size, long long rows, int sms) {
  const long long bytes = vocab * size + 32;  // with both ends' granules
  RowPlan p{1, 0, 0};
  while (p.ctas < kMaxCluster && bytes / p.ctas > kHalfSmem) p.ctas *= 2;
  if (bytes / p.ctas > kFullSmem) return RowPlan{0, kDistillThreads, 0};
  // few rows: more CTAs a row, as long as each keeps a few granules per thread
  while (p.ctas < kMaxCluster && rows * p.ctas * 2 <= sms && bytes / p.ctas >= 16 * 1024) p.ctas *= 2;
  const long long granules = bytes / 16 / p.ctas + 2;
  p.smem = (size_t)granules * 16;
  p.threads = (int)std::min<long long>(kDistillThreads, std::max<long long>(64, (granules / 4 + 31) / 32 * 32));
  return p;
}

template <typename Z, bool ALIGNED> cudaError_t launch_chip(const DistillArgs& a, const RowPlan& p, int device, cudaStream_t st) {
  static std::atomic<unsigned long long> raised{0};  // devices whose shared-memory limit is raised
  const unsigned long long bit = 1ull << device;
  cudaError_t e = cudaSuccess;
  if (!(raised.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(k_distill_chip<Z, ALIGNED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFullSmem + 64);
    if (e != cudaSuccess) return e;
    raised.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.rows * p.ctas));
  cfg.blockDim = dim3(p.threads);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = p.ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = p.ctas > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k_distill_chip<Z, ALIGNED>, a, p.ctas);
}

template <typename Z> cudaError_t launch_distill(const DistillArgs& a, int device, int sms, cudaStream_t st) {
  const RowPlan p = plan_row(a.vocab, (int)sizeof(Z), a.rows, sms);
  if (p.ctas == 0) {
    k_distill_long<Z><<<(unsigned)a.rows, kDistillThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  const bool aligned = !a.dz || ((((uintptr_t)a.z ^ (uintptr_t)a.dz) & 15) == 0 &&
                                 (a.rows == 1 || ((a.zs - a.dzs) * (long long)sizeof(Z)) % 16 == 0));
  return aligned ? launch_chip<Z, true>(a, p, device, st) : launch_chip<Z, false>(a, p, device, st);
}

// Multiprocessors of a device (looked up once).
int sm_count(int device) {
  static std::atomic<int> count[64];
  int n = count[device].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) {
      cudaGetLastError();
      return 1;
    }
    count[device].store(n, std::memory_order_relaxed);
  }
  return n;
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
                            int64_t dlogits_stride, int32_t device, void* stream) {
  const char* who = "psgd_distill";
  if (!dtype_ok(dtype) || !dtype_ok(teacher_dtype)) return fail(PSGD_EINVAL, "psgd_distill: unknown dtype");
  if (index_bits != 32 && index_bits != 64) return fail(PSGD_EINVAL, "psgd_distill: index_bits must be 32 or 64");
  if (rows < 0 || rows > 0xfffffff) return fail(PSGD_EINVAL, "psgd_distill: rows must be in [0, 2^28 - 1]");
  if (vocab < 1 || vocab > (1 << 30)) return fail(PSGD_EINVAL, "psgd_distill: vocab must be in [1, 2^30]");
  if (k < 1 || k > PSGD_DISTILL_MAX_K) return fail(PSGD_EINVAL, "psgd_distill: k must be in [1, PSGD_DISTILL_MAX_K]");
  if (!(temperature > 0.f) || !isfinite(temperature))
    return fail(PSGD_EINVAL, "psgd_distill: temperature must be finite and > 0");
  if (device < 0 || device >= 64) return fail(PSGD_EINVAL, "psgd_distill: device ordinal must be in [0, 63]");
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
  DeviceScope scope(device);
  const cudaStream_t st = (cudaStream_t)stream;
  const int sms = sm_count(device);
  const cudaError_t e = dtype == PSGD_F32   ? launch_distill<float>(a, device, sms, st)
                        : dtype == PSGD_F16 ? launch_distill<__half>(a, device, sms, st)
                                            : launch_distill<__nv_bfloat16>(a, device, sms, st);
  return e == cudaSuccess ? PSGD_OK : cuda_fail(who, e);
}
