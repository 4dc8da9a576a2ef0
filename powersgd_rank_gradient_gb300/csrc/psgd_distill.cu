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
#include <type_traits>

#include "psgd_ops.cuh"

namespace cg = cooperative_groups;

namespace psgd {
namespace ops {
namespace {

constexpr int kDistillThreads = 512;
constexpr int kDistillWarps = kDistillThreads / 32;
constexpr int kStages = 4;               // groups of copies a slice arrives in
constexpr int kMaxCluster = 8;           // CTAs of a row
constexpr int kHalfSmem = 112 * 1024;    // of a CTA, two of which fit an SM
constexpr int kFullSmem = 224 * 1024;    // of a CTA alone on its SM

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
  float inv_t;  // 1 / temperature
  float c;      // log2(e) / temperature
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kFar = 1048576.f;  // 2^20

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
// 2^(c z_j - r) over its sum, r the largest c z_j, rounded.  One fused operation
// gives an exponent; r's rounding is in every term and cancels, as long as it
// is small: up to |r| = kFar it is below 2^-4.  A row further out (masks of the
// type's lowest value and nothing else, or enormous logits) takes its sums
// again with the difference first, 2^(c (z_j - max)).
//
// The teacher's entries of one row: validity (at[k], -1 where not), and their
// softmax p[k].  Returns whether the row counts at all.  The largest logit comes
// off before the temperature: a rounding is then relative to the distance
// between two logits, however far from zero both are, and none overflows.
__device__ __forceinline__ bool teacher_softmax(const DistillArgs& a, long long row, float w, float* p, int* at,
                                                float* buf) {
  const float inv_t = a.inv_t;
  float m = -INFINITY;
  bool mass = false;
  for (int k = threadIdx.x; k < a.k; k += blockDim.x) {
    const long long i = a.index64 ? __ldg((const long long*)a.index + row * a.is + k)
                                  : (long long)__ldg((const int*)a.index + row * a.is + k);
    const bool valid = i >= 0 && i < a.vocab;
    const float t = valid ? load_any(a.t, a.tdtype, row * a.ts + k) : -INFINITY;
    at[k] = valid ? (int)i : -1;
    p[k] = t;
    m = fmaxf(m, t);
    mass |= t != -INFINITY;
  }
  if (!__syncthreads_or(mass) || w == 0.f) return false;
  m = block_max(m, buf);
  float s = 0.f;
  for (int k = threadIdx.x; k < a.k; k += blockDim.x) {
    const float e = at[k] >= 0 ? expf((p[k] - m) * inv_t) : 0.f;
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

// The largest element of a 16-byte granule.
template <typename Z> __device__ __forceinline__ float top_of(const uint4& u);
template <> __device__ __forceinline__ float top_of<float>(const uint4& u) {
  return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
}
template <> __device__ __forceinline__ float top_of<__half>(const uint4& u) {
  const __half2* h = reinterpret_cast<const __half2*>(&u);
  const __half2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
  return fmaxf(__low2float(m), __high2float(m));
}
template <> __device__ __forceinline__ float top_of<__nv_bfloat16>(const uint4& u) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
  const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
  return fmaxf(__low2float(m), __high2float(m));
}

// Slots of the table in which a row's entries look for equal indices: a power
// of two, at least twice the entries.
__host__ __device__ constexpr int table_slots(int k) {
  int n = 64;
  while (n < 2 * k) n *= 2;
  return n;
}

// One warp's work on a row's teacher entries: validity (at[k], -1 where not),
// their softmax p[k], whether the row counts (state bit 0) and whether two of
// its indices are equal (bit 1).
__device__ __forceinline__ int teacher_warp(const DistillArgs& a, long long row, float* p, int* at, int* table) {
  const int lane = threadIdx.x & 31;
  const float inv_t = a.inv_t;
  const int slots = table_slots(a.k);
  for (int i = lane; i < slots; i += 32) table[i] = -1;
  __syncwarp();
  float m = -INFINITY;
  bool mass = false, twice = false;
  for (int k = lane; k < a.k; k += 32) {
    const long long i = a.index64 ? __ldg((const long long*)a.index + row * a.is + k)
                                  : (long long)__ldg((const int*)a.index + row * a.is + k);
    const float tk = load_any(a.t, a.tdtype, row * a.ts + k);
    const bool valid = i >= 0 && i < a.vocab;
    const float t = valid ? tk : -INFINITY;
    at[k] = valid ? (int)i : -1;
    p[k] = t;
    m = fmaxf(m, t);
    mass |= t != -INFINITY;
    if (valid) {
      // open addressing: there are more slots than entries, so a free one or the index itself is met
      unsigned h = ((unsigned)i * 2654435761u) & (slots - 1);
      for (;;) {
        const int old = atomicCAS(&table[h], -1, (int)i);
        if (old == (int)i) twice = true;
        if (old == -1 || old == (int)i) break;
        h = (h + 1) & (slots - 1);
      }
    }
  }
  mass = __any_sync(0xffffffffu, mass);
  twice = __any_sync(0xffffffffu, twice);
  if (!mass) return 0;
  m = warp_max(m);
  float s = 0.f;
  for (int k = lane; k < a.k; k += 32) {
    const float e = at[k] >= 0 ? expf((p[k] - m) * inv_t) : 0.f;
    p[k] = e;
    s += e;
  }
  const float inv_p = 1.f / warp_sum(s);
  for (int k = lane; k < a.k; k += 32) p[k] *= inv_p;
  return twice ? 3 : 1;
}

// Maximum and sum over all warps of a CTA, the same in every thread.
__device__ __forceinline__ float cta_max(float v, float* buf, int warps) {
  const int lane = threadIdx.x & 31;
  v = warp_max(v);
  __syncthreads();
  if (lane == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_max(lane < warps ? buf[lane] : -INFINITY);
}
__device__ __forceinline__ float cta_sum(float v, float* buf, int warps) {
  const int lane = threadIdx.x & 31;
  v = warp_sum(v);
  __syncthreads();
  if (lane == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(lane < warps ? buf[lane] : 0.f);
}
// A CTA's value joined over the cluster by `join`, a reduction over a warp.
template <typename J>
__device__ __forceinline__ float cluster_join(float v, float2* peers, int ctas, int rank, J join, float none) {
  if (ctas == 1) return v;
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();  // nobody reads `peers` any more
  if ((int)threadIdx.x < ctas) *cluster.map_shared_rank(&peers[rank].x, threadIdx.x) = v;
  cluster.sync();
  const int lane = threadIdx.x & 31;
  return join(lane < ctas ? peers[lane].x : none);
}

// One cluster per row; CTA r of C holds the row's granules [r n / C, (r + 1) n / C)
// in shared memory, n the number of aligned 16-byte granules that the row
// touches (its first and last may be shared with the neighbouring rows).  The
// last warp of a CTA works on the teacher's entries while the others take the
// softmax's sums, so neither waits for the other's loads.  ALIGNED: the
// gradient's rows start at the same place of a granule as the logits' do, so
// whole granules are stored.
//
// Two slices of about 100 KB to an SM (rows of more than that are cut over a
// cluster), one CTA's loads and stores under the other's arithmetic.  8192 rows
// of 50257 bf16 logits take 285 us (5.79 TB/s, 86 % of the copy bandwidth), 2458
// rows of 30522 fp32 ones 105 us (5.4 TB/s, 80 %); with the logits read twice
// from memory 995 and 202 us.  What is left is the instructions (about 16 an
// element, the issue slots 60 % full) in the phases that both CTAs of an SM meet
// in.  Few rows: a row over up to 8 CTAs, five rows of 50257 fp32 5.1 us.
template <typename Z, bool ALIGNED>
__global__ void __launch_bounds__(kDistillThreads + 32, 2) k_distill_chip(DistillArgs a, int log_ctas, int slice_granules,
                                                                         int per, int early) {
  constexpr int NE = Vec16<Z>::N;
  constexpr int NP = NE / 2;
  constexpr int U = NE == 8 ? 2 : 4;  // granules a thread takes at a time
  extern __shared__ uint4 slice[];
  __shared__ float bufm[kDistillWarps + 1], bufs[kDistillWarps + 1];
  __shared__ float2 peers[kMaxCluster];
  __shared__ float parts[kMaxCluster];
  __shared__ int state_shared;
  float* p = reinterpret_cast<float*>(slice + slice_granules);  // k each, and the table
  float* pm = p + a.k;
  int* at = reinterpret_cast<int*>(pm + a.k);
  int* table = at + a.k;
  const int threads = blockDim.x - 32;  // of the row's warps
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = threads >> 5;
  const bool entries = warp == warps;
  const int ctas = 1 << log_ctas;
  const int row = blockIdx.x >> log_ctas, rank = blockIdx.x & (ctas - 1);
  const Z* z = (const Z*)a.z + row * a.zs;
  Z* dz = a.dz ? (Z*)a.dz + row * a.dzs : nullptr;
  const int head = (int)(((uintptr_t)z & 15) / sizeof(Z));  // elements of the first granule before the row
  const int granules = (head + a.vocab + NE - 1) / NE;
  // (a row's granules times 8 fit 32 bits: its CTAs hold at most 8 x 224 KB of them)
  const int g0 = granules * rank >> log_ctas, n = (granules * (rank + 1) >> log_ctas) - g0;
  // granules of the slice that lie inside the row: [whole0, whole0 + whole)
  const int whole0 = max(0, (head ? 1 : 0) - g0);
  const unsigned whole = (unsigned)max(0, min(n, (head + a.vocab) / NE - g0) - whole0);
  const Z* zs = z + ((long long)g0 * NE - head);  // the slice's first granule (its first elements may lie before the row)
  const int j0 = g0 * NE - head;                  // its first element
  if (early) {
    after_previous();
    next_may_launch();
  }
  const float w = a.weights ? __ldg(a.weights + row) : 1.f;
  if (ctas > 1) cluster_arrive();  // a peer's shared memory is written once all have started

  auto store = [&](int g, const float* f) {
    if (ALIGNED && (unsigned)(g - whole0) < whole) {
      store_pack<Z, NE>(dz + j0 + g * NE, f);
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (j0 + g * NE + i >= 0 && j0 + g * NE + i < a.vocab) dz[j0 + g * NE + i] = from_f<Z>(f[i]);
    }
  };
  auto store_zeros = [&]() {
    float zero[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) zero[i] = 0.f;
    if (dz && !entries)
      for (int g = tid; g < n; g += threads) store(g, zero);
    if (rank == 0 && tid == 0) a.losses[row] = 0.f;
  };

  if (w == 0.f) {  // the same for every CTA of the cluster
    store_zeros();
    if (ctas > 1) cluster_wait();
    return;
  }

  const float c = a.c;
  if (entries) {
    const int state = teacher_warp(a, row, p, at, table);
    if (lane == 0) state_shared = state;
  } else {
    // The slice is copied by the threads that will use it (granule tid, tid +
    // threads, ...), in kStages groups of `per` copies that are all under way at once.
#pragma unroll
    for (int q = 0; q < kStages; ++q) {
      const int last = min(n, (q + 1) * per * threads);
      for (int g = q * per * threads + tid; g < last; g += threads) {
        if ((unsigned)(g - whole0) < whole) {
          copy16(&slice[g], zs + (long long)g * NE);
        } else {
          uint4 v;
          Z* e = reinterpret_cast<Z*>(&v);
#pragma unroll
          for (int i = 0; i < NE; ++i) {
            const int j = j0 + g * NE + i;
            e[i] = j >= 0 && j < a.vocab ? z[j] : from_f<Z>(-INFINITY);
          }
          slice[g] = v;
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    float r = -kFar;
    F2 sums[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
    const F2 cc = f2(c, c);
    auto take = [&](const uint4* v, auto count) {
      constexpr int N = decltype(count)::value;
      float top = top_of<Z>(v[0]);
#pragma unroll
      for (int i = 1; i < N; ++i) top = fmaxf(top, top_of<Z>(v[i]));
      if (top * c > r) {
        const float down = exp2_fast(r - top * c);
        sums[0] = mul(sums[0], f2(down, down));
        sums[1] = mul(sums[1], f2(down, down));
        r = top * c;
      }
      const F2 bb = f2(-r, -r);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        F2 f[NP];
        to_pairs<Z>(v[i], f);
#pragma unroll
        for (int h = 0; h < NP; ++h) {
          float x, y;
          split(fma(f[h], cc, bb), x, y);
          sums[h & 1] = add(sums[h & 1], f2(exp2_fast(x), exp2_fast(y)));
        }
      }
    };
#pragma unroll
    for (int q = 0; q < kStages; ++q) {
      wait_copies<kStages - 1>(q);
      const int last = min(n, (q + 1) * per * threads);
      int g = q * per * threads + tid;
      for (; g + (U - 1) * threads < last; g += threads * U) {
        uint4 v[U];
#pragma unroll
        for (int i = 0; i < U; ++i) v[i] = slice[g + i * threads];
        take(v, std::integral_constant<int, U>());
      }
      for (; g < last; g += threads) take(&slice[g], std::integral_constant<int, 1>());
    }
    float x, y;
    split(add(sums[0], sums[1]), x, y);
    float s = x + y;
    // over the warp
    const float top = warp_max(r);
    s = warp_sum(s * exp2_fast(r - top));
    if (lane == 0) {
      bufm[warp] = top;
      bufs[warp] = s;
    }
  }
  __syncthreads();
  // over the CTA, then the cluster
  float top, s;
  top = warp_max(lane < warps ? bufm[lane] : -kFar);
  s = warp_sum(lane < warps ? bufs[lane] * exp2_fast(bufm[lane] - top) : 0.f);
  if (ctas > 1) {
    cg::cluster_group cluster = cg::this_cluster();
    cluster_wait();
    if (tid < ctas) *cluster.map_shared_rank(&peers[rank], tid) = make_float2(top, s);
    cluster.sync();
    top = warp_max(lane < ctas ? peers[lane].x : -kFar);
    s = warp_sum(lane < ctas ? peers[lane].y * exp2_fast(peers[lane].x - top) : 0.f);
  }
  const int state = state_shared;
  if (state == 0) {  // the same for every CTA of the cluster
    store_zeros();
    return;
  }
  // the exponent of a logit is c (z - shift) - base; one of shift and base is 0
  float shift = 0.f, base = top;
  if (!(fabsf(top) < kFar)) {  // the same for every CTA of the cluster
    float m = -INFINITY;
    for (int g = tid; g < n; g += blockDim.x) m = fmaxf(m, top_of<Z>(slice[g]));
    m = cta_max(m, bufm, warps + 1);
    m = cluster_join(m, peers, ctas, rank, [](float v) { return warp_max(v); }, -INFINITY);
    shift = m == -INFINITY ? 0.f : m;
    base = 0.f;
    s = 0.f;
    for (int g = tid; g < n; g += blockDim.x) {
      F2 x[NP];
      to_pairs<Z>(slice[g], x);
#pragma unroll
      for (int h = 0; h < NP; ++h) {
        float u, v;
        split(x[h], u, v);
        s += exp2_fast((u - shift) * c) + exp2_fast((v - shift) * c);
      }
    }
    s = cta_sum(s, bufs, warps + 1);
    s = cluster_join(s, peers, ctas, rank, [](float v) { return warp_sum(v); }, 0.f);
  }
  const float f = w * a.temperature * a.scale, fq = f / s;
  if (state & 2) {
    for (int k = tid; k < a.k; k += blockDim.x) pm[k] = mass_at(p, at, a.k, k);
    __syncthreads();
  }
  const Z* held = reinterpret_cast<const Z*>(slice) - j0;
  if (entries) {
    // the entries that fall into this CTA's slice: their part of the loss, and their gradients
    const float log2_s = log2f(s);
    float part = 0.f;
    for (int k = lane; k < a.k; k += 32) {
      const int j = at[k];
      const float pk = p[k];
      if (j >= 0 && (unsigned)(j - j0) < (unsigned)(n * NE)) {
        const float x = fmaf(to_f(held[j]) - shift, c, -base);
        if (!(pk == 0.f)) part += pk * (logf(pk) - kLn2 * (x - log2_s));
        pm[k] = exp2_fast(x) * fq - (state & 2 ? pm[k] : pk) * f;
      } else {
        at[k] = -1;
      }
    }
    part = warp_sum(part);
    if (ctas == 1) {
      if (lane == 0) a.losses[row] = w * (a.temperature * a.temperature) * part;
    } else if (lane == 0) {
      *cg::this_cluster().map_shared_rank(&parts[rank], 0) = part;
    }
  } else if (dz) {
    const F2 cc = f2(c, c), ff = f2(fq, fq), bb = f2(-base, -base), ss = f2(-shift, -shift);
    auto gradient = [&](auto far) {
      for (int g = tid; g < n; g += threads) {
        F2 x[NP];
        float q[NE];
        to_pairs<Z>(slice[g], x);
#pragma unroll
        for (int h = 0; h < NP; ++h) {
          float u, v;
          split(decltype(far)::value ? mul(add(x[h], ss), cc) : fma(x[h], cc, bb), u, v);
          split(mul(f2(exp2_fast(u), exp2_fast(v)), ff), q[2 * h], q[2 * h + 1]);
        }
        store(g, q);
      }
    };
    if (fabsf(top) < kFar) gradient(std::false_type());
    else gradient(std::true_type());
  }
  if (ctas > 1) {
    cg::this_cluster().sync();
    if (rank == 0 && tid == 0) {
      float part = 0.f;
      for (int v = 0; v < ctas; ++v) part += parts[v];
      a.losses[row] = w * (a.temperature * a.temperature) * part;
    }
  } else if (dz) {
    __syncthreads();
  }
  if (dz && entries)
    for (int k = lane; k < a.k; k += 32)
      if (at[k] >= 0) dz[at[k]] = from_f<Z>(pm[k]);
}

// Rows larger than a cluster's shared memory (1.7 MB): one CTA per row, which
// reads the logits twice, element by element: bound by its one SM's loads.
template <typename Z> __global__ void __launch_bounds__(kDistillThreads) k_distill_long(DistillArgs a) {
  __shared__ float buf[kDistillWarps];
  __shared__ float p[PSGD_DISTILL_MAX_K];
  __shared__ int at[PSGD_DISTILL_MAX_K];
  const int tid = threadIdx.x;
  const long long row = blockIdx.x;
  const Z* z = (const Z*)a.z + row * a.zs;
  Z* dz = a.dz ? (Z*)a.dz + row * a.dzs : nullptr;
  after_previous();
  next_may_launch();
  const float w = a.weights ? __ldg(a.weights + row) : 1.f;
  if (!teacher_softmax(a, row, w, p, at, buf)) {
    if (tid == 0) a.losses[row] = 0.f;
    if (dz)
      for (int j = tid; j < a.vocab; j += kDistillThreads) dz[j] = from_f<Z>(0.f);
    return;
  }
  const float c = a.c;
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

// How a row is spread: CTAs of its cluster (0: too long for one), threads of
// the row's warps, granules of a slice, shared memory with the entries'.
struct RowPlan {
  int ctas;
  int log_ctas;
  int threads;
  int granules;
  size_t smem;
};

RowPlan plan_row(long long vocab, int size, int k, long long rows, int sms) {
  const long long extra = 12LL * k + 4LL * table_slots(k) + 16;
  const long long bytes = vocab * size + 32;  // with both ends' granules
  RowPlan p{1, 0, kDistillThreads, 0, 0};
  while (p.ctas < kMaxCluster && bytes / p.ctas + extra > kHalfSmem) p.ctas *= 2;
  if (bytes / p.ctas + extra > kFullSmem) return RowPlan{0, 0, kDistillThreads, 0, 0};
  // few rows: more CTAs a row, as long as each keeps a few granules per thread
  while (p.ctas < kMaxCluster && rows * p.ctas * 2 <= sms && bytes / p.ctas >= 16 * 1024) p.ctas *= 2;
  while (1 << p.log_ctas < p.ctas) ++p.log_ctas;
  p.granules = (int)(bytes / 16 / p.ctas + 2);
  p.smem = (size_t)p.granules * 16 + extra;
  // threads: 512 where two slices fill an SM, 256 where three and more do (4000
  // bf16 rows of 38000 logits, 76 KB a slice: 113.4 us with 512, 116.0 with 256;
  // of 35000, 70 KB: 104.9 and 93.4), and fewer for short rows, eight granules
  // each: an SM then has more rows, each waiting for its own loads (of 8000
  // logits 33.5 us so, 41.0 with four granules each; from 32 KB a slice on the
  // limit above is what counts)
  const int most = p.smem > 72 * 1024 ? kDistillThreads : kDistillThreads / 2;
  p.threads = (int)std::min<long long>(most, std::max<long long>(64, (p.granules / 8 + 31) / 32 * 32));
  return p;
}

template <typename Z, bool ALIGNED> cudaError_t launch_chip(const DistillArgs& a, const RowPlan& p, int device, int sms, cudaStream_t st) {
  static std::atomic<unsigned long long> raised{0};
  const cudaError_t e = raise_smem(k_distill_chip<Z, ALIGNED>, raised, device, kFullSmem + 64);
  if (e != cudaSuccess) return e;
  const int per = ((p.granules + p.threads - 1) / p.threads + kStages - 1) / kStages;  // granules per thread and group of copies
  // set up early only where the launch itself counts: in many waves of CTAs it costs 2 % (289 against 283 us at 8192 rows)
  const bool early = a.rows * p.ctas <= 8LL * sms;
  return launch(early, k_distill_chip<Z, ALIGNED>, (unsigned)(a.rows * p.ctas), p.threads + 32, p.smem, p.ctas, st, a,
                p.log_ctas, p.granules, per, early);
}

template <typename Z> cudaError_t launch_distill(const DistillArgs& a, int device, int sms, cudaStream_t st) {
  const RowPlan p = plan_row(a.vocab, (int)sizeof(Z), a.k, a.rows, sms);
  if (p.ctas == 0) {
    return launch_early(k_distill_long<Z>, (unsigned)a.rows, kDistillThreads, 0, 1, st, a);
  }
  const bool aligned = !a.dz || ((((uintptr_t)a.z ^ (uintptr_t)a.dz) & 15) == 0 &&
                                 (a.rows == 1 || ((a.zs - a.dzs) * (long long)sizeof(Z)) % 16 == 0));
  return aligned ? launch_chip<Z, true>(a, p, device, sms, st) : launch_chip<Z, false>(a, p, device, sms, st);
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
  if (!(temperature > 0.f) || !isfinite(temperature) || !isfinite(kLog2e / temperature))
    return fail(PSGD_EINVAL, "psgd_distill: temperature must be finite and > 0, and so must its reciprocal");
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
                losses, rows, (int)vocab, k, (int)teacher_dtype, index_bits == 64, temperature, grad_scale, 1.f / temperature,
                kLog2e / temperature};
  DeviceScope scope(device);
  const cudaStream_t st = (cudaStream_t)stream;
  const int sms = sm_count(device);
  const cudaError_t e = dtype == PSGD_F32   ? launch_distill<float>(a, device, sms, st)
                        : dtype == PSGD_F16 ? launch_distill<__half>(a, device, sms, st)
                                            : launch_distill<__nv_bfloat16>(a, device, sms, st);
  return e == cudaSuccess ? PSGD_OK : cuda_fail(who, e);
}
