// What the norms' kernels share: rows that groups of threads hold in registers.
#pragma once

#include "psgd_ops.cuh"

namespace psgd {
namespace ops {

constexpr int kRowThreads = 512;  // of a CTA

// N values (a power of two up to 8) summed over a warp with N - 1 + log2(32 / N)
// shuffles: while there is more than one value, half of the lanes keep one half
// of them and send the other.  Returns the sum of value fold_index(lane).
template <int N> __device__ __forceinline__ float fold_sum(float (&v)[N], int lane) {
#pragma unroll
  for (int k = 0; k < 5; ++k) {
    const int off = 16 >> k, n = N >> (k + 1);
    if (n >= 1) {
      const bool upper = lane & off;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float send = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
      }
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
    }
  }
  return v[0];
}
template <int N> __device__ __forceinline__ int fold_index(int lane) {
  return N == 8 ? (lane >> 2) : N == 4 ? (lane >> 3) : N == 2 ? (lane >> 4) : 0;
}

// Sums of N values over the `warps` warps of one thread group, returned to all
// of its threads.  `buf` holds warps * N floats of this group; the caller
// alternates between two of them, so one barrier per call suffices.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float* buf, int warps, int warp, int lane, int group,
                                          int threads) {
  float x = fold_sum<N>(v, lane);
  if (warps == 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, x, i * (32 / N));
    return;
  }
  if ((lane & (32 / N - 1)) == 0) buf[warp * N + fold_index<N>(lane)] = x;
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(threads) : "memory");
  x = 0.f;
  constexpr int kMaxWarps = kRowThreads / 32;
#pragma unroll
  for (int k = 0; k < (kMaxWarps * N + 31) / 32; ++k)  // value lane % N of warp lane / N + k * 32 / N
    if (k * 32 + lane < warps * N) x += buf[k * 32 + lane];
#pragma unroll
  for (int off = N; off < 32; off *= 2) x += __shfl_xor_sync(0xffffffffu, x, off);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, x, i);
}

// N elements of a parameter from column c on, `none` where there is no
// parameter or no column.  One branch on the type, so that all loads are under
// way together.
template <int N> __device__ __forceinline__ void load_param(const void* w, int dtype, long long c, bool in, float none, float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = in ? none : 0.f;
  if (!w || !in) return;
  if (dtype == PSGD_F32) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = __ldg((const float*)w + c + i);
  } else if (dtype == PSGD_F16) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = __half2float(__ldg((const __half*)w + c + i));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = __bfloat162float(__ldg((const __nv_bfloat16*)w + c + i));
  }
}
template <int NE> __device__ __forceinline__ void load_param(const void* w, int dtype, long long c, bool in, float none, F2 (&f)[NE]) {
  float v[2 * NE];
  load_param<2 * NE>(w, dtype, c, in, none, v);
#pragma unroll
  for (int h = 0; h < NE; ++h) f[h] = f2(v[2 * h], v[2 * h + 1]);
}

// How the warps of a group share the copies of `items` rows: warp w takes the
// items first, first + step, ..., and of each the granules of part `part` of
// `parts`.
struct CopyShare {
  int first, step, part, parts;
  __device__ __forceinline__ CopyShare(int items, int warps, int warp) {
    parts = warps >= items ? warps / items : 1;
    first = parts > 1 ? warp / parts : warp;
    part = parts > 1 ? warp - first * parts : 0;
    step = parts > 1 ? items : warps;  // (with parts, warps that are left over have first >= items)
  }
};

__device__ __forceinline__ void group_barrier(int group, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(threads) : "memory");
}

// Where in its first granule row `index` of an array begins, in bytes.
__device__ __forceinline__ int row_phase(const void* base, int index, long long stride, int size) {
  return ((unsigned)(uintptr_t)base + (unsigned)index * ((unsigned)stride * (unsigned)size)) & 15;
}
}  // namespace ops
}  // namespace psgd
