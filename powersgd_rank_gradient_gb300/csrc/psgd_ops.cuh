// Shared pieces of the training operators (embedding, layer norm,
// distillation): element types, vector accesses, host-side argument checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <string>

#include "../../include/psgd.h"

int psgd_internal_set_error(int code, const char* msg);

namespace psgd {
namespace ops {

// ---- host side ---------------------------------------------------------------

inline int fail(int code, const std::string& msg) { return psgd_internal_set_error(code, msg.c_str()); }

inline int cuda_fail(const char* where, cudaError_t e) {
  cudaGetLastError();
  return fail(e == cudaErrorMemoryAllocation ? PSGD_ENOMEM : PSGD_ECUDA,
              std::string(where) + ": " + cudaGetErrorString(e));
}

// Makes `dev` current for the enclosing scope.
struct DeviceScope {
  int prev = -1;
  explicit DeviceScope(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
    if (prev != dev) cudaSetDevice(dev);
    else prev = -1;
  }
  ~DeviceScope() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

inline bool dtype_ok(int32_t d) { return d == PSGD_F32 || d == PSGD_F16 || d == PSGD_BF16; }
inline int dtype_size(int32_t d) { return d == PSGD_F32 ? 4 : 2; }
inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// How many units of `of` hold n (of both at least 1).  In 64 bits: n may be as
// large as its type, and n + of - 1 then needs more.
__host__ __device__ inline long long units(long long n, long long of) { return (n + of - 1) / of; }

// Whether [a, a + an) and [b, b + bn) share a byte (NULL ranges share none).
inline bool overlap(const void* a, long long an, const void* b, long long bn) {
  if (!a || !b || an <= 0 || bn <= 0) return false;
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + (uintptr_t)bn && y < x + (uintptr_t)an;
}

// Bytes from the first to one past the last element of `rows` rows of `cols`
// elements, `stride` elements apart.
inline long long extent(long long rows, long long cols, long long stride, int32_t dtype) {
  return rows > 0 && cols > 0 ? ((rows - 1) * stride + cols) * dtype_size(dtype) : 0;
}

// Largest element count of one operand that the checks accept: extents in
// bytes and row x stride products then stay far inside 64 bits.
constexpr long long kMaxElems = 1LL << 46;

// rows x stride stays inside kMaxElems (both non-negative).
inline bool span_ok(long long rows, long long stride) {
  return rows >= 0 && stride >= 0 && (rows == 0 || stride <= kMaxElems / rows);
}

// ---- device side -------------------------------------------------------------

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Elements of T in 16 bytes.
template <typename T> struct Vec16 { static constexpr int N = 16 / (int)sizeof(T); };

// V consecutive elements: V * sizeof(T) bytes in one access (V = 1: one
// element of any alignment; otherwise the address is a multiple of the size).
template <typename T, int V> struct Pack {
  T v[V];
};
template <> struct __align__(16) Pack<float, 4> { float v[4]; };
template <> struct __align__(16) Pack<__half, 8> { __half v[8]; };
template <> struct __align__(16) Pack<__nv_bfloat16, 8> { __nv_bfloat16 v[8]; };

template <typename T, int V> __device__ __forceinline__ Pack<T, V> load_pack(const T* p) {
  Pack<T, V> r;
  if constexpr (V == 1) {
    r.v[0] = __ldg(p);
  } else {
    static_assert(V * sizeof(T) == 16, "one 16-byte access");
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    r = *reinterpret_cast<const Pack<T, V>*>(&u);
  }
  return r;
}

// Two values rounded to T, as the 32 bits of a pair (one conversion for both).
template <typename T> __device__ __forceinline__ unsigned pack2(float x, float y);
template <> __device__ __forceinline__ unsigned pack2<__half>(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const unsigned*>(&h);
}
template <> __device__ __forceinline__ unsigned pack2<__nv_bfloat16>(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const unsigned*>(&h);
}

template <typename T, int V> __device__ __forceinline__ void store_pack(T* p, const float* f) {
  if constexpr (V == 1) {
    p[0] = from_f<T>(f[0]);
  } else if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  } else {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
  }
}

// V values into V consecutive elements, 16 bytes at a time (8 where they are
// no more): the address is a multiple of that.
template <typename T, int V> __device__ __forceinline__ void store_run(T* p, const float* f) {
  constexpr int N = Vec16<T>::N;
  if constexpr (V == 1) {
    p[0] = from_f<T>(f[0]);
  } else if constexpr (V >= N) {
#pragma unroll
    for (int i = 0; i < V; i += N) store_pack<T, N>(p + i, f + i);
  } else {
    static_assert(V == 4 && sizeof(T) == 2, "8 bytes");
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]));
  }
}
// The alignment in bytes that store_run of V elements of `size` bytes asks for.
inline int run_alignment(int v, int size) { return v == 1 ? size : (v * size >= 16 ? 16 : v * size); }

// Launches a kernel that may be set up while the one before it in the stream
// still runs: it must begin with after_previous(), before it touches any memory
// (the kernel before may be anyone's).  cluster: CTAs of a cluster, 1: none;
// early = false: after the kernel before, as usual.
template <typename... P, typename... A>
cudaError_t launch(bool early, void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t st,
                   A&&... args) {
  cudaLaunchAttribute attrs[2];
  int n = 0;
  if (early) {
    attrs[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    attrs[n].id = cudaLaunchAttributeClusterDimension;
    attrs[n].val.clusterDim.x = cluster;
    attrs[n].val.clusterDim.y = 1;
    attrs[n++].val.clusterDim.z = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attrs;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t st, A&&... args) {
  return launch(true, kernel, grid, block, smem, cluster, st, static_cast<A&&>(args)...);
}
// Raises a kernel's shared-memory limit, once per device.
template <typename K> cudaError_t raise_smem(K kernel, std::atomic<unsigned long long>& raised, int device, int bytes) {
  const unsigned long long bit = 1ull << device;
  if (raised.load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) raised.fetch_or(bit, std::memory_order_release);
  return e;
}
// Waits until everything the previous kernel of the stream wrote is visible.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next kernel of the stream be set up.
__device__ __forceinline__ void next_may_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Element i of an array of runtime type.
__device__ __forceinline__ float load_any(const void* p, int dtype, long long i) {
  if (dtype == PSGD_F32) return __ldg((const float*)p + i);
  if (dtype == PSGD_F16) return __half2float(__ldg((const __half*)p + i));
  return __bfloat162float(__ldg((const __nv_bfloat16*)p + i));
}
// Its current value, where the kernel itself writes the array.
__device__ __forceinline__ float read_any(const void* p, int dtype, long long i) {
  if (dtype == PSGD_F32) return ((const float*)p)[i];
  if (dtype == PSGD_F16) return __half2float(((const __half*)p)[i]);
  return __bfloat162float(((const __nv_bfloat16*)p)[i]);
}
__device__ __forceinline__ void store_any(void* p, int dtype, long long i, float v) {
  if (dtype == PSGD_F32) ((float*)p)[i] = v;
  else if (dtype == PSGD_F16) ((__half*)p)[i] = __float2half_rn(v);
  else ((__nv_bfloat16*)p)[i] = __float2bfloat16_rn(v);
}

// Two floats in one register pair: one instruction for both.
struct F2 {
  float2 p;
};
__device__ __forceinline__ F2 f2(float x, float y) { F2 r; r.p = make_float2(x, y); return r; }
__device__ __forceinline__ void split(F2 a, float& x, float& y) { x = a.p.x; y = a.p.y; }
__device__ __forceinline__ F2 add(F2 a, F2 b) { F2 r; r.p = __fadd2_rn(a.p, b.p); return r; }
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) { F2 r; r.p = __ffma2_rn(a.p, b.p, c.p); return r; }
__device__ __forceinline__ F2 mul(F2 a, F2 b) { F2 r; r.p = __fmul2_rn(a.p, b.p); return r; }

// 16 bytes of elements as pairs of floats.
template <typename T> __device__ __forceinline__ void to_pairs(const uint4& u, F2* f);
template <> __device__ __forceinline__ void to_pairs<float>(const uint4& u, F2* f) {
  f[0] = f2(__uint_as_float(u.x), __uint_as_float(u.y));
  f[1] = f2(__uint_as_float(u.z), __uint_as_float(u.w));
}
template <> __device__ __forceinline__ void to_pairs<__half>(const uint4& u, F2* f) {
  const __half2* h = reinterpret_cast<const __half2*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = __half22float2(h[i]);
    f[i] = f2(x.x, x.y);
  }
}
template <> __device__ __forceinline__ void to_pairs<__nv_bfloat16>(const uint4& u, F2* f) {
  const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

// Asynchronous copies into shared memory, of 16, 8 and 4 bytes.
__device__ __forceinline__ void copy16(uint4* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy8(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Waits for the first q + 1 of LAST + 1 groups of copies.
template <int LAST> __device__ __forceinline__ void wait_copies(int q) {
  if (q == LAST) asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (q == LAST - 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else if (q == LAST - 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else asm volatile("cp.async.wait_group 3;" ::: "memory");
}

// Starts the copy of row `index` of an array: granule u, u + step, ... into
// `slot`.  The bytes in front of a row within its first granule are the array's
// own where the row begins that far into it; elsewhere there may be nothing to
// read, and the granule's elements are copied one by one.
template <typename T>
__device__ __forceinline__ void copy_row(unsigned char* slot, const T* base, int index, long long stride, int dim, int u,
                                         int step) {
  const T* row = base + index * stride;
  const int before = (int)((uintptr_t)row & 15);
  const int bytes = before + dim * (int)sizeof(T);
  const unsigned char* src = (const unsigned char*)row - before;
  if (u == 0 && index * stride * (long long)sizeof(T) < before) {
    for (int e = before; e < min(16, bytes); e += (int)sizeof(T)) *(T*)(slot + e) = *(const T*)(src + e);
    u += step;
  }
  unsigned to = (unsigned)__cvta_generic_to_shared(slot) + u * 16;
  src += u * 16;
  for (int left = bytes - u * 16; left > 0; left -= step * 16) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src), "r"(min(16, left)) : "memory");
    to += step * 16;
    src += step * 16;
  }
}
// Bytes of a row's place in shared memory: `columns` elements (the columns of
// all threads) from any place of the first granule on.
__host__ __device__ inline int slot_bytes(int columns, int size) { return (columns * size + 15 + 15) / 16 * 16; }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

}  // namespace ops
}  // namespace psgd
