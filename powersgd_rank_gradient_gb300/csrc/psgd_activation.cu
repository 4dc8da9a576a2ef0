// Activation checkpoints in 8 bits (psgd_eight.cuh): saving and restoring.
//
// Both move data and do a few operations an element.  The lanes that hold a
// block of 128 elements are neighbours (16 lanes of 8 elements of a 16-bit type,
// 32 of 4 otherwise), so a block's largest magnitude takes four or five shuffles
// and every access is 16 bytes where the rows allow it.
#include <algorithm>
#include <type_traits>

#include "psgd_eight.cuh"

namespace psgd {
namespace ops {
namespace {

constexpr int kThreads8 = 256;

struct EightArgs {
  const void* x;  // save: source; restore: result
  long long xs;
  unsigned char* codes;
  float* scales;
  long long rows;
  long long pieces;  // blocks of all rows
  int dim, blocks;
  int e5;
};

// A thread takes U units of E elements: unit i of thread t is lane t % LANES of block (t / LANES) + i * step.
template <typename T, int V, int U> __global__ void __launch_bounds__(kThreads8) k_save(EightArgs a) {
  constexpr int E = V == 1 ? 4 : V, LANES = kBlock8 / E;
  const int lane = threadIdx.x & (LANES - 1);
  const long long first = ((long long)blockIdx.x * kThreads8 + threadIdx.x) / LANES;
  const long long step = (long long)gridDim.x * (kThreads8 / LANES);
  after_previous();
  next_may_launch();
  float v[U][E];
  long long row[U];
  int block[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const long long piece = first + i * step;
    row[i] = piece < a.pieces ? piece / a.blocks : a.rows;
    block[i] = (int)(piece - row[i] * a.blocks);
    const T* src = (const T*)a.x + row[i] * a.xs;
    const int c = block[i] * kBlock8 + (V == 1 ? lane : lane * E);
#pragma unroll
    for (int e = 0; e < E; ++e) v[i][e] = 0.f;
    if (row[i] == a.rows) continue;
    if constexpr (V == 1) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (c + 32 * e < a.dim) v[i][e] = to_f(__ldg(src + c + 32 * e));
    } else if (c < a.dim) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(src + c));
      F2 p[E / 2];
      to_pairs<T>(q, p);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) split(p[e], v[i][2 * e], v[i][2 * e + 1]);
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    unsigned code[E / 4];
    float scale;
    encode<E, LANES>(a.e5, v[i], code, scale);
    if (row[i] == a.rows) continue;
    unsigned char* dst = a.codes + row[i] * a.dim;
    const int c = block[i] * kBlock8 + (V == 1 ? lane : lane * E);
    if constexpr (V == 1) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (c + 32 * e < a.dim) dst[c + 32 * e] = (unsigned char)(code[0] >> (8 * e));
    } else if (c < a.dim) {
      if constexpr (E == 8) *reinterpret_cast<uint2*>(dst + c) = make_uint2(code[0], code[1]);
      else *reinterpret_cast<unsigned*>(dst + c) = code[0];
    }
    if (lane == 0) a.scales[row[i] * a.blocks + block[i]] = scale;
  }
}

template <typename T, int V, int U> __global__ void __launch_bounds__(kThreads8) k_restore(EightArgs a) {
  constexpr int E = V == 1 ? 4 : V, LANES = kBlock8 / E;
  const int lane = threadIdx.x & (LANES - 1);
  const long long first = ((long long)blockIdx.x * kThreads8 + threadIdx.x) / LANES;
  const long long step = (long long)gridDim.x * (kThreads8 / LANES);
  after_previous();
  next_may_launch();
  unsigned code[U][E / 4];
  float scale[U];
  long long row[U];
  int block[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const long long piece = first + i * step;
    row[i] = piece < a.pieces ? piece / a.blocks : a.rows;
    block[i] = (int)(piece - row[i] * a.blocks);
    const unsigned char* src = a.codes + row[i] * a.dim;
    const int c = block[i] * kBlock8 + (V == 1 ? lane : lane * E);
#pragma unroll
    for (int e = 0; e < E / 4; ++e) code[i][e] = 0;
    scale[i] = 1.f;
    if (row[i] == a.rows) continue;
    scale[i] = __ldg(a.scales + row[i] * a.blocks + block[i]);
    if constexpr (V == 1) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (c + 32 * e < a.dim) code[i][0] |= (unsigned)__ldg(src + c + 32 * e) << (8 * e);
    } else if (c < a.dim) {
      if constexpr (E == 8) {
        const uint2 q = __ldg(reinterpret_cast<const uint2*>(src + c));
        code[i][0] = q.x;
        code[i][1] = q.y;
      } else {
        code[i][0] = __ldg(reinterpret_cast<const unsigned*>(src + c));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (row[i] == a.rows) continue;
    float f[E];
#pragma unroll
    for (int e = 0; e < E / 4; ++e) decode4(a.e5, code[i][e], scale[i], f + 4 * e);
    T* dst = (T*)const_cast<void*>(a.x) + row[i] * a.xs;
    const int c = block[i] * kBlock8 + (V == 1 ? lane : lane * E);
    if constexpr (V == 1) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (c + 32 * e < a.dim) dst[c + 32 * e] = from_f<T>(f[e]);
    } else if (c < a.dim) {
      store_pack<T, V>(dst + c, f);
    }
  }
}

int check(const std::string& who, const void* x, int32_t dtype, int64_t stride, int64_t rows, int64_t dim, const void* codes,
          int32_t code, const void* scales, bool save, int32_t device) {
  if (!dtype_ok(dtype)) return fail(PSGD_EINVAL, who + ": unknown dtype");
  if (code != PSGD_E4M3 && code != PSGD_E5M2) return fail(PSGD_EINVAL, who + ": unknown 8-bit format");
  if (rows < 0 || rows > (1 << 30)) return fail(PSGD_EINVAL, who + ": rows must be in [0, 2^30]");
  if (dim < 1 || dim > (1 << 30)) return fail(PSGD_EINVAL, who + ": dim must be in [1, 2^30]");
  if (device < 0 || device >= 64) return fail(PSGD_EINVAL, who + ": device ordinal must be in [0, 63]");
  if (!span_ok(rows, stride) || !span_ok(rows, dim)) return fail(PSGD_EINVAL, who + ": bad row stride");
  if (!save && rows > 1 && stride < dim) return fail(PSGD_EINVAL, who + ": rows overlap");
  if (rows > 0 && (!x || !codes || !scales)) return fail(PSGD_EINVAL, who + ": NULL operand");
  const long long xb = extent(rows, dim, stride, dtype), cb = rows * dim, sb = rows * blocks8(dim) * 4;
  if (overlap(x, xb, codes, cb) || overlap(x, xb, scales, sb) || overlap(codes, cb, scales, sb))
    return fail(PSGD_EINVAL, who + ": an output overlaps another operand");
  return PSGD_OK;
}

template <bool SAVE, typename T, int V>
cudaError_t go(EightArgs a, cudaStream_t st) {
  constexpr int E = V == 1 ? 4 : V, LANES = kBlock8 / E, U = 2;
  const long long per = kThreads8 / LANES * U;
  // (a grid of at most 2^31 - 1 CTAs holds 2^46 / 128 blocks of one CTA's 16 or 32)
  const unsigned grid = (unsigned)units(a.pieces, per);
  return launch_early(SAVE ? k_save<T, V, U> : k_restore<T, V, U>, grid, kThreads8, 0, 1, st, a);
}

template <bool SAVE> int run(const std::string& who, const void* x, int32_t dtype, int64_t stride, int64_t rows, int64_t dim,
                             void* codes, int32_t code, float* scales, int32_t device, void* stream) {
  const int rc = check(who, x, dtype, stride, rows, dim, codes, code, scales, SAVE, device);
  if (rc) return rc;
  if (rows == 0) return PSGD_OK;
  const long long blocks = blocks8(dim);
  if (units(rows * blocks, 16) > 0x7fffffffLL) return fail(PSGD_EINVAL, who + ": too many elements");
  DeviceScope scope(device);
  EightArgs a{x, stride, (unsigned char*)codes, scales, rows, rows * blocks, (int)dim, (int)blocks, code == PSGD_E5M2};
  const cudaStream_t st = (cudaStream_t)stream;
  const int full = 16 / dtype_size(dtype);
  const bool vec = dim % full == 0 && aligned16(x) && (stride * dtype_size(dtype)) % 16 == 0 && (uintptr_t)codes % full == 0;
  cudaError_t e;
  if (dtype == PSGD_F32) e = vec ? go<SAVE, float, 4>(a, st) : go<SAVE, float, 1>(a, st);
  else if (dtype == PSGD_F16) e = vec ? go<SAVE, __half, 8>(a, st) : go<SAVE, __half, 1>(a, st);
  else e = vec ? go<SAVE, __nv_bfloat16, 8>(a, st) : go<SAVE, __nv_bfloat16, 1>(a, st);
  return e == cudaSuccess ? PSGD_OK : cuda_fail(who.c_str(), e);
}

}  // namespace
}  // namespace ops
}  // namespace psgd

using namespace psgd::ops;

extern "C" int psgd_activation_save(const void* x, psgd_dtype dtype, int64_t x_stride, int64_t rows, int64_t dim, void* codes,
                                    psgd_code code, float* scales, int32_t device, void* stream) {
  return run<true>("psgd_activation_save", x, dtype, x_stride, rows, dim, codes, code, scales, device, stream);
}

extern "C" int psgd_activation_restore(const void* codes, psgd_code code, const float* scales, int64_t rows, int64_t dim,
                                       void* out, psgd_dtype dtype, int64_t out_stride, int32_t device, void* stream) {
  return run<false>("psgd_activation_restore", out, dtype, out_stride, rows, dim, const_cast<void*>(codes), code,
                    const_cast<float*>(scales), device, stream);
}
