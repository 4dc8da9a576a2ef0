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
  unsigned pieces;   // blocks of all rows
  unsigned long long by;  // 2^64 / blocks, rounded up (0: one block a row)
  int dim, blocks;
  int e5;
};

// piece / blocks without a division (exact for 32-bit numbers).
__device__ __forceinline__ long long row_of(const EightArgs& a, unsigned piece) {
  return a.by ? (long long)__umul64hi(piece, a.by) : piece;
}
// Where a piece's elements of this lane are: its row and column.  ONE: of one row, all in 32 bits.
template <bool ONE> struct Place {
  std::conditional_t<ONE, int, long long> row, scale;
  int c;
  bool in;
  __device__ __forceinline__ Place(const EightArgs& a, long long piece, int lane, int e) {
    if constexpr (ONE) {
      row = 0;
      scale = (int)piece;
      c = (int)piece * kBlock8 + lane * e;
    } else {
      row = row_of(a, (unsigned)piece);
      scale = piece;  // (scales have no gaps)
      c = (int)(piece - row * a.blocks) * kBlock8 + lane * e;
    }
    in = piece < a.pieces && c < a.dim;
  }
};

// The largest magnitude's bits, as fp32, among 16 bytes of elements: of 16-bit types two at a time.
template <typename T> __device__ __forceinline__ unsigned magnitude(const uint4& u) {
  if constexpr (sizeof(T) == 4) {
    return max(max(u.x & 0x7fffffffu, u.y & 0x7fffffffu), max(u.z & 0x7fffffffu, u.w & 0x7fffffffu));
  } else {
    const unsigned k = 0x7fff7fffu;
    return __vmaxu2(__vmaxu2(u.x & k, u.y & k), __vmaxu2(u.z & k, u.w & k));
  }
}
template <typename T> __device__ __forceinline__ unsigned wider(unsigned a, unsigned b) {
  if constexpr (sizeof(T) == 4) return max(a, b);
  else return __vmaxu2(a, b);
}
template <typename T> __device__ __forceinline__ unsigned as_f32(unsigned m) {
  if constexpr (sizeof(T) == 4) return m;
  const unsigned short h = (unsigned short)max(m & 0xffffu, m >> 16);
  if constexpr (std::is_same_v<T, __half>) return __float_as_uint(__half2float(__ushort_as_half(h)));
  else return (unsigned)h << 16;
}

// Rows of whole 16-byte units.  A thread takes U of them: unit i of thread t is lane t % LANES of block (t / LANES) +
// i * step.  What is under way waits in its own type, and the largest magnitude of a block is found in it.  16384 x 4096
// bf16 saved and restored: 61 us, 404 MB at 6.6 TB/s (90 us with maxima in fp32 and a division a unit, 74 with a
// multiplication in its place and places in 64 bits): bound by HBM.
template <typename T, bool E5, int U, bool ONE> __global__ void __launch_bounds__(kThreads8) k_save_vec(EightArgs a) {
  constexpr int E = Vec16<T>::N, LANES = kBlock8 / E;
  const int lane = threadIdx.x & (LANES - 1);
  const long long first = ((long long)blockIdx.x * kThreads8 + threadIdx.x) / LANES;
  const long long step = (long long)gridDim.x * (kThreads8 / LANES);
  after_previous();
  next_may_launch();
  uint4 raw[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const long long piece = first + i * step;
    const Place<ONE> at(a, piece, lane, E);
    raw[i] = at.in ? __ldg(reinterpret_cast<const uint4*>((const T*)a.x + at.row * a.xs + at.c)) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    unsigned top = magnitude<T>(raw[i]);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) top = wider<T>(top, __shfl_xor_sync(0xffffffffu, top, o));
    top = as_f32<T>(top);
    F2 p[E / 2];
    to_pairs<T>(raw[i], p);
    unsigned code[E / 4];
    float scale;
    if (top < 0x7f800000u) {
      const int e = scale_exponent<E5>(top);
      const float inv = power2(-e);
      scale = power2(e);
#pragma unroll
      for (int k = 0; k < E / 4; ++k) {
        float v[4];
        split(mul(p[2 * k], f2(inv, inv)), v[0], v[1]);
        split(mul(p[2 * k + 1], f2(inv, inv)), v[2], v[3]);
        code[k] = codes2<E5>(v[0], v[1]) | codes2<E5>(v[2], v[3]) << 16;
      }
    } else {  // something infinite or NaN (for all lanes of the block)
      float v[E];
#pragma unroll
      for (int k = 0; k < E / 2; ++k) split(p[k], v[2 * k], v[2 * k + 1]);
      encode_special<E, LANES, E5>(v, code, scale);
    }
    const Place<ONE> at(a, first + i * step, lane, E);
    if (!at.in) continue;
    unsigned char* dst = a.codes + (long long)at.row * a.dim + at.c;
    if constexpr (E == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(code[0], code[1]);
    else *reinterpret_cast<unsigned*>(dst) = code[0];
    if (lane == 0) a.scales[at.scale] = scale;
  }
}

template <typename T, bool E5, int U, bool ONE> __global__ void __launch_bounds__(kThreads8) k_restore_vec(EightArgs a) {
  constexpr int E = Vec16<T>::N, LANES = kBlock8 / E;
  const int lane = threadIdx.x & (LANES - 1);
  const long long first = ((long long)blockIdx.x * kThreads8 + threadIdx.x) / LANES;
  const long long step = (long long)gridDim.x * (kThreads8 / LANES);
  after_previous();
  next_may_launch();
  unsigned code[U][E / 4];
  float scale[U];
  T* dst[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const Place<ONE> at(a, first + i * step, lane, E);
    dst[i] = nullptr;
    if (!at.in) continue;
    dst[i] = (T*)const_cast<void*>(a.x) + at.row * a.xs + at.c;
    scale[i] = __ldg(a.scales + at.scale);
    const unsigned char* src = a.codes + (long long)at.row * a.dim + at.c;
    if constexpr (E == 8) {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(src));
      code[i][0] = q.x;
      code[i][1] = q.y;
    } else {
      code[i][0] = __ldg(reinterpret_cast<const unsigned*>(src));
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (!dst[i]) continue;
    float f[E];
#pragma unroll
    for (int e = 0; e < E / 4; ++e) decode4(E5, code[i][e], scale[i], f + 4 * e);
    store_pack<T, E>(dst[i], f);
  }
}

// Rows of any length and alignment: a warp a block, lane by lane, U blocks of a warp.
template <typename T, bool SAVE, int U> __global__ void __launch_bounds__(kThreads8) k_eight_any(EightArgs a) {
  const int lane = threadIdx.x & 31;
  const long long first = ((long long)blockIdx.x * kThreads8 + threadIdx.x) / 32, step = (long long)gridDim.x * (kThreads8 / 32);
  after_previous();
  next_may_launch();
  T* x = (T*)const_cast<void*>(a.x);
  float v[U][4];
  unsigned code[U];
  float scale[U];
  long long row[U];
  int c[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const long long piece = first + i * step;
    row[i] = piece < a.pieces ? row_of(a, (unsigned)piece) : -1;
    const int block = (int)(piece - row[i] * a.blocks);
    c[i] = block * kBlock8 + lane;
    code[i] = 0;
    scale[i] = 1.f;
    if (!SAVE && row[i] >= 0) scale[i] = __ldg(a.scales + row[i] * a.blocks + block);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[i][e] = 0.f;
      if (row[i] < 0 || c[i] + 32 * e >= a.dim) continue;
      if constexpr (SAVE) v[i][e] = to_f(__ldg(x + row[i] * a.xs + c[i] + 32 * e));
      else code[i] |= (unsigned)__ldg(a.codes + row[i] * a.dim + c[i] + 32 * e) << (8 * e);
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if constexpr (SAVE) {
      unsigned packed[1];
      encode<4, 32>(a.e5, v[i], packed, scale[i]);
      code[i] = packed[0];
    } else {
      decode4(a.e5, code[i], scale[i], v[i]);
    }
    if (row[i] < 0) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (c[i] + 32 * e >= a.dim) continue;
      if constexpr (SAVE) a.codes[row[i] * a.dim + c[i] + 32 * e] = (unsigned char)(code[i] >> (8 * e));
      else x[row[i] * a.xs + c[i] + 32 * e] = from_f<T>(v[i][e]);
    }
    if (SAVE && lane == 0) a.scales[row[i] * a.blocks + c[i] / kBlock8] = scale[i];
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

// Four units a thread; one where that would leave SMs without a CTA (a weight gradient from 509 x 1024: 13.0 -> 10.4 us).
template <bool SAVE, typename T> cudaError_t go(const EightArgs& a, bool vec, cudaStream_t st) {
  const long long per = kThreads8 / (vec ? kBlock8 / Vec16<T>::N : 32);
  const auto with = [&](auto u) {
    constexpr int U = decltype(u)::value;
    const unsigned grid = (unsigned)units(a.pieces, per * U);
    if (!vec) return launch_early(k_eight_any<T, SAVE, U>, grid, kThreads8, 0, 1, st, a);
    const auto of = [&](auto one) {
      constexpr bool ONE = decltype(one)::value;
      if constexpr (SAVE) return launch_early(a.e5 ? k_save_vec<T, true, U, ONE> : k_save_vec<T, false, U, ONE>, grid, kThreads8, 0, 1, st, a);
      else return launch_early(a.e5 ? k_restore_vec<T, true, U, ONE> : k_restore_vec<T, false, U, ONE>, grid, kThreads8, 0, 1, st, a);
    };
    return a.rows == 1 ? of(std::true_type()) : of(std::false_type());
  };
  return a.pieces > per * 4 * 512 ? with(std::integral_constant<int, 4>()) : with(std::integral_constant<int, 1>());
}

template <bool SAVE> int run(const std::string& who, const void* x, int32_t dtype, int64_t stride, int64_t rows, int64_t dim,
                             void* codes, int32_t code, float* scales, int32_t device, void* stream) {
  const int rc = check(who, x, dtype, stride, rows, dim, codes, code, scales, SAVE, device);
  if (rc) return rc;
  if (rows == 0) return PSGD_OK;
  // rows without gaps of whole blocks are one long row
  if (dim % kBlock8 == 0 && (stride == dim || rows == 1) && rows * dim < (1LL << 30)) {
    dim *= rows;
    rows = 1;
    stride = dim;
  }
  const long long blocks = blocks8(dim);
  if (rows * blocks > 0xffffffffLL) return fail(PSGD_EINVAL, who + ": too many elements");
  DeviceScope scope(device);
  EightArgs a{x, stride, (unsigned char*)codes, scales, rows, (unsigned)(rows * blocks),
              blocks == 1 ? 0 : ~0ull / (unsigned long long)blocks + 1, (int)dim, (int)blocks, code == PSGD_E5M2};
  const cudaStream_t st = (cudaStream_t)stream;
  const int full = 16 / dtype_size(dtype);
  const bool vec = dim % full == 0 && aligned16(x) && (stride * dtype_size(dtype)) % 16 == 0 && (uintptr_t)codes % full == 0;
  const cudaError_t e = dtype == PSGD_F32   ? go<SAVE, float>(a, vec, st)
                        : dtype == PSGD_F16 ? go<SAVE, __half>(a, vec, st)
                                            : go<SAVE, __nv_bfloat16>(a, vec, st);
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
