// Root-mean-square norm over the last dimension, forward and backward.
//
//   forward   s = x + residual (rounded to x's type: it is what is kept), r = (mean(s^2) + eps)^-1/2,
//             y = s r w, in x's type or in 8 bits (psgd_eight.cuh)
//   backward  xh = s r, a = g w, dx = r (a - xh mean(a xh)) + gs, dw = sum_rows g xh
//             with s as it was kept: in its type, or 8-bit codes and scales
//
// One group of threads takes a whole row, which stays in registers between its
// sum and its result, so every operand is read once and every result written
// once.  While a row is summed, the loads of the group's next row are under way.
// In the backward pass a thread owns the same columns of every row it meets and
// keeps their dw sums in fp32 registers; a CTA leaves one partial row and a
// second kernel adds the partial rows in a fixed order.
#include <algorithm>
#include <atomic>
#include <new>
#include <type_traits>

#include "psgd_eight.cuh"
#include "psgd_rows.cuh"

struct psgd_rmsnorm {
  int device = 0;
  int sms = 0;
  long long dim = 0;
  int max_ctas = 0;       // partial rows
  float* part = nullptr;  // max_ctas x dim
  size_t bytes = 0;
};

namespace psgd {
namespace ops {
namespace {

constexpr int kThreadsMost = kRowThreads;  // of a CTA
constexpr int kCtasPerSm = 2;      // at most; one where a thread holds 16 elements of a row
constexpr int kElements = 16;      // of a row that a thread holds, at most

struct RmsArgs {
  const void* x;         // forward: x; backward: s where it was kept in its type
  const void* residual;  // forward, may be NULL; backward: gs, may be NULL
  const void* g;         // backward
  const void* w;         // may be NULL
  void* y;               // forward: y (NULL for 8 bits); backward: dx (may be NULL)
  void* summed;          // forward, may be NULL
  float* rstd;
  unsigned char* codes;  // 8 bits: of y (forward), of s (backward); else NULL
  float* scales;
  float* part;           // backward: partial rows of dw, may be NULL
  long long xs, rs, gs, ys, ss;  // row strides of x, residual, g, y, summed
  long long rows;
  int dim, blocks;       // blocks of 128 in a row
  int pdtype, e5;
  float eps;
};

// How a thread's columns lie.  V > 1: unit j of thread t is the 16 bytes t + j * threads of a row.  V = 1, rows of
// any alignment: a warp's unit is a block of 128 columns, lane by lane.  Either way the lanes of a block of 128 are
// neighbours.
template <typename T, int V> struct Unit {
  static constexpr int E = V == 1 ? 4 : V;              // elements
  static constexpr int LANES = kBlock8 / E;             // lanes of a block
  int first;  // column of element 0 of unit 0
  int step;   // columns between units
  __device__ __forceinline__ Unit(int t, int threads)
      : first(V == 1 ? (t >> 5) * kBlock8 + (t & 31) : t * V), step(V == 1 ? threads / 32 * kBlock8 : threads * V) {}
  __device__ __forceinline__ int col(int j, int e) const { return first + j * step + (V == 1 ? 32 * e : e); }
  // V > 1: a unit is in the row or not (a row is whole units)
  __device__ __forceinline__ bool in(int j, int e, int dim) const { return col(j, V == 1 ? e : 0) < dim; }
};

// A unit's raw elements, so that a load may be under way while nothing waits for it.
template <typename T, int V> struct Raw {
  static constexpr int E = Unit<T, V>::E;
  std::conditional_t<V == 1, T, uint4> v[V == 1 ? E : 1];
  __device__ __forceinline__ void load(const T* row, const Unit<T, V>& u, int j, int dim) {
    if constexpr (V == 1) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (u.in(j, e, dim)) v[e] = row[u.col(j, e)];
        else v[e] = from_f<T>(0.f);
    } else {
      v[0] = u.in(j, 0, dim) ? *reinterpret_cast<const uint4*>(row + u.col(j, 0)) : make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ void get(float (&f)[E]) const {
    if constexpr (V == 1) {
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = to_f(v[e]);
    } else {
      F2 p[E / 2];
      to_pairs<T>(v[0], p);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) split(p[i], f[2 * i], f[2 * i + 1]);
    }
  }
};
template <typename T, int V>
__device__ __forceinline__ void put(T* row, const Unit<T, V>& u, int j, int dim, const float (&f)[Unit<T, V>::E]) {
  if constexpr (V == 1) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (u.in(j, e, dim)) row[u.col(j, e)] = from_f<T>(f[e]);
  } else {
    if (u.in(j, 0, dim)) store_pack<T, V>(row + u.col(j, 0), f);
  }
}
// Codes of a unit: E bytes side by side (V > 1; the address is a multiple of E), or one by one.
template <typename T, int V> struct RawCodes {
  static constexpr int E = Unit<T, V>::E;
  unsigned v[E / 4];
  float scale;
  __device__ __forceinline__ void load(const unsigned char* row, const float* scales, const Unit<T, V>& u, int j, int dim) {
    scale = u.in(j, 0, dim) ? __ldg(scales + u.col(j, 0) / kBlock8) : 1.f;
    if constexpr (V == 1) {
      v[0] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (u.in(j, e, dim)) v[0] |= (unsigned)__ldg(row + u.col(j, e)) << (8 * e);
    } else if constexpr (E == 8) {
      const uint2 c = u.in(j, 0, dim) ? __ldg(reinterpret_cast<const uint2*>(row + u.col(j, 0))) : make_uint2(0, 0);
      v[0] = c.x;
      v[1] = c.y;
    } else {
      v[0] = u.in(j, 0, dim) ? __ldg(reinterpret_cast<const unsigned*>(row + u.col(j, 0))) : 0u;
    }
  }
  __device__ __forceinline__ void get(bool e5, float (&f)[E]) const {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) decode4(e5, v[i], scale, f + 4 * i);
  }
};
template <typename T, int V>
__device__ __forceinline__ void put_codes(unsigned char* row, float* scales, const Unit<T, V>& u, int j, int dim,
                                          const unsigned (&c)[Unit<T, V>::E / 4], float scale) {
  if constexpr (V == 1) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (u.in(j, e, dim)) row[u.col(j, e)] = (unsigned char)(c[0] >> (8 * e));
  } else if (u.in(j, 0, dim)) {
    if constexpr (Unit<T, V>::E == 8) *reinterpret_cast<uint2*>(row + u.col(j, 0)) = make_uint2(c[0], c[1]);
    else *reinterpret_cast<unsigned*>(row + u.col(j, 0)) = c[0];
  }
  if ((threadIdx.x & (Unit<T, V>::LANES - 1)) == 0 && u.in(j, 0, dim)) scales[u.col(j, 0) / kBlock8] = scale;
}
// A unit of a parameter of any type and alignment (`none` where there is no parameter).
template <typename T, int V>
__device__ __forceinline__ void load_weight(const void* w, int dtype, const Unit<T, V>& u, int j, int dim, float (&f)[Unit<T, V>::E]) {
#pragma unroll
  for (int e = 0; e < Unit<T, V>::E; ++e) f[e] = u.in(j, e, dim) ? (w ? load_any(w, dtype, u.col(j, e)) : 1.f) : 0.f;
}

// The sum of v over a group's threads, returned to all of them.  `buf` holds a float per warp of the group; the
// caller alternates between two of them, so that one barrier a call suffices.
__device__ __forceinline__ float row_sum(float v, float* buf, int warps, int warp, int lane, int group, int threads) {
  v = warp_sum(v);
  if (warps == 1) return v;
  if (lane == 0) buf[warp] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(threads) : "memory");
  return warp_sum(lane < warps ? buf[lane] : 0.f);
}

template <typename T, int V, int NV>
__global__ void __launch_bounds__(kThreadsMost, (Unit<T, V>::E * NV < kElements ? kCtasPerSm : 1)) k_rms_forward(RmsArgs a) {
  constexpr int E = Unit<T, V>::E;
  __shared__ float red[2][kThreadsMost / 32];
  const int t = threadIdx.x, group = threadIdx.y, threads = blockDim.x;
  const int warps = threads / 32, warp = t >> 5, lane = t & 31;
  const Unit<T, V> u(t, threads);
  const float inv = 1.f / (float)a.dim;
  const long long step = (long long)gridDim.x * blockDim.y;
  long long row = (long long)blockIdx.x * blockDim.y + group;
  Raw<T, V> x[NV], res[NV];
  auto fetch = [&](long long r) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      x[j].load((const T*)a.x + r * a.xs, u, j, a.dim);
      if (a.residual) res[j].load((const T*)a.residual + r * a.rs, u, j, a.dim);
    }
  };
  after_previous();
  next_may_launch();
  if (row < a.rows) fetch(row);
  float w[NV][E];
#pragma unroll
  for (int j = 0; j < NV; ++j) load_weight<T, V>(a.w, a.pdtype, u, j, a.dim, w[j]);
  int flip = 0;
  for (; row < a.rows; row += step, flip ^= 1) {
    float s[NV][E], sum = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      x[j].get(s[j]);
      if (a.residual) {
        float r[E];
        res[j].get(r);
#pragma unroll
        for (int e = 0; e < E; ++e) s[j][e] = to_f(from_f<T>(s[j][e] + r[e]));
      }
#pragma unroll
      for (int e = 0; e < E; ++e) sum = fmaf(s[j][e], s[j][e], sum);
    }
    if (row + step < a.rows) fetch(row + step);
    if (a.summed) {
#pragma unroll
      for (int j = 0; j < NV; ++j) put<T, V>((T*)a.summed + row * a.ss, u, j, a.dim, s[j]);
    }
    sum = row_sum(sum, red[flip] + group * warps, warps, warp, lane, group, threads);
    const float rstd = rsqrtf(fmaf(sum, inv, a.eps));
    if (t == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float y[E];
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = s[j][e] * rstd * w[j][e];
      if (a.codes) {
        unsigned c[E / 4];
        float scale;
        encode<E, Unit<T, V>::LANES>(a.e5, y, c, scale);
        put_codes<T, V>(a.codes + row * a.dim, a.scales + row * a.blocks, u, j, a.dim, c, scale);
      } else {
        put<T, V>((T*)a.y + row * a.ys, u, j, a.dim, y);
      }
    }
  }
}

template <typename T, int V, int NV, bool SAVED>
__global__ void __launch_bounds__(kThreadsMost, (Unit<T, V>::E * NV < kElements ? kCtasPerSm : 1)) k_rms_backward(RmsArgs a) {
  constexpr int E = Unit<T, V>::E;
  extern __shared__ float cols[];
  __shared__ float red[2][kThreadsMost / 32];
  const int t = threadIdx.x, group = threadIdx.y, threads = blockDim.x;
  const int warps = threads / 32, warp = t >> 5, lane = t & 31;
  const Unit<T, V> u(t, threads);
  const float inv = 1.f / (float)a.dim;
  const long long step = (long long)gridDim.x * blockDim.y;
  long long row = (long long)blockIdx.x * blockDim.y + group;
  Raw<T, V> g[NV], gs[NV];
  std::conditional_t<SAVED, RawCodes<T, V>, Raw<T, V>> x[NV];
  float rstd = 0.f;
  auto fetch = [&](long long r) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      g[j].load((const T*)a.g + r * a.gs, u, j, a.dim);
      if constexpr (SAVED) x[j].load(a.codes + r * a.dim, a.scales + r * a.blocks, u, j, a.dim);
      else x[j].load((const T*)a.x + r * a.xs, u, j, a.dim);
    }
    rstd = __ldg(a.rstd + r);
  };
  after_previous();
  if (row < a.rows) fetch(row);
  float w[NV][E], dw[NV][E];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    load_weight<T, V>(a.w, a.pdtype, u, j, a.dim, w[j]);
#pragma unroll
    for (int e = 0; e < E; ++e) dw[j][e] = 0.f;
  }
  int flip = 0;
  for (; row < a.rows; row += step, flip ^= 1) {
    float xh[NV][E], ga[NV][E], sum = 0.f;
    const float rs = rstd;
    if (a.residual && a.y) {
#pragma unroll
      for (int j = 0; j < NV; ++j) gs[j].load((const T*)a.residual + row * a.rs, u, j, a.dim);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if constexpr (SAVED) x[j].get(a.e5, xh[j]);
      else x[j].get(xh[j]);
      g[j].get(ga[j]);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        xh[j][e] *= rs;
        dw[j][e] = fmaf(ga[j][e], xh[j][e], dw[j][e]);
        ga[j][e] *= w[j][e];
        sum = fmaf(ga[j][e], xh[j][e], sum);
      }
    }
    if (row + step < a.rows) fetch(row + step);
    if (!a.y) continue;
    sum = row_sum(sum, red[flip] + group * warps, warps, warp, lane, group, threads);
    const float m = -sum * inv;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float d[E], add[E];
      if (a.residual) gs[j].get(add);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        d[e] = fmaf(xh[j][e], m, ga[j][e]) * rs;
        if (a.residual) d[e] += add[e];
      }
      put<T, V>((T*)a.y + row * a.ys, u, j, a.dim, d);
    }
  }
  next_may_launch();
  if (!a.part) return;
  // the groups' sums in group order
  float* out = a.part + (long long)blockIdx.x * a.dim;
  for (int y = 0; y < (int)blockDim.y; ++y) {
    __syncthreads();
    if (group != y) continue;
    float* dst = y + 1 < (int)blockDim.y ? cols : out;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (u.in(j, e, a.dim)) dst[u.col(j, e)] = (y ? cols[u.col(j, e)] : 0.f) + dw[j][e];
  }
}

// The kernels for rows of whole 16-byte units.  A group takes R rows at a time, which share the barriers and shuffles
// of one reduction; the rows of the next two turns are copied ahead into shared memory, by the thread that will use
// them, so that neither a register nor a barrier waits for what is under way.
constexpr int kAhead = 3;  // turns: the one in use and those under way
// CTAs of an SM: two where a turn's rows leave the room (and 64 registers a thread suffice).
constexpr int ctas_of(int nv, int r) { return nv == 1 && r <= 2 ? 2 : 1; }

template <typename T, int NV, int R>
__global__ void __launch_bounds__(kThreadsMost, ctas_of(NV, R)) k_rms_forward_vec(RmsArgs a) {
  constexpr int E = Vec16<T>::N, NP = E / 2;
  extern __shared__ __align__(16) uint4 staged[];
  __shared__ float red[2][kThreadsMost / 32 * R];
  const int t = threadIdx.x, group = threadIdx.y, threads = blockDim.x;
  const int warps = threads / 32, warp = t >> 5, lane = t & 31;
  const int arrays = a.residual ? 2 : 1;
  const float inv = 1.f / (float)a.dim;
  uint4* mine = staged + group * threads + t;
  bool in[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) in[j] = (t + j * threads) * E < a.dim;
  const int step = gridDim.x * blockDim.y * R;
  int row = ((int)blockIdx.x * blockDim.y + group) * R;  // the turn's first row
  int left = (int)a.rows - row;                          // rows from the next turn to copy on
  const T* from_x = (const T*)a.x + row * a.xs + t * E;
  const T* from_r = (const T*)a.residual + row * a.rs + t * E;
  auto issue = [&](int stage) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (r < left && in[j]) {
          uint4* dst = mine + ((stage * R + r) * NV + j) * arrays * kThreadsMost;
          copy16(dst, from_x + r * a.xs + j * threads * E);
          if (a.residual) copy16(dst + kThreadsMost, from_r + r * a.rs + j * threads * E);
        }
    commit_copies();
    left -= step;
    from_x += step * a.xs;
    from_r += step * a.rs;
  };
  after_previous();
  next_may_launch();
#pragma unroll
  for (int k = 0; k < kAhead - 1; ++k) issue(k);
  F2 w[NV][NP];
#pragma unroll
  for (int j = 0; j < NV; ++j) load_param<NP>(a.w, a.pdtype, (long long)(t + j * threads) * E, in[j], 1.f, w[j]);
  int stage = 0, flip = 0;
  for (; row < (int)a.rows; row += step, flip ^= 1) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 2) : "memory");
    // (in the place of the turn before, which is used up)
    issue(stage == 0 ? kAhead - 1 : stage - 1);
    const int rows = min(R, (int)a.rows - row);
    F2 s[R][NV][NP];
    float sum[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      F2 squares = f2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const uint4* src = mine + ((stage * R + r) * NV + j) * arrays * kThreadsMost;
        const bool live = in[j] && r < rows;
        uint4 raw = live ? src[0] : make_uint4(0, 0, 0, 0);
        to_pairs<T>(raw, s[r][j]);
        if (a.residual) {
          F2 add2[NP];
          to_pairs<T>(live ? src[kThreadsMost] : make_uint4(0, 0, 0, 0), add2);
          float f[E];
#pragma unroll
          for (int h = 0; h < NP; ++h) {
            s[r][j][h] = add(s[r][j][h], add2[h]);
            split(s[r][j][h], f[2 * h], f[2 * h + 1]);
          }
          // rounded as it is kept
          if constexpr (sizeof(T) == 2) {
            raw = make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
            to_pairs<T>(raw, s[r][j]);
          } else {
            raw = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
          }
        }
        if (a.summed && live) *reinterpret_cast<uint4*>((T*)a.summed + (row + r) * a.ss + (t + j * threads) * E) = raw;
#pragma unroll
        for (int h = 0; h < NP; ++h) squares = fma(s[r][j][h], s[r][j][h], squares);
      }
      float u, v;
      split(squares, u, v);
      sum[r] = u + v;
    }
    stage = stage + 1 == kAhead ? 0 : stage + 1;
    group_sum<R>(sum, red[flip] + group * warps * R, warps, warp, lane, group, threads);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r >= rows) break;
      const float rstd = rsqrtf(fmaf(sum[r], inv, a.eps));
      if (t == 0) a.rstd[row + r] = rstd;
      const F2 rs = f2(rstd, rstd);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float y[E];
#pragma unroll
        for (int h = 0; h < NP; ++h) split(mul(mul(s[r][j][h], rs), w[j][h]), y[2 * h], y[2 * h + 1]);
        const int c = (t + j * threads) * E;
        if (a.codes) {
          unsigned code[E / 4];
          float scale;
          encode<E, kBlock8 / E>(a.e5, y, code, scale);
          if (!in[j]) continue;
          unsigned char* to = a.codes + (long long)(row + r) * a.dim + c;
          if constexpr (E == 8) *reinterpret_cast<uint2*>(to) = make_uint2(code[0], code[1]);
          else *reinterpret_cast<unsigned*>(to) = code[0];
          if (c % kBlock8 == 0) a.scales[(long long)(row + r) * a.blocks + c / kBlock8] = scale;
        } else if (in[j]) {
          store_pack<T, E>((T*)a.y + (row + r) * a.ys + c, y);
        }
      }
    }
  }
}

// SAVED: s is in 8 bits.
template <typename T, int NV, int R, bool SAVED>
__global__ void __launch_bounds__(kThreadsMost, 1) k_rms_backward_vec(RmsArgs a) {
  constexpr int E = Vec16<T>::N, NP = E / 2, LANES = kBlock8 / E;
  extern __shared__ __align__(16) uint4 staged[];
  __shared__ float red[2][kThreadsMost / 32 * R];
  __shared__ float stats[kAhead][kThreadsMost / 32][R];  // each warp's own copy of the rows' rstd
  __shared__ float scales[kAhead][R * NV][kThreadsMost / LANES];
  const int t = threadIdx.x, group = threadIdx.y, threads = blockDim.x;
  const int warps = threads / 32, warp = t >> 5, lane = t & 31, cta_warp = group * warps + warp;
  const int arrays = a.residual && a.y ? 3 : 2, mine_8 = (group * threads + t) / LANES;
  const float inv = 1.f / (float)a.dim;
  uint4* mine = staged + group * threads + t;
  bool in[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) in[j] = (t + j * threads) * E < a.dim;
  const int step = gridDim.x * blockDim.y * R;
  int row = ((int)blockIdx.x * blockDim.y + group) * R, ahead = row;
  auto issue = [&](int stage) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (ahead + r < (int)a.rows && in[j]) {
          const int c = (t + j * threads) * E;
          uint4* dst = mine + ((stage * R + r) * NV + j) * arrays * kThreadsMost;
          copy16(dst, (const T*)a.g + (ahead + r) * a.gs + c);
          if constexpr (SAVED) {
            const unsigned char* code = a.codes + (long long)(ahead + r) * a.dim + c;
            if constexpr (E == 8) copy8(dst + kThreadsMost, code);
            else copy4(dst + kThreadsMost, code);
            if (t % LANES == 0) copy4(&scales[stage][r * NV + j][mine_8], a.scales + (long long)(ahead + r) * a.blocks + c / kBlock8);
          } else {
            copy16(dst + kThreadsMost, (const T*)a.x + (ahead + r) * a.xs + c);
          }
          if (arrays == 3) copy16(dst + 2 * kThreadsMost, (const T*)a.residual + (ahead + r) * a.rs + c);
        }
    if (lane < R && ahead + lane < (int)a.rows) copy4(&stats[stage][cta_warp][lane], a.rstd + ahead + lane);
    commit_copies();
    ahead = ahead < (int)a.rows ? ahead + step : ahead;
  };
  after_previous();
#pragma unroll
  for (int k = 0; k < kAhead - 1; ++k) issue(k);
  F2 w[NV][NP], dw[NV][NP];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    load_param<NP>(a.w, a.pdtype, (long long)(t + j * threads) * E, in[j], 1.f, w[j]);
#pragma unroll
    for (int h = 0; h < NP; ++h) dw[j][h] = f2(0.f, 0.f);
  }
  int stage = 0, flip = 0;
  for (; row < (int)a.rows; row += step, flip ^= 1) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 2) : "memory");
    __syncwarp();  // the other lanes' copies of scales and statistics
    issue(stage == 0 ? kAhead - 1 : stage - 1);
    const int rows = min(R, (int)a.rows - row);
    const uint4* data = mine + stage * R * NV * arrays * kThreadsMost;
    F2 xh[R][NV][NP], ga[R][NV][NP];
    float sum[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      F2 along = f2(0.f, 0.f);
      rstd[r] = stats[stage][cta_warp][r];
      const F2 rs = f2(rstd[r], rstd[r]);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const uint4* src = data + (r * NV + j) * arrays * kThreadsMost;
        if (!in[j] || r >= rows) {
#pragma unroll
          for (int h = 0; h < NP; ++h) xh[r][j][h] = ga[r][j][h] = f2(0.f, 0.f);
          continue;
        }
        to_pairs<T>(src[0], ga[r][j]);
        if constexpr (SAVED) {
          const float scale = scales[stage][r * NV + j][mine_8];
          float f[E];
          const unsigned* code = reinterpret_cast<const unsigned*>(src + kThreadsMost);
#pragma unroll
          for (int k = 0; k < E / 4; ++k) decode4(a.e5, code[k], scale, f + 4 * k);
#pragma unroll
          for (int h = 0; h < NP; ++h) xh[r][j][h] = f2(f[2 * h], f[2 * h + 1]);
        } else {
          to_pairs<T>(src[kThreadsMost], xh[r][j]);
        }
#pragma unroll
        for (int h = 0; h < NP; ++h) {
          xh[r][j][h] = mul(xh[r][j][h], rs);
          dw[j][h] = fma(ga[r][j][h], xh[r][j][h], dw[j][h]);
          ga[r][j][h] = mul(ga[r][j][h], w[j][h]);
          along = fma(ga[r][j][h], xh[r][j][h], along);
        }
      }
      float u, v;
      split(along, u, v);
      sum[r] = u + v;
    }
    if (a.y) {
      group_sum<R>(sum, red[flip] + group * warps * R, warps, warp, lane, group, threads);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r >= rows) break;
        const float m = -sum[r] * inv;
        const F2 ms = f2(m, m), rs = f2(rstd[r], rstd[r]);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          if (!in[j]) continue;
          F2 more[NP];
          if (arrays == 3) to_pairs<T>(data[((r * NV + j) * 3 + 2) * kThreadsMost], more);
          float d[E];
#pragma unroll
          for (int h = 0; h < NP; ++h) {
            F2 x = mul(fma(xh[r][j][h], ms, ga[r][j][h]), rs);
            if (arrays == 3) x = add(x, more[h]);
            split(x, d[2 * h], d[2 * h + 1]);
          }
          store_pack<T, E>((T*)a.y + (row + r) * a.ys + (t + j * threads) * E, d);
        }
      }
    }
    stage = stage + 1 == kAhead ? 0 : stage + 1;
  }
  next_may_launch();
  if (!a.part) return;
  // the groups' sums in group order, through the rows' memory
  float* out = a.part + (long long)blockIdx.x * a.dim;
  float* cols = reinterpret_cast<float*>(staged);
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  for (int y = 0; y < (int)blockDim.y; ++y) {
    __syncthreads();
    if (group != y) continue;
    float* dst = y + 1 < (int)blockDim.y ? cols : out;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!in[j]) continue;
      const int c = (t + j * threads) * E;
#pragma unroll
      for (int h = 0; h < NP; ++h) {
        float u, v;
        split(dw[j][h], u, v);
        if (y) {
          u += cols[c + 2 * h];
          v += cols[c + 2 * h + 1];
        }
        *reinterpret_cast<float2*>(dst + c + 2 * h) = make_float2(u, v);
      }
    }
  }
}

// Rows too long for registers: one CTA a row, a warp a block of 128 at a time; read again (from L2) for the result.
__device__ __forceinline__ float cta_sum(float v, float* buf) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum((threadIdx.x & 31) < blockDim.x / 32 ? buf[threadIdx.x & 31] : 0.f);
}
template <typename T> __global__ void __launch_bounds__(kThreadsMost) k_rms_forward_long(RmsArgs a) {
  __shared__ float buf[kThreadsMost / 32];
  const Unit<T, 1> u(threadIdx.x, blockDim.x);
  const int rounds = (a.blocks + (int)blockDim.x / 32 - 1) / ((int)blockDim.x / 32);
  auto sum_of = [&](long long row, int j, float (&s)[4]) {
    Raw<T, 1> x;
    x.load((const T*)a.x + row * a.xs, u, j, a.dim);
    x.get(s);
    if (!a.residual) return;
    float r[4];
    x.load((const T*)a.residual + row * a.rs, u, j, a.dim);
    x.get(r);
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = to_f(from_f<T>(s[e] + r[e]));
  };
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float sum = 0.f;
    for (int j = 0; j < rounds; ++j) {
      float s[4];
      sum_of(row, j, s);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum = fmaf(s[e], s[e], sum);
    }
    const float rstd = rsqrtf(fmaf(cta_sum(sum, buf), 1.f / (float)a.dim, a.eps));
    if (threadIdx.x == 0) a.rstd[row] = rstd;
    for (int j = 0; j < rounds; ++j) {
      float s[4], w[4], y[4];
      sum_of(row, j, s);  // before the sum is written: it may take x's or the residual's place
      if (a.summed) put<T, 1>((T*)a.summed + row * a.ss, u, j, a.dim, s);
      load_weight<T, 1>(a.w, a.pdtype, u, j, a.dim, w);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = s[e] * rstd * w[e];
      if (a.codes) {
        unsigned c[1];
        float scale;
        encode<4, 32>(a.e5, y, c, scale);
        put_codes<T, 1>(a.codes + row * a.dim, a.scales + row * a.blocks, u, j, a.dim, c, scale);
      } else {
        put<T, 1>((T*)a.y + row * a.ys, u, j, a.dim, y);
      }
    }
  }
}
template <typename T> __device__ __forceinline__ void kept(const RmsArgs& a, long long row, const Unit<T, 1>& u, int j, float (&s)[4]) {
  if (a.codes) {
    RawCodes<T, 1> c;
    c.load(a.codes + row * a.dim, a.scales + row * a.blocks, u, j, a.dim);
    c.get(a.e5, s);
  } else {
    Raw<T, 1> x;
    x.load((const T*)a.x + row * a.xs, u, j, a.dim);
    x.get(s);
  }
}
template <typename T> __global__ void __launch_bounds__(kThreadsMost) k_rms_dx_long(RmsArgs a) {
  __shared__ float buf[kThreadsMost / 32];
  const Unit<T, 1> u(threadIdx.x, blockDim.x);
  const int rounds = (a.blocks + (int)blockDim.x / 32 - 1) / ((int)blockDim.x / 32);
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float rs = a.rstd[row];
    float sum = 0.f;
    for (int pass = 0; pass < 2; ++pass) {
      const float m = -sum / (float)a.dim;
      for (int j = 0; j < rounds; ++j) {
        float s[4], g[4], w[4];
        Raw<T, 1> raw;
        kept<T>(a, row, u, j, s);
        raw.load((const T*)a.g + row * a.gs, u, j, a.dim);
        raw.get(g);
        load_weight<T, 1>(a.w, a.pdtype, u, j, a.dim, w);
        if (pass == 0) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sum = fmaf(g[e] * w[e], s[e] * rs, sum);
          continue;
        }
        float d[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] = fmaf(s[e] * rs, m, g[e] * w[e]) * rs;
        if (a.residual) {
          float add[4];
          raw.load((const T*)a.residual + row * a.rs, u, j, a.dim);
          raw.get(add);
#pragma unroll
          for (int e = 0; e < 4; ++e) d[e] += add[e];
        }
        put<T, 1>((T*)a.y + row * a.ys, u, j, a.dim, d);
      }
      if (pass == 0) sum = cta_sum(sum, buf);
    }
  }
}
// Partial rows of dw: gridDim.y of them, each over a run of rows; a thread a column.
template <typename T> __global__ void k_rms_dw_long(RmsArgs a) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= a.dim) return;
  const long long per = (a.rows + gridDim.y - 1) / gridDim.y, lo = per * blockIdx.y, hi = min(a.rows, lo + per);
  float sum = 0.f;
  for (long long row = lo; row < hi; ++row) {
    const float s = a.codes ? decode1(a.e5, a.codes[row * a.dim + c], a.scales[row * a.blocks + c / kBlock8])
                            : to_f(((const T*)a.x)[row * a.xs + c]);
    sum = fmaf(to_f(((const T*)a.g)[row * a.gs + c]), s * a.rstd[row], sum);
  }
  a.part[(long long)blockIdx.y * a.dim + c] = sum;
}

// dw from the partial rows: a CTA takes 32 columns, its warps share the rows.
constexpr int kColumnWarps = 16;
__global__ void __launch_bounds__(32 * kColumnWarps) k_rms_columns(const float* part, int parts, long long dim, void* dweight,
                                                                    int dtype, int accumulate) {
  __shared__ float sums[kColumnWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long c = (long long)blockIdx.x * 32 + lane;
  after_previous();
  next_may_launch();
  float sum = 0.f;
  if (c < dim)
    for (int p = warp; p < parts; p += kColumnWarps) sum += __ldcg(part + p * dim + c);
  sums[warp][lane] = sum;
  __syncthreads();
  if (warp || c >= dim) return;
  sum = 0.f;
#pragma unroll
  for (int k = 0; k < kColumnWarps; ++k) sum += sums[k][lane];
  store_any(dweight, dtype, c, accumulate ? read_any(dweight, dtype, c) + sum : sum);
}

template <typename F> void by_dtype(int32_t d, F&& f) {
  switch (d) {
    case PSGD_F32: f((float*)nullptr); break;
    case PSGD_F16: f((__half*)nullptr); break;
    default: f((__nv_bfloat16*)nullptr); break;
  }
}
template <int N> using Int = std::integral_constant<int, N>;
// A turn's memory: at most four units of a row (of 16 bytes), of two arrays or (backward) two of three, for each thread.
constexpr int kMostStaged = kAhead * 8 * kThreadsMost * 16;

// Threads of a group, groups of a CTA and units of a thread (0: the row is too long).
struct Plan {
  int threads = 0, groups = 0, nv = 0;
};
Plan plan_of(long long dim, int e) {
  Plan p;
  for (int nv = 1; nv * e <= kElements; nv *= 2) {
    const long long threads = units(units(dim, (long long)e * nv), 32) * 32;
    if (threads > kThreadsMost) continue;
    p.threads = (int)threads;
    p.groups = kThreadsMost / (int)threads;
    if (p.groups > 15) p.groups = 15;  // named barriers 1 to 15
    p.nv = nv;
    break;
  }
  return p;
}
// f(units of a thread, rows of a turn) for rows of whole units: `r1` rows where a thread has one unit of each, or one
// row where there are few; f(units) for any rows.
template <typename T, int R1, typename F> void by_vec_plan(const Plan& p, bool few, F&& f) {
  if (p.nv == 1) few ? f(Int<1>(), Int<1>()) : f(Int<1>(), Int<R1>());
  else if (p.nv == 2) f(Int<2>(), Int<(R1 + 1) / 2>());
  else if constexpr (Vec16<T>::N * 4 <= kElements) f(Int<4>(), Int<1>());
}
template <typename F> void by_any_plan(const Plan& p, F&& f) {
  if (p.nv == 1) f(Int<1>());
  else if (p.nv == 2) f(Int<2>());
  else f(Int<4>());
}
// Rows in one turn of a launch of one CTA an SM, and its CTAs.
unsigned turns_of(const Plan& p, int r, long long rows, int sms) {
  return (unsigned)std::min<long long>(units(rows, (long long)p.groups * r), sms);
}
template <typename K> cudaError_t launch_vec(K kernel, std::atomic<unsigned long long>& raised, const Plan& p, int stage_units, unsigned grid,
                                             int device, cudaStream_t st, const RmsArgs& a) {
  const cudaError_t e = raise_smem(kernel, raised, device, kMostStaged);
  if (e != cudaSuccess) return e;
  return launch_early(kernel, grid, dim3(p.threads, p.groups), (size_t)kAhead * stage_units * kThreadsMost * 16, 1, st, a);
}
template <typename T, int NV, int R>
cudaError_t forward_vec(const RmsArgs& a, const Plan& p, int sms, int device, cudaStream_t st) {
  static std::atomic<unsigned long long> raised{0};
  return launch_vec(k_rms_forward_vec<T, NV, R>, raised, p, R * NV * (a.residual ? 2 : 1), turns_of(p, R, a.rows, sms * ctas_of(NV, R)), device, st, a);
}
template <typename T, int NV, int R, bool SAVED>
cudaError_t backward_vec(const RmsArgs& a, const Plan& p, unsigned grid, int device, cudaStream_t st) {
  static std::atomic<unsigned long long> raised{0};
  return launch_vec(k_rms_backward_vec<T, NV, R, SAVED>, raised, p, R * NV * (a.residual && a.y ? 3 : 2), grid, device, st, a);
}

bool vec_ok(const void* p, long long stride, int dtype) {
  return !p || (aligned16(p) && (stride * dtype_size(dtype)) % 16 == 0);
}

int check_common(const std::string& w, const psgd_rmsnorm* h, int32_t dtype, int32_t pdtype, int64_t rows, int32_t code) {
  if (!h) return fail(PSGD_EINVAL, w + ": NULL norm");
  if (!dtype_ok(dtype) || !dtype_ok(pdtype)) return fail(PSGD_EINVAL, w + ": unknown dtype");
  if (code != PSGD_E4M3 && code != PSGD_E5M2) return fail(PSGD_EINVAL, w + ": unknown 8-bit format");
  if (rows < 0 || rows > (1 << 30)) return fail(PSGD_EINVAL, w + ": rows must be in [0, 2^30]");
  return PSGD_OK;
}
int check_operand(const std::string& who, const char* what, const void* p, int64_t rows, int64_t dim, int64_t stride, bool written) {
  const std::string w = who + ": " + what;
  if (rows > 0 && !p) return fail(PSGD_EINVAL, w + " is NULL");
  if (!span_ok(rows, stride)) return fail(PSGD_EINVAL, w + ": bad row stride");
  if (written && rows > 1 && stride < dim) return fail(PSGD_EINVAL, w + ": rows overlap");
  return PSGD_OK;
}
struct Range {
  const void* p;
  long long bytes;
};
// Whether one of `outs` shares a byte with one of `ins` or with another of `outs`.
template <size_t N, size_t M> bool any_overlap(const Range (&outs)[N], const Range (&ins)[M]) {
  for (size_t i = 0; i < N; ++i) {
    for (size_t k = 0; k < M; ++k)
      if (overlap(outs[i].p, outs[i].bytes, ins[k].p, ins[k].bytes)) return true;
    for (size_t k = 0; k < i; ++k)
      if (overlap(outs[i].p, outs[i].bytes, outs[k].p, outs[k].bytes)) return true;
  }
  return false;
}

}  // namespace
}  // namespace ops
}  // namespace psgd

using namespace psgd;
using namespace psgd::ops;

extern "C" int psgd_rmsnorm_create(int64_t dim, int32_t device, psgd_rmsnorm** out) {
  if (!out) return fail(PSGD_EINVAL, "psgd_rmsnorm_create: out is NULL");
  *out = nullptr;
  if (dim < 1 || dim > (1 << 20)) return fail(PSGD_EINVAL, "psgd_rmsnorm_create: dim must be in [1, 2^20]");
  if (device < 0 || device >= 64) return fail(PSGD_EINVAL, "psgd_rmsnorm_create: device ordinal must be in [0, 63]");
  int count = 0;
  cudaError_t e = cudaGetDeviceCount(&count);
  if (e != cudaSuccess) return cuda_fail("psgd_rmsnorm_create: cudaGetDeviceCount", e);
  if (device >= count) return fail(PSGD_ECUDA, "psgd_rmsnorm_create: no such device");
  psgd_rmsnorm* h = new (std::nothrow) psgd_rmsnorm;
  if (!h) return fail(PSGD_ENOMEM, "psgd_rmsnorm_create: out of host memory");
  DeviceScope scope(device);
  h->device = device;
  h->dim = dim;
  e = cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, device);
  if (e == cudaSuccess) {
    h->max_ctas = h->sms * kCtasPerSm;
    h->bytes = (size_t)h->max_ctas * dim * 4;
    e = cudaMalloc((void**)&h->part, h->bytes);
  }
  if (e != cudaSuccess) {
    const int rc = cuda_fail("psgd_rmsnorm_create", e);
    h->part = nullptr;
    psgd_rmsnorm_destroy(h);
    return rc;
  }
  *out = h;
  return PSGD_OK;
}

extern "C" void psgd_rmsnorm_destroy(psgd_rmsnorm* h) {
  if (!h) return;
  {
    DeviceScope scope(h->device);
    if (h->part) cudaFree(h->part);
  }
  delete h;
}

extern "C" size_t psgd_rmsnorm_workspace_bytes(const psgd_rmsnorm* h) { return h ? h->bytes : 0; }

extern "C" int psgd_rmsnorm_forward(psgd_rmsnorm* h, const void* x, psgd_dtype dtype, int64_t x_stride, int64_t rows,
                                    const void* residual, int64_t residual_stride, const void* weight,
                                    psgd_dtype param_dtype, float eps, void* y, int64_t y_stride, void* codes,
                                    psgd_code code, float* scales, void* summed, int64_t summed_stride, float* rstd,
                                    void* stream) {
  const std::string who = "psgd_rmsnorm_forward";
  int rc = check_common(who, h, dtype, param_dtype, rows, code);
  if (rc) return rc;
  if (!(eps >= 0.f) || !isfinite(eps)) return fail(PSGD_EINVAL, who + ": eps must be finite and >= 0");
  const long long dim = h->dim;
  rc = check_operand(who, "x", x, rows, dim, x_stride, false);
  if (!rc && residual) rc = check_operand(who, "residual", residual, rows, dim, residual_stride, false);
  if (!rc && !codes) rc = check_operand(who, "y", y, rows, dim, y_stride, true);
  if (!rc && summed) rc = check_operand(who, "summed", summed, rows, dim, summed_stride, true);
  if (rc) return rc;
  if (codes && y) return fail(PSGD_EINVAL, who + ": y and codes are both given");
  if (codes && rows > 0 && !scales) return fail(PSGD_EINVAL, who + ": scales is NULL");
  if (rows > 0 && !rstd) return fail(PSGD_EINVAL, who + ": rstd is NULL");
  const long long xb = extent(rows, dim, x_stride, dtype), rb = residual ? extent(rows, dim, residual_stride, dtype) : 0;
  const Range outs[] = {{y, y ? extent(rows, dim, y_stride, dtype) : 0}, {codes, rows * dim}, {scales, codes ? rows * blocks8(dim) * 4 : 0},
                        {rstd, rows * 4}};
  const Range sum[] = {{summed, summed ? extent(rows, dim, summed_stride, dtype) : 0}};
  const Range ins[] = {{x, xb}, {residual, rb}, {weight, dim * dtype_size(param_dtype)}, sum[0]};
  // the sum may take x's or the residual's place, and nothing else's
  const bool on_x = summed && summed == x && (summed_stride == x_stride || rows < 2);
  const bool on_residual = summed && summed == residual && (summed_stride == residual_stride || rows < 2);
  const Range kept[] = {{on_x ? nullptr : x, xb}, {on_residual ? nullptr : residual, rb}, ins[2]};
  if (any_overlap(outs, ins) || any_overlap(sum, kept)) return fail(PSGD_EINVAL, who + ": an output overlaps another operand");
  if (rows == 0) return PSGD_OK;
  DeviceScope scope(h->device);
  const cudaStream_t st = (cudaStream_t)stream;
  RmsArgs a{};
  a.x = x, a.residual = residual, a.w = weight, a.y = y, a.summed = summed, a.rstd = rstd;
  a.codes = (unsigned char*)codes, a.scales = scales;
  a.xs = x_stride, a.rs = residual_stride, a.ys = y_stride, a.ss = summed_stride;
  a.rows = rows, a.dim = (int)dim, a.blocks = (int)blocks8(dim), a.pdtype = param_dtype, a.e5 = code == PSGD_E5M2, a.eps = eps;
  const int full = 16 / dtype_size(dtype);
  const bool vec = dim % full == 0 && vec_ok(x, x_stride, dtype) && vec_ok(residual, residual_stride, dtype) &&
                   vec_ok(y, y_stride, dtype) && vec_ok(summed, summed_stride, dtype) && (uintptr_t)codes % full == 0;
  const Plan p = plan_of(dim, vec ? full : 4);
  cudaError_t e = cudaSuccess;
  by_dtype(dtype, [&](auto* tt) {
    using T = std::remove_pointer_t<decltype(tt)>;
    if (p.nv == 0) {
      k_rms_forward_long<T><<<(unsigned)std::min<long long>(rows, h->sms * 4), kThreadsMost, 0, st>>>(a);
      e = cudaGetLastError();
      return;
    }
    if (vec) {
      by_vec_plan<T, 2>(p, rows <= 4LL * h->sms * p.groups, [&](auto nv, auto r) {
        e = forward_vec<T, decltype(nv)::value, decltype(r)::value>(a, p, h->sms, h->device, st);
      });
      return;
    }
    const unsigned grid = (unsigned)std::min<long long>(units(rows, p.groups), h->sms * kCtasPerSm);
    by_any_plan(p, [&](auto nv) {
      e = launch_early(k_rms_forward<T, 1, decltype(nv)::value>, grid, dim3(p.threads, p.groups), 0, 1, st, a);
    });
  });
  return e == cudaSuccess ? PSGD_OK : cuda_fail(who.c_str(), e);
}

extern "C" int psgd_rmsnorm_backward(psgd_rmsnorm* h, const void* grad, psgd_dtype dtype, int64_t grad_stride, int64_t rows,
                                     const void* summed, int64_t summed_stride, const void* codes, psgd_code code,
                                     const float* scales, const float* rstd, const void* weight, psgd_dtype param_dtype,
                                     const void* grad_summed, int64_t grad_summed_stride, void* dx, int64_t dx_stride,
                                     void* dweight, psgd_dtype dparam_dtype, int32_t accumulate, void* stream) {
  const std::string who = "psgd_rmsnorm_backward";
  int rc = check_common(who, h, dtype, param_dtype, rows, code);
  if (rc) return rc;
  if (!dtype_ok(dparam_dtype)) return fail(PSGD_EINVAL, who + ": unknown dtype");
  const long long dim = h->dim;
  rc = check_operand(who, "grad", grad, rows, dim, grad_stride, false);
  if (!rc && !codes) rc = check_operand(who, "summed", summed, rows, dim, summed_stride, false);
  if (!rc && grad_summed) rc = check_operand(who, "grad_summed", grad_summed, rows, dim, grad_summed_stride, false);
  if (!rc && dx) rc = check_operand(who, "dx", dx, rows, dim, dx_stride, true);
  if (rc) return rc;
  if (codes && summed) return fail(PSGD_EINVAL, who + ": summed and codes are both given");
  if (codes && rows > 0 && !scales) return fail(PSGD_EINVAL, who + ": scales is NULL");
  if (rows > 0 && !rstd) return fail(PSGD_EINVAL, who + ": rstd is NULL");
  const long long gb = extent(rows, dim, grad_stride, dtype), ab = grad_summed ? extent(rows, dim, grad_summed_stride, dtype) : 0;
  const Range outs[] = {{dx, dx ? extent(rows, dim, dx_stride, dtype) : 0}, {dweight, dim * dtype_size(dparam_dtype)}};
  // dx may take the place of a gradient, and nothing else's
  const bool on_grad = dx && dx == grad && (dx_stride == grad_stride || rows < 2);
  const bool on_add = dx && dx == grad_summed && (dx_stride == grad_summed_stride || rows < 2);
  const Range fixed[] = {{summed, summed ? extent(rows, dim, summed_stride, dtype) : 0}, {codes, rows * dim},
                         {scales, codes ? rows * blocks8(dim) * 4 : 0}, {rstd, rows * 4}, {weight, dim * dtype_size(param_dtype)}};
  const Range grads[] = {{grad, gb}, {grad_summed, ab}};
  const Range dxs[] = {outs[0]}, dws[] = {outs[1]};
  const Range other[] = {{on_grad ? nullptr : grad, gb}, {on_add ? nullptr : grad_summed, ab}};
  if (any_overlap(outs, fixed) || any_overlap(dws, grads) || any_overlap(dxs, other))
    return fail(PSGD_EINVAL, who + ": an output overlaps another operand");
  if (!dweight && (!dx || rows == 0)) return PSGD_OK;
  DeviceScope scope(h->device);
  const cudaStream_t st = (cudaStream_t)stream;
  RmsArgs a{};
  a.x = summed, a.residual = grad_summed, a.g = grad, a.w = weight, a.y = dx, a.rstd = const_cast<float*>(rstd);
  a.codes = (unsigned char*)const_cast<void*>(codes), a.scales = const_cast<float*>(scales), a.part = dweight ? h->part : nullptr;
  a.xs = summed_stride, a.rs = grad_summed_stride, a.gs = grad_stride, a.ys = dx_stride;
  a.rows = rows, a.dim = (int)dim, a.blocks = (int)blocks8(dim), a.pdtype = param_dtype, a.e5 = code == PSGD_E5M2;
  const int full = 16 / dtype_size(dtype);
  const bool vec = dim % full == 0 && vec_ok(grad, grad_stride, dtype) && vec_ok(summed, summed_stride, dtype) &&
                   vec_ok(grad_summed, grad_summed_stride, dtype) && vec_ok(dx, dx_stride, dtype) && (uintptr_t)codes % full == 0;
  const Plan p = plan_of(dim, vec ? full : 4);
  int parts = 0;
  cudaError_t e = cudaSuccess;
  if (rows > 0)
    by_dtype(dtype, [&](auto* tt) {
      using T = std::remove_pointer_t<decltype(tt)>;
      if (p.nv == 0) {
        // (dx may take g's place: dw first)
        if (dweight) {
          parts = (int)std::min<long long>(units(rows, 32), h->max_ctas);
          k_rms_dw_long<T><<<dim3((unsigned)units(dim, 256), parts), 256, 0, st>>>(a);
          e = cudaGetLastError();
        }
        if (dx && e == cudaSuccess) {
          k_rms_dx_long<T><<<(unsigned)std::min<long long>(rows, h->sms * 4), kThreadsMost, 0, st>>>(a);
          e = cudaGetLastError();
        }
        return;
      }
      if (vec && p.nv < 4) {  // (three arrays of four units have no room for their turns)
        by_vec_plan<T, 2>(p, rows <= 4LL * h->sms * p.groups, [&](auto nv, auto r) {
          constexpr int NV = decltype(nv)::value, R = decltype(r)::value;
          parts = (int)turns_of(p, R, rows, h->sms);
          e = codes ? backward_vec<T, NV, R, true>(a, p, parts, h->device, st) : backward_vec<T, NV, R, false>(a, p, parts, h->device, st);
        });
        return;
      }
      parts = (int)std::min<long long>(units(rows, p.groups), h->max_ctas);
      const size_t smem = p.groups > 1 ? (size_t)dim * 4 : 0;
      by_any_plan(p, [&](auto nv) {
        auto go = [&](auto saved) {
          e = launch_early(k_rms_backward<T, 1, decltype(nv)::value, decltype(saved)::value>, (unsigned)parts, dim3(p.threads, p.groups), smem, 1,
                           st, a);
        };
        if (codes) go(std::true_type());
        else go(std::false_type());
      });
    });
  if (e == cudaSuccess && dweight)
    e = launch_early(k_rms_columns, (unsigned)units(dim, 32), 32 * kColumnWarps, 0, 1, st, h->part, parts, dim, dweight,
                     dparam_dtype, accumulate);
  return e == cudaSuccess ? PSGD_OK : cuda_fail(who.c_str(), e);
}
