// Root-mean-square norm over the last dimension, forward and backward.
//
//   forward   s = x + residual (rounded to x's type: it is what is kept), r = (mean(s^2) + eps)^-1/2,
//             y = s r w, in x's type or in 8 bits (psgd_eight.cuh)
//   backward  xh = s r, a = g w, dx = r (a - xh mean(a xh)) + gs, dw = sum_rows g xh
//             with s as it was kept: in its type, or 8-bit codes and scales
//
// One group of threads takes a whole row, which stays in registers between its
// sum and its result, so every operand is read once and every result written
// once.  In the backward pass a thread owns the same columns of every row it meets and
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
constexpr int kPartsPerSm = 2;     // partial rows of dw, at most
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

// Rows of any length and alignment: a warp's unit is a block of 128 columns, four a lane, 32 apart.
__device__ __forceinline__ void load_unit(const void* w, int dtype, int c, int dim, float none, float (&f)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = c + 32 * e < dim ? (w ? load_any(w, dtype, c + 32 * e) : none) : 0.f;
}
template <typename T> __device__ __forceinline__ void load_unit(const T* row, int c, int dim, float (&f)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = c + 32 * e < dim ? to_f(row[c + 32 * e]) : 0.f;
}
template <typename T> __device__ __forceinline__ void put_unit(T* row, int c, int dim, const float (&f)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (c + 32 * e < dim) row[c + 32 * e] = from_f<T>(f[e]);
}
__device__ __forceinline__ void put_codes(unsigned char* row, float* scales, int c, int dim, bool e5, const float (&f)[4]) {
  unsigned code[1];
  float scale;
  encode<4, 32>(e5, f, code, scale);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (c + 32 * e < dim) row[c + 32 * e] = (unsigned char)(code[0] >> (8 * e));
  if (c % kBlock8 == 0 && c < dim) scales[c / kBlock8] = scale;
}

// The kernels for rows of whole 16-byte units.  A group takes R rows at a time, which share the barriers and shuffles
// of one reduction; the rows of the next two turns are copied ahead into shared memory, by the thread that will use
// them, so that neither a register nor a barrier waits for what is under way.  Forward 32768 x 1600 bf16 with a residual
// 73 us (5.8 TB/s, 85 % of the copy rate; 77 with plain loads a row ahead), 16384 x 1024 into 8 bits 23: HBM, and
// instructions at 58 % of the issue slots.  Backward 65536 x 1600 bf16 from 8 bits with a residual's gradient 131 us
// (5.6 TB/s; 246 with plain loads, 144 with one row a turn and two CTAs an SM).
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
          // (a scale is a power of two: its product with rstd is exact, and one multiplication an element does for both)
          const float scale = scales[stage][r * NV + j][mine_8] * rstd[r];
          float f[E];
          const unsigned* code = reinterpret_cast<const unsigned*>(src + kThreadsMost);
#pragma unroll
          for (int k = 0; k < E / 4; ++k) decode4(a.e5, code[k], scale, f + 4 * k);
#pragma unroll
          for (int h = 0; h < NP; ++h) xh[r][j][h] = f2(f[2 * h], f[2 * h + 1]);
        } else {
          to_pairs<T>(src[kThreadsMost], xh[r][j]);
#pragma unroll
          for (int h = 0; h < NP; ++h) xh[r][j][h] = mul(xh[r][j][h], rs);
        }
#pragma unroll
        for (int h = 0; h < NP; ++h) {
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

// The kernels for rows of any length and alignment.  The rows' aligned 16-byte granules are copied ahead into shared
// memory, at the rows' own places within their first granules, and read from there element by element; a barrier of the
// group follows each wait, as a granule is used by other threads than the one that copied it.  Backward 4099 x 1023 f16
// 13.5 us with the columns' sums (17.0 with plain loads): four turns of four rows a group, of which the last is 37 % full, and
// two launches.
// Bytes of one turn of a group: R rows of `arrays` arrays, and (backward) the rows' scales.
__host__ __device__ inline int any_turn(int r, int arrays, int slot, int blocks) { return r * (arrays * slot + units(blocks, 4) * 16); }

template <typename T, int NB, int R>
__global__ void __launch_bounds__(kThreadsMost, 1) k_rms_forward_any(RmsArgs a) {
  extern __shared__ __align__(16) unsigned char slots[];
  __shared__ float red[2][kThreadsMost / 32 * R];
  const int t = threadIdx.x, group = threadIdx.y, threads = blockDim.x;
  const int warps = threads / 32, warp = t >> 5, lane = t & 31;
  const int arrays = a.residual ? 2 : 1, slot = slot_bytes(warps * NB * kBlock8, sizeof(T)), turn = R * arrays * slot;
  unsigned char* mine = slots + group * kAhead * turn;
  const int first = warp * NB * kBlock8 + lane;
  const float inv = 1.f / (float)a.dim;
  const int step = gridDim.x * blockDim.y * R;
  int row = ((int)blockIdx.x * blockDim.y + group) * R, ahead = row;
  const CopyShare share(R * arrays, warps, warp);
  auto issue = [&](int stage) {
    for (int i = share.first; i < R * arrays; i += share.step) {
      const bool second = i >= R;
      const int r = ahead + (second ? i - R : i);
      if (r < (int)a.rows)
        copy_row(mine + stage * turn + i * slot, (const T*)(second ? a.residual : a.x), r, second ? a.rs : a.xs, a.dim,
                 share.part * 32 + lane, share.parts * 32);
    }
    commit_copies();
    ahead = ahead < (int)a.rows ? ahead + step : ahead;
  };
  after_previous();
  next_may_launch();
#pragma unroll
  for (int k = 0; k < kAhead - 1; ++k) issue(k);
  float w[NB][4];
#pragma unroll
  for (int b = 0; b < NB; ++b) load_unit(a.w, a.pdtype, first + b * kBlock8, a.dim, 1.f, w[b]);
  int stage = 0, flip = 0;
  for (; row < (int)a.rows; row += step, flip ^= 1) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 2) : "memory");
    group_barrier(group, threads);
    issue(stage == 0 ? kAhead - 1 : stage - 1);
    const int rows = min(R, (int)a.rows - row);
    float s[R][NB][4], sum[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      sum[r] = 0.f;
      const unsigned char* at = mine + stage * turn + r * slot;
      const T* x = (const T*)(at + row_phase(a.x, row + r, a.xs, sizeof(T)));
      const T* res = (const T*)(at + R * slot + row_phase(a.residual, row + r, a.rs, sizeof(T)));
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int c = first + b * kBlock8;
        load_unit(x, c, r < rows ? a.dim : 0, s[r][b]);
        if (a.residual) {
          float more[4];
          load_unit(res, c, r < rows ? a.dim : 0, more);
#pragma unroll
          for (int e = 0; e < 4; ++e) s[r][b][e] = to_f(from_f<T>(s[r][b][e] + more[e]));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[r] = fmaf(s[r][b][e], s[r][b][e], sum[r]);
        if (a.summed && r < rows) put_unit((T*)a.summed + (row + r) * a.ss, c, a.dim, s[r][b]);
      }
    }
    stage = stage + 1 == kAhead ? 0 : stage + 1;
    group_sum<R>(sum, red[flip] + group * warps * R, warps, warp, lane, group, threads);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r >= rows) break;
      const float rstd = rsqrtf(fmaf(sum[r], inv, a.eps));
      if (t == 0) a.rstd[row + r] = rstd;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int c = first + b * kBlock8;
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = s[r][b][e] * rstd * w[b][e];
        if (a.codes) put_codes(a.codes + (long long)(row + r) * a.dim, a.scales + (long long)(row + r) * a.blocks, c, a.dim, a.e5, y);
        else put_unit((T*)a.y + (row + r) * a.ys, c, a.dim, y);
      }
    }
  }
}

template <typename T, int NB, int R, bool SAVED>
__global__ void __launch_bounds__(kThreadsMost, 1) k_rms_backward_any(RmsArgs a) {
  extern __shared__ __align__(16) unsigned char slots[];
  __shared__ float red[2][kThreadsMost / 32 * R];
  __shared__ float stats[kAhead][kThreadsMost / 32][R];  // each warp's own copy of the rows' rstd
  const int t = threadIdx.x, group = threadIdx.y, threads = blockDim.x;
  const int warps = threads / 32, warp = t >> 5, lane = t & 31, cta_warp = group * warps + warp;
  const int arrays = a.residual && a.y ? 3 : 2, slot = slot_bytes(warps * NB * kBlock8, sizeof(T));
  const int turn = any_turn(R, arrays, slot, SAVED ? a.blocks : 0);
  unsigned char* mine = slots + group * kAhead * turn;
  const int first = warp * NB * kBlock8 + lane;
  const float inv = 1.f / (float)a.dim;
  const int step = gridDim.x * blockDim.y * R;
  int row = ((int)blockIdx.x * blockDim.y + group) * R, ahead = row;
  const CopyShare share(R * arrays, warps, warp);
  auto scales_of = [&](int stage, int r) { return reinterpret_cast<float*>(mine + stage * turn + R * arrays * slot) + r * (int)units(a.blocks, 4) * 4; };
  auto issue = [&](int stage) {
    for (int i = share.first; i < R * arrays; i += share.step) {
      const int array = i / R, r = ahead + i - array * R;
      if (r >= (int)a.rows) continue;
      unsigned char* to = mine + stage * turn + i * slot;
      const int u = share.part * 32 + lane, by = share.parts * 32;
      if (SAVED && array == 1) copy_row(to, (const unsigned char*)a.codes, r, a.dim, a.dim, u, by);
      else copy_row(to, (const T*)(array == 0 ? a.g : array == 1 ? a.x : a.residual), r, array == 0 ? a.gs : array == 1 ? a.xs : a.rs, a.dim, u, by);
    }
    if constexpr (SAVED)
      for (int r = 0; r < R; ++r)
        for (int b = t; b < a.blocks; b += threads)
          if (ahead + r < (int)a.rows) copy4(scales_of(stage, r) + b, a.scales + (long long)(ahead + r) * a.blocks + b);
    if (lane < R && ahead + lane < (int)a.rows) copy4(&stats[stage][cta_warp][lane], a.rstd + ahead + lane);
    commit_copies();
    ahead = ahead < (int)a.rows ? ahead + step : ahead;
  };
  after_previous();
#pragma unroll
  for (int k = 0; k < kAhead - 1; ++k) issue(k);
  float w[NB][4], dw[NB][4];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    load_unit(a.w, a.pdtype, first + b * kBlock8, a.dim, 1.f, w[b]);
#pragma unroll
    for (int e = 0; e < 4; ++e) dw[b][e] = 0.f;
  }
  int stage = 0, flip = 0;
  for (; row < (int)a.rows; row += step, flip ^= 1) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 2) : "memory");
    group_barrier(group, threads);
    issue(stage == 0 ? kAhead - 1 : stage - 1);
    const int rows = min(R, (int)a.rows - row);
    const unsigned char* data = mine + stage * turn;
    float xh[R][NB][4], ga[R][NB][4], sum[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      sum[r] = 0.f;
      rstd[r] = stats[stage][cta_warp][r];
      const int dim = r < rows ? a.dim : 0;
      const T* g = (const T*)(data + r * slot + row_phase(a.g, row + r, a.gs, sizeof(T)));
      const unsigned char* kept = data + (R + r) * slot;
      kept += SAVED ? row_phase(a.codes, row + r, a.dim, 1) : row_phase(a.x, row + r, a.xs, sizeof(T));
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int c = first + b * kBlock8;
        load_unit(g, c, dim, ga[r][b]);
        if constexpr (SAVED) {
          unsigned code = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c + 32 * e < dim) code |= (unsigned)kept[c + 32 * e] << (8 * e);
          decode4(a.e5, code, c < dim ? scales_of(stage, r)[c / kBlock8] : 1.f, xh[r][b]);
        } else {
          load_unit((const T*)kept, c, dim, xh[r][b]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // (a row that is none: its rstd may be anything)
          xh[r][b][e] = r < rows ? xh[r][b][e] * rstd[r] : 0.f;
          dw[b][e] = fmaf(ga[r][b][e], xh[r][b][e], dw[b][e]);
          ga[r][b][e] *= w[b][e];
          sum[r] = fmaf(ga[r][b][e], xh[r][b][e], sum[r]);
        }
      }
    }
    if (a.y) {
      group_sum<R>(sum, red[flip] + group * warps * R, warps, warp, lane, group, threads);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r >= rows) break;
        const float m = -sum[r] * inv;
        const T* more = (const T*)(data + (2 * R + r) * slot + row_phase(a.residual, row + r, a.rs, sizeof(T)));
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const int c = first + b * kBlock8;
          float d[4], f[4];
          if (arrays == 3) load_unit(more, c, a.dim, f);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            d[e] = fmaf(xh[r][b][e], m, ga[r][b][e]) * rstd[r];
            if (arrays == 3) d[e] += f[e];
          }
          put_unit((T*)a.y + (row + r) * a.ys, c, a.dim, d);
        }
      }
    }
    stage = stage + 1 == kAhead ? 0 : stage + 1;
  }
  next_may_launch();
  if (!a.part) return;
  // the groups' sums in group order, through the rows' memory
  float* out = a.part + (long long)blockIdx.x * a.dim;
  float* cols = reinterpret_cast<float*>(slots);
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  for (int y = 0; y < (int)blockDim.y; ++y) {
    __syncthreads();
    if (group != y) continue;
    float* dst = y + 1 < (int)blockDim.y ? cols : out;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = first + b * kBlock8 + 32 * e;
        if (c < a.dim) dst[c] = (y ? cols[c] : 0.f) + dw[b][e];
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
  const int first = ((int)threadIdx.x >> 5) * kBlock8 + (threadIdx.x & 31), step = (int)blockDim.x / 32 * kBlock8;
  // (all lanes of a warp take part in a block or none does: encode() is a matter of the warp)
  const int end = a.blocks * kBlock8;
  auto sum_of = [&](long long row, int c, float (&s)[4]) {
    load_unit((const T*)a.x + row * a.xs, c, a.dim, s);
    if (!a.residual) return;
    float r[4];
    load_unit((const T*)a.residual + row * a.rs, c, a.dim, r);
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = to_f(from_f<T>(s[e] + r[e]));
  };
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float sum = 0.f;
    for (int c = first; c < end; c += step) {
      float s[4];
      sum_of(row, c, s);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum = fmaf(s[e], s[e], sum);
    }
    const float rstd = rsqrtf(fmaf(cta_sum(sum, buf), 1.f / (float)a.dim, a.eps));
    if (threadIdx.x == 0) a.rstd[row] = rstd;
    for (int c = first; c < end; c += step) {
      float s[4], w[4], y[4];
      sum_of(row, c, s);  // before the sum is written: it may take x's or the residual's place
      if (a.summed) put_unit((T*)a.summed + row * a.ss, c, a.dim, s);
      load_unit(a.w, a.pdtype, c, a.dim, 1.f, w);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = s[e] * rstd * w[e];
      if (a.codes) put_codes(a.codes + row * a.dim, a.scales + row * a.blocks, c, a.dim, a.e5, y);
      else put_unit((T*)a.y + row * a.ys, c, a.dim, y);
    }
  }
}
template <typename T> __global__ void __launch_bounds__(kThreadsMost) k_rms_dx_long(RmsArgs a) {
  __shared__ float buf[kThreadsMost / 32];
  const int first = ((int)threadIdx.x >> 5) * kBlock8 + (threadIdx.x & 31), step = (int)blockDim.x / 32 * kBlock8;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float rs = a.rstd[row];
    float sum = 0.f;
    for (int pass = 0; pass < 2; ++pass) {
      const float m = -sum / (float)a.dim;
      for (int c = first; c < a.dim; c += step) {
        float s[4], g[4], w[4];
        if (a.codes) {
          const float scale = a.scales[row * a.blocks + c / kBlock8];
#pragma unroll
          for (int e = 0; e < 4; ++e) s[e] = c + 32 * e < a.dim ? decode1(a.e5, a.codes[row * a.dim + c + 32 * e], scale) : 0.f;
        } else {
          load_unit((const T*)a.x + row * a.xs, c, a.dim, s);
        }
        load_unit((const T*)a.g + row * a.gs, c, a.dim, g);
        load_unit(a.w, a.pdtype, c, a.dim, 1.f, w);
        if (pass == 0) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sum = fmaf(g[e] * w[e], s[e] * rs, sum);
          continue;
        }
        float d[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] = fmaf(s[e] * rs, m, g[e] * w[e]) * rs;
        if (a.residual) {
          float more[4];
          load_unit((const T*)a.residual + row * a.rs, c, a.dim, more);
#pragma unroll
          for (int e = 0; e < 4; ++e) d[e] += more[e];
        }
        put_unit((T*)a.y + row * a.ys, c, a.dim, d);
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
  if (c < dim) {
#pragma unroll 4
    for (int p = warp; p < parts; p += kColumnWarps) sum += __ldcg(part + p * dim + c);
  }
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
// f(units of a thread, rows of a turn) for rows of whole units: `r1` rows where a thread has one unit of each, or one row
// where there are few, that is, no more than groups on all SMs: 300 x 1024 bf16 forward 2.1 us (two rows 2.5), backward 4.6
// (4.9), but 1216 x 1600 3.3 with two rows (3.6 with one), backward 7.0 (7.8), and 9728 x 1600 backward 23.7 (28.5).
template <typename T, int R1, typename F> void by_vec_plan(const Plan& p, bool few, F&& f) {
  if (p.nv == 1) few ? f(Int<1>(), Int<1>()) : f(Int<1>(), Int<R1>());
  else if (p.nv == 2) f(Int<2>(), Int<(R1 + 1) / 2>());
  else if constexpr (Vec16<T>::N * 4 <= kElements) f(Int<4>(), Int<1>());
}
// The same for any rows (300 x 1023 bf16 forward 3.0 us one row a turn, 4.3 four, backward 6.1 and 6.5; 1216 rows 5.8 and 4.4, 10.3
// and 7.1), whose `arrays` (and scales) have to fit into shared memory; false where not even one row of each does.
template <typename F> bool by_any_plan(const Plan& p, bool few, int size, int arrays, int blocks, int& bytes, F&& f) {
  const int slot = slot_bytes(p.threads / 32 * p.nv * kBlock8, size);
  const auto fits = [&](int r) {
    bytes = p.groups * kAhead * any_turn(r, arrays, slot, blocks);
    return bytes <= kMostStaged;
  };
  if (p.nv == 1 && !few && fits(4)) f(Int<1>(), Int<4>());
  else if (p.nv == 2 && !few && fits(2)) f(Int<2>(), Int<2>());
  else if (!fits(1)) return false;
  else if (p.nv == 1) f(Int<1>(), Int<1>());
  else if (p.nv == 2) f(Int<2>(), Int<1>());
  else f(Int<4>(), Int<1>());
  return true;
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
template <typename K> cudaError_t launch_any(K kernel, std::atomic<unsigned long long>& raised, const Plan& p, int bytes, unsigned grid, int device,
                                             cudaStream_t st, const RmsArgs& a) {
  const cudaError_t e = raise_smem(kernel, raised, device, kMostStaged);
  return e != cudaSuccess ? e : launch_early(kernel, grid, dim3(p.threads, p.groups), bytes, 1, st, a);
}
template <typename T, int NB, int R>
cudaError_t forward_any(const RmsArgs& a, const Plan& p, int bytes, int sms, int device, cudaStream_t st) {
  static std::atomic<unsigned long long> raised{0};
  return launch_any(k_rms_forward_any<T, NB, R>, raised, p, bytes, turns_of(p, R, a.rows, sms), device, st, a);
}
template <typename T, int NB, int R, bool SAVED>
cudaError_t backward_any(const RmsArgs& a, const Plan& p, int bytes, unsigned grid, int device, cudaStream_t st) {
  static std::atomic<unsigned long long> raised{0};
  return launch_any(k_rms_backward_any<T, NB, R, SAVED>, raised, p, bytes, grid, device, st, a);
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
    h->max_ctas = h->sms * kPartsPerSm;
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
    const bool few = rows <= (long long)h->sms * std::max(p.groups, 1);
    int bytes = 0;
    if (p.nv && vec) {
      by_vec_plan<T, 2>(p, few, [&](auto nv, auto r) {
        e = forward_vec<T, decltype(nv)::value, decltype(r)::value>(a, p, h->sms, h->device, st);
      });
    } else if (!p.nv || !by_any_plan(p, few, sizeof(T), residual ? 2 : 1, 0, bytes, [&](auto nb, auto r) {
                 e = forward_any<T, decltype(nb)::value, decltype(r)::value>(a, p, bytes, h->sms, h->device, st);
               })) {
      k_rms_forward_long<T><<<(unsigned)std::min<long long>(rows, h->sms * 4), kThreadsMost, 0, st>>>(a);
      e = cudaGetLastError();
    }
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
      const bool few = rows <= (long long)h->sms * std::max(p.groups, 1);
      int bytes = 0;
      if (vec && p.nv && p.nv < 4) {  // (three arrays of four units have no room for their turns)
        by_vec_plan<T, 2>(p, few, [&](auto nv, auto r) {
          constexpr int NV = decltype(nv)::value, R = decltype(r)::value;
          parts = (int)turns_of(p, R, rows, h->sms);
          e = codes ? backward_vec<T, NV, R, true>(a, p, parts, h->device, st) : backward_vec<T, NV, R, false>(a, p, parts, h->device, st);
        });
      } else if (!p.nv || !by_any_plan(p, few, sizeof(T), grad_summed && dx ? 3 : 2, codes ? a.blocks : 0, bytes, [&](auto nb, auto r) {
                   constexpr int NB = decltype(nb)::value, R = decltype(r)::value;
                   parts = (int)turns_of(p, R, rows, h->sms);
                   e = codes ? backward_any<T, NB, R, true>(a, p, bytes, parts, h->device, st)
                             : backward_any<T, NB, R, false>(a, p, bytes, parts, h->device, st);
                 })) {
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
      }
    });
  if (e == cudaSuccess && dweight)
    e = launch_early(k_rms_columns, (unsigned)units(dim, 32), 32 * kColumnWarps, 0, 1, st, h->part, parts, dim, dweight,
                     dparam_dtype, accumulate);
  return e == cudaSuccess ? PSGD_OK : cuda_fail(who.c_str(), e);
}
