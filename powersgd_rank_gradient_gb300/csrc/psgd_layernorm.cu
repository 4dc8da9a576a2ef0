// Layer norm over the last dimension, forward and backward.
//
//   forward   mu = mean(x), r = (mean((x - mu)^2) + eps)^-1/2, y = (x - mu) r w + b
//   backward  xh = (x - mu) r, a = g w
//             dx = r (a - mean(a) - xh mean(a xh)),  dw = sum_rows g xh,  db = sum_rows g
//
// One group of threads takes a whole row, which is copied into shared memory
// ahead of its use, so every operand is read from memory once.  The variance is
// the mean of the squared deviations from the mean (a second reduction over
// registers, no cancellation).  In the backward pass each thread owns the same
// columns of every row it meets and keeps their dw and db sums in fp32
// registers; a CTA leaves one partial row and a second kernel adds the partial
// rows in a fixed order.  Rows longer than a CTA's threads can hold (8192
// elements, 16384 of whole units of a 16-bit type) have kernels of their own,
// which read a row once per reduction.
#include <algorithm>
#include <atomic>
#include <new>
#include <type_traits>

#include "psgd_rows.cuh"

struct psgd_layernorm {
  int device = 0;
  int sms = 0;
  long long dim = 0;
  int max_ctas = 0;       // partial rows
  float* part = nullptr;  // max_ctas x 2 x dim
  size_t bytes = 0;
};

namespace psgd {
namespace ops {
namespace {

constexpr int kMaxThreads = kRowThreads;  // of a register kernel's CTA

struct RowsArgs {
  const void* x;
  const void* g;   // backward
  const void* w;
  const void* b;
  void* y;         // y (forward) or dx (backward)
  float* mean;
  float* rstd;
  float* part;     // backward
  long long xs, gs, ys;
  long long rows;
  int dim;
  int pdtype;
  float eps;
};

// The kernels for rows of whole 16-byte units.  blockDim = (threads of a group,
// groups); a group takes R rows at a time, thread t the vectors t, t + threads,
// ... (NV of them) of each.  The rows are copied kStages - 1 steps ahead into
// shared memory, by the thread that will use them, so no barrier is needed for
// them and no register holds what is under way.  Both are bound by HBM once
// there is enough of it: forward 65536 x 1024 bf16 41 us (6.5 TB/s), 16384 rows
// 12.9 us, three of which are the launch and the first rows' way; backward 65536
// x 1600 bf16 96 us with the columns' sums (6.6 TB/s, 97 % of the copy
// bandwidth; 173 us with plain loads one batch at a time, whose instructions and
// latency bound it).  Four rows at a time share the barriers and shuffles of one
// reduction (forward: 14.8 us with two).
constexpr int kStages = 3;

template <typename T, int NV, int R>
__global__ void __launch_bounds__(kMaxThreads, NV == 1 && R == 1 ? 2 : 1) k_norm_forward_vec(RowsArgs a) {
  constexpr int NE = Vec16<T>::N, NP = NE / 2;
  constexpr int kStep = R * NV;  // vectors of a stage per thread, kMaxThreads apart
  extern __shared__ __align__(16) uint4 staged[];
  __shared__ float red[2][kMaxThreads / 32 * R];
  const int t = threadIdx.x, group = threadIdx.y, threads = blockDim.x;
  const int warps = threads / 32, warp = t >> 5, lane = t & 31;
  float* buf[2] = {red[0] + group * warps * R, red[1] + group * warps * R};
  const int nvec = a.dim / NE;
  const float inv = 1.f / (float)a.dim;
  const int step = gridDim.x * blockDim.y * R;
  uint4* mine = staged + group * threads + t;
  bool in[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) in[j] = t + j * threads < nvec;
  int row = ((int)blockIdx.x * blockDim.y + group) * R;  // the batch's first row
  // rows left from the next batch to copy on, and this thread's first vector of it
  int left = (int)a.rows - row;
  const T* from = (const T*)a.x + row * a.xs + t * NE;
  const long long from_step = step * a.xs, to_step = step * a.ys;
  auto issue = [&](int stage) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (r < left && in[j])
          copy16(mine + ((stage * R + r) * NV + j) * kMaxThreads, from + r * a.xs + j * threads * NE);
    commit_copies();
    left -= step;
    from += from_step;
  };
  after_previous();
  next_may_launch();
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) issue(k);
  F2 w[NV][NP], bias[NV][NP];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int v = t + j * threads;
    load_param<NP>(a.w, a.pdtype, (long long)v * NE, in[j], 1.f, w[j]);
    load_param<NP>(a.b, a.pdtype, (long long)v * NE, in[j], 0.f, bias[j]);
  }
  T* to = (T*)a.y + row * a.ys + t * NE;
  int stage = 0;
  for (; row < (int)a.rows; row += step, to += to_step) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    issue(stage == 0 ? kStages - 1 : stage - 1);
    const int rows = min(R, (int)a.rows - row);
    F2 x[R][NV][NP];
    float s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      F2 sum = f2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        to_pairs<T>(in[j] ? mine[((stage * R + r) * NV + j) * kMaxThreads] : make_uint4(0, 0, 0, 0), x[r][j]);
#pragma unroll
        for (int h = 0; h < NP; ++h) sum = add(sum, x[r][j][h]);
      }
      float u, v;
      split(sum, u, v);
      s[r] = u + v;
    }
    stage = stage + 1 == kStages ? 0 : stage + 1;
    group_sum<R>(s, buf[0], warps, warp, lane, group, threads);
    float mean[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = s[r] * inv;
      const F2 nm = f2(-mean[r], -mean[r]);
      F2 sum = f2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int h = 0; h < NP; ++h) {
          x[r][j][h] = add(x[r][j][h], nm);
          if (in[j]) sum = fma(x[r][j][h], x[r][j][h], sum);
        }
      }
      float u, v;
      split(sum, u, v);
      s[r] = u + v;
    }
    group_sum<R>(s, buf[1], warps, warp, lane, group, threads);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r >= rows) break;
      const float rstd = rsqrtf(fmaf(s[r], inv, a.eps));
      if (t == 0) {
        if (a.mean) a.mean[row + r] = mean[r];
        if (a.rstd) a.rstd[row + r] = rstd;
      }
      const F2 rs = f2(rstd, rstd);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float f[NE];
#pragma unroll
        for (int h = 0; h < NP; ++h) split(fma(mul(x[r][j][h], rs), w[j][h], bias[j][h]), f[2 * h], f[2 * h + 1]);
        if (in[j]) store_pack<T, NE>(to + r * a.ys + j * threads * NE, f);
      }
    }
  }
}

// dx = rstd a - rstd m0 - xh rstd m1, with m0 = mean(a) and m1 = mean(a xh).  The
// mean comes off x first, so rows far from zero lose nothing, and rstd meets each
// deviation before anything else does: products of gradients and deviations, or
// powers of rstd, would leave fp32's range where the result does not (rstd is
// 1e19 and more where eps is 0 and a row hardly varies).
template <typename T, int NV, int R>
__global__ void __launch_bounds__(kMaxThreads, 1) k_norm_backward_vec(RowsArgs a) {
  constexpr int NE = Vec16<T>::N, NP = NE / 2;
  extern __shared__ __align__(16) uint4 staged[];
  __shared__ float red[2][kMaxThreads / 32 * 2 * R];
  __shared__ float stats[kStages][kMaxThreads / 32][2 * R];  // each warp's own copy of the rows' mean and rstd
  const int t = threadIdx.x, group = threadIdx.y, threads = blockDim.x;
  const int warps = threads / 32, warp = t >> 5, lane = t & 31, cta_warp = group * warps + warp;
  const int nvec = a.dim / NE;
  const float inv = 1.f / (float)a.dim;
  const int step = gridDim.x * blockDim.y * R;
  uint4* mine = staged + group * threads + t;
  bool in[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) in[j] = t + j * threads < nvec;
  int row = ((int)blockIdx.x * blockDim.y + group) * R;  // the batch's first row
  // rows left from the next batch to copy on, and this thread's first vectors of it
  int left = (int)a.rows - row;
  const T* from_x = (const T*)a.x + row * a.xs + t * NE;
  const T* from_g = (const T*)a.g + row * a.gs + t * NE;
  const float* from_s = (lane & 1 ? a.rstd : a.mean) + row + lane / 2;
  const long long x_step = step * a.xs, g_step = step * a.gs, y_step = step * a.ys;
  auto issue = [&](int stage) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (r < left && in[j]) {
          uint4* dst = mine + ((stage * R + r) * NV + j) * 2 * kMaxThreads;
          copy16(dst, from_x + r * a.xs + j * threads * NE);
          copy16(dst + kMaxThreads, from_g + r * a.gs + j * threads * NE);
        }
    if (lane < 2 * R && lane / 2 < left) copy4(&stats[stage][cta_warp][lane], from_s);
    commit_copies();
    left -= step;
    from_x += x_step;
    from_g += g_step;
    from_s += step;
  };
  after_previous();
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) issue(k);
  F2 dw[NV][NP], db[NV][NP], w[NV][NP];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int v = t + j * threads;
    load_param<NP>(a.w, a.pdtype, (long long)v * NE, in[j], 1.f, w[j]);
#pragma unroll
    for (int h = 0; h < NP; ++h) dw[j][h] = db[j][h] = f2(0.f, 0.f);
  }
  T* to = (T*)a.y + row * a.ys + t * NE;
  int stage = 0, flip = 0;
  for (; row < (int)a.rows; row += step, to += y_step) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();  // the other lanes' copies of the statistics
    issue(stage == 0 ? kStages - 1 : stage - 1);
    const uint4* data = mine + stage * R * NV * 2 * kMaxThreads;
    const float* stat = stats[stage][cta_warp];
    auto rows_of = [&](auto full) {
      const int rows = decltype(full)::value ? R : (int)a.rows - row;
      float s[2 * R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        F2 s0 = f2(0.f, 0.f), s1 = f2(0.f, 0.f);
        if (r < rows) {
          const F2 nm = f2(-stat[2 * r], -stat[2 * r]), rs = f2(stat[2 * r + 1], stat[2 * r + 1]);
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            if (!in[j]) continue;
            F2 x[NP], g[NP];
            to_pairs<T>(data[(r * NV + j) * 2 * kMaxThreads], x);
            to_pairs<T>(data[((r * NV + j) * 2 + 1) * kMaxThreads], g);
#pragma unroll
            for (int h = 0; h < NP; ++h) {
              const F2 gx = mul(g[h], mul(add(x[h], nm), rs));
              s0 = fma(g[h], w[j][h], s0);
              s1 = fma(gx, w[j][h], s1);
              dw[j][h] = add(dw[j][h], gx);
              db[j][h] = add(db[j][h], g[h]);
            }
          }
        }
        float u, v;
        split(s0, u, v);
        s[2 * r] = u + v;
        split(s1, u, v);
        s[2 * r + 1] = u + v;
      }
      if (!a.y) return;
      group_sum<2 * R>(s, red[flip] + group * warps * 2 * R, warps, warp, lane, group, threads);
      flip ^= 1;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r >= rows) break;
        const float mean = stat[2 * r], rstd = stat[2 * r + 1];
        const float c0 = -s[2 * r] * inv * rstd, c1 = -s[2 * r + 1] * inv * rstd;
        const F2 nm = f2(-mean, -mean), rs = f2(rstd, rstd), k0 = f2(c0, c0), k1 = f2(c1, c1);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          if (!in[j]) continue;
          F2 x[NP], g[NP];
          to_pairs<T>(data[(r * NV + j) * 2 * kMaxThreads], x);
          to_pairs<T>(data[((r * NV + j) * 2 + 1) * kMaxThreads], g);
          float f[NE];
#pragma unroll
          for (int h = 0; h < NP; ++h)
            split(fma(mul(g[h], w[j][h]), rs, fma(mul(add(x[h], nm), rs), k1, k0)), f[2 * h], f[2 * h + 1]);
          store_pack<T, NE>(to + r * a.ys + j * threads * NE, f);
        }
      }
    };
    if (row + R <= (int)a.rows) rows_of(std::true_type());
    else rows_of(std::false_type());
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  next_may_launch();
  if (!a.part) return;
  float* out = a.part + (long long)blockIdx.x * 2 * a.dim;
  // the groups' sums in group order, through the staging memory
  float* cols = reinterpret_cast<float*>(staged);
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  for (int y = 0; y < (int)blockDim.y; ++y) {
    __syncthreads();
    if (group != y) continue;
    float* dst = y + 1 < (int)blockDim.y ? cols : out;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = t + j * threads;
      if (v >= nvec) continue;
#pragma unroll
      for (int h = 0; h < NP; ++h) {
        float u0, u1, v0, v1;
        split(dw[j][h], u0, u1);
        split(db[j][h], v0, v1);
        const int c = v * NE + 2 * h;
        if (y > 0) {
          u0 += cols[c];
          u1 += cols[c + 1];
          v0 += cols[a.dim + c];
          v1 += cols[a.dim + c + 1];
        }
        *reinterpret_cast<float2*>(dst + c) = make_float2(u0, u1);
        *reinterpret_cast<float2*>(dst + a.dim + c) = make_float2(v0, v1);
      }
    }
  }
}

// The kernels for rows of any length and alignment.  A row's aligned 16-byte
// granules are copied ahead into shared memory at the row's own place within
// its first granule, and read from there element by element.  Bound by the
// instructions that takes: backward 30001 x 1023 fp16 45 us (4.1 TB/s), fp32 67 us
// (5.5 TB/s).  A barrier of the group follows each wait, as a granule is used by
// other threads than the one that copied it.

// `a` where `keep` is not 0, else 0 (not a product: what lies behind a row may
// be anything).
__device__ __forceinline__ F2 only(F2 a, F2 keep) {
  float x, y, k, l;
  split(a, x, y);
  split(keep, k, l);
  return f2(k != 0.f ? x : 0.f, l != 0.f ? y : 0.f);
}

// Elements 0 and 32 from a place in a row in shared memory, as a pair; they may
// lie behind the row's end, where the slot's last bytes are read.
template <typename T> __device__ __forceinline__ F2 pair_at(const T* row) { return f2(to_f(row[0]), to_f(row[32])); }

template <typename T, int NV, int R>
__global__ void __launch_bounds__(kMaxThreads, 1) k_norm_forward_any(RowsArgs a) {
  constexpr int NP = NV / 2;  // pairs of columns
  extern __shared__ __align__(16) unsigned char slots[];
  __shared__ float red[2][kMaxThreads / 32 * R];
  const int t = threadIdx.x, group = threadIdx.y, threads = blockDim.x;
  const int warps = threads / 32, warp = t >> 5, lane = t & 31;
  float* buf[2] = {red[0] + group * warps * R, red[1] + group * warps * R};
  // a warp owns 32 NV columns, lane by lane: first, first + 32, ...; `left` of them and of what follows are in the row
  const int first = warp * 32 * NV + lane, left = a.dim - warp * 32 * NV;
  const int slot = slot_bytes(threads * NV, sizeof(T));
  unsigned char* mine = slots + group * kStages * R * slot;
  const float inv = 1.f / (float)a.dim;
  const int step = gridDim.x * blockDim.y * R;
  int row = ((int)blockIdx.x * blockDim.y + group) * R, ahead = row;
  const CopyShare share(R, warps, warp);
  auto issue = [&](int stage) {
    for (int r = share.first; r < R; r += share.step)
      if (ahead + r < (int)a.rows)
        copy_row(mine + (stage * R + r) * slot, (const T*)a.x, ahead + r, a.xs, a.dim, share.part * 32 + lane, share.parts * 32);
    commit_copies();
    ahead = ahead < (int)a.rows ? ahead + step : ahead;
  };
  after_previous();
  next_may_launch();
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) issue(k);
  F2 w[NP], bias[NP], keep[NP];  // keep: 1 in a column of the row, 0 behind its end
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    float v[2], u[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = first + (2 * j + i) * 32;
      float one[1];
      load_param<1>(a.w, a.pdtype, c, c < a.dim, 1.f, one);
      v[i] = one[0];
      load_param<1>(a.b, a.pdtype, c, c < a.dim, 0.f, one);
      u[i] = one[0];
    }
    w[j] = f2(v[0], v[1]);
    bias[j] = f2(u[0], u[1]);
    keep[j] = f2(first + 2 * j * 32 < a.dim ? 1.f : 0.f, first + (2 * j + 1) * 32 < a.dim ? 1.f : 0.f);
  }
  T* to = (T*)a.y + row * a.ys + first;
  const long long to_step = step * a.ys;
  int stage = 0;
  for (; row < (int)a.rows; row += step, to += to_step) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    group_barrier(group, threads);
    issue(stage == 0 ? kStages - 1 : stage - 1);
    const int rows = min(R, (int)a.rows - row);
    F2 x[R][NP];
    float s[R], mean[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const T* src = (const T*)(mine + (stage * R + r) * slot + row_phase(a.x, row + r, a.xs, sizeof(T))) + first;
      F2 sum = f2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        x[r][j] = pair_at(src + 2 * j * 32);
        if ((2 * j + 2) * 32 > left) x[r][j] = only(x[r][j], keep[j]);
        sum = add(sum, x[r][j]);
      }
      float u, v;
      split(sum, u, v);
      s[r] = u + v;
    }
    stage = stage + 1 == kStages ? 0 : stage + 1;
    group_sum<R>(s, buf[0], warps, warp, lane, group, threads);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = s[r] * inv;
      const F2 nm = f2(-mean[r], -mean[r]);
      F2 sum = f2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        x[r][j] = add(x[r][j], nm);
        if ((2 * j + 2) * 32 > left) x[r][j] = only(x[r][j], keep[j]);
        sum = fma(x[r][j], x[r][j], sum);
      }
      float u, v;
      split(sum, u, v);
      s[r] = u + v;
    }
    group_sum<R>(s, buf[1], warps, warp, lane, group, threads);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r >= rows) break;
      const float rstd = rsqrtf(fmaf(s[r], inv, a.eps));
      if (t == 0) {
        if (a.mean) a.mean[row + r] = mean[r];
        if (a.rstd) a.rstd[row + r] = rstd;
      }
      const F2 rs = f2(rstd, rstd);
      T* dst = to + r * a.ys;
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        float u, v;
        split(fma(mul(x[r][j], rs), w[j], bias[j]), u, v);
        if (lane + 2 * j * 32 < left) dst[2 * j * 32] = from_f<T>(u);
        if (lane + (2 * j + 1) * 32 < left) dst[(2 * j + 1) * 32] = from_f<T>(v);
      }
    }
  }
}

template <typename T, int NV, int R>
__global__ void __launch_bounds__(kMaxThreads, 1) k_norm_backward_any(RowsArgs a) {
  constexpr int NP = NV / 2;
  extern __shared__ __align__(16) unsigned char slots[];
  __shared__ float red[2][kMaxThreads / 32 * 2 * R];
  __shared__ float stats[kStages][kMaxThreads / 32][2 * R];  // a group's
  const int t = threadIdx.x, group = threadIdx.y, threads = blockDim.x;
  const int warps = threads / 32, warp = t >> 5, lane = t & 31;
  // a warp owns 32 NV columns, lane by lane: first, first + 32, ...; `left` of them and of what follows are in the row
  const int first = warp * 32 * NV + lane, left = a.dim - warp * 32 * NV;
  const int slot = slot_bytes(threads * NV, sizeof(T));
  unsigned char* mine = slots + group * kStages * R * 2 * slot;
  const float inv = 1.f / (float)a.dim;
  const int step = gridDim.x * blockDim.y * R;
  int row = ((int)blockIdx.x * blockDim.y + group) * R, ahead = row;
  const CopyShare share(2 * R, warps, warp);
  auto issue = [&](int stage) {
    for (int i = share.first; i < 2 * R; i += share.step)
      if (ahead + i / 2 < (int)a.rows)
        copy_row(mine + (stage * 2 * R + i) * slot, (const T*)(i & 1 ? a.g : a.x), ahead + i / 2, i & 1 ? a.gs : a.xs,
                 a.dim, share.part * 32 + lane, share.parts * 32);
    if (t < 2 * R && ahead + t / 2 < (int)a.rows) copy4(&stats[stage][group][t], (t & 1 ? a.rstd : a.mean) + ahead + t / 2);
    commit_copies();
    ahead = ahead < (int)a.rows ? ahead + step : ahead;
  };
  after_previous();
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) issue(k);
  F2 dw[NP], db[NP], w[NP], keep[NP];
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    float v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = first + (2 * j + i) * 32;
      float one[1];
      load_param<1>(a.w, a.pdtype, c, c < a.dim, 1.f, one);
      v[i] = one[0];
    }
    w[j] = f2(v[0], v[1]);
    dw[j] = db[j] = f2(0.f, 0.f);
    keep[j] = f2(first + 2 * j * 32 < a.dim ? 1.f : 0.f, first + (2 * j + 1) * 32 < a.dim ? 1.f : 0.f);
  }
  T* to = (T*)a.y + row * a.ys + first;
  const long long to_step = step * a.ys;
  int stage = 0, flip = 0;
  for (; row < (int)a.rows; row += step, to += to_step) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    group_barrier(group, threads);
    issue(stage == 0 ? kStages - 1 : stage - 1);
    const float* stat = stats[stage][group];
    const int rows = min(R, (int)a.rows - row);
    F2 xh[R][NP], g[R][NP];
    float s[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      F2 s0 = f2(0.f, 0.f), s1 = f2(0.f, 0.f);
      if (r < rows) {
        const unsigned char* at = mine + (stage * R + r) * 2 * slot;
        const T* x = (const T*)(at + row_phase(a.x, row + r, a.xs, sizeof(T))) + first;
        const T* y = (const T*)(at + slot + row_phase(a.g, row + r, a.gs, sizeof(T))) + first;
        const F2 nm = f2(-stat[2 * r], -stat[2 * r]), rs = f2(stat[2 * r + 1], stat[2 * r + 1]);
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          xh[r][j] = mul(add(pair_at(x + 2 * j * 32), nm), rs);
          g[r][j] = pair_at(y + 2 * j * 32);
          if ((2 * j + 2) * 32 > left) {
            xh[r][j] = only(xh[r][j], keep[j]);
            g[r][j] = only(g[r][j], keep[j]);
          }
          const F2 gx = mul(g[r][j], xh[r][j]);
          s0 = fma(g[r][j], w[j], s0);
          s1 = fma(gx, w[j], s1);
          dw[j] = add(dw[j], gx);
          db[j] = add(db[j], g[r][j]);
        }
      }
      float u, v;
      split(s0, u, v);
      s[2 * r] = u + v;
      split(s1, u, v);
      s[2 * r + 1] = u + v;
    }
    stage = stage + 1 == kStages ? 0 : stage + 1;
    if (!a.y) continue;
    group_sum<2 * R>(s, red[flip] + group * warps * 2 * R, warps, warp, lane, group, threads);
    flip ^= 1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r >= rows) break;
      const float rstd = stat[2 * r + 1];
      const float c0 = -s[2 * r] * inv * rstd, c1 = -s[2 * r + 1] * inv * rstd;
      const F2 rs = f2(rstd, rstd), k0 = f2(c0, c0), k1 = f2(c1, c1);
      T* dst = to + r * a.ys;
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        float u, v;
        split(fma(mul(g[r][j], w[j]), rs, fma(xh[r][j], k1, k0)), u, v);
        if (lane + 2 * j * 32 < left) dst[2 * j * 32] = from_f<T>(u);
        if (lane + (2 * j + 1) * 32 < left) dst[(2 * j + 1) * 32] = from_f<T>(v);
      }
    }
  }
  next_may_launch();
  if (!a.part) return;
  float* out = a.part + (long long)blockIdx.x * 2 * a.dim;
  // the groups' sums in group order, through the rows' memory
  float* cols = reinterpret_cast<float*>(slots);
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  for (int y = 0; y < (int)blockDim.y; ++y) {
    __syncthreads();
    if (group != y) continue;
    float* dst = y + 1 < (int)blockDim.y ? cols : out;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = first + j * 32;
      if (c >= a.dim) continue;
      float u[2], v[2];
      split(dw[j / 2], u[0], u[1]);
      split(db[j / 2], v[0], v[1]);
      dst[c] = (y ? cols[c] : 0.f) + u[j & 1];
      dst[a.dim + c] = (y ? cols[a.dim + c] : 0.f) + v[j & 1];
    }
  }
}

// Rows too long for registers: one CTA a row, the row read once per reduction
// (from L2 after the first).
__device__ __forceinline__ float block_sum(float v, float* buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_sum(v);
  __syncthreads();
  if (lane == 0) buf[warp] = v;
  __syncthreads();
  v = 0.f;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) v += buf[w];
  return v;
}

template <typename T> __global__ void __launch_bounds__(kMaxThreads) k_norm_forward_long(RowsArgs a) {
  __shared__ float buf[kMaxThreads / 32];
  const float inv = 1.f / (float)a.dim;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = (const T*)a.x + row * a.xs;
    float s = 0.f;
    for (int c = threadIdx.x; c < a.dim; c += blockDim.x) s += to_f(__ldg(x + c));
    const float mean = block_sum(s, buf) * inv;
    s = 0.f;
    for (int c = threadIdx.x; c < a.dim; c += blockDim.x) {
      const float d = to_f(__ldg(x + c)) - mean;
      s = fmaf(d, d, s);
    }
    const float rstd = rsqrtf(fmaf(block_sum(s, buf), inv, a.eps));
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    T* y = (T*)a.y + row * a.ys;
    for (int c = threadIdx.x; c < a.dim; c += blockDim.x)
      y[c] = from_f<T>(fmaf((to_f(__ldg(x + c)) - mean) * rstd, a.w ? load_any(a.w, a.pdtype, c) : 1.f,
                            a.b ? load_any(a.b, a.pdtype, c) : 0.f));
  }
}

template <typename T> __global__ void __launch_bounds__(kMaxThreads) k_norm_dx_long(RowsArgs a) {
  __shared__ float buf[kMaxThreads / 32];
  const float inv = 1.f / (float)a.dim;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = (const T*)a.x + row * a.xs;
    const T* g = (const T*)a.g + row * a.gs;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s0 = 0.f, s1 = 0.f;
    for (int c = threadIdx.x; c < a.dim; c += blockDim.x) {
      const float av = to_f(__ldg(g + c)) * (a.w ? load_any(a.w, a.pdtype, c) : 1.f);
      s0 += av;
      s1 = fmaf(av, (to_f(__ldg(x + c)) - mean) * rstd, s1);
    }
    const float m0 = block_sum(s0, buf) * inv, m1 = block_sum(s1, buf) * inv;
    T* y = (T*)a.y + row * a.ys;
    for (int c = threadIdx.x; c < a.dim; c += blockDim.x) {
      const float xh = (to_f(__ldg(x + c)) - mean) * rstd;
      y[c] = from_f<T>((to_f(__ldg(g + c)) * (a.w ? load_any(a.w, a.pdtype, c) : 1.f) - m0 - xh * m1) * rstd);
    }
  }
}

// dw and db of long rows: gridDim.y partial rows, each the sum of a
// contiguous share of the rows in row order.
template <typename T> __global__ void __launch_bounds__(256) k_norm_columns_long(RowsArgs a) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= a.dim) return;
  const long long per = (a.rows + gridDim.y - 1) / gridDim.y;
  const long long r0 = blockIdx.y * per, r1 = min(a.rows, r0 + per);
  float dw = 0.f, db = 0.f;
  for (long long r = r0; r < r1; ++r) {
    const float g = to_f(__ldg((const T*)a.g + r * a.gs + c));
    const float xh = (to_f(__ldg((const T*)a.x + r * a.xs + c)) - __ldg(a.mean + r)) * __ldg(a.rstd + r);
    dw = fmaf(g, xh, dw);
    db += g;
  }
  a.part[(long long)blockIdx.y * 2 * a.dim + c] = dw;
  a.part[(long long)blockIdx.y * 2 * a.dim + a.dim + c] = db;
}

// dw and db: the partial rows' sums, 32 columns a CTA, its warps over
// interleaved partial rows, then the warps' sums in order.  Bound by latency (3 us
// behind the pass that leaves 152 partial rows; 8 us with loads one by one).
constexpr int kColumnWarps = 16;
__global__ void __launch_bounds__(32 * kColumnWarps) k_norm_columns(const float* __restrict__ part, int parts, int dim,
                                                                    void* dw, void* db, int dtype, int accumulate) {
  __shared__ float sums[kColumnWarps][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const long long c = (long long)blockIdx.x * 32 + x;
  after_previous();
  next_may_launch();
  float s = 0.f;
  if (c < 2LL * dim) {
    constexpr int kAtOnce = 10;  // loads under way; 152 SMs' partial rows take one turn
    for (int p0 = y; p0 < parts; p0 += kAtOnce * kColumnWarps) {
      float v[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int p = p0 + k * kColumnWarps;
        v[k] = p < parts ? __ldcg(part + (long long)p * 2 * dim + c) : 0.f;
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) s += v[k];
    }
  }
  sums[y][x] = s;
  __syncthreads();
  if (y != 0 || c >= 2LL * dim) return;
  s = sums[0][x];
#pragma unroll
  for (int w = 1; w < kColumnWarps; ++w) s += sums[w][x];
  void* out = c < dim ? dw : db;
  if (!out) return;
  const long long i = c < dim ? c : c - dim;
  if (accumulate) s += read_any(out, dtype, i);
  store_any(out, dtype, i, s);
}

// How a row is spread over threads.
struct RowPlan {
  int nv;       // accesses per thread and row; 0: the row does not fit
  int threads;  // of a group
  int groups;   // of a CTA
};

// vec: elements per access; groups fill a CTA of up to kMaxThreads.  The
// fewest accesses per thread that leave at most a quarter of those without work.
RowPlan plan_rows(long long dim, int vec) {
  const int max_nv = vec == 1 ? 16 : 4;
  const long long nvec = dim / vec;
  // (single elements: 4 a thread and 4 rows at a time, or 8 and 2.  Backward,
  // fp16: 1023 columns 51 us so and 45, 30001 rows; 333 columns 19 and 23, 20000
  // rows)
  const int min_nv = vec != 1 ? 1 : dim > 768 ? 8 : 4;
  RowPlan best{0, 0, 1};
  double best_share = 0.0;
  for (int nv = min_nv; nv <= max_nv; nv *= 2) {
    const long long threads = ((nvec + nv - 1) / nv + 31) / 32 * 32;
    if (threads > kMaxThreads) continue;
    RowPlan p{nv, (int)threads, 0};
    p.groups = std::max(1, std::min(8, kMaxThreads / p.threads));
    const double share = (double)nvec * p.groups / ((double)nv * kMaxThreads);
    if (share > best_share) {
      best = p;
      best_share = share;
    }
    if (share >= 0.75) break;
  }
  return best;
}

template <int V> struct Int {
  static constexpr int value = V;
};
// f(NV, R) as compile-time constants: R1 rows at a time where a thread has one
// vector of each, fewer where it has more, one where there are few rows.
template <int R1, typename F> void with_vec_plan(const RowPlan& p, bool few, F&& f) {
  if (p.nv == 1 && few) f(Int<1>(), Int<1>());
  else if (p.nv == 1) f(Int<1>(), Int<R1>());
  else if (p.nv == 2) f(Int<2>(), Int<2>());
  else f(Int<4>(), Int<1>());
}
// Few rows: one at a time, so that more CTAs have some.  Forward, one row at a
// time against four: up to a row for every group of an SM's CTA 0.73 to 0.96 of
// the time (304 x 1600 bf16 2.4 us, 3.0 with four), at two and more 1.1 to 1.5
// times (608 x 1600 3.7 and 2.9, 608 x 4096 5.4 and 3.5; 64 columns 1.8 and 2.1
// at two, 2.3 and 2.1 at four).  Backward: up to two rows 0.8 to 0.98, at four 0.88 to 1.09 (1216 x 1600 7.0 and 7.8, 608 x 2048 fp32 6.1
// and 5.6), from eight on 1.0 to 1.2 (4864 x 1600 15.6 and 15.0, 4864 x 4096 30 and 25).
bool few_forward(const RowPlan& p, long long rows, int sms) { return rows <= (long long)sms * p.groups; }
bool few_backward(const RowPlan& p, long long rows, int sms) { return rows <= 4LL * sms * p.groups; }
int vec_rows(const RowPlan& p, int r1, bool few) { return p.nv == 1 ? (few ? 1 : r1) : p.nv == 2 ? 2 : 1; }
template <typename F> void with_scalar_plan(const RowPlan& p, F&& f) {
  if (p.nv == 4) f(Int<4>(), Int<4>());
  else if (p.nv == 8) f(Int<8>(), Int<2>());
  else f(Int<16>(), Int<1>());
}
int scalar_rows(const RowPlan& p) { return 16 / p.nv; }

// Shared memory of the kernels for any rows, one CTA of which an SM gets.
size_t any_smem(const RowPlan& p, int size, int arrays) {
  return (size_t)p.groups * kStages * scalar_rows(p) * arrays * slot_bytes(p.threads * p.nv, size);
}

template <typename T, int NV, int R>
cudaError_t launch_forward_any(const RowsArgs& a, const RowPlan& p, unsigned grid, size_t smem, int device, cudaStream_t st) {
  static std::atomic<unsigned long long> raised{0};
  const cudaError_t e = raise_smem(k_norm_forward_any<T, NV, R>, raised, device, 220 * 1024);
  if (e != cudaSuccess) return e;
  return launch_early(k_norm_forward_any<T, NV, R>, grid, dim3(p.threads, p.groups), smem, 1, st, a);
}
template <typename T, int NV, int R>
cudaError_t launch_backward_any(const RowsArgs& a, const RowPlan& p, unsigned grid, size_t smem, int device, cudaStream_t st) {
  static std::atomic<unsigned long long> raised{0};
  const cudaError_t e = raise_smem(k_norm_backward_any<T, NV, R>, raised, device, 220 * 1024);
  if (e != cudaSuccess) return e;
  return launch_early(k_norm_backward_any<T, NV, R>, grid, dim3(p.threads, p.groups), smem, 1, st, a);
}

template <typename T, int NV, int R>
cudaError_t launch_forward(const RowsArgs& a, const RowPlan& p, unsigned grid, int device, cudaStream_t st) {
  static std::atomic<unsigned long long> raised{0};
  const cudaError_t e = raise_smem(k_norm_forward_vec<T, NV, R>, raised, device, kStages * R * NV * kMaxThreads * 16);
  if (e != cudaSuccess) return e;
  return launch_early(k_norm_forward_vec<T, NV, R>, grid, dim3(p.threads, p.groups),
                      (size_t)kStages * R * NV * kMaxThreads * 16, 1, st, a);
}
template <typename T, int NV, int R>
cudaError_t launch_backward(const RowsArgs& a, const RowPlan& p, unsigned grid, int device, cudaStream_t st) {
  static std::atomic<unsigned long long> raised{0};
  const cudaError_t e = raise_smem(k_norm_backward_vec<T, NV, R>, raised, device, kStages * R * NV * kMaxThreads * 32);
  if (e != cudaSuccess) return e;
  return launch_early(k_norm_backward_vec<T, NV, R>, grid, dim3(p.threads, p.groups),
                      (size_t)kStages * R * NV * kMaxThreads * 32, 1, st, a);
}

template <typename F> void by_dtype(int32_t d, F&& f) {
  switch (d) {
    case PSGD_F32: f((float*)nullptr); break;
    case PSGD_F16: f((__half*)nullptr); break;
    default: f((__nv_bfloat16*)nullptr); break;
  }
}

bool vec_ok(const void* p, long long stride, int dtype) {
  return !p || (aligned16(p) && (stride * dtype_size(dtype)) % 16 == 0);
}

int check_common(const char* who, const psgd_layernorm* h, int32_t dtype, int32_t pdtype, int64_t rows) {
  const std::string w(who);
  if (!h) return fail(PSGD_EINVAL, w + ": NULL layer norm");
  if (!dtype_ok(dtype) || !dtype_ok(pdtype)) return fail(PSGD_EINVAL, w + ": unknown dtype");
  if (rows < 0 || rows > (1 << 30)) return fail(PSGD_EINVAL, w + ": rows must be in [0, 2^30]");
  return PSGD_OK;
}

int check_operand(const char* who, const char* what, const void* p, int64_t rows, int64_t dim, int64_t stride,
                  bool written) {
  const std::string w = std::string(who) + ": " + what;
  if (rows > 0 && !p) return fail(PSGD_EINVAL, w + " is NULL");
  if (!span_ok(rows, stride)) return fail(PSGD_EINVAL, w + ": bad row stride");
  if (written && rows > 1 && stride < dim) return fail(PSGD_EINVAL, w + ": rows overlap");
  return PSGD_OK;
}

}  // namespace
}  // namespace ops
}  // namespace psgd

using namespace psgd;
using namespace psgd::ops;

extern "C" int psgd_layernorm_create(int64_t dim, int32_t device, psgd_layernorm** out) {
  if (!out) return fail(PSGD_EINVAL, "psgd_layernorm_create: out is NULL");
  *out = nullptr;
  if (dim < 1 || dim > (1 << 20)) return fail(PSGD_EINVAL, "psgd_layernorm_create: dim must be in [1, 2^20]");
  if (device < 0 || device >= 64) return fail(PSGD_EINVAL, "psgd_layernorm_create: device ordinal must be in [0, 63]");
  int count = 0;
  cudaError_t e = cudaGetDeviceCount(&count);
  if (e != cudaSuccess) return cuda_fail("psgd_layernorm_create: cudaGetDeviceCount", e);
  if (device >= count) return fail(PSGD_ECUDA, "psgd_layernorm_create: no such device");
  psgd_layernorm* h = new (std::nothrow) psgd_layernorm;
  if (!h) return fail(PSGD_ENOMEM, "psgd_layernorm_create: out of host memory");
  DeviceScope scope(device);
  h->device = device;
  h->dim = dim;
  e = cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, device);
  if (e == cudaSuccess) {
    h->max_ctas = h->sms * 2;
    h->bytes = (size_t)h->max_ctas * 2 * dim * 4;
    e = cudaMalloc((void**)&h->part, h->bytes);
  }
  if (e != cudaSuccess) {
    const int rc = cuda_fail("psgd_layernorm_create", e);
    h->part = nullptr;
    psgd_layernorm_destroy(h);
    return rc;
  }
  *out = h;
  return PSGD_OK;
}

extern "C" void psgd_layernorm_destroy(psgd_layernorm* h) {
  if (!h) return;
  {
    DeviceScope scope(h->device);
    if (h->part) cudaFree(h->part);
  }
  delete h;
}

extern "C" size_t psgd_layernorm_workspace_bytes(const psgd_layernorm* h) { return h ? h->bytes : 0; }

extern "C" int psgd_layernorm_forward(psgd_layernorm* h, const void* x, psgd_dtype dtype, int64_t x_stride,
                                      int64_t rows, const void* weight, const void* bias, psgd_dtype param_dtype,
                                      float eps, void* y, int64_t y_stride, float* mean, float* rstd, void* stream) {
  const char* who = "psgd_layernorm_forward";
  int rc = check_common(who, h, dtype, param_dtype, rows);
  if (!rc) rc = check_operand(who, "x", x, rows, h->dim, x_stride, false);
  if (!rc) rc = check_operand(who, "y", y, rows, h->dim, y_stride, true);
  if (rc) return rc;
  if (!(eps >= 0.f) || !isfinite(eps)) return fail(PSGD_EINVAL, "psgd_layernorm_forward: eps must be finite and >= 0");
  if (rows == 0) return PSGD_OK;
  const long long yb = extent(rows, h->dim, y_stride, dtype), xb = extent(rows, h->dim, x_stride, dtype);
  const long long pb = h->dim * dtype_size(param_dtype), sb = rows * 4;
  for (const auto& o : {std::pair<const void*, long long>(y, yb), {mean, sb}, {rstd, sb}})
    if (overlap(o.first, o.second, x, xb) || overlap(o.first, o.second, weight, pb) || overlap(o.first, o.second, bias, pb))
      return fail(PSGD_EINVAL, "psgd_layernorm_forward: an output overlaps an input");
  if (overlap(y, yb, mean, sb) || overlap(y, yb, rstd, sb) || overlap(mean, sb, rstd, sb))
    return fail(PSGD_EINVAL, "psgd_layernorm_forward: the outputs overlap");
  DeviceScope scope(h->device);
  const cudaStream_t st = (cudaStream_t)stream;
  RowsArgs a{x, nullptr, weight, bias, y, mean, rstd, nullptr, x_stride, 0, y_stride, rows, (int)h->dim,
             (int)param_dtype, eps};
  const int full = 16 / dtype_size(dtype);
  const bool vec = h->dim % full == 0 && vec_ok(x, x_stride, dtype) && vec_ok(y, y_stride, dtype);
  const RowPlan p = plan_rows(h->dim, vec ? full : 1);
  cudaError_t e = cudaSuccess;
  by_dtype(dtype, [&](auto* tt) {
    using T = std::remove_pointer_t<decltype(tt)>;
    if (p.nv == 0) {
      k_norm_forward_long<T><<<(unsigned)std::min<long long>(rows, h->sms * 4), kMaxThreads, 0, st>>>(a);
      e = cudaGetLastError();
    } else if (vec) {
      const bool few = few_forward(p, rows, h->sms);
      const long long per = (long long)p.groups * vec_rows(p, 4, few);
      const unsigned grid = (unsigned)std::min<long long>((rows + per - 1) / per, h->sms);
      with_vec_plan<4>(p, few, [&](auto nv, auto r) {
        e = launch_forward<T, decltype(nv)::value, decltype(r)::value>(a, p, grid, h->device, st);
      });
    } else {
      const long long per = (long long)p.groups * scalar_rows(p);
      const size_t smem = any_smem(p, (int)sizeof(T), 1);
      const unsigned grid = (unsigned)std::min<long long>((rows + per - 1) / per, h->sms);
      with_scalar_plan(p, [&](auto nv, auto r) {
        e = launch_forward_any<T, decltype(nv)::value, decltype(r)::value>(a, p, grid, smem, h->device, st);
      });
    }
  });
  return e == cudaSuccess ? PSGD_OK : cuda_fail(who, e);
}

extern "C" int psgd_layernorm_backward(psgd_layernorm* h, const void* grad, int64_t grad_stride, const void* x,
                                       psgd_dtype dtype, int64_t x_stride, int64_t rows, const float* mean,
                                       const float* rstd, const void* weight, psgd_dtype param_dtype, void* dx,
                                       int64_t dx_stride, void* dweight, void* dbias, psgd_dtype dparam_dtype,
                                       int32_t accumulate, void* stream) {
  const char* who = "psgd_layernorm_backward";
  int rc = check_common(who, h, dtype, param_dtype, rows);
  if (!rc) rc = check_operand(who, "grad", grad, rows, h->dim, grad_stride, false);
  if (!rc) rc = check_operand(who, "x", x, rows, h->dim, x_stride, false);
  if (!rc && dx) rc = check_operand(who, "dx", dx, rows, h->dim, dx_stride, true);
  if (rc) return rc;
  if (!dtype_ok(dparam_dtype)) return fail(PSGD_EINVAL, "psgd_layernorm_backward: unknown dtype");
  if (rows > 0 && (!mean || !rstd)) return fail(PSGD_EINVAL, "psgd_layernorm_backward: mean or rstd is NULL");
  const long long gb = extent(rows, h->dim, grad_stride, dtype), xb = extent(rows, h->dim, x_stride, dtype);
  const long long db = dx ? extent(rows, h->dim, dx_stride, dtype) : 0, wb = h->dim * dtype_size(param_dtype);
  const long long ob = h->dim * dtype_size(dparam_dtype);
  for (const auto& o : {std::pair<const void*, long long>(dx, db), {dweight, ob}, {dbias, ob}})
    if (overlap(o.first, o.second, grad, gb) || overlap(o.first, o.second, x, xb) ||
        overlap(o.first, o.second, mean, rows * 4) || overlap(o.first, o.second, rstd, rows * 4) ||
        overlap(o.first, o.second, weight, wb))
      return fail(PSGD_EINVAL, "psgd_layernorm_backward: an output overlaps an input");
  if (overlap(dx, db, dweight, ob) || overlap(dx, db, dbias, ob) || overlap(dweight, ob, dbias, ob))
    return fail(PSGD_EINVAL, "psgd_layernorm_backward: the outputs overlap");
  const bool params = dweight || dbias;
  if (!params && (!dx || rows == 0)) return PSGD_OK;
  DeviceScope scope(h->device);
  const cudaStream_t st = (cudaStream_t)stream;
  RowsArgs a{x, grad, weight, nullptr, dx, const_cast<float*>(mean), const_cast<float*>(rstd),
             params ? h->part : nullptr, x_stride, grad_stride, dx_stride, rows, (int)h->dim, (int)param_dtype, 0.f};
  const int full = 16 / dtype_size(dtype);
  const bool vec = h->dim % full == 0 && vec_ok(x, x_stride, dtype) && vec_ok(grad, grad_stride, dtype) &&
                   vec_ok(dx, dx_stride, dtype);
  const RowPlan p = plan_rows(h->dim, vec ? full : 1);
  int parts = 0;
  cudaError_t e = cudaSuccess;
  if (rows > 0)
    by_dtype(dtype, [&](auto* tt) {
      using T = std::remove_pointer_t<decltype(tt)>;
      if (p.nv == 0) {
        if (dx) k_norm_dx_long<T><<<(unsigned)std::min<long long>(rows, h->sms * 4), kMaxThreads, 0, st>>>(a);
        if (params) {
          parts = (int)std::min<long long>((rows + 31) / 32, h->max_ctas);
          k_norm_columns_long<T><<<dim3((unsigned)((h->dim + 255) / 256), parts), 256, 0, st>>>(a);
        }
        e = cudaGetLastError();
      } else if (vec) {
        const bool few = few_backward(p, rows, h->sms);
        const long long per = (long long)p.groups * vec_rows(p, 4, few);
        parts = (int)std::min<long long>((rows + per - 1) / per, h->sms);
        with_vec_plan<4>(p, few, [&](auto nv, auto r) {
          e = launch_backward<T, decltype(nv)::value, decltype(r)::value>(a, p, (unsigned)parts, h->device, st);
        });
      } else {
        const long long per = (long long)p.groups * scalar_rows(p);
        const size_t smem = any_smem(p, (int)sizeof(T), 2);
        parts = (int)std::min<long long>((rows + per - 1) / per, h->sms);
        with_scalar_plan(p, [&](auto nv, auto r) {
          e = launch_backward_any<T, decltype(nv)::value, decltype(r)::value>(a, p, (unsigned)parts, smem, h->device, st);
        });
      }
    });
  if (e == cudaSuccess && params) {
    e = launch_early(k_norm_columns, (unsigned)((2 * h->dim + 31) / 32), 32 * kColumnWarps, 0, 1, st, h->part, parts, h->dim,
                     dweight, dbias, dparam_dtype, accumulate);
  }
  return e == cudaSuccess ? PSGD_OK : cuda_fail(who, e);
}
