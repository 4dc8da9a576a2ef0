// Matrix products on the tensor cores (psgd_mma.cuh), with what follows a product
// in the same kernel: the pieces of a log-sum-exp, the gradient of a softmax cross
// entropy, or the sums' rounding into a bucket.
//
// Persistent pairs of CTAs.  In each, one thread loads (TMA, 160 KB in five stages, or up to ten of fewer rows or columns),
// one thread of the first CTA multiplies (tcgen05, both CTAs' tensor memory), and
// sixteen warps take finished tiles, 32 rows of 64 columns each, out of tensor
// memory while the next tile is summed in its other half.
#include <algorithm>
#include <type_traits>

#include "psgd_mma.cuh"

namespace psgd {
namespace mma {
namespace {

using ops::after_previous;
using ops::next_may_launch;

struct Shared {
  uint64_t full[kMostStages], empty[kMostStages], done[2], drained[2];
  uint32_t tmem;
  volatile int dead;
  int m;
  Schedule schedule;
};

// One run of a pair: steps [k0, k1) of tile (tm, tn); slot < 0: the whole tile.
struct Run {
  int tm, tn, k0, k1, slot, width;
};
// A pair's i-th run; false behind the last.  The schedule is in shared memory: in the registers of the warps that drain
// it pushed some of their 64 sums out into local memory, which cost up to 10 us a tile (one word of an OUT kernel still is).
__device__ __forceinline__ bool run_of(const Product& p, const Schedule& s, int pairs, int pair, int i, Run& r) {
  int tile = pair + i * pairs;
  r.k0 = 0;
  r.k1 = s.kb;
  r.slot = -1;
  if (tile >= s.whole) {
    if (pair >= s.workers) return false;
    const int j = i - (s.whole > pair ? (s.whole - pair + pairs - 1) / pairs : 0);
    if (s.cuts) {
      if (j > 0) return false;
      tile = s.whole + pair % s.rest;
      r.k0 = first_of_cut(s, pair / s.rest);
      r.k1 = first_of_cut(s, pair / s.rest + 1);
      r.slot = 2 * pair;
    } else {
      // a run of steps reaches into two tiles at most
      const long long from = first_step(s, pair), to = first_step(s, pair + 1);
      const int first = (int)(from / s.kb);
      const long long border = (long long)(first + 1) * s.kb;
      if (j > 1 || (j == 1 && to <= border)) return false;
      tile = s.whole + first + j;
      r.k0 = j ? 0 : (int)(from - (border - s.kb));
      r.k1 = (int)((j ? to - border : (to < border ? to : border) - (border - s.kb)));
      r.slot = r.k0 == 0 && r.k1 == s.kb ? -1 : 2 * pair + j;
    }
  }
  r.tm = p.m_fast ? tile % s.mt : tile / s.nt;
  r.tn = p.m_fast ? tile / s.mt : tile % s.nt;
  r.width = width_of(p.n, p.bn, r.tn);
  return true;
}

__device__ __forceinline__ float exp_of(float x) {
  // 2 ulp of ex2 and the product's rounding, |x| 2^-24 of the result at most
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}

// Four elements of one row, side by side, at a multiple of their size.
template <typename T> __device__ __forceinline__ float4 load4(const T* p) {
  if constexpr (sizeof(T) == 4) {
    return *reinterpret_cast<const float4*>(p);
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    const T* e = reinterpret_cast<const T*>(&u);
    return make_float4(ops::to_f(e[0]), ops::to_f(e[1]), ops::to_f(e[2]), ops::to_f(e[3]));
  }
}
template <typename T> __device__ __forceinline__ void store4(T* p, float4 v) {
  if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(p) = v;
  else *reinterpret_cast<uint2*>(p) = make_uint2(ops::pack2<T>(v.x, v.y), ops::pack2<T>(v.z, v.w));
}
__device__ __forceinline__ float4 plus(float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }

// A staged 32 x 32 block into rows of `to`.  Aligned rows: eight lanes a row, four rows at a time; others: a row at a
// time.  What is there already is read for several rows together.
template <typename T>
__device__ __forceinline__ void put_rows(const float4* st, int lane, T* to, long long ldo, int rows, int cols, bool vec, bool add) {
  if (vec && cols >= 32) {
    const int r = lane >> 3, c = lane & 7;
    T* at = to + r * ldo + 4 * c;
#pragma unroll 1
    for (int r0 = r; r0 < rows; r0 += 8, at += 8 * ldo) {
      const bool second = r0 + 4 < rows;
      float4 y0 = st[r0 * 8 + (c ^ (r0 & 7))], y1 = st[(r0 + 4) * 8 + (c ^ ((r0 + 4) & 7))];
      if (add) {
        const float4 x0 = load4(at), x1 = second ? load4(at + 4 * ldo) : make_float4(0.f, 0.f, 0.f, 0.f);
        y0 = plus(x0, y0);
        y1 = plus(x1, y1);
      }
      store4(at, y0);
      if (second) store4(at + 4 * ldo, y1);
    }
  } else if (lane < cols) {
    const float* s = reinterpret_cast<const float*>(st);
    T* at = to + lane;
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += 4, at += 4 * ldo) {
      float old[4], y[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        old[r] = add && r0 + r < rows ? ops::to_f(at[r * ldo]) : 0.f;
        y[r] = s[(r0 + r) * 32 + (((lane >> 2) ^ ((r0 + r) & 7)) << 2 | (lane & 3))];
      }
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r0 + r < rows) at[r * ldo] = ops::from_f<T>(add ? old[r] + y[r] : y[r]);
    }
  }
}
// A 32 x 32 block (lane = row) through a warp's staging into `out`, from (row0, col0) on.
template <typename T>
__device__ __forceinline__ void put_block(const float* v, float4* st, int lane, const Product& p, int row0, int rows, int col0, int cols,
                                          float scale) {
  if (rows <= 0 || cols <= 0) return;
#pragma unroll
  for (int c = 0; c < 8; ++c)
    st[lane * 8 + (c ^ (lane & 7))] = make_float4(v[4 * c] * scale, v[4 * c + 1] * scale, v[4 * c + 2] * scale, v[4 * c + 3] * scale);
  __syncwarp();
  put_rows((const float4*)st, lane, (T*)p.out + (long long)row0 * p.ldo + col0, p.ldo, rows, cols, p.vec, p.accumulate);
  __syncwarp();
}

// T: OUT: out's type, GRAD: the operands', LSE: any.
template <int KIND, typename T>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1) k_product(const __grid_constant__ Product p) {
  extern __shared__ __align__(1024) unsigned char raw[];
  __shared__ Shared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  // the stages begin at a multiple of 1024 bytes, at the same place in both CTAs
  unsigned char* stages = raw + ((1024 - (saddr(raw) & 1023)) & 1023);
  unsigned char* staging = stages + kStages * kStageBytes;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMostStages; ++i) {
      bar_init(&sh.full[i], 1);
      bar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&sh.done[i], 1);
      bar_init(&sh.drained[i], 2 * kEpilogueWarps);
    }
    sh.dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kEpilogueWarps + 1) tmem_alloc(&sh.tmem);
  if (warp == kEpilogueWarps && lane == 0) {
    fetch_map(&p.a);
    fetch_map(&p.b);
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sh.tmem;
  cluster_sync();
  after_previous();
  next_may_launch();
  if (threadIdx.x == 0) {
    const int live = p.live ? *p.live : 0;
    sh.m = p.live_is == 1 ? live : p.m;
    sh.schedule = schedule_of(sh.m, p.n, p.bn, p.live_is == 2 ? live : p.k, pairs, p.slots != nullptr);
  }
  __syncthreads();
  const int m = sh.m;
  const Schedule& plan = sh.schedule;
  Run run;
  volatile int* dead = &sh.dead;

  if (warp == kEpilogueWarps) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (int i = 0; run_of(p, plan, pairs, pair, i, run); ++i) {
        const int row = run.tm * kTile + (int)rank * kHalf, col = run.tn * p.bn + (int)rank * (run.width / 2);
        // Of A with K rows, no more than the rows that there are: fewer bytes into the SMs, and room for more stages.  What lies in the
        // others' place gives rows that nobody takes.
        const int rows_here = min(kHalf, m - row), rows_0 = min(kHalf, m - run.tm * kTile), rows_1 = min(kHalf, m - run.tm * kTile - kHalf);
        const bool few = !p.a_m_rows && rows_1 < kHalf;
        const int boxes = (max(rows_here, 0) + kFew - 1) / kFew;
        // of B with M rows, 64 columns more or not (with K rows, a box has bn / 2)
        const bool wide = run.width > 128;
        const uint32_t bytes = (!p.b_m_rows ? p.bn * (kStep * 2) : (wide ? 2 : 1) * kOperand) + (few ? ((rows_0 + kFew - 1) / kFew + (max(rows_1, 0) + kFew - 1) / kFew) *
                                                                     (kFew * kStep * 2)
                                                               : 2 * kOperand);
        for (int kb = run.k0; kb < run.k1; ++kb) {
          if (!bar_wait(&sh.empty[stage], phase ^ 1, dead)) break;
          const uint32_t a = saddr(stages + stage * p.stage_bytes), b = a + p.a_bytes, bar = at_rank(saddr(&sh.full[stage]), 0);
          if (rank == 0) bar_expect(&sh.full[stage], bytes);
          const int x = kb * kStep;
          if (p.a_m_rows) {
            load_box(a, &p.a, row, x, bar);
            load_box(a + kOperand / 2, &p.a, row + 64, x, bar);
          } else if (few) {
            for (int i = 0; i < boxes; ++i) load_box(a + i * (kFew * kStep * 2), &p.a_few, x, row + i * kFew, bar);
          } else {
            load_box(a, &p.a, x, row, bar);
          }
          if (p.b_m_rows) {
            load_box(b, &p.b, col, p.b_y0 + x, bar);
            if (wide) load_box(b + kOperand / 2, &p.b, col + 64, p.b_y0 + x, bar);
          } else {
            load_box(b, &p.b, x, p.b_y0 + col, bar);
          }
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (*dead) break;
      }
    }
  } else if (warp == kEpilogueWarps + 1) {
    if (rank == 0 && lane == 0) {
      const uint32_t a_step = step_bytes(p.a_m_rows) >> 4, b_step = step_bytes(p.b_m_rows) >> 4;
      int stage = 0, buf = 0;
      uint32_t phase = 0, turn = 0;
      for (int i = 0; !*dead && run_of(p, plan, pairs, pair, i, run); ++i) {
        const uint32_t idesc = instruction(p.bf16, p.a_m_rows, p.b_m_rows, run.width);
        for (int kb = run.k0; kb < run.k1;) {
          if (!bar_wait(&sh.drained[buf], turn ^ 1, dead)) break;
          fence_after();
          const uint32_t d = tmem + buf * kTile;
          const int from = kb, to = p.chunk ? min(run.k1, kb + p.chunk) : run.k1;
          for (; kb < to; ++kb) {
            if (!bar_wait(&sh.full[stage], phase, dead)) break;
            fence_after();
            const uint32_t at = saddr(stages + stage * p.stage_bytes);
            const uint64_t a = describe(at, p.a_m_rows), b = describe(at + p.a_bytes, p.b_m_rows);
#pragma unroll
            for (int i = 0; i < kStep / 16; ++i) multiply(d, a + i * a_step, b + i * b_step, idesc, kb > from || i > 0);
            commit_both(&sh.empty[stage]);
            if (++stage == p.stages) {
              stage = 0;
              phase ^= 1;
            }
          }
          if (*dead) break;
          commit_both(&sh.done[buf]);
          buf ^= 1;
          turn ^= buf == 0;
        }
      }
    }
  } else {
    const int quarter = warp & 3, group = warp >> 2;  // 32 lanes of tensor memory, 64 columns
    float4* st = reinterpret_cast<float4*>(staging + warp * kStaging);
    int buf = 0;
    uint32_t turn = 0, flip = 0;
    bool alive = true;
    for (int i = 0; run_of(p, plan, pairs, pair, i, run); ++i) {
      const int row0 = run.tm * kTile + (int)rank * kHalf + quarter * 32, row = row0 + lane;
      const int col0 = run.tn * p.bn + group * kCols;
      // (loaded while the tile is summed)
      int tgt = -1;
      float lse = 0.f, factor = 0.f, own = 0.f;
      if constexpr (KIND != kOut) {
        if (row < m) tgt = p.target[row] - p.column0 - col0;
      }
      if constexpr (KIND == kGrad) {
        if (row < m) {
          lse = p.lse[row];
          factor = p.factor[row];
          own = p.at_target[row];
        }
      }
      float v[kCols];  // this lane's row, 64 columns of it
#pragma unroll
      for (int i = 0; i < kCols; ++i) v[i] = 0.f;
      for (int kb = run.k0; kb < run.k1; kb = p.chunk ? kb + p.chunk : run.k1) {
        alive = alive && warp_wait(&sh.done[buf], turn, dead);
        if (!alive) break;
        fence_after();
        const uint32_t t = tmem + buf * kTile + group * kCols + ((uint32_t)(quarter * 32) << 16);
#pragma unroll
        for (int c = 0; c < kCols; c += 8) {
          float x[8];
          tmem_load8(t + c, x);
          tmem_wait();
#pragma unroll
          for (int e = 0; e < 8; ++e) v[c + e] += x[e];
        }
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive_at(at_rank(saddr(&sh.drained[buf]), 0));
        buf ^= 1;
        turn ^= buf == 0;
      }
      if (KIND != kLse && !alive) break;  // (kLse: on to the barriers that the other warps are at)
      if constexpr (KIND == kOut) {
        if (group * kCols >= run.width) continue;
        if (run.slot >= 0) {
          // groups of four columns, row by row: neighbouring lanes write neighbouring 16 bytes
          float4* to = reinterpret_cast<float4*>(p.slots + run.slot * kSlotFloats) + (long long)rank * kHalf * kTile / 4 +
                       (long long)(group * (kCols / 4)) * kHalf + quarter * 32 + lane;
#pragma unroll
          for (int i = 0; i < kCols / 4; ++i) to[i * kHalf] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        } else {
          const int end = min(p.n, run.tn * p.bn + run.width);
          const float scale = p.scale ? __ldg(p.scale) : 1.f;
          put_block<T>(v, st, lane, p, row0, min(32, m - row0), col0, min(32, end - col0), scale);
          put_block<T>(v + 32, st, lane, p, row0, min(32, m - row0), col0 + 32, min(32, end - col0 - 32), scale);
        }
      } else if constexpr (KIND == kLse) {
        // columns that are in the tile and the vocabulary
        const int left = min(p.vocab - p.column0 - run.tn * p.bn, run.width) - group * kCols;
        if (left < kCols) {
#pragma unroll
          for (int i = 0; i < kCols; ++i)
            if (i >= left) v[i] = -INFINITY;
        }
        // without the target's, which is added with more care at the end
        if (__any_sync(0xffffffffu, tgt >= 0 && tgt < kCols)) {
#pragma unroll
          for (int i = 0; i < kCols; ++i) v[i] = tgt == i ? -INFINITY : v[i];
        }
        float most[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          most[c] = v[c];
#pragma unroll
          for (int i = 1; i < kCols / 4; ++i) most[c] = fmaxf(most[c], v[4 * i + c]);
        }
        const float top = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3])), from = top == -INFINITY ? 0.f : top;
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kCols; ++i) s[i & 3] += exp_of(v[i] - from);
        // the four warps of these rows join their columns, through each other's staging; two halves of it in turn, so that
        // one barrier a tile is enough
        float2* mine = reinterpret_cast<float2*>(staging + warp * kStaging) + flip * 32;
        mine[lane] = make_float2(top, (s[0] + s[1]) + (s[2] + s[3]));
        asm volatile("bar.sync %0, 128;" ::"r"(1 + quarter) : "memory");
        if (group == 0 && row < m) {
          float2 x[4];
          float most_of = -INFINITY, sum = 0.f;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            x[g] = (reinterpret_cast<const float2*>(staging + (g * 4 + quarter) * kStaging) + flip * 32)[lane];
            most_of = fmaxf(most_of, x[g].x);
          }
          // (columns without a logit above -infinity have a sum of 0, or NaN, which stays)
#pragma unroll
          for (int g = 0; g < 4; ++g) sum += x[g].y * (x[g].x == -INFINITY ? 0.f : exp_of(x[g].x - most_of));
          p.part[(long long)run.tn * p.part_rows + row] = make_float2(most_of, sum);
        }
        flip ^= 1;
      } else {
        // (rows of zeros up to a whole step of the sum over tokens, and none behind them)
        if (group * kCols >= run.width || row0 >= (m + kStep - 1) / kStep * kStep) continue;
        const int left = row < m ? p.vocab - p.column0 - col0 : 0;
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the staging's last box is out
        __syncwarp();
        uint4* to = reinterpret_cast<uint4*>(st);
#pragma unroll
        for (int i = 0; i < kCols / 8; ++i) {
          unsigned w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float g[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int at = 8 * i + 2 * e + k;
              // a row or column that is none: 0 whatever was summed there
              g[k] = at < left ? exp_of(v[at] - lse) * factor : 0.f;
            }
            w[e] = ops::pack2<T>(g[0], g[1]);
          }
          to[lane * 8 + (i ^ (lane & 7))] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        // the target's, which is a difference, from elsewhere: the sum here has drifted more than 1 - p of a likely one.
        // (Chosen with each element, it took the kernel for 6000 tokens over 8000 x 512 from 60 to 65 us.)
        if (tgt >= 0 && tgt < kCols)
          reinterpret_cast<T*>(to + lane * 8 + ((tgt >> 3) ^ (lane & 7)))[tgt & 7] = ops::from_f<T>(own * factor);
        fence_async();
        __syncwarp();
        if (lane == 0) {
          store_box(&p.store, col0, row0, saddr(st));
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
      }
    }
    if (KIND == kGrad && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncwarp();
  if (*dead) {
    // a wait gave up: let copies and products in flight end before their memory is let go
    for (int i = 0; i < 2000; ++i) __nanosleep(1000);
    if (lane == 0) atomicExch(p.error, 1);
  }
  __syncthreads();
  cluster_sync();
  if (warp == kEpilogueWarps + 1) tmem_free(tmem);
}

// The sum of a split tile's parts, in the order of the summed dimension.  A CTA takes 32 rows of 64 columns: two warps
// side by side, in kJoin rows of warps that share the parts.
constexpr int kJoin = 4;
template <typename T> __global__ void __launch_bounds__(64 * kJoin) k_join(const __grid_constant__ Product p, int pairs) {
  __shared__ float4 st[kJoin][2][32 * 8];
  after_previous();
  next_may_launch();
  const int live = p.live ? *p.live : 0;
  const int m = p.live_is == 1 ? live : p.m, k = p.live_is == 2 ? live : p.k;
  const Schedule s = schedule_of(m, p.n, p.bn, k, pairs, true);
  const int i = blockIdx.y;  // of the tiles that are cut
  if (i >= s.tiles - s.whole) return;
  const int tile = s.whole + i;
  const int tm = p.m_fast ? tile % s.mt : tile / s.nt, tn = p.m_fast ? tile / s.mt : tile % s.nt;
  const int warp = threadIdx.x >> 5 & 1, turn = threadIdx.x >> 6, lane = threadIdx.x & 31;
  const int rows32 = blockIdx.x >> 2, cols64 = blockIdx.x & 3;  // of 8 and of 4
  const int row0 = tm * kTile + rows32 * 32, col0 = tn * p.bn + cols64 * 64 + warp * 32;
  const int end = min(p.n, tn * p.bn + p.bn);
  if (cols64 * 64 >= p.bn || row0 >= m || tn * p.bn + cols64 * 64 >= end) return;
  // the parts: `parts` of them, part j in slot first + j * step, but for the first one's
  int parts, first, step, slot0;
  if (s.cuts) {
    parts = s.cuts;
    first = slot0 = 2 * i;
    step = 2 * s.rest;
  } else {
    const long long lo = (long long)i * s.kb, hi = lo + s.kb;
    int w = (int)(lo * s.workers / s.steps);
    while (w > 0 && first_step(s, w) > lo) --w;
    while (first_step(s, w + 1) <= lo) ++w;
    int last = w;
    while (last + 1 < s.workers && first_step(s, last + 1) < hi) ++last;
    parts = last - w + 1;
    if (parts == 1) return;  // one pair did all of it
    first = 2 * w;
    slot0 = first + (first_step(s, w) < lo ? 1 : 0);
    step = 2;
  }
  float v[32];
#pragma unroll
  for (int c = 0; c < 32; ++c) v[c] = 0.f;
  for (int j = turn; j < parts; j += kJoin) {
    const int slot = j == 0 ? slot0 : first + j * step;
    const float4* from = reinterpret_cast<const float4*>(p.slots + slot * kSlotFloats) + (long long)(rows32 >> 2) * kHalf * kTile / 4 +
                         (long long)(cols64 * 16 + warp * 8) * kHalf + (rows32 & 3) * 32 + lane;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float4 x = __ldcg(from + c * kHalf);
      v[4 * c] += x.x;
      v[4 * c + 1] += x.y;
      v[4 * c + 2] += x.z;
      v[4 * c + 3] += x.w;
    }
  }
  if (turn > 0) {
#pragma unroll
    for (int c = 0; c < 8; ++c) st[turn][warp][c * 32 + lane] = make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
  }
  __syncthreads();
  if (turn > 0) return;
#pragma unroll
  for (int t = 1; t < kJoin; ++t)
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float4 x = st[t][warp][c * 32 + lane];
      v[4 * c] += x.x;
      v[4 * c + 1] += x.y;
      v[4 * c + 2] += x.z;
      v[4 * c + 3] += x.w;
    }
  put_block<T>(v, st[0][warp], lane, p, row0, min(32, m - row0), col0, min(32, end - col0), p.scale ? *p.scale : 1.f);
}

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                            const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                            CUtensorMapFloatOOBfill);
Encode encode_function() {
  static Encode f = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<Encode>(p);
  }();
  return f;
}

}  // namespace

cudaError_t make_map(CUtensorMap* map, const void* p, long long rows, long long cols, long long stride, int box_rows, bool bf16) {
  const Encode encode = encode_function();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)std::max(rows, 1LL)}, strides[1] = {(cuuint64_t)stride * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, step[2] = {1, 1};
  const CUresult r = encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(p), dims,
                            strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

namespace {
template <int KIND, typename T> cudaError_t raise(int device) {
  static std::atomic<unsigned long long> raised{0};
  return ops::raise_smem(k_product<KIND, T>, raised, device, kSmem);
}
template <int KIND, typename T> cudaError_t go(const Product& p, unsigned pairs, int device, cudaStream_t st) {
  const cudaError_t e = raise<KIND, T>(device);
  return e != cudaSuccess ? e : ops::launch_early(k_product<KIND, T>, 2 * pairs, kThreads, kSmem, 1, st, p);
}
template <typename F> cudaError_t by_type(int dtype, F&& f) {
  return dtype == PSGD_F32 ? f((float*)nullptr) : dtype == PSGD_F16 ? f((__half*)nullptr) : f((__nv_bfloat16*)nullptr);
}
}  // namespace

cudaError_t pairs_of(int device, int* pairs) {
  cudaError_t e = raise<kOut, float>(device);
  if (e != cudaSuccess) return e;
  int sms = 0;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = sms / 2 * 2;
  cfg.blockDim = kThreads;
  cfg.dynamicSmemBytes = kSmem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {2, 1, 1};
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaOccupancyMaxActiveClusters(pairs, k_product<kOut, float>, &cfg);
  if (e == cudaSuccess && *pairs < 1) e = cudaErrorLaunchOutOfResources;
  return e;
}

// Columns of an OUT product's tiles.  A step costs about as long as its lines take into an SM, 0.33 us for 256 + 256
// rows and columns, and what is drained after a pair's last step, 2.5 us for 256 columns, is waited for.  So where the tiles
// do not occupy the pairs (and cannot be cut along k), narrower ones end earlier: 1024 x 1024 from 509 rows, 16 tiles of 256
// columns 12.2 us, 64 of 64 columns 11.4.
static int columns_of(const Product& p, int pairs) {
  int best = kTile;
  double least = 1e30;
  for (int bn = kTile; bn >= 64; bn /= 2) {
    const Schedule s = schedule_of(p.m, p.n, bn, p.k, pairs, p.slots != nullptr);
    const double step = 0.33 * (kTile + bn) / (2 * kTile), steps = (double)s.kb;
    double us = (double)(s.whole / pairs + (s.whole % pairs ? 1 : 0)) * steps * step + 2.5 * bn / kTile;
    if (s.workers) us += (double)s.steps / s.workers * step + 4.0;
    if (us < 0.95 * least) {
      least = us;
      best = bn;
    }
  }
  return best;
}

// A step costs as its rows and columns; the last turn's pairs without a tile idle.  For up to 256 tokens over 50257 columns,
// 197 tiles of 256 on 76 pairs are 3 turns, 225 of 224 as many.  GRAD leaves boxes of 64 columns.
int logits_columns(Epilogue kind, long long rows, long long n, int pairs) {
  int best = kTile;
  long long least = 0;
  for (int bn = kTile; bn >= 128; bn -= kind == kGrad ? 64 : 32) {
    const long long turns = ops::units(ops::units(rows, kTile) * ops::units(n, bn), pairs), cost = turns * (std::min<long long>(rows, kTile) + bn);
    if (bn == kTile || cost * 20 < least * 19) {
      least = cost;
      best = bn;
    }
  }
  return best;
}

cudaError_t enqueue(Epilogue kind, Product p, int device, int pairs, cudaStream_t st) {
  if (kind == kOut) {  // (the others' callers know theirs, of which B's boxes have half)
    p.bn = columns_of(p, pairs);
    const int size = 4 * ops::dtype_size(p.dtype);
    p.vec = (uintptr_t)p.out % size == 0 && (p.ldo % 4 == 0 || p.m == 1);
  }
  // where A with K rows has fewer rows than a CTA's part, or B fewer columns, there are more stages
  p.a_bytes = p.a_m_rows || p.m > kHalf ? kOperand : (int)ops::units(std::max(p.m, 1), kFew) * kFew * kStep * 2;
  p.stage_bytes = p.a_bytes + (p.b_m_rows ? (p.bn > 128 ? kOperand : kOperand / 2) : p.bn * kStep);
  p.stages = std::min(kMostStages, kStages * kStageBytes / p.stage_bytes);
  // (extents that the device knows are at most these)
  const long long tiles = ops::units(p.m, kTile) * ops::units(p.n, p.bn);
  if (tiles == 0) return cudaSuccess;
  // split tiles want every pair, also where there are few of them
  const unsigned grid = (unsigned)(p.slots ? pairs : std::min<long long>(pairs, tiles));
  cudaError_t e;
  if (kind == kLse) e = go<kLse, float>(p, grid, device, st);
  else if (kind == kGrad) e = p.bf16 ? go<kGrad, __nv_bfloat16>(p, grid, device, st) : go<kGrad, __half>(p, grid, device, st);
  else e = by_type(p.dtype, [&](auto* t) { return go<kOut, std::remove_pointer_t<decltype(t)>>(p, grid, device, st); });
  if (e != cudaSuccess || kind != kOut || !p.slots) return e;
  // Which tiles are cut goes by the extents that the device knows.  Few steps are never cut, and of one row of tiles there
  // is either that or nothing.
  const Schedule s = schedule_of(p.m, p.n, p.bn, p.k, pairs, true);
  if (s.kb < 2 * kMinSplit || ((!p.live || (p.live_is == 1 && s.mt == 1)) && s.workers == 0)) return e;
  const dim3 parts(32, (unsigned)std::min<long long>(tiles, pairs - 1));
  return by_type(p.dtype, [&](auto* t) {
    return ops::launch_early(k_join<std::remove_pointer_t<decltype(t)>>, parts, 64 * kJoin, 0, 1, st, p, pairs);
  });
}

}  // namespace mma
}  // namespace psgd
