// Matrix products on the tensor cores (psgd_mma.cuh), with what follows a product
// in the same kernel: the pieces of a log-sum-exp, the gradient of a softmax cross
// entropy, or the sums' rounding into a bucket.
//
// Persistent pairs of CTAs.  In each, one thread loads (TMA, six stages of 32 KB), one
// thread of the first CTA multiplies (tcgen05, both CTAs' tensor memory), eight warps take finished tiles out
// of tensor memory while the next tile is summed in its other half.
#include <algorithm>
#include <mutex>

#include "psgd_mma.cuh"

namespace psgd {
namespace mma {
namespace {

using ops::after_previous;
using ops::next_may_launch;

struct Shared {
  uint64_t full[kStages], empty[kStages], done[2], drained[2];
  uint32_t tmem;
  volatile int dead;
};

// One run of a pair: steps [k0, k1) of tile (tm, tn); slot < 0: the whole tile.
struct Run {
  int tm, tn, k0, k1, slot;
};
struct Walk {
  Schedule s;
  int pairs, pair, m_fast, next;
  long long at, end;
  int piece;
  __device__ Walk(const Product& p, int m, int k, int pairs_, int pair_)
      : s(schedule_of(m, p.n, k, pairs_, p.slots != nullptr)), pairs(pairs_), pair(pair_), m_fast(p.m_fast), next(pair_), piece(0) {
    at = pair < s.workers ? first_step(s, pair) : 0;
    end = pair < s.workers ? first_step(s, pair + 1) : 0;
  }
  __device__ bool take(Run& r) {
    int tile;
    if (next < s.whole) {
      tile = next;
      next += pairs;
      r.k0 = 0;
      r.k1 = s.kb;
      r.slot = -1;
    } else if (at < end) {
      const int i = (int)(at / s.kb);
      tile = s.whole + i;
      r.k0 = (int)(at - (long long)i * s.kb);
      r.k1 = (int)min((long long)s.kb, r.k0 + (end - at));
      r.slot = r.k0 == 0 && r.k1 == s.kb ? -1 : 2 * pair + piece;
      at += r.k1 - r.k0;
      ++piece;
    } else {
      return false;
    }
    r.tm = m_fast ? tile % s.mt : tile / s.nt;
    r.tn = m_fast ? tile / s.mt : tile % s.nt;
    return true;
  }
};

__device__ __forceinline__ float exp_of(float x) {
  // 2 ulp of ex2 and the product's rounding, |x| 2^-24 of the result at most
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}

// A 32 x 32 block (lane = row) through a warp's staging into rows of `out`, 32 elements side by side.
__device__ __forceinline__ void put_block(const float (&v)[32], float* st, int lane, void* out, int dtype, long long ldo, long long row0,
                                          int rows, long long col0, int cols, float scale, int accumulate) {
#pragma unroll
  for (int c = 0; c < 32; ++c) st[lane * 32 + (c ^ lane)] = v[c] * scale;
  __syncwarp();
  if (lane < cols) {
    for (int r = 0; r < rows; ++r) {
      const long long i = (row0 + r) * ldo + col0 + lane;
      const float x = st[r * 32 + (lane ^ r)];
      ops::store_any(out, dtype, i, accumulate ? ops::read_any(out, dtype, i) + x : x);
    }
  }
  __syncwarp();
}

template <int KIND>
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
    for (int i = 0; i < kStages; ++i) {
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
  const int live = p.live ? *p.live : 0;
  const int m = p.live_is == 1 ? live : p.m, k = p.live_is == 2 ? live : p.k;
  Walk walk(p, m, k, pairs, pair);
  Run run;
  volatile int* dead = &sh.dead;

  if (warp == kEpilogueWarps) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      while (walk.take(run)) {
        const int row = run.tm * kTile + (int)rank * kHalf, col = run.tn * kTile + (int)rank * kHalf;
        for (int kb = run.k0; kb < run.k1; ++kb) {
          if (!bar_wait(&sh.empty[stage], phase ^ 1, dead)) break;
          const uint32_t a = saddr(stages + stage * kStageBytes), b = a + kOperand, bar = at_rank(saddr(&sh.full[stage]), 0);
          if (rank == 0) bar_expect(&sh.full[stage], 2 * kStageBytes);
          const int x = kb * kStep;
          if (p.a_m_rows) {
            load_box(a, &p.a, row, x, bar);
            load_box(a + kOperand / 2, &p.a, row + 64, x, bar);
          } else {
            load_box(a, &p.a, x, row, bar);
          }
          if (p.b_m_rows) {
            load_box(b, &p.b, col, p.b_y0 + x, bar);
            load_box(b + kOperand / 2, &p.b, col + 64, p.b_y0 + x, bar);
          } else {
            load_box(b, &p.b, x, p.b_y0 + col, bar);
          }
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (*dead) break;
      }
    }
  } else if (warp == kEpilogueWarps + 1) {
    if (rank == 0 && lane == 0) {
      const uint32_t idesc = instruction(p.bf16, p.a_m_rows, p.b_m_rows);
      const uint32_t a_step = step_bytes(p.a_m_rows) >> 4, b_step = step_bytes(p.b_m_rows) >> 4;
      int stage = 0, buf = 0;
      uint32_t phase = 0, turn = 0;
      while (walk.take(run)) {
        if (!bar_wait(&sh.drained[buf], turn ^ 1, dead)) break;
        fence_after();
        const uint32_t d = tmem + buf * kTile;
        for (int kb = run.k0; kb < run.k1; ++kb) {
          if (!bar_wait(&sh.full[stage], phase, dead)) break;
          fence_after();
          const uint32_t at = saddr(stages + stage * kStageBytes);
          const uint64_t a = describe(at, p.a_m_rows), b = describe(at + kOperand, p.b_m_rows);
#pragma unroll
          for (int i = 0; i < kStep / 16; ++i) multiply(d, a + i * a_step, b + i * b_step, idesc, kb > run.k0 || i > 0);
          commit_both(&sh.empty[stage]);
          if (++stage == kStages) {
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
  } else {
    const int quarter = warp & 3, half = warp >> 2;
    float* st = reinterpret_cast<float*>(staging + warp * kStaging);
    const float scale = KIND == kOut && p.scale ? *p.scale : 1.f;
    int buf = 0;
    uint32_t turn = 0;
    while (walk.take(run)) {
      if (!warp_wait(&sh.done[buf], turn, dead)) break;
      fence_after();
      const uint32_t t = tmem + buf * kTile + half * kHalf + ((uint32_t)(quarter * 32) << 16);
      const int row0 = run.tm * kTile + (int)rank * kHalf + quarter * 32, row = row0 + lane;
      const int col0 = run.tn * kTile + half * kHalf;
      float v[32];
      if constexpr (KIND == kOut) {
        for (int c = 0; c < 4; ++c) {
          if (run.k1 > run.k0) {
            tmem_load32(t + c * 32, v);
          } else {  // a sum of nothing
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.f;
          }
          if (run.slot >= 0) {
            // groups of four columns, row by row: neighbouring lanes write neighbouring 16 bytes
            float4* to = reinterpret_cast<float4*>(p.slots + run.slot * kSlotFloats) + (long long)rank * kHalf * kTile / 4 +
                         (long long)(half * 32 + c * 8) * kHalf + quarter * 32 + lane;
#pragma unroll
            for (int i = 0; i < 8; ++i) to[i * kHalf] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          } else {
            put_block(v, st, lane, p.out, p.dtype, p.ldo, row0, min(32, m - row0), col0 + c * 32, min(32, p.n - col0 - c * 32), scale,
                      p.accumulate);
          }
        }
      } else if constexpr (KIND == kLse) {
        const int tgt = row < m ? p.target[row] - p.column0 - col0 : -1;
        const int left = p.vocab - p.column0 - col0;  // columns that are in the vocabulary
        float top = -INFINITY, sum = 0.f;
        for (int c = 0; c < 4; ++c) {
          tmem_load32(t + c * 32, v);
          if (left < c * 32 + 32) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (c * 32 + i >= left) v[i] = -INFINITY;
          }
          float most = v[0];
#pragma unroll
          for (int i = 1; i < 32; ++i) most = fmaxf(most, v[i]);
          if (tgt >= c * 32 && tgt < c * 32 + 32) {
            float z = 0.f;
#pragma unroll
            for (int i = 0; i < 32; ++i) z = tgt - c * 32 == i ? v[i] : z;
            p.at_target[row] = z;
          }
          const float now = fmaxf(top, most), from = now == -INFINITY ? 0.f : now;
          sum *= top == -INFINITY ? 0.f : exp_of(top - now);
          top = now;
          float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 32; ++i) s[i & 3] += exp_of(v[i] - from);
          sum += (s[0] + s[1]) + (s[2] + s[3]);
        }
        if (row < m) p.part[(long long)((p.column0 + col0) / kHalf) * p.part_rows + row] = make_float2(top, sum);
      } else {
        const bool in = row < m;
        const float lse = in ? p.lse[row] : 0.f, factor = in ? p.factor[row] : 0.f;
        const int tgt = in ? p.target[row] - p.column0 - col0 : -1;
        const int left = in ? p.vocab - p.column0 - col0 : 0;
        uint4* to = reinterpret_cast<uint4*>(st);
        for (int box = 0; box < 2; ++box) {
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the staging's last box is out
          __syncwarp();
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int at = box * 64 + c * 32;
            tmem_load32(t + at, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              // a row or column that is none: 0 whatever was summed there
              const float g = (exp_of(v[i] - lse) - (at + i == tgt ? 1.f : 0.f)) * factor;
              v[i] = at + i < left ? g : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint4 u;
              unsigned* w = &u.x;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = p.bf16 ? ops::pack2<__nv_bfloat16>(v[8 * i + 2 * e], v[8 * i + 2 * e + 1])
                              : ops::pack2<__half>(v[8 * i + 2 * e], v[8 * i + 2 * e + 1]);
              to[lane * 8 + ((c * 4 + i) ^ (lane & 7))] = u;
            }
          }
          fence_async();
          __syncwarp();
          if (lane == 0) {
            store_box(&p.store, col0 + box * 64, row0, saddr(st));
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive_at(at_rank(saddr(&sh.drained[buf]), 0));
      buf ^= 1;
      turn ^= buf == 0;
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
  next_may_launch();
  cluster_sync();
  if (warp == kEpilogueWarps + 1) tmem_free(tmem);
}

// The sum of a split tile's parts, in the order of the summed dimension.  A CTA takes 32 rows of 64 columns.
__global__ void __launch_bounds__(64) k_join(const __grid_constant__ Product p, int pairs) {
  __shared__ float st[2][32 * 32];
  after_previous();
  next_may_launch();
  const int live = p.live ? *p.live : 0;
  const int m = p.live_is == 1 ? live : p.m, k = p.live_is == 2 ? live : p.k;
  const Schedule s = schedule_of(m, p.n, k, pairs, true);
  const int i = blockIdx.y;  // of the tiles that are cut
  if (i >= s.tiles - s.whole) return;
  const int tile = s.whole + i;
  const int tm = p.m_fast ? tile % s.mt : tile / s.nt, tn = p.m_fast ? tile / s.mt : tile % s.nt;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows32 = blockIdx.x >> 2, cols64 = blockIdx.x & 3;  // of 8 and of 4
  const int row0 = tm * kTile + rows32 * 32, col0 = tn * kTile + cols64 * 64 + warp * 32;
  if (row0 >= m || col0 >= p.n) return;
  const long long lo = (long long)i * s.kb, hi = lo + s.kb;
  int w = (int)(lo * s.workers / s.steps);
  while (w > 0 && first_step(s, w) > lo) --w;
  while (first_step(s, w + 1) <= lo) ++w;
  if (first_step(s, w) <= lo && first_step(s, w + 1) >= hi) return;  // one pair did all of it
  float v[32];
#pragma unroll
  for (int c = 0; c < 32; ++c) v[c] = 0.f;
  for (; w < s.workers && first_step(s, w) < hi; ++w) {
    const int slot = 2 * w + (first_step(s, w) < lo ? 1 : 0);
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
  put_block(v, st[warp], lane, p.out, p.dtype, p.ldo, row0, min(32, m - row0), col0, min(32, p.n - col0), p.scale ? *p.scale : 1.f,
            p.accumulate);
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
template <int KIND> cudaError_t raise(int device) {
  static std::atomic<unsigned long long> raised{0};
  return ops::raise_smem(k_product<KIND>, raised, device, kSmem);
}
template <int KIND> cudaError_t go(const Product& p, unsigned pairs, int device, cudaStream_t st) {
  const cudaError_t e = raise<KIND>(device);
  return e != cudaSuccess ? e : ops::launch_early(k_product<KIND>, 2 * pairs, kThreads, kSmem, 1, st, p);
}
}  // namespace

cudaError_t pairs_of(int device, int* pairs) {
  cudaError_t e = raise<kOut>(device);
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
  e = cudaOccupancyMaxActiveClusters(pairs, k_product<kOut>, &cfg);
  if (e == cudaSuccess && *pairs < 1) e = cudaErrorLaunchOutOfResources;
  return e;
}

cudaError_t enqueue(Epilogue kind, const Product& p, int device, int pairs, cudaStream_t st) {
  // (extents that the device knows are at most these)
  const long long tiles = ops::units(p.m, kTile) * ops::units(p.n, kTile);
  if (tiles == 0) return cudaSuccess;
  // split tiles want every pair, also where there are few of them
  const unsigned grid = (unsigned)(p.slots ? pairs : std::min<long long>(pairs, tiles));
  cudaError_t e;
  if (kind == kLse) e = go<kLse>(p, grid, device, st);
  else if (kind == kGrad) e = go<kGrad>(p, grid, device, st);
  else e = go<kOut>(p, grid, device, st);
  if (e != cudaSuccess || kind != kOut || !p.slots) return e;
  // which tiles are cut goes by the extents that the device knows; with those of the host there may be none
  if (!p.live && schedule_of(p.m, p.n, p.k, pairs, true).workers == 0) return e;
  return ops::launch_early(k_join, dim3(32, (unsigned)std::min<long long>(tiles, pairs - 1)), 64, 0, 1, st, p, pairs);
}

}  // namespace mma
}  // namespace psgd
