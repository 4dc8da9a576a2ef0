// Embedding: lookup with scaling, and the dense gradient of the table.
//
//   forward   y_i = s * W[id_i]
//   backward  dW_v = [dW_v +] s * sum over the tokens i with id_i = v of g_i
//
// The gradient sorts the tokens by id (stable, so by position within an id),
// cuts the sorted list into chunks of equal length and lets each CTA add its
// chunk's rows in order, in fp32.  A row whose tokens lie in one chunk is
// written there; a row that crosses a chunk's end leaves one fp32 partial per
// chunk, and a last kernel adds those in chunk order.  Few tokens take one
// launch without a sort (k_rows_direct).  No sum depends on the order in which
// CTAs run.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>
#include <new>
#include <type_traits>

#include "psgd_ops.cuh"

namespace cg = cooperative_groups;

struct psgd_embedding {
  int device = 0;
  int sms = 0;
  bool many_sort_ctas = false;  // this device runs clusters of 16 CTAs
  long long vocab = 0, dim = 0, max_tokens = 0;
  void* memory = nullptr;  // all of the following
  // the sorted tokens: two (id, position) buffers the radix passes alternate between
  int2* sorted[2] = {nullptr, nullptr};
  float* part = nullptr;  // per chunk: the partial rows of its first and its last id
  int4* crossing = nullptr;  // rows that cross a chunk's end: (chunk where they begin, id, chunks that follow)
  int* counts = nullptr;     // of few partials; sorted tokens; of many partials
  unsigned char* named = nullptr;  // per row of the table: a token names it
  int* ready = nullptr;            // the map is complete (0 between calls)
  int* d_flag = nullptr;  // an id outside [0, vocab) was seen
  size_t bytes = 0;
};

namespace psgd {
namespace ops {
namespace {

constexpr int kMaxChunk = 32;       // sorted tokens per CTA of the row sums, at most
constexpr int kFewParts = 8;        // partials of a row that one warp adds
constexpr int kJoinWarps = 8;
// Zeroing CTAs of 256 threads to an SM, at most.  BERT-large's table (125 MB,
// 16384 tokens) takes 45.8, 44.4 and 44.0 us with 1, 2 and 4 of them, with 32
// tokens 34.8, 29.7 and 27.2: fewer leave room for the row sums' CTAs, but do
// not reach the write rate alone.
constexpr int kZeroCtas = 4;
constexpr int kSortCtas = 8;        // CTAs of the sort's cluster
constexpr int kManySortCtas = 16;   // the same for many tokens: more than 8 is not portable
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;

// Tokens in an (outer, inner) layout: token i = o * inner + n at o * os + n * is,
// in units of the operand's elements.  inner = 0: all tokens are `is` apart,
// and no division is needed to find one.
struct Layout2 {
  long long os, is;
  int inner;
  Layout2(int64_t outer, int64_t inner_, int64_t os_, int64_t is_)
      : os(os_), is(inner_ == 1 ? os_ : is_), inner(outer == 1 || inner_ == 1 || os_ == inner_ * is_ ? 0 : (int)inner_) {}
  __device__ __forceinline__ long long at(int i) const {
    if (inner == 0) return i * is;
    const int o = i / inner;
    return o * os + (i - o * inner) * is;
  }
};

__device__ __forceinline__ long long load_id(const void* ids, int id64, long long at) {
  return id64 ? __ldg((const long long*)ids + at) : (long long)__ldg((const int*)ids + at);
}

// A group of threads (blockDim = (threads of a group, groups)) takes one token;
// thread t owns the vectors t, t + threads, ... (NV of them) of a tile of
// columns, all of them under way at once.  What finding a token's row costs is
// paid once per NV vectors.  Bound by the rows' way from L2 and the output's to
// it: 16384 tokens of a 30522 x 1024 fp32 table 15.5 us (89 MB from and to HBM,
// 85 % of the copy bandwidth; 134 MB through L2); with one vector a thread and
// four tokens at a time 25 us, with two tokens 17.5.
template <typename W, typename O, int VEC, int NV>
__global__ void __launch_bounds__(256) k_lookup(const W* __restrict__ weight, long long wstride, long long vocab,
                                                int dim, const void* __restrict__ ids, int id64, Layout2 il, int n,
                                                float scale, O* __restrict__ out, Layout2 ol, int* flag) {
  // (single elements: a warp's are next to each other, at constant distances)
  const int c0 = VEC > 1 ? (blockIdx.y * blockDim.x * NV + threadIdx.x) * VEC
                         : (blockIdx.y * blockDim.x + threadIdx.x / 32 * 32) * NV + threadIdx.x % 32;
  const int step = VEC > 1 ? blockDim.x * VEC : 32;
  const long long token = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  if (token >= n) return;
  after_previous();
  next_may_launch();
  const int i = (int)token;
  const long long id = load_id(ids, id64, il.at(i));
  const bool ok = id >= 0 && id < vocab;
  if (!ok && threadIdx.x == 0) *flag = 1;
  const W* src = weight + (ok ? id : 0) * wstride + c0;
  O* dst = out + ol.at(i) + c0;
  Pack<W, VEC> v[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (c0 + j * step < dim) v[j] = load_pack<W, VEC>(src + j * step);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (c0 + j * step >= dim) continue;
    float f[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = ok ? to_f(v[j].v[e]) * scale : 0.f;
    store_run<O, VEC>(dst + j * step, f);
  }
}

struct SortArgs {
  const void* ids;
  int id64;
  Layout2 il;
  int n, vocab;
  long long padding;
  int passes;
  int2* sorted[2];       // (id, position); pass p writes buffer p & 1
  int* flag;
  int* counts;           // out: [0] = [2] = 0 (crossing rows found so far), [1] = tokens with a gradient
  // NULL, or one byte a row: 1 where a token with a gradient names it.  It is
  // complete once *ready is 1, early in the first pass.
  unsigned char* named;
  int* ready;
};

template <int CTAS, int BITS> struct SortShared {
  // a CTA's counts fit 16 bits where a digit has 10 (the host sees to it)
  using Count = typename std::conditional<(BITS > 8), unsigned short, int>::type;
  static constexpr int kDigits = 1 << BITS;
  static constexpr int kParts = kSortThreads / kDigits;  // threads per digit of the scan over the warps
  Count cnt[kSortWarps][kDigits];
  int part[kParts][kDigits];
  int totals[CTAS][kDigits];  // every CTA's digit totals, pushed by the peers
  int base[kDigits];
  int scan[32];
  int all;
};

// Stable least-significant-digit radix sort of (id, position) by one cluster of
// CTAS.  Tokens without a gradient (padding, or an id outside the table) are
// dropped by the first pass.  Each warp owns a contiguous share of the list, so
// that digit counts per (CTA, warp), scanned in list order, give every element
// its place; each CTA writes its digit totals into its peers' shared memory.  A
// warp loads 32 x ITEMS elements of its share at a time; a share of no more stays
// in registers between counting and placing.  The time is the chain of
// latencies of a pass (a load, the barriers, a scan, a scattered store), so
// tables of up to 1024 rows take one pass of 10 bits in place of two of 8, and
// up to 2048 tokens one CTA without a cluster's barriers.  Digits are counted by
// shared-memory atomics; when elements are placed, a warp's equal digits are
// found by a ballot per bit.  16384 tokens of 30522 rows take 14 us profiled
// alone from a cold cache, on 16 of the SMs while the others zero the rows that
// no token names (17 us on 8 SMs).
template <int CTAS, int ITEMS, int BITS> __global__ void __launch_bounds__(kSortThreads) k_sort_tokens(SortArgs a) {
  using Shared = SortShared<CTAS, BITS>;
  constexpr int D = Shared::kDigits, PARTS = Shared::kParts, PER = kSortWarps / PARTS;
  extern __shared__ __align__(16) unsigned char raw[];
  Shared& s = *reinterpret_cast<Shared*>(raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = CTAS > 1 ? (int)cluster.block_rank() : 0;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  after_previous();  // and with it the row sums' kernel, which starts when this one lets it
  if (a.named) {  // (its size is rounded up to 16 bytes)
    uint4* v = reinterpret_cast<uint4*>(a.named);
    for (int i = rank * kSortThreads + t; i < (int)units(a.vocab, 16); i += CTAS * kSortThreads) v[i] = make_uint4(0, 0, 0, 0);
  }
  if constexpr (CTAS > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  const unsigned below = (1u << lane) - 1u;
  int n = a.n;
  for (int p = 0; p < a.passes; ++p) {
    const int shift = BITS * p;
    const int2* src = p & 1 ? a.sorted[0] : a.sorted[1];
    int2* dst = p & 1 ? a.sorted[1] : a.sorted[0];
    const int per = (int)((n + (long long)CTAS * kSortThreads - 1) / ((long long)CTAS * kSortThreads)) * 32;
    const long long first = ((long long)rank * kSortWarps + warp) * per;
    const int share = (int)max(0LL, min((long long)n - first, (long long)per));  // of this warp
    // a token's id, or -1 if it has no gradient, and its position
    auto id_at = [&](long long i) -> int {
      const long long id = load_id(a.ids, a.id64, a.il.at((int)i));
      if (id < 0 || id >= a.vocab) {
        *a.flag = 1;
        return -1;
      }
      return id == a.padding ? -1 : (int)id;
    };
    auto digit = [&](int key) { return key < 0 ? D : (key >> shift) & (D - 1); };
    auto count = [&](int d) {  // (a warp's own counts; two of 16 bits to a word)
      if (d >= D) return;
      if constexpr (sizeof(typename Shared::Count) == 2)
        atomicAdd(reinterpret_cast<unsigned*>(&s.cnt[warp][d & ~1]), 1u << (16 * (d & 1)));
      else
        atomicAdd(&s.cnt[warp][d], 1);
    };
    // the lanes with the same digit, bit by bit (__match_any_sync takes several times as long)
    auto same_digit = [&](int d) {
      unsigned same = 0xffffffffu;
#pragma unroll
      for (int b = 0; b <= BITS; ++b) {
        const bool bit = d >> b & 1;
        const unsigned set = __ballot_sync(0xffffffffu, bit);
        same &= bit ? set : ~set;
      }
      return same;
    };
    auto place = [&](int d, int key, int pos) {
      const unsigned same = same_digit(d);
      const int ahead = __popc(same & below);
      int at = 0;
      if (d < D) {
        at = s.cnt[warp][d];
        dst[s.base[d] + at + ahead] = make_int2(key, pos);
      }
      __syncwarp();
      if (d < D && ahead == 0) s.cnt[warp][d] = at + __popc(same);
      __syncwarp();
    };
    int key[ITEMS], pos[ITEMS];
    auto load = [&](int e0) {  // the elements e0 .. e0 + 32 ITEMS of the share
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int e = e0 + i * 32 + lane;
        if (e >= share) {
          key[i] = -1;
        } else if (p == 0) {
          key[i] = id_at(first + e);
          pos[i] = (int)first + e;
        } else {
          const int2 v = __ldcg(src + first + e);
          key[i] = v.x;
          pos[i] = v.y;
        }
      }
    };
    load(0);
    {
      uint4* z = reinterpret_cast<uint4*>(&s.cnt[0][0]);
      for (int i = t; i < (int)(sizeof(s.cnt) / 16); i += kSortThreads) z[i] = make_uint4(0, 0, 0, 0);
    }
    if constexpr (CTAS > 1) {
      // all have started, and the map is clear
      if (p == 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    __syncthreads();
    const bool mark = p == 0 && a.named;
    for (int e0 = 0; e0 < share; e0 += 32 * ITEMS) {
      if (e0 > 0) load(e0);
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
        if (e0 + i * 32 < share) {
          if (mark && key[i] >= 0) a.named[key[i]] = 1;
          count(digit(key[i]));
        }
    }
    __syncthreads();
    // exclusive counts over the warps, PER of them per thread
    const int d = t & (D - 1), q = t / D;
    int total = 0;
#pragma unroll
    for (int w = 0; w < PER; ++w) {
      const int c = s.cnt[q * PER + w][d];
      s.cnt[q * PER + w][d] = total;
      total += c;
    }
    if constexpr (PARTS > 1) {
      s.part[q][d] = total;
      __syncthreads();
      int ahead = 0;
      total = 0;
#pragma unroll
      for (int k = 0; k < PARTS; ++k) {
        const int c = s.part[k][d];
        if (k < q) ahead += c;
        total += c;
      }
      if (q > 0) {
#pragma unroll
        for (int w = 0; w < PER; ++w) s.cnt[q * PER + w][d] += ahead;
      }
    }
    if constexpr (CTAS > 1) {
#pragma unroll
      for (int k = 0; k < CTAS / PARTS; ++k)
        cluster.map_shared_rank(&s.totals[rank][0], q * (CTAS / PARTS) + k)[d] = total;
      cluster.sync();
    }
    if (p == 0) {
      if (CTAS == 1) __syncthreads();
      if (mark && rank == 0 && t == 0)
        asm volatile("st.release.gpu.global.s32 [%0], 1;" ::"l"(a.ready) : "memory");
      next_may_launch();
    }
    int before = 0, all = 0, inc = 0;
    if (t < D) {
      if constexpr (CTAS > 1) {
#pragma unroll
        for (int r = 0; r < CTAS; ++r) {
          const int c = s.totals[r][t];
          if (r < rank) before += c;
          all += c;
        }
      } else {
        all = total;
      }
      inc = all;  // inclusive scan over the digits of a warp
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (lane == 31) s.scan[warp] = inc;
    }
    __syncthreads();
    if (t < D) {
      const int mine = lane < D / 32 ? s.scan[lane] : 0;
      const int ahead = __reduce_add_sync(0xffffffffu, lane < warp ? mine : 0);
      s.base[t] = ahead + inc - all + before;
      if (t == D - 1) s.all = ahead + inc;
    }
    __syncthreads();
    for (int e0 = 0; e0 < share; e0 += 32 * ITEMS) {
      if (share > 32 * ITEMS) load(e0);
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
        if (e0 + i * 32 < share) place(digit(key[i]), key[i], pos[i]);
    }
    n = s.all;
    if (p + 1 < a.passes) {
      // this pass's output, for every CTA of the cluster; the totals are free again
      if constexpr (CTAS > 1) cluster.sync();
      else __syncthreads();
    }
  }
  if (rank == 0 && t == 0) {
    a.counts[0] = a.counts[2] = 0;
    a.counts[1] = n;
  }
}

// One warp zeroes `bytes` bytes, 16 at a time between the first and the last boundary.
__device__ __forceinline__ void zero_bytes(char* p, long long bytes, int lane) {
  const long long head = min(bytes, (long long)((16 - ((uintptr_t)p & 15)) & 15));
  const long long vecs = (bytes - head) / 16, tail = bytes - head - vecs * 16;
  uint4* v = reinterpret_cast<uint4*>(p + head);
  for (long long i = lane; i < vecs; i += 32) v[i] = make_uint4(0, 0, 0, 0);
  if (lane < head) p[lane] = 0;
  if (lane < tail) p[head + vecs * 16 + lane] = 0;
}

// The whole table, where there is no token.
__global__ void __launch_bounds__(256) k_zero_table(char* __restrict__ w, long long rows, long long bytes, long long stride) {
  after_previous();
  next_may_launch();
  const int warps = blockDim.x / 32;
  for (long long r = (long long)blockIdx.x * warps + threadIdx.x / 32; r < rows; r += (long long)gridDim.x * warps)
    zero_bytes(w + r * stride, bytes, threadIdx.x & 31);
}

// The rows that no token names, which the CTAs before the row sums' zero while
// the sort runs.
struct ZeroArgs {
  int ctas;                 // 0: rows without a token keep what they hold
  char* table;
  long long bytes, stride;  // of a row
  int vocab;
  const unsigned char* named;
  const int* ready;
};

__device__ __forceinline__ void zero_unnamed(const ZeroArgs& z) {
  // This kernel starts once the sort has let it, after it set *ready: seen as
  // 1, the map is complete and visible.  If it is not seen, the sort's end is
  // waited for, which makes everything visible.
  int ready;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(ready) : "l"(z.ready) : "memory");
  if (!ready) after_previous();
  // a contiguous share of the table, 32 flags at a time and one step ahead
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5, warp = threadIdx.x >> 5;
  const int first = (int)((long long)z.vocab * blockIdx.x / z.ctas), last = (int)((long long)z.vocab * (blockIdx.x + 1) / z.ctas);
  auto unnamed = [&](long long r0) { return r0 + lane < last && __ldcg(z.named + r0 + lane) == 0; };
  bool next = unnamed(first);
  int turn = 0;  // a row per warp
  for (long long r0 = first; r0 < last; r0 += 32) {
    unsigned todo = __ballot_sync(0xffffffffu, next);
    next = unnamed(r0 + 32);
    for (; todo; todo &= todo - 1) {
      if (turn == warp) zero_bytes(z.table + (r0 + __ffs(todo) - 1) * z.stride, z.bytes, lane);
      turn = turn + 1 == warps ? 0 : turn + 1;
    }
  }
}

// A finished sum into its row of the table: as VEC elements if they are
// aligned for that, else one by one.
template <typename O, int VEC>
__device__ __forceinline__ void write_row(O* dst, const float* acc, float scale, int accumulate, bool aligned) {
  float f[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    f[i] = acc[i] * scale;
    if (accumulate) f[i] += to_f(dst[i]);
  }
  if (VEC > 1 && aligned) {
    store_run<O, VEC>(dst, f);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) dst[i] = from_f<O>(f[i]);
  }
}

// The rows of one chunk of sorted tokens (CTAs zero.ctas + chunk), for one tile of columns: thread t
// owns the vectors t, t + threads, ... (NV of them).  kBatch rows are loaded at
// a time, then added in order; a sum ends with its id's last token.  Bound by
// HBM: with the zeroing, 192 MB of BERT-large's table gradient in 31 us (6.2
// TB/s, 92 % of the copy bandwidth).  One column a thread and one row at a time
// it took 48 us for the sums alone.  32 tokens a chunk: a row's partials then
// cost at most two fp32 rows for 32 read.  Rows at any alignment (VEC 1): all
// granules of the chunk's rows are copied into shared memory at once, and read
// from there element by element: 32768 tokens of 30000 x 1601 bf16 77 us with
// the sort (80 before its cluster had 16 CTAs, 109 then with single loads into
// registers, which leave too few under way).
template <typename G, typename O, int VEC, int NV>
__global__ void __launch_bounds__(256, VEC == 1 ? 3 : 4) k_row_sums(const int2* __restrict__ sorted, const G* __restrict__ grad, Layout2 gl, int dim,
                                                  float scale, int accumulate, O* __restrict__ dw, long long stride,
                                                  int dw_aligned, float* __restrict__ part, int chunk, int4* __restrict__ crossing, int* __restrict__ counts, ZeroArgs zero) {
  constexpr int kBatch = VEC == 8 ? 4 : 8;
  extern __shared__ __align__(16) unsigned char slots[];  // the chunk's rows, if VEC is 1
  __shared__ long long s_off[kMaxChunk];
  __shared__ int s_key[kMaxChunk + 2];  // with the tokens on both sides (-1: none)
  next_may_launch();
  if ((int)blockIdx.x < zero.ctas) {
    if (blockIdx.y == 0) zero_unnamed(zero);
    return;
  }
  const int block = blockIdx.x - zero.ctas;  // the chunk
  after_previous();
  const int n = __ldcg(counts + 1);  // sorted tokens
  const int e0 = block * chunk, m = min(n - e0, chunk);
  if (m <= 0) return;
  const int t = threadIdx.x;
  if (t < m + 2) {
    const int e = e0 + t - 1;
    const int2 v = e >= 0 && e < n ? __ldcg(sorted + e) : make_int2(-1, 0);
    s_key[t] = v.x;
    if (t >= 1 && t <= m) s_off[t - 1] = gl.at(v.y);
  }
  __syncthreads();
  const int tile = blockIdx.y * blockDim.x * NV, slot = slot_bytes(blockDim.x * NV, sizeof(G));
  if constexpr (VEC == 1) {
    const int columns = min((int)blockDim.x * NV, dim - tile);
#pragma unroll
    for (int b = 0; b < kMaxChunk; b += kBatch) {
      for (int k = b + t / 32; k < min(b + kBatch, m); k += blockDim.x / 32)
        copy_row(slots + k * slot, grad, 1, s_off[k] + tile, columns, t & 31, 32);
      commit_copies();
    }
  }
  if (t < 32 && blockIdx.y == 0 && s_key[m + 1] == s_key[m] && s_key[0] != s_key[m]) {
    // a row begins here and goes on: into how many chunks, each of which begins with its id
    int more = 0;
    for (;;) {
      const long long e = ((long long)block + 1 + more + t) * chunk;
      const int found = __popc(__ballot_sync(0xffffffffu, e < n && __ldcg(sorted + e).x == s_key[m]));
      more += found;
      if (found < 32) break;
    }
    if (t == 0) {
      const bool few = more <= kFewParts - 1;
      const int at = atomicAdd(counts + (few ? 0 : 2), 1);
      crossing[few ? at : (int)gridDim.x - zero.ctas - 1 - at] = make_int4(block, s_key[m], more, 0);
    }
  }
  const int c0 = (blockIdx.y * blockDim.x * NV + t) * VEC, step = blockDim.x * VEC;
  if (VEC > 1 && c0 >= dim) return;
  float acc[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[j][i] = 0.f;
  bool open = s_key[0] == s_key[1];  // the first id's tokens began in an earlier chunk
  for (int b = 0; b < m; b += kBatch) {
    Pack<G, VEC> v[kBatch][NV];
    if constexpr (VEC == 1) {
      wait_copies<kMaxChunk / kBatch - 1>(b / kBatch);
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (b + k < m) {
        const G* row = grad + s_off[b + k];
        if constexpr (VEC == 1) {
          const G* mine = (const G*)(slots + (b + k) * slot + ((uintptr_t)(row + tile) & 15)) + t;
#pragma unroll
          for (int j = 0; j < NV; ++j) v[k][j].v[0] = mine[j * step];
        } else {
#pragma unroll
          for (int j = 0; j < NV; ++j)
            if (c0 + j * step < dim) v[k][j] = load_pack<G, VEC>(row + c0 + j * step);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int e = b + k;
      if (e >= m) break;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[j][i] += to_f(v[k][j].v[i]);
      const bool more = s_key[e + 2] == s_key[e + 1];
      if (more && e + 1 < m) continue;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = c0 + j * step;
        if (c < dim) {
          if (open || more) {
            float* dst = part + ((long long)block * 2 + (open ? 0 : 1)) * dim + c;
            if (VEC > 1 && dim % 4 == 0) {
#pragma unroll
              for (int i = 0; i < VEC; i += 4) store_pack<float, 4>(dst + i, acc[j] + i);
            } else {
#pragma unroll
              for (int i = 0; i < VEC; ++i) dst[i] = acc[j][i];
            }
          } else {
            write_row<O, VEC>(dw + (long long)s_key[e + 1] * stride + c, acc[j], scale, accumulate, dw_aligned);
          }
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[j][i] = 0.f;
      }
      open = false;
    }
  }
}

// The whole gradient in one launch, for few tokens: each CTA owns `span` rows of
// the table, looks at every token's id itself, and lists the tokens of its rows
// by row and position.  A row of up to kAlone tokens is summed by one group of
// threads, the others by all groups, each over a contiguous part of the row's
// tokens.  blockDim = (threads of a group, groups).  Shared memory: per token a
// byte and two integers, and the groups' partial sums.  Bound by latency, or by
// writing the table: 64 tokens of 300 rows of 1024 fp32 columns 3.5 us, of 30522
// rows 22.1 us (125 MB, 5.7 TB/s).
constexpr int kAlone = 16;
constexpr int kMaxSpan = 32;

__host__ __device__ inline int direct_bytes(int n) { return (n + 15) / 16 * 16; }

template <typename G, typename O, int VEC, int NV>
__global__ void __launch_bounds__(512) k_rows_direct(const void* __restrict__ ids, int id64, Layout2 il, int n, int vocab,
                                                     long long padding, int* flag, const G* __restrict__ grad, Layout2 gl,
                                                     int dim, float scale, int accumulate, O* __restrict__ dw,
                                                     long long stride, int dw_aligned, int span) {
  constexpr int kBatch = VEC == 8 ? 4 : 8;
  extern __shared__ __align__(16) unsigned char mark[];  // row within the span, 255: another's token
  __shared__ int count[kMaxSpan], first[kMaxSpan + 1], warp_total[16];
  int* found = reinterpret_cast<int*>(mark + direct_bytes(n));  // position | row << 16, by position
  int* list = found + n;                                        // positions, by row and position
  float* sums = reinterpret_cast<float*>(list + n);
  const int threads = blockDim.x, groups = blockDim.y, group = threadIdx.y;
  const int all = threads * groups, t = group * threads + threadIdx.x, lane = t & 31, warp = t >> 5, warps = all >> 5;
  const int base = blockIdx.x * span, rows = min(span, vocab - base);
  after_previous();
  next_may_launch();
  if (t < kMaxSpan) count[t] = 0;
  __syncthreads();
  for (int i0 = t; i0 < n; i0 += all * 8) {
    long long id[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) id[k] = i0 + k * all < n ? load_id(ids, id64, il.at(i0 + k * all)) : padding;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (i0 + k * all >= n) break;
      const bool mine = id[k] >= base && id[k] < base + rows && id[k] != padding;
      mark[i0 + k * all] = mine ? (unsigned char)(id[k] - base) : 255;
      if (mine) atomicAdd(&count[id[k] - base], 1);
      if ((id[k] < 0 || id[k] >= vocab) && blockIdx.x == 0) *flag = 1;
    }
  }
  __syncthreads();
  // first place of each row in the list (one warp's scan)
  if (warp == 0) {
    const int c = count[lane];
    int inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    first[lane] = inc - c;
    if (lane == 31) first[32] = inc;
  }
  __syncthreads();
  const int total = first[kMaxSpan];
  if (total > 0) {
    // the tokens found, by position: each thread's share of the marks in order
    const int share = ((n + all - 1) / all + 3) / 4 * 4, b = min(n, t * share), e = min(n, b + share);
    int mine = 0;
    for (int i = b; i < e; ++i) mine += mark[i] != 255;
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) warp_total[warp] = inc;
    __syncthreads();
    int at = inc - mine;
    for (int w = 0; w < warp; ++w) at += warp_total[w];
    if (mine)
      for (int i = b; i < e; ++i)
        if (mark[i] != 255) found[at++] = i | mark[i] << 16;
    __syncthreads();
    // then by row, one warp keeping the order within each
    if (warp == 0) {
      for (int i0 = 0; i0 < total; i0 += 32) {
        const int v = i0 + lane < total ? found[i0 + lane] : -1;
        const int row = v >= 0 ? v >> 16 : kMaxSpan;
        const unsigned same = __match_any_sync(0xffffffffu, row);
        const int ahead = __popc(same & ((1u << lane) - 1));
        int start = 0;
        if (v >= 0) start = first[row];
        __syncwarp();
        if (v >= 0) {
          list[start + ahead] = v & 0xffff;
          if (ahead == 0) first[row] = start + __popc(same);  // (ends at the row's end)
        }
        __syncwarp();
      }
    }
    __syncthreads();
  }
  const int c0 = (blockIdx.y * threads * NV + threadIdx.x) * VEC, step = threads * VEC;
  float acc[NV][VEC];
  auto clear = [&]() {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[j][i] = 0.f;
  };
  // adds the tokens list[b, e) in order
  auto sum = [&](int b, int e) {
    for (int i0 = b; i0 < e; i0 += kBatch) {
      Pack<G, VEC> v[kBatch][NV];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (i0 + k >= e) continue;
        const G* src = grad + gl.at(list[i0 + k]);
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (c0 + j * step < dim) v[k][j] = load_pack<G, VEC>(src + c0 + j * step);
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (i0 + k >= e) continue;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < VEC; ++i) acc[j][i] += to_f(v[k][j].v[i]);
      }
    }
  };
  auto write = [&](int u) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (c0 + j * step < dim)
        write_row<O, VEC>(dw + (long long)(base + u) * stride + c0 + j * step, acc[j], scale, accumulate, dw_aligned);
  };
  // (first[u] is now the end of row u's tokens)
  for (int u = group; u < rows; u += groups) {
    const int m = count[u];
    if (m > kAlone || (m == 0 && accumulate)) continue;
    clear();
    sum(first[u] - m, first[u]);
    write(u);
  }
  if (total <= kAlone) return;
  for (int u = 0; u < rows; ++u) {
    const int m = count[u];
    if (m <= kAlone) continue;  // the same for the whole CTA
    const int b = first[u] - m;
    clear();
    sum(b + (int)((long long)m * group / groups), b + (int)((long long)m * (group + 1) / groups));
    if (groups > 1) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) sums[(group * NV * VEC + j * VEC + i) * threads + threadIdx.x] = acc[j][i];
      __syncthreads();
      if (group == 0) {
        for (int g = 1; g < groups; ++g)
#pragma unroll
          for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[j][i] += sums[(g * NV * VEC + j * VEC + i) * threads + threadIdx.x];
      }
    }
    if (group == 0) write(u);
  }
}

// The rows that cross a chunk's end, as listed by the chunks where they begin:
// (chunk, id, chunks that follow), those of at most kFewParts partials from the
// list's front, the others from its back.  A row's partials are added in chunk
// order, by one warp per 128 columns if they are few (all loaded at once), else
// by a CTA, whose warps take interleaved partials and whose sums are then added
// in order: the list's own order does not matter.  Bound by its chain of four
// loads: 5 us for BERT-large's 250 rows (a CTA for every chunk end that looked
// for its own rows: 14 us).
template <typename O>
__global__ void __launch_bounds__(32 * kJoinWarps) k_join_rows(int dim, float scale, int accumulate,
                                                               O* __restrict__ dw, long long stride,
                                                               const float* __restrict__ part,
                                                               const int4* __restrict__ crossing, int chunks,
                                                               const int* __restrict__ counts, int* ready) {
  __shared__ float sums[kJoinWarps][32][4];
  after_previous();
  next_may_launch();
  if (blockIdx.x == 0 && threadIdx.x == 0 && threadIdx.y == 0) *ready = 0;  // for the next call
  const int lane = threadIdx.x, warp = threadIdx.y;
  const bool vec = dim % 4 == 0;
  const int tiles = (dim + 127) / 128;
  const int few = __ldcg(counts), many = __ldcg(counts + 2);
  auto load = [&](const float* src, int c, float (&v)[4]) {
    if (vec && c < dim) {
      const float4 u = __ldcg(reinterpret_cast<const float4*>(src + c));
      v[0] = u.x;
      v[1] = u.y;
      v[2] = u.z;
      v[3] = u.w;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = c + k < dim ? __ldcg(src + c + k) : 0.f;
    }
  };
  auto write = [&](int id, int c, const float (&acc)[4]) {
    O* dst = dw + (long long)id * stride + c;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c + k < dim) {
        float v = acc[k] * scale;
        if (accumulate) v += to_f(dst[k]);
        dst[k] = from_f<O>(v);
      }
  };
  // (items x 1 KB of partials fit a GPU's memory: 32 bits count them)
  for (int i = blockIdx.x; i < many * tiles; i += gridDim.x) {
    const int4 who = __ldcg(crossing + (chunks - 1 - i / tiles));
    const int c = (i % tiles * 32 + lane) * 4;
    const float* first = part + (long long)who.x * 2 * dim;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int j = warp; j <= who.z; j += kJoinWarps) {
      float v[4];
      load(first + (j == 0 ? dim : (long long)j * 2 * dim), c, v);
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[k] += v[k];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) sums[warp][lane][k] = acc[k];
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int w = 1; w < kJoinWarps; ++w)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] += sums[w][lane][k];
      write(who.y, c, acc);
    }
    __syncthreads();
  }
  for (int i = blockIdx.x * kJoinWarps + warp; i < few * tiles; i += gridDim.x * kJoinWarps) {
    const int4 who = __ldcg(crossing + i / tiles);
    const int c = (i % tiles * 32 + lane) * 4;
    const float* first = part + (long long)who.x * 2 * dim;
    float v[kFewParts][4];
#pragma unroll
    for (int j = 0; j < kFewParts; ++j)
      if (j <= who.z) load(first + (j == 0 ? dim : (long long)j * 2 * dim), c, v[j]);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < kFewParts; ++j)
      if (j <= who.z) {
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] += v[j][k];
      }
    write(who.y, c, acc);
  }
}

template <typename F> int by_dtype(int32_t d, F&& f) {
  switch (d) {
    case PSGD_F32: return f((float*)nullptr);
    case PSGD_F16: return f((__half*)nullptr);
    default: return f((__nv_bfloat16*)nullptr);
  }
}

template <int CTAS, int ITEMS, int BITS> cudaError_t allow_sort(int device) {
  static std::atomic<unsigned long long> raised{0}, large{0};
  cudaError_t e = raise_smem(k_sort_tokens<CTAS, ITEMS, BITS>, raised, device, (int)sizeof(SortShared<CTAS, BITS>));
  const unsigned long long bit = 1ull << device;
  if (CTAS > 8 && e == cudaSuccess && !(large.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(k_sort_tokens<CTAS, ITEMS, BITS>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) large.fetch_or(bit, std::memory_order_release);
  }
  return e;
}

template <int CTAS, int ITEMS, int BITS> cudaError_t launch_sort(const SortArgs& a, int device, cudaStream_t st) {
  constexpr int bytes = (int)sizeof(SortShared<CTAS, BITS>);
  const cudaError_t e = allow_sort<CTAS, ITEMS, BITS>(device);
  return e != cudaSuccess ? e : launch_early(k_sort_tokens<CTAS, ITEMS, BITS>, CTAS, kSortThreads, bytes, CTAS, st, a);
}

// Whether a cluster of kManySortCtas of the sort's largest CTAs can run.
bool runs_many_sort_ctas(int device) {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = kManySortCtas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = kManySortCtas;
  cfg.blockDim = kSortThreads;
  cfg.dynamicSmemBytes = sizeof(SortShared<kManySortCtas, 10>);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  const bool ok = allow_sort<kManySortCtas, 8, 10>(device) == cudaSuccess &&
                  cudaOccupancyMaxActiveClusters(&clusters, k_sort_tokens<kManySortCtas, 8, 10>, &cfg) == cudaSuccess;
  if (!ok) cudaGetLastError();  // not an error: clusters of 8 do it too
  return ok && clusters > 0;
}

// Sorted tokens per CTA of the row sums: 32, or 8 to 16 where that would leave
// multiprocessors idle.
int chunk_for(long long n, int sms) {
  int c = kMaxChunk;
  while (c > 8 && n < (long long)c * sms * 2) c /= 2;
  return c;
}

// The most chunks that up to n tokens make.
long long max_chunks(long long n, int sms) {
  long long most = (n + chunk_for(n, sms) - 1) / chunk_for(n, sms);
  // fewer tokens in smaller chunks can make more of them: at the sizes where the length halves
  for (int c = kMaxChunk / 2; c >= 8; c /= 2) {
    const long long last = std::min(n, (long long)2 * c * sms * 2 - 1);  // the most tokens that get chunks of c or less
    if (last > 0) most = std::max(most, (last + c - 1) / c);
  }
  return std::max<long long>(most, 1);
}

// Whether rows at two strides all begin at multiples of `to` bytes.
bool aligned_rows(const void* p, long long s0, long long s1, int size, int to) {
  return (uintptr_t)p % to == 0 && s0 * size % to == 0 && s1 * size % to == 0;
}

// How a row is spread over threads: tiles of columns (grid.y), threads of a
// group, groups of a CTA.
constexpr int kScalarNv = 4;   // elements per thread and row of the one-launch gradient where accesses are single elements
constexpr int kLookupNv = 16;  // the same in a lookup
struct TilePlan {
  int threads, groups, tiles;
};
TilePlan plan_tile(long long dim, int vec, int nv) {
  const long long per = (long long)vec * nv;  // elements per thread
  const long long want = ((dim + per - 1) / per + 31) / 32 * 32;
  TilePlan p;
  p.threads = (int)std::min<long long>(256, want);
  p.groups = std::max(1, 256 / p.threads);
  p.tiles = (int)((dim + p.threads * per - 1) / (p.threads * per));
  return p;
}

// Rows of the table per CTA of the one-launch gradient (8 CTAs to an SM, or
// kMaxSpan rows), or 0 where the sorted one is used: every CTA looks at all ids,
// 2^18 of them together at most, and a row's tokens are not split over CTAs.  On
// 152 SMs up to 1024 tokens take it where a table has 64 to 256 rows, up to 512
// of 512 rows, 223 of 30522 and 166 of 50257.  GPU time of one launch against the sorted three, 1024 fp32
// columns: 16 tokens of a 300-row table 3.1 and 7.2 us, 512 6.8 and 9.3, 2048
// 19.1 and 13.5; 256 tokens of 3000 rows 8.9 and 10.8; 64 tokens of 30522 rows
// 22.1 and 26.3 (with 640 bf16 columns 12.6 and 14.3).
int direct_span(int n, int vocab, int sms) {
  if (n > 1024 || n > 16LL * vocab) return 0;
  const int span = (int)std::min<long long>(kMaxSpan, units(vocab, 8LL * sms));
  return units(vocab, span) * n <= (1 << 18) ? span : 0;
}

int check_ids(const char* who, const psgd_embedding* e, const void* ids, int32_t id_bits, int64_t outer, int64_t inner,
              int64_t os, int64_t is) {
  const std::string w(who);
  if (!e) return fail(PSGD_EINVAL, w + ": NULL embedding");
  if (id_bits != 32 && id_bits != 64) return fail(PSGD_EINVAL, w + ": id_bits must be 32 or 64");
  if (outer < 0 || inner < 0) return fail(PSGD_EINVAL, w + ": negative token count");
  if (outer > 0 && inner > e->max_tokens / outer)
    return fail(PSGD_EINVAL, w + ": more tokens than the embedding was created for (max_tokens)");
  if (outer * inner > 0 && !ids) return fail(PSGD_EINVAL, w + ": ids is NULL");
  if (!span_ok(outer, os) || !span_ok(inner, is)) return fail(PSGD_EINVAL, w + ": bad ids stride");
  return PSGD_OK;
}

// An (outer, inner) operand of dim-wide rows, with rows that do not overlap
// when it is written.
int check_rows(const char* who, const char* what, const void* p, int32_t dtype, int64_t outer, int64_t inner,
               int64_t dim, int64_t os, int64_t is, bool written) {
  const std::string w = std::string(who) + ": " + what;
  if (!dtype_ok(dtype)) return fail(PSGD_EINVAL, w + ": unknown dtype");
  if (outer * inner > 0 && !p) return fail(PSGD_EINVAL, w + " is NULL");
  if (!span_ok(outer, os) || !span_ok(inner, is)) return fail(PSGD_EINVAL, w + ": bad stride");
  if (!written || outer == 0 || inner == 0) return PSGD_OK;
  // rows apart: all inner ones before the next outer one, or all outer ones before the next inner one
  const bool inner_first = (inner == 1 || is >= dim) && (outer == 1 || os >= (inner - 1) * is + dim);
  const bool outer_first = (outer == 1 || os >= dim) && (inner == 1 || is >= (outer - 1) * os + dim);
  if (!inner_first && !outer_first) return fail(PSGD_EINVAL, w + ": rows overlap");
  return PSGD_OK;
}

long long extent2(int64_t outer, int64_t inner, int64_t dim, int64_t os, int64_t is, int32_t dtype) {
  return outer > 0 && inner > 0 ? ((outer - 1) * os + (inner - 1) * is + dim) * dtype_size(dtype) : 0;
}

}  // namespace
}  // namespace ops
}  // namespace psgd

using namespace psgd;
using namespace psgd::ops;

extern "C" int psgd_embedding_create(int64_t vocab, int64_t dim, int64_t max_tokens, int32_t device,
                                     psgd_embedding** out) {
  if (!out) return fail(PSGD_EINVAL, "psgd_embedding_create: out is NULL");
  *out = nullptr;
  if (vocab < 1 || vocab > 0x7ffffffe) return fail(PSGD_EINVAL, "psgd_embedding_create: vocab must be in [1, 2^31 - 2]");
  if (dim < 1 || dim > (1 << 20)) return fail(PSGD_EINVAL, "psgd_embedding_create: dim must be in [1, 2^20]");
  if (max_tokens < 0 || max_tokens > 0x7fffff00)
    return fail(PSGD_EINVAL, "psgd_embedding_create: max_tokens must be in [0, 2^31 - 256]");
  if (device < 0 || device >= 64) return fail(PSGD_EINVAL, "psgd_embedding_create: device ordinal must be in [0, 63]");
  int count = 0;
  cudaError_t e = cudaGetDeviceCount(&count);
  if (e != cudaSuccess) return cuda_fail("psgd_embedding_create: cudaGetDeviceCount", e);
  if (device >= count) return fail(PSGD_ECUDA, "psgd_embedding_create: no such device");
  psgd_embedding* h = new (std::nothrow) psgd_embedding;
  if (!h) return fail(PSGD_ENOMEM, "psgd_embedding_create: out of host memory");
  DeviceScope scope(device);
  h->device = device;
  h->vocab = vocab;
  h->dim = dim;
  h->max_tokens = max_tokens;
  e = cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, device);
  if (e == cudaSuccess) h->many_sort_ctas = runs_many_sort_ctas(device);
  const long long n = std::max<long long>(1, max_tokens);
  const long long chunks = max_chunks(n, h->sms);
  // one allocation, cut into 256-byte aligned parts
  long long bytes = 0;
  auto part = [&](long long size) {
    const long long at = bytes;
    bytes += (size + 255) / 256 * 256;
    return at;
  };
  const long long words = part(16), sorted0 = part(n * 8), sorted1 = part(n * 8), sums = part(chunks * 2 * dim * 4), crossing = part(chunks * 16), counts = part(12),
                  named = part((vocab + 15) / 16 * 16);
  if (e == cudaSuccess) e = cudaMalloc(&h->memory, (size_t)bytes);
  if (e != cudaSuccess) h->memory = nullptr;
  if (e == cudaSuccess) e = cudaMemset(h->memory, 0, 16);
  if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);  // before any stream may use the handle
  if (e != cudaSuccess) {
    const int rc = cuda_fail("psgd_embedding_create", e);
    psgd_embedding_destroy(h);
    return rc;
  }
  char* base = (char*)h->memory;
  h->bytes = (size_t)bytes;
  h->d_flag = (int*)(base + words);
  h->ready = h->d_flag + 1;
  h->sorted[0] = (int2*)(base + sorted0);
  h->sorted[1] = (int2*)(base + sorted1);
  h->part = (float*)(base + sums);
  h->crossing = (int4*)(base + crossing);
  h->counts = (int*)(base + counts);
  h->named = (unsigned char*)(base + named);
  *out = h;
  return PSGD_OK;
}

extern "C" void psgd_embedding_destroy(psgd_embedding* h) {
  if (!h) return;
  {
    DeviceScope scope(h->device);
    if (h->memory) cudaFree(h->memory);
  }
  delete h;
}

extern "C" size_t psgd_embedding_workspace_bytes(const psgd_embedding* h) { return h ? h->bytes : 0; }

extern "C" int psgd_embedding_forward(psgd_embedding* h, const void* weight, psgd_dtype weight_dtype,
                                      int64_t weight_stride, const void* ids, int32_t id_bits, int64_t outer,
                                      int64_t inner, int64_t ids_outer_stride, int64_t ids_inner_stride, float scale,
                                      void* out, psgd_dtype out_dtype, int64_t out_outer_stride,
                                      int64_t out_inner_stride, void* stream) {
  const char* who = "psgd_embedding_forward";
  int rc = check_ids(who, h, ids, id_bits, outer, inner, ids_outer_stride, ids_inner_stride);
  if (rc) return rc;
  if (!weight) return fail(PSGD_EINVAL, "psgd_embedding_forward: weight is NULL");
  if (!dtype_ok(weight_dtype)) return fail(PSGD_EINVAL, "psgd_embedding_forward: weight: unknown dtype");
  if (weight_stride < h->dim || !span_ok(h->vocab, weight_stride))
    return fail(PSGD_EINVAL, "psgd_embedding_forward: bad weight stride");
  rc = check_rows(who, "out", out, out_dtype, outer, inner, h->dim, out_outer_stride, out_inner_stride, true);
  if (rc) return rc;
  const int n = (int)(outer * inner);
  if (n == 0) return PSGD_OK;
  const long long ob = extent2(outer, inner, h->dim, out_outer_stride, out_inner_stride, out_dtype);
  if (overlap(out, ob, weight, extent(h->vocab, h->dim, weight_stride, weight_dtype)) ||
      overlap(out, ob, ids, ((outer - 1) * ids_outer_stride + (inner - 1) * ids_inner_stride + 1) * (id_bits / 8)))
    return fail(PSGD_EINVAL, "psgd_embedding_forward: out overlaps an input");
  DeviceScope scope(h->device);
  const Layout2 il(outer, inner, ids_outer_stride, ids_inner_stride), ol(outer, inner, out_outer_stride, out_inner_stride);
  const cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  by_dtype(weight_dtype, [&](auto* wt) {
    using W = std::remove_pointer_t<decltype(wt)>;
    return by_dtype(out_dtype, [&](auto* ot) {
      using O = std::remove_pointer_t<decltype(ot)>;
      constexpr int V = Vec16<W>::N;
      const int align = run_alignment(V, sizeof(O));
      const bool vec = h->dim % V == 0 && aligned_rows(weight, weight_stride, 0, sizeof(W), 16) &&
                       aligned_rows(out, out_outer_stride, out_inner_stride, sizeof(O), align);
      // rows of 64 vectors and more: four of them to a thread
      const bool wide = vec && h->dim >= 64 * V;
      const TilePlan p = plan_tile(h->dim, vec ? V : 1, wide ? 4 : vec ? 1 : kLookupNv);
      const dim3 grid((unsigned)((n + (long long)p.groups - 1) / p.groups), p.tiles);
      const dim3 block(p.threads, p.groups);
      auto kernel = wide ? k_lookup<W, O, V, 4> : vec ? k_lookup<W, O, V, 1> : k_lookup<W, O, 1, kLookupNv>;
      e = launch_early(kernel, grid, block, 0, 1, st, (const W*)weight, weight_stride, h->vocab, h->dim, ids,
                       id_bits == 64, il, n, scale, (O*)out, ol, h->d_flag);
      return 0;
    });
  });
  return e == cudaSuccess ? PSGD_OK : cuda_fail(who, e);
}

extern "C" int psgd_embedding_backward(psgd_embedding* h, const void* ids, int32_t id_bits, int64_t outer,
                                       int64_t inner, int64_t ids_outer_stride, int64_t ids_inner_stride,
                                       const void* grad, psgd_dtype grad_dtype, int64_t grad_outer_stride,
                                       int64_t grad_inner_stride, float scale, int64_t padding_idx, int32_t accumulate,
                                       void* dweight, psgd_dtype dweight_dtype, int64_t dweight_stride, void* stream) {
  const char* who = "psgd_embedding_backward";
  int rc = check_ids(who, h, ids, id_bits, outer, inner, ids_outer_stride, ids_inner_stride);
  if (rc) return rc;
  rc = check_rows(who, "grad", grad, grad_dtype, outer, inner, h->dim, grad_outer_stride, grad_inner_stride, false);
  if (rc) return rc;
  if (!dweight) return fail(PSGD_EINVAL, "psgd_embedding_backward: dweight is NULL");
  if (!dtype_ok(dweight_dtype)) return fail(PSGD_EINVAL, "psgd_embedding_backward: dweight: unknown dtype");
  if (dweight_stride < h->dim || !span_ok(h->vocab, dweight_stride))
    return fail(PSGD_EINVAL, "psgd_embedding_backward: bad dweight stride");
  if (padding_idx < -1 || padding_idx >= h->vocab)
    return fail(PSGD_EINVAL, "psgd_embedding_backward: padding_idx must be -1 or a row of the table");
  const int n = (int)(outer * inner);
  const long long wb = extent(h->vocab, h->dim, dweight_stride, dweight_dtype);
  if (n > 0 &&
      (overlap(dweight, wb, grad, extent2(outer, inner, h->dim, grad_outer_stride, grad_inner_stride, grad_dtype)) ||
       overlap(dweight, wb, ids, ((outer - 1) * ids_outer_stride + (inner - 1) * ids_inner_stride + 1) * (id_bits / 8))))
    return fail(PSGD_EINVAL, "psgd_embedding_backward: dweight overlaps an input");
  DeviceScope scope(h->device);
  const cudaStream_t st = (cudaStream_t)stream;
  const Layout2 il(outer, inner, ids_outer_stride, ids_inner_stride), gl(outer, inner, grad_outer_stride, grad_inner_stride);
  const int dim = (int)h->dim, vocab = (int)h->vocab;
  const int osize = dtype_size(dweight_dtype);
  cudaError_t e = cudaSuccess;
  if (n == 0) {
    if (!accumulate)
      e = launch_early(k_zero_table, (unsigned)std::min<long long>(units(vocab, 8), h->sms * 8), 256, 0, 1, st,
                       (char*)dweight, vocab, (long long)dim * osize, dweight_stride * osize);
  } else if (const int span = direct_span(n, vocab, h->sms)) {
    by_dtype(grad_dtype, [&](auto* gt) {
      using G = std::remove_pointer_t<decltype(gt)>;
      return by_dtype(dweight_dtype, [&](auto* ot) {
        using O = std::remove_pointer_t<decltype(ot)>;
        constexpr int V = Vec16<G>::N;
        const bool vec = dim % V == 0 && aligned_rows(grad, grad_outer_stride, grad_inner_stride, sizeof(G), 16);
        const int dw_aligned = aligned_rows(dweight, dweight_stride, 0, sizeof(O), run_alignment(V, sizeof(O)));
        const TilePlan p = plan_tile(dim, vec ? V : 1, vec ? 1 : kScalarNv);
        const int groups = std::min(8, 512 / p.threads);
        const size_t smem = direct_bytes(n) + 8 * (size_t)n + (size_t)groups * p.threads * (vec ? V : kScalarNv) * 4;
        auto kernel = vec ? k_rows_direct<G, O, V, 1> : k_rows_direct<G, O, 1, kScalarNv>;
        static std::atomic<unsigned long long> raised[2];
        e = raise_smem(kernel, raised[vec], h->device, 64 * 1024);
        if (e == cudaSuccess)
          e = launch_early(kernel, dim3((unsigned)units(vocab, span), p.tiles), dim3(p.threads, groups), smem, 1, st, ids,
                           id_bits == 64, il, n, vocab, padding_idx, h->d_flag, (const G*)grad, gl, dim, scale, accumulate,
                           (O*)dweight, dweight_stride, dw_aligned, span);
        return 0;
      });
    });
  } else {
    const bool wide = vocab > 256 && vocab <= 1024 && n <= (1 << 18);  // one pass of 10 bits; a CTA's counts fit 16
    int passes = 1;
    while (!wide && passes < 4 && ((vocab - 1) >> (8 * passes)) != 0) ++passes;
    SortArgs a{ids, id_bits == 64, il, n, vocab, padding_idx, passes, {h->sorted[0], h->sorted[1]},
               h->d_flag, h->counts, accumulate ? nullptr : h->named, h->ready};
    // A cluster of 16 where each CTA has enough to do.  GPU time of the gradient
    // with 8 and 16: 4491 tokens of 512 rows 13.9 and 15.4 us, 16384 of 600 x 64
    // bf16 18.0 and 18.9, 65536 34.2 and 33.0; of 30000 x 64 4096 18.1 and 17.6,
    // 16384 24.8 and 21.8, 65536 46.0 and 38.5.
    const bool many = h->many_sort_ctas && n > (wide ? 16384 : 8192);
    auto sort = [&](auto bits) {
      constexpr int BITS = decltype(bits)::value;
      if (n <= 2 * kSortThreads) return launch_sort<1, 2, BITS>(a, h->device, st);
      if (!many) return launch_sort<kSortCtas, 2, BITS>(a, h->device, st);
      return n <= 2 * kSortThreads * kManySortCtas ? launch_sort<kManySortCtas, 2, BITS>(a, h->device, st)
                                                   : launch_sort<kManySortCtas, 8, BITS>(a, h->device, st);
    };
    e = wide ? sort(std::integral_constant<int, 10>{}) : sort(std::integral_constant<int, 8>{});
    const int chunk = chunk_for(n, h->sms);
    const unsigned chunks = (unsigned)((n + (long long)chunk - 1) / chunk);
    const int2* sorted = h->sorted[(passes - 1) & 1];
    by_dtype(grad_dtype, [&](auto* gt) {
      using G = std::remove_pointer_t<decltype(gt)>;
      return by_dtype(dweight_dtype, [&](auto* ot) {
        using O = std::remove_pointer_t<decltype(ot)>;
        constexpr int V = Vec16<G>::N;
        const bool vec = dim % V == 0 && aligned_rows(grad, grad_outer_stride, grad_inner_stride, sizeof(G), 16);
        const int dw_aligned = aligned_rows(dweight, dweight_stride, 0, sizeof(O), run_alignment(V, sizeof(O)));
        constexpr int NV = 8 / sizeof(G);  // columns per thread, if single: a slot is about 2 KB then
        TilePlan p = plan_tile(dim, vec ? V : 1, vec ? 1 : NV);
        if (!vec) p.threads = (int)(((long long)(dim + p.tiles - 1) / p.tiles + 32 * NV - 1) / (32 * NV)) * 32;  // even tiles
        const int threads = std::max(p.threads, 64);
        const size_t smem = vec ? 0 : (size_t)chunk * slot_bytes(threads * NV, sizeof(G));
        auto kernel = vec ? k_row_sums<G, O, V, 1> : k_row_sums<G, O, 1, NV>;
        static std::atomic<unsigned long long> raised{0};
        if (e == cudaSuccess && !vec) e = raise_smem(kernel, raised, h->device, kMaxChunk * slot_bytes(256 * NV, sizeof(G)));
        // zeroing: about 64 KB or 32 rows a CTA, up to kZeroCtas CTAs of 256 threads to an SM
        ZeroArgs zero{0, (char*)dweight, (long long)dim * osize, dweight_stride * osize, vocab, h->named, h->ready};
        if (!accumulate)
          zero.ctas = (int)std::min<long long>(std::max<long long>(vocab * zero.bytes / 65536, units(vocab, 32)),
                                               (long long)h->sms * kZeroCtas * (256 / threads));
        if (e == cudaSuccess)
          e = launch_early(kernel, dim3(zero.ctas + chunks, p.tiles), threads, smem, 1, st, sorted, (const G*)grad, gl, dim, scale, accumulate, (O*)dweight,
                           dweight_stride, dw_aligned, h->part, chunk, h->crossing, h->counts, zero);
        if ((chunks > 1 || !accumulate) && e == cudaSuccess) {
          const long long items = std::max<long long>(1, chunks - 1) * ((dim + 127) / 128);
          e = launch_early(k_join_rows<O>,
                           (unsigned)std::min<long long>((items + kJoinWarps - 1) / kJoinWarps, h->sms * 4),
                           dim3(32, kJoinWarps), 0, 1, st, dim, scale, accumulate, (O*)dweight, dweight_stride, h->part,
                           h->crossing, chunks, h->counts, h->ready);
        }
        return 0;
      });
    });
    if (e != cudaSuccess) cudaMemsetAsync(h->ready, 0, 4, st);  // the kernel that does so may not have been launched
  }
  return e == cudaSuccess ? PSGD_OK : cuda_fail(who, e);
}

extern "C" int psgd_embedding_status(psgd_embedding* h, void* stream) {
  if (!h) return fail(PSGD_EINVAL, "psgd_embedding_status: NULL embedding");
  DeviceScope scope(h->device);
  const cudaStream_t st = (cudaStream_t)stream;
  int flag = 0;
  cudaError_t e = cudaMemcpyAsync(&flag, h->d_flag, 4, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaMemsetAsync(h->d_flag, 0, 4, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail("psgd_embedding_status", e);
  return flag ? PSGD_BAD_TOKEN : PSGD_OK;
}
