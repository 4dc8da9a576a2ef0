// Embedding: lookup with scaling, and the dense gradient of the table.
//
//   forward   y_i = s * W[id_i]
//   backward  dW_v = [dW_v +] s * sum over the tokens i with id_i = v of g_i
//
// The gradient sorts the tokens by id (stable, so by position within an id),
// cuts the sorted list into chunks of equal length and lets each CTA add its
// chunk's rows in order, in fp32.  A row whose tokens lie in one chunk is
// written there; a row that crosses a chunk's end leaves one fp32 partial per
// chunk, and a last kernel adds those in chunk order.  No sum depends on the
// order in which CTAs run.
#include <cooperative_groups.h>

#include <algorithm>
#include <new>

#include "psgd_ops.cuh"

namespace cg = cooperative_groups;

struct psgd_embedding {
  int device = 0;
  int sms = 0;
  long long vocab = 0, dim = 0, max_tokens = 0;
  // the sorted tokens: two (key, position) buffers the radix passes alternate between
  int* key[2] = {nullptr, nullptr};
  int* pos[2] = {nullptr, nullptr};
  float* part = nullptr;  // per chunk: the partial rows of its first and its last id
  int* d_flag = nullptr;  // an id outside [0, vocab) was seen
  int* h_flag = nullptr;  // pinned
  size_t bytes = 0;
};

namespace psgd {
namespace ops {
namespace {

constexpr int kChunk = 32;          // sorted tokens per CTA of the row sums
constexpr int kSortCtas = 8;        // CTAs of the sort's cluster
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigits = 256;        // 8 bits a radix pass

// Tokens in an (outer, inner) layout: token i = o * inner + n, at
// o * os + n * is in units of the operand's elements.
struct Layout2 {
  long long os, is;
  int inner;
  __device__ __forceinline__ long long at(int i) const {
    const int o = i / inner;
    return o * os + (i - o * inner) * is;
  }
};

__device__ __forceinline__ long long load_id(const void* ids, int id64, long long at) {
  return id64 ? __ldg((const long long*)ids + at) : (long long)__ldg((const int*)ids + at);
}

// A group of threads (blockDim = (threads of a group, groups)) takes kLookup
// tokens at a time, so that as many row loads are in flight per thread; thread
// t owns the vectors t, t + threads, ... (NV of them) of a tile of columns.
template <typename W, typename O, int VEC, int NV>
__global__ void __launch_bounds__(256) k_lookup(const W* __restrict__ weight, long long wstride, long long vocab,
                                                int dim, const void* __restrict__ ids, int id64, Layout2 il, int n,
                                                float scale, O* __restrict__ out, Layout2 ol, int* flag) {
  constexpr int T = VEC == 1 ? 2 : 4;  // tokens at a time
  const int c0 = (blockIdx.y * blockDim.x * NV + threadIdx.x) * VEC, step = blockDim.x * VEC;
  const int group = blockIdx.x * blockDim.y + threadIdx.y, groups = gridDim.x * blockDim.y;
  for (long long i0 = (long long)group * T; i0 < n; i0 += groups * T) {
    long long id[T];
    bool ok[T];
#pragma unroll
    for (int k = 0; k < T; ++k) {
      id[k] = i0 + k < n ? load_id(ids, id64, il.at((int)i0 + k)) : 0;
      ok[k] = id[k] >= 0 && id[k] < vocab;
      if (!ok[k] && threadIdx.x == 0) *flag = 1;
    }
    Pack<W, VEC> v[T][NV];
#pragma unroll
    for (int k = 0; k < T; ++k) {
      const W* src = weight + (ok[k] ? id[k] : 0) * wstride;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (c0 + j * step < dim) v[k][j] = load_pack<W, VEC>(src + c0 + j * step);
    }
#pragma unroll
    for (int k = 0; k < T; ++k) {
      if (i0 + k >= n) break;
      O* dst = out + ol.at((int)i0 + k);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (c0 + j * step >= dim) continue;
        float f[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = ok[k] ? to_f(v[k][j].v[e]) * scale : 0.f;
        store_run<O, VEC>(dst + c0 + j * step, f);
      }
    }
  }
}

struct SortArgs {
  const void* ids;
  int id64;
  Layout2 il;
  int n, vocab;
  long long padding;
  int passes;
  int *key[2], *pos[2];  // pass p writes buffer p & 1
  int* flag;
  // the table to zero beside the sort (NULL: none): a run of bytes
  void* zero;
  long long zero_bytes;
};

struct SortShared {
  int cnt[kSortWarps][kDigits];
  int quarter[4][kDigits];
  int totals[kSortCtas][kDigits];  // every CTA's digit totals, pushed by the peers
  int base[kDigits];
  int scan[kDigits / 32];
};

// Stable least-significant-digit radix sort of (key, position) by one cluster:
// key = id, or `vocab` for a token without a gradient (padding, or an id
// outside the table), which sorts behind every row.  Each warp owns a
// contiguous share of the list, so that digit counts per (CTA, warp), scanned
// in list order, give every element its place; each CTA writes its digit totals
// into its peers' shared memory.  A share of at most 32 x ITEMS elements stays
// in registers between counting and placing (ITEMS = 0: any share, read twice).
template <int ITEMS> __device__ __forceinline__ void sort_tokens(const SortArgs& a, SortShared& s) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const unsigned below = (1u << lane) - 1u;
  const int per = (int)((a.n + (long long)kSortCtas * kSortThreads - 1) / ((long long)kSortCtas * kSortThreads)) * 32;
  const long long first = ((long long)rank * kSortWarps + warp) * per;
  const int share = (int)max(0LL, min((long long)a.n - first, (long long)per));  // of this warp
  for (int p = 0; p < a.passes; ++p) {
    const int shift = 8 * p;
    const int *sk = p & 1 ? a.key[0] : a.key[1], *sp = p & 1 ? a.pos[0] : a.pos[1];
    int *dk = p & 1 ? a.key[1] : a.key[0], *dp = p & 1 ? a.pos[1] : a.pos[0];
    auto key_at = [&](long long i) -> int {
      if (p > 0) return __ldcg(sk + i);
      const long long id = load_id(a.ids, a.id64, a.il.at((int)i));
      if (id < 0 || id >= a.vocab) {
        *a.flag = 1;
        return a.vocab;
      }
      return id == a.padding ? a.vocab : (int)id;
    };
    auto count = [&](int d) {
      const unsigned same = __match_any_sync(0xffffffffu, d);
      if (d < kDigits && (same & below) == 0) s.cnt[warp][d] += __popc(same);
      __syncwarp();
    };
    auto place = [&](int d, int key, int pos) {
      const unsigned same = __match_any_sync(0xffffffffu, d);
      int at = 0;
      if (d < kDigits) {
        at = s.base[d] + s.cnt[warp][d] + __popc(same & below);
        dk[at] = key;
        dp[at] = pos;
      }
      __syncwarp();
      if (d < kDigits && (same & below) == 0) s.cnt[warp][d] += __popc(same);
      __syncwarp();
    };
    int key[ITEMS > 0 ? ITEMS : 1], pos[ITEMS > 0 ? ITEMS : 1];
    if constexpr (ITEMS > 0) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int e = i * 32 + lane;
        key[i] = e < share ? key_at(first + e) : 0;
        pos[i] = e < share ? (p > 0 ? __ldcg(sp + first + e) : (int)first + e) : 0;
      }
    }
    for (int i = t; i < kSortWarps * kDigits; i += kSortThreads) (&s.cnt[0][0])[i] = 0;
    __syncthreads();
    if constexpr (ITEMS > 0) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
        if (i * 32 < share) count(i * 32 + lane < share ? (key[i] >> shift) & (kDigits - 1) : kDigits);
    } else {
      for (int e = lane; e - lane < share; e += 32)
        count(e < share ? (key_at(first + e) >> shift) & (kDigits - 1) : kDigits);
    }
    __syncthreads();
    // exclusive counts over the warps, a quarter of them per thread
    const int d = t & (kDigits - 1), q = t / kDigits;
    {
      int sum = 0;
#pragma unroll
      for (int w = 0; w < kSortWarps / 4; ++w) {
        const int c = s.cnt[q * (kSortWarps / 4) + w][d];
        s.cnt[q * (kSortWarps / 4) + w][d] = sum;
        sum += c;
      }
      s.quarter[q][d] = sum;
    }
    __syncthreads();
    int ahead = 0, total = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = s.quarter[k][d];
      if (k < q) ahead += c;
      total += c;
    }
    if (q > 0) {
#pragma unroll
      for (int w = 0; w < kSortWarps / 4; ++w) s.cnt[q * (kSortWarps / 4) + w][d] += ahead;
    }
    // two of the peers each
#pragma unroll
    for (int k = 0; k < kSortCtas / 4; ++k) {
      const int peer = q * (kSortCtas / 4) + k;
      cluster.map_shared_rank(&s.totals[rank][0], peer)[d] = total;
    }
    cluster.sync();
    if (t < kDigits) {
      int before = 0, all = 0;
#pragma unroll
      for (int r = 0; r < kSortCtas; ++r) {
        const int c = s.totals[r][t];
        if (r < rank) before += c;
        all += c;
      }
      int inc = all;  // inclusive scan over the digits
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (lane == 31) s.scan[warp] = inc;
      s.base[t] = inc - all + before;
    }
    __syncthreads();
    if (t < kDigits) {
      int add = 0;
      for (int w = 0; w < warp; ++w) add += s.scan[w];
      s.base[t] += add;
    }
    __syncthreads();
    if constexpr (ITEMS > 0) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
        if (i * 32 < share)
          place(i * 32 + lane < share ? (key[i] >> shift) & (kDigits - 1) : kDigits, key[i], pos[i]);
    } else {
      for (int e = lane; e - lane < share; e += 32) {
        const bool in = e < share;
        const int k = in ? key_at(first + e) : 0;
        place(in ? (k >> shift) & (kDigits - 1) : kDigits, k,
              in ? (p > 0 ? __ldcg(sp + first + e) : (int)first + e) : 0);
      }
    }
    cluster.sync();  // this pass's output, for every CTA of the cluster; the totals are free again
  }
}

// The first cluster sorts the tokens; the others, if any, zero the table.
template <int ITEMS>
__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortThreads) k_sort_and_zero(SortArgs a) {
  __shared__ SortShared s;
  next_may_launch();
  if (blockIdx.x < kSortCtas) {
    cg::this_cluster().sync();  // all have started: their shared memory may be written
    sort_tokens<ITEMS>(a, s);
    return;
  }
  // 16 bytes at a time between the first and the last boundary, the ends by bytes
  const long long t = (long long)(blockIdx.x - kSortCtas) * kSortThreads + threadIdx.x;
  const long long step = (long long)(gridDim.x - kSortCtas) * kSortThreads;
  char* p = (char*)a.zero;
  const long long head = min(a.zero_bytes, (long long)((16 - ((uintptr_t)p & 15)) & 15));
  const long long vecs = (a.zero_bytes - head) / 16, tail = a.zero_bytes - head - vecs * 16;
  uint4* v = reinterpret_cast<uint4*>(p + head);
  for (long long i = t; i < vecs; i += step) v[i] = make_uint4(0, 0, 0, 0);
  if (t < head) p[t] = 0;
  if (t < tail) p[head + vecs * 16 + t] = 0;
}

// Zeroes `rows` rows of `dim` elements, `stride` apart.
template <typename O>
__global__ void __launch_bounds__(256) k_zero_rows(O* __restrict__ w, long long rows, long long dim, long long stride) {
  const O zero = from_f<O>(0.f);
  for (long long r = blockIdx.x; r < rows; r += gridDim.x)
    for (long long c = threadIdx.x; c < dim; c += blockDim.x) w[r * stride + c] = zero;
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

// The rows of one chunk of sorted tokens, for one tile of columns: thread t
// owns the vectors t, t + threads, ... (NV of them).  kBatch rows are loaded at
// a time, then added in order; a sum ends with its id's last token.
template <typename G, typename O, int VEC, int NV>
__global__ void __launch_bounds__(256) k_row_sums(const int* __restrict__ key, const int* __restrict__ pos, int n,
                                                  int vocab, const G* __restrict__ grad, Layout2 gl, int dim,
                                                  float scale, int accumulate, O* __restrict__ dw, long long stride,
                                                  int dw_aligned, float* __restrict__ part) {
  constexpr int kBatch = 8;
  __shared__ long long s_off[kChunk];
  __shared__ int s_key[kChunk + 2];  // with the tokens on both sides (-1: none)
  after_previous();
  next_may_launch();
  const int e0 = blockIdx.x * kChunk, m = min(n - e0, kChunk);
  const int t = threadIdx.x;
  if (t < kChunk + 2) {
    const int e = e0 + t - 1;
    s_key[t] = t <= m + 1 && e >= 0 && e < n ? __ldcg(key + e) : -1;
  }
  if (t < m) s_off[t] = gl.at(__ldcg(pos + e0 + t));
  __syncthreads();
  const int c0 = (blockIdx.y * blockDim.x * NV + t) * VEC, step = blockDim.x * VEC;
  if (c0 >= dim) return;
  float acc[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[j][i] = 0.f;
  bool open = s_key[0] == s_key[1];  // the first id's tokens began in an earlier chunk
  for (int b = 0; b < m; b += kBatch) {
    if (s_key[b + 1] >= vocab) return;  // only tokens without a gradient from here on
    Pack<G, VEC> v[kBatch][NV];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (b + k < m && s_key[b + k + 1] < vocab) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (c0 + j * step < dim) v[k][j] = load_pack<G, VEC>(grad + s_off[b + k] + c0 + j * step);
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int e = b + k;
      if (e >= m || s_key[e + 1] >= vocab) break;
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
            float* dst = part + ((long long)blockIdx.x * 2 + (open ? 0 : 1)) * dim + c;
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

// One past the last sorted token whose key is `k`, known to be >= lo.
__device__ __forceinline__ int upper_bound(const int* __restrict__ key, int lo, int n, int k) {
  int hi = n;
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (__ldcg(key + mid) <= k) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

constexpr int kJoinGroups = 8;

// The rows that cross a chunk's end: the chunk where such a row begins adds
// its partials in chunk order (kJoinGroups interleaved sums, then those in
// order).  blockDim = (32 lanes of 4 columns, kJoinGroups); a CTA looks at the
// chunk ends blockIdx.x, blockIdx.x + gridDim.x, ...
template <typename O>
__global__ void __launch_bounds__(32 * kJoinGroups) k_join_rows(const int* __restrict__ key, int n, int vocab, int dim,
                                                                float scale, int accumulate, O* __restrict__ dw,
                                                                long long stride, const float* __restrict__ part) {
  __shared__ float sums[kJoinGroups][32][4];
  after_previous();
  const int x = threadIdx.x, y = threadIdx.y;
  const int c = (blockIdx.y * 32 + x) * 4;
  const bool vec = dim % 4 == 0;
  for (int chunk = blockIdx.x; (chunk + 1) * (long long)kChunk < n; chunk += gridDim.x) {
    const int e0 = chunk * kChunk, e1 = e0 + kChunk;
    const int k = __ldcg(key + e1 - 1);
    const bool crosses = k < vocab && __ldcg(key + e1) == k;
    const bool began = !(e0 > 0 && __ldcg(key + e0) == k && __ldcg(key + e0 - 1) == k);
    if (!crosses || !began) continue;  // the same for the whole CTA
    const int end = upper_bound(key, e1, n, k);
    const int chunks = (end - 1) / kChunk - chunk;  // chunks after this one
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    auto take = [&](const float* src) {
      if (vec && c < dim) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
        acc[0] += v.x;
        acc[1] += v.y;
        acc[2] += v.z;
        acc[3] += v.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c + i < dim) acc[i] += __ldcg(src + i);
      }
    };
    if (y == 0) take(part + ((long long)chunk * 2 + 1) * dim + c);
#pragma unroll 4
    for (int j = 1 + y; j <= chunks; j += kJoinGroups) take(part + ((long long)chunk + j) * 2 * dim + c);
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[y][x][i] = acc[i];
    __syncthreads();
    if (y == 0) {
#pragma unroll
      for (int w = 1; w < kJoinGroups; ++w)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += sums[w][x][i];
      O* dst = dw + (long long)k * stride + c;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < dim) {
          float v = acc[i] * scale;
          if (accumulate) v += to_f(dst[i]);
          dst[i] = from_f<O>(v);
        }
    }
    __syncthreads();
  }
}

template <typename F> int by_dtype(int32_t d, F&& f) {
  switch (d) {
    case PSGD_F32: return f((float*)nullptr);
    case PSGD_F16: return f((__half*)nullptr);
    default: return f((__nv_bfloat16*)nullptr);
  }
}

// Whether rows at two strides all begin at multiples of `to` bytes.
bool aligned_rows(const void* p, long long s0, long long s1, int size, int to) {
  return (uintptr_t)p % to == 0 && s0 * size % to == 0 && s1 * size % to == 0;
}

// How a row is spread over threads: tiles of columns (grid.y), threads of a
// group, groups of a CTA.
constexpr int kScalarNv = 4;  // elements per thread and row where accesses are single elements
struct TilePlan {
  int threads, groups, tiles;
};
TilePlan plan_tile(long long dim, int vec) {
  const long long per = vec > 1 ? vec : kScalarNv;  // elements per thread
  const long long want = ((dim + per - 1) / per + 31) / 32 * 32;
  TilePlan p;
  p.threads = (int)std::min<long long>(256, want);
  p.groups = std::max(1, 128 / p.threads);
  p.tiles = (int)((dim + p.threads * per - 1) / (p.threads * per));
  return p;
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
  if (written && ((inner > 1 && is < dim) || (outer > 1 && os < (inner - 1) * is + dim)))
    return fail(PSGD_EINVAL, w + ": rows overlap");
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
  const long long n = std::max<long long>(1, max_tokens);
  const long long chunks = (n + kChunk - 1) / kChunk;
  auto alloc = [&](void** p, long long bytes) {
    if (e != cudaSuccess) return;
    e = cudaMalloc(p, (size_t)bytes);
    if (e == cudaSuccess) h->bytes += (size_t)bytes;
    else *p = nullptr;
  };
  e = cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, device);
  for (int i = 0; i < 2; ++i) {
    alloc((void**)&h->key[i], n * 4);
    alloc((void**)&h->pos[i], n * 4);
  }
  alloc((void**)&h->part, chunks * 2 * dim * 4);
  alloc((void**)&h->d_flag, 4);
  if (e == cudaSuccess) e = cudaMemset(h->d_flag, 0, 4);
  if (e == cudaSuccess) e = cudaMallocHost((void**)&h->h_flag, 4);
  if (e != cudaSuccess) {
    const int rc = cuda_fail("psgd_embedding_create", e);
    psgd_embedding_destroy(h);
    return rc;
  }
  *out = h;
  return PSGD_OK;
}

extern "C" void psgd_embedding_destroy(psgd_embedding* h) {
  if (!h) return;
  {
    DeviceScope scope(h->device);
    for (int i = 0; i < 2; ++i) {
      if (h->key[i]) cudaFree(h->key[i]);
      if (h->pos[i]) cudaFree(h->pos[i]);
    }
    if (h->part) cudaFree(h->part);
    if (h->d_flag) cudaFree(h->d_flag);
    if (h->h_flag) cudaFreeHost(h->h_flag);
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
  const Layout2 il{ids_outer_stride, ids_inner_stride, (int)inner}, ol{out_outer_stride, out_inner_stride, (int)inner};
  const cudaStream_t st = (cudaStream_t)stream;
  by_dtype(weight_dtype, [&](auto* wt) {
    using W = std::remove_pointer_t<decltype(wt)>;
    return by_dtype(out_dtype, [&](auto* ot) {
      using O = std::remove_pointer_t<decltype(ot)>;
      constexpr int V = Vec16<W>::N;
      const int align = run_alignment(V, sizeof(O));
      const bool vec = h->dim % V == 0 && aligned_rows(weight, weight_stride, 0, sizeof(W), 16) &&
                       aligned_rows(out, out_outer_stride, out_inner_stride, sizeof(O), align);
      const TilePlan p = plan_tile(h->dim, vec ? V : 1);
      const int tokens = (vec ? 4 : 2) * p.groups;
      const dim3 grid((unsigned)std::min<long long>((n + tokens - 1) / tokens, (long long)h->sms * 8), p.tiles);
      const dim3 block(p.threads, p.groups);
      if (vec)
        k_lookup<W, O, V, 1><<<grid, block, 0, st>>>((const W*)weight, weight_stride, h->vocab, (int)h->dim, ids,
                                                     id_bits == 64, il, n, scale, (O*)out, ol, h->d_flag);
      else
        k_lookup<W, O, 1, kScalarNv><<<grid, block, 0, st>>>((const W*)weight, weight_stride, h->vocab, (int)h->dim,
                                                             ids, id_bits == 64, il, n, scale, (O*)out, ol, h->d_flag);
      return 0;
    });
  });
  const cudaError_t e = cudaGetLastError();
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
  const Layout2 il{ids_outer_stride, ids_inner_stride, (int)inner}, gl{grad_outer_stride, grad_inner_stride, (int)inner};
  const int dim = (int)h->dim, vocab = (int)h->vocab;
  int passes = 1;
  while (passes < 4 && (vocab >> (8 * passes)) != 0) ++passes;
  cudaError_t e = cudaSuccess;
  // A table without gaps is zeroed beside the sort, in one launch.
  const bool beside = !accumulate && n > 0 && (dweight_stride == dim || vocab == 1);
  if (!accumulate && !beside) {
    by_dtype(dweight_dtype, [&](auto* ot) {
      using O = std::remove_pointer_t<decltype(ot)>;
      k_zero_rows<O><<<(unsigned)std::min<long long>(vocab, h->sms * 8), 256, 0, st>>>((O*)dweight, vocab, dim,
                                                                                     dweight_stride);
      return 0;
    });
    e = cudaGetLastError();
  }
  if (n > 0 && e == cudaSuccess) {
    SortArgs a{ids, id_bits == 64, il, n, vocab, padding_idx, passes, {h->key[0], h->key[1]}, {h->pos[0], h->pos[1]},
               h->d_flag, beside ? dweight : nullptr, beside ? wb : 0};
    // a cluster of zeroing CTAs per 512 KB, up to one wave of them
    const unsigned zero = beside ? (unsigned)std::min<long long>((wb + (1 << 19) - 1) >> 19, (h->sms - kSortCtas) / kSortCtas) : 0;
    const unsigned grid = kSortCtas * (1 + zero);
    if (n <= kSortCtas * kSortThreads * 2) k_sort_and_zero<2><<<grid, kSortThreads, 0, st>>>(a);
    else k_sort_and_zero<0><<<grid, kSortThreads, 0, st>>>(a);
    e = cudaGetLastError();
    const unsigned chunks = (unsigned)((n + kChunk - 1) / kChunk);
    const int *key = h->key[(passes - 1) & 1], *pos = h->pos[(passes - 1) & 1];
    cudaLaunchAttribute early = early_launch();
    cudaLaunchConfig_t cfg = {};
    cfg.stream = st;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    by_dtype(grad_dtype, [&](auto* gt) {
      using G = std::remove_pointer_t<decltype(gt)>;
      return by_dtype(dweight_dtype, [&](auto* ot) {
        using O = std::remove_pointer_t<decltype(ot)>;
        constexpr int V = Vec16<G>::N;
        const bool vec = dim % V == 0 && aligned_rows(grad, grad_outer_stride, grad_inner_stride, sizeof(G), 16);
        const int dw_aligned = aligned_rows(dweight, dweight_stride, 0, sizeof(O), run_alignment(V, sizeof(O)));
        const TilePlan p = plan_tile(dim, vec ? V : 1);
        cfg.gridDim = dim3(chunks, p.tiles);
        cfg.blockDim = dim3(std::max(p.threads, 64));
        if (e == cudaSuccess)
          e = cudaLaunchKernelEx(&cfg, vec ? k_row_sums<G, O, V, 1> : k_row_sums<G, O, 1, kScalarNv>, key, pos, n, vocab,
                                 (const G*)grad, gl, dim, scale, (int)accumulate, (O*)dweight, (long long)dweight_stride,
                                 dw_aligned, h->part);
        if (chunks > 1 && e == cudaSuccess) {
          cfg.gridDim = dim3(std::min(chunks - 1, (unsigned)h->sms), (dim + 127) / 128);
          cfg.blockDim = dim3(32, kJoinGroups);
          e = cudaLaunchKernelEx(&cfg, k_join_rows<O>, key, n, vocab, dim, scale, (int)accumulate, (O*)dweight,
                                 (long long)dweight_stride, (const float*)h->part);
        }
        return 0;
      });
    });
  }
  return e == cudaSuccess ? PSGD_OK : cuda_fail(who, e);
}

extern "C" int psgd_embedding_status(psgd_embedding* h, void* stream) {
  if (!h) return fail(PSGD_EINVAL, "psgd_embedding_status: NULL embedding");
  DeviceScope scope(h->device);
  const cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaMemcpyAsync(h->h_flag, h->d_flag, 4, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaMemsetAsync(h->d_flag, 0, 4, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail("psgd_embedding_status", e);
  return *h->h_flag ? PSGD_BAD_TOKEN : PSGD_OK;
}
