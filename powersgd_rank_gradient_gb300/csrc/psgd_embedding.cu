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

// One CTA per token: its row of W times the scale.
template <typename W, typename O, int VEC>
__global__ void __launch_bounds__(256) k_lookup(const W* __restrict__ weight, long long wstride, long long vocab,
                                                int dim, const void* __restrict__ ids, int id64, Layout2 il, int n,
                                                float scale, O* __restrict__ out, Layout2 ol, int* flag) {
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const long long id = load_id(ids, id64, il.at(i));
    const bool ok = id >= 0 && id < vocab;
    if (!ok && threadIdx.x == 0) *flag = 1;
    const W* src = weight + (ok ? id : 0) * wstride;
    O* dst = out + ol.at(i);
    for (int c = threadIdx.x * VEC; c < dim; c += blockDim.x * VEC) {
      float f[VEC];
#pragma unroll
      for (int k = 0; k < VEC; ++k) f[k] = 0.f;
      if (ok) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) f[k] = to_f(__ldg(src + c + k)) * scale;
      }
#pragma unroll
      for (int k = 0; k < VEC; ++k) dst[c + k] = from_f<O>(f[k]);
    }
  }
}

// Stable least-significant-digit radix sort of (key, position) by one cluster:
// key = id, or `vocab` for a token without a gradient (padding, or an id
// outside the table), which sorts behind every row.  Each warp owns a
// contiguous share of the list, so that digit counts per (CTA, warp), scanned
// in list order, give every element its place; the CTAs read one another's
// digit totals through distributed shared memory.
__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortThreads)
    k_sort_tokens(const void* __restrict__ ids, int id64, Layout2 il, int n, int vocab, long long padding, int passes,
                  int* keyA, int* posA, int* keyB, int* posB, int* flag) {
  __shared__ int cnt[kSortWarps][kDigits];
  __shared__ int total[kDigits];
  __shared__ int base[kDigits];
  __shared__ int scan[kDigits / 32];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const unsigned below = (1u << lane) - 1u;
  // elements per warp: a multiple of 32
  const long long per = ((n + (long long)kSortCtas * kSortThreads - 1) / ((long long)kSortCtas * kSortThreads)) * 32;
  const long long first = ((long long)rank * kSortWarps + warp) * per;
  const long long last = min((long long)n, first + per);
  int *sk = keyB, *sp = posB, *dk = keyA, *dp = posA;
  for (int p = 0; p < passes; ++p) {
    const int shift = 8 * p;
    auto key_at = [&](long long i) -> int {
      if (p > 0) return __ldcg(sk + i);
      const long long id = load_id(ids, id64, il.at((int)i));
      if (id < 0 || id >= vocab) {
        *flag = 1;
        return vocab;
      }
      return id == padding ? vocab : (int)id;
    };
    for (int i = t; i < kSortWarps * kDigits; i += kSortThreads) (&cnt[0][0])[i] = 0;
    __syncthreads();
    for (long long i0 = first; i0 < last; i0 += 32) {
      const long long i = i0 + lane;
      const int d = i < last ? (key_at(i) >> shift) & (kDigits - 1) : kDigits;
      const unsigned same = __match_any_sync(0xffffffffu, d);
      if (d < kDigits && (same & below) == 0) cnt[warp][d] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
    if (t < kDigits) {
      int run = 0;
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = cnt[w][t];
        cnt[w][t] = run;
        run += c;
      }
      total[t] = run;
    }
    cluster.sync();
    int before = 0, all = 0;
    if (t < kDigits) {
      for (int r = 0; r < kSortCtas; ++r) {
        const int c = cluster.map_shared_rank(total, r)[t];
        if (r < rank) before += c;
        all += c;
      }
      // exclusive scan of `all` over the digits
      int inc = all;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (lane == 31) scan[warp] = inc;
      base[t] = inc - all + before;
    }
    __syncthreads();
    if (t < kDigits) {
      int add = 0;
      for (int w = 0; w < warp; ++w) add += scan[w];
      base[t] += add;
    }
    __syncthreads();
    for (long long i0 = first; i0 < last; i0 += 32) {
      const long long i = i0 + lane;
      const int key = i < last ? key_at(i) : 0;
      const int ps = i < last ? (p > 0 ? __ldcg(sp + i) : (int)i) : 0;
      const int d = i < last ? (key >> shift) & (kDigits - 1) : kDigits;
      const unsigned same = __match_any_sync(0xffffffffu, d);
      if (d < kDigits) {
        const int at = base[d] + cnt[warp][d] + __popc(same & below);
        dk[at] = key;
        dp[at] = ps;
      }
      __syncwarp();
      if (d < kDigits && (same & below) == 0) cnt[warp][d] += __popc(same);
      __syncwarp();
    }
    cluster.sync();  // this pass's output, for every CTA of the cluster; its totals are free again
    int* x = sk; sk = dk; dk = x;
    x = sp; sp = dp; dp = x;
  }
}

// Zeroes `rows` rows of `dim` elements, `stride` apart.
template <typename O>
__global__ void __launch_bounds__(256) k_zero_rows(O* __restrict__ w, long long rows, long long dim, long long stride) {
  const O zero = from_f<O>(0.f);
  for (long long r = blockIdx.x; r < rows; r += gridDim.x)
    for (long long c = threadIdx.x; c < dim; c += blockDim.x) w[r * stride + c] = zero;
}

// The rows of one chunk of sorted tokens, for one tile of columns.
template <typename G, typename O>
__global__ void __launch_bounds__(256) k_row_sums(const int* __restrict__ key, const int* __restrict__ pos, int n,
                                                  int vocab, const G* __restrict__ grad, Layout2 gl, int dim,
                                                  float scale, int accumulate, O* __restrict__ dw, long long stride,
                                                  float* __restrict__ part) {
  const int e0 = blockIdx.x * kChunk, e1 = min(n, e0 + kChunk);
  const int c = blockIdx.y * blockDim.x + threadIdx.x;
  if (c >= dim) return;
  float acc = 0.f;
  bool open = e0 > 0 && key[e0 - 1] == key[e0];  // the first id's tokens began in an earlier chunk
  for (int e = e0; e < e1; ++e) {
    const int k = key[e];
    if (k >= vocab) return;
    acc += to_f(__ldg(grad + gl.at(pos[e]) + c));
    const bool more = e + 1 < n && key[e + 1] == k;
    if (more && e + 1 < e1) continue;
    if (open || more) {
      part[((long long)blockIdx.x * 2 + (open ? 0 : 1)) * dim + c] = acc;
    } else {
      O* dst = dw + (long long)k * stride + c;
      float v = acc * scale;
      if (accumulate) v += to_f(*dst);
      *dst = from_f<O>(v);
    }
    acc = 0.f;
    open = false;
  }
}

// One past the last sorted token whose key is `k`, known to be >= lo.
__device__ __forceinline__ int upper_bound(const int* __restrict__ key, int lo, int n, int k) {
  int hi = n;
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (key[mid] <= k) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// The rows that cross a chunk's end: the chunk where such a row begins adds
// its partials in chunk order (eight interleaved sums, then those in order).
template <typename O>
__global__ void __launch_bounds__(256) k_join_rows(const int* __restrict__ key, int n, int vocab, int dim, float scale,
                                                   int accumulate, O* __restrict__ dw, long long stride,
                                                   const float* __restrict__ part) {
  __shared__ float sums[8][32];
  const int e0 = blockIdx.x * kChunk, e1 = min(n, e0 + kChunk);
  if (e1 >= n) return;
  const int k = key[e1 - 1];
  if (k >= vocab || key[e1] != k) return;                       // nothing crosses this end
  if (key[e0] == k && e0 > 0 && key[e0 - 1] == k) return;       // began earlier: not this chunk's
  const int end = upper_bound(key, e1, n, k);
  const int chunks = (end - 1) / kChunk - (int)blockIdx.x;      // chunks after this one
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int c = blockIdx.y * 32 + x;
  float acc = 0.f;
  if (c < dim) {
    if (y == 0) acc = part[((long long)blockIdx.x * 2 + 1) * dim + c];
    for (int j = 1 + y; j <= chunks; j += 8) acc += part[((long long)blockIdx.x + j) * 2 * dim + c];
  }
  sums[y][x] = acc;
  __syncthreads();
  if (y != 0 || c >= dim) return;
  acc = sums[0][x];
#pragma unroll
  for (int w = 1; w < 8; ++w) acc += sums[w][x];
  O* dst = dw + (long long)k * stride + c;
  float v = acc * scale;
  if (accumulate) v += to_f(*dst);
  *dst = from_f<O>(v);
}

template <typename F> int by_dtype(int32_t d, F&& f) {
  switch (d) {
    case PSGD_F32: return f((float*)nullptr);
    case PSGD_F16: return f((__half*)nullptr);
    default: return f((__nv_bfloat16*)nullptr);
  }
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
      const int grid = (int)std::min<long long>(n, (long long)h->sms * 8);
      k_lookup<W, O, 1><<<grid, 256, 0, st>>>((const W*)weight, weight_stride, h->vocab, (int)h->dim, ids,
                                              id_bits == 64, il, n, scale, (O*)out, ol, h->d_flag);
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
  // pass p writes buffer p % 2
  const int last = (passes - 1) & 1;
  if (!accumulate) {
    by_dtype(dweight_dtype, [&](auto* ot) {
      using O = std::remove_pointer_t<decltype(ot)>;
      k_zero_rows<O><<<(unsigned)std::min<long long>(vocab, h->sms * 8), 256, 0, st>>>((O*)dweight, vocab, dim,
                                                                                     dweight_stride);
      return 0;
    });
  }
  if (n > 0) {
    k_sort_tokens<<<kSortCtas, kSortThreads, 0, st>>>(ids, id_bits == 64, il, n, vocab, padding_idx, passes, h->key[0],
                                                      h->pos[0], h->key[1], h->pos[1], h->d_flag);
    const unsigned chunks = (unsigned)((n + kChunk - 1) / kChunk);
    const int *key = h->key[last], *pos = h->pos[last];
    by_dtype(grad_dtype, [&](auto* gt) {
      using G = std::remove_pointer_t<decltype(gt)>;
      return by_dtype(dweight_dtype, [&](auto* ot) {
        using O = std::remove_pointer_t<decltype(ot)>;
        k_row_sums<G, O><<<dim3(chunks, (dim + 255) / 256), 256, 0, st>>>(key, pos, n, vocab, (const G*)grad, gl, dim,
                                                                         scale, accumulate, (O*)dweight,
                                                                         dweight_stride, h->part);
        if (chunks > 1)
          k_join_rows<O><<<dim3(chunks, (dim + 31) / 32), 256, 0, st>>>(key, n, vocab, dim, scale, accumulate,
                                                                       (O*)dweight, dweight_stride, h->part);
        return 0;
      });
    });
  }
  const cudaError_t e = cudaGetLastError();
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
