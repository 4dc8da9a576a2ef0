// Softmax cross entropy of a linear output layer without its logits.
//
//   z = h W^T (tokens x vocabulary),  lse_t = log sum_v exp z_tv,  loss_t = w_t (lse_t - z_t,target)
//   G_tv = scale w_t (exp(z_tv - lse_t) - [v = target_t]),  dh = G W,  dW = [dW +] G^T h
//
// The logits are made tile by tile on the tensor cores and used where they are
// made (psgd_gemm.cu): the forward pass leaves the largest logit and the sum of
// exponentials of every tile's columns of a row, the backward pass makes them again
// and leaves G, rounded to 16 bits, for a piece of the vocabulary at a time; both
// gradients are products of that piece.  Those pieces are bounded, as are those of a
// weight that is copied; what grows with tokens x vocabulary are eight bytes for every 128 logits.
//
// Tokens that count (a target in the vocabulary, a weight that is not 0) are moved
// together first, so that padding costs nothing, and what its rows hold touches
// nothing.  A weight is split, w_t = s r_t 2^e_t with s the largest one's significand and 1 <= |r_t| < 2:
// G's rows are rounded with r_t (and 2^14 for f16, whose smallest step is 6e-8),
// dh's rows are multiplied by the power of two at the end, and h's rows by
// 2^(e_t - max e) for dW, which is exact where the weights are of one size.  So G
// is rounded once, at its own size, in either type.
#include <limits.h>

#include <algorithm>
#include <atomic>
#include <new>
#include <type_traits>

#include "psgd_mma.cuh"

struct psgd_linear_ce {
  int device = 0, pairs = 0;
  long long vocab = 0, dim = 0, most = 0;
  long long dp = 0;          // row stride of h, W and dh in the workspace
  long long cap = 0;         // rows of the workspace: max_tokens up to a multiple of 64
  long long piece = 0;       // columns of the vocabulary that G holds, a multiple of 256
  long long gp = 0;          // row stride of G
  void *h = nullptr, *hs = nullptr;  // the tokens that count, and them times 2^(e - max e)
  long long copied = 0;      // rows that w holds, a multiple of 256 and at most `piece`
  void* w = nullptr;         // a piece of a weight that TMA cannot read in place
  void* g = nullptr;
  float* dh = nullptr;       // cap x dp
  float* slots = nullptr;
  float2* part = nullptr;    // cap for every tile's columns
  float *lse = nullptr, *factor = nullptr, *at_target = nullptr;
  int *row = nullptr, *target = nullptr, *exponent = nullptr;  // of the tokens that count
  int* place = nullptr;      // of a token among them, or -1
  int* count = nullptr;      // [0]: tokens that count, [1]: largest exponent, [2]: error, [3]: CTAs that are done
  float* scale = nullptr;    // [0]: dW's, [1]: a row of dh's without its power of two
  size_t bytes = 0;
};

namespace psgd {
namespace ops {
namespace {

constexpr long long kMostTokens = 1 << 20, kMostVocab = 1 << 24;
// Of G.  (Every piece is three products with ends of their own: 2458 tokens' gradients over 30522 x 1024 with all of G, 157 MB,
// 394 us, in halves 521, in quarters 685.)
constexpr long long kPieceBytes = 256LL << 20;
// Of a weight that TMA cannot read in place.  Rows of whole 16-byte units seldom need it, and a handle for one token should
// not hold a table; others mostly do (50257 x 1601 in pieces of 32 MB: 8 tokens' losses 166 us, 128 whole, 2458 tokens'
// gradients 1445 and 1075).
constexpr long long kCopyBytes = 32LL << 20, kOddCopyBytes = 256LL << 20;
constexpr int kF16Shift = 14;  // G's values are at most 2 in size: 2^15 with it

struct Tokens {
  const void* targets;
  int bits;
  const float* weights;  // may be NULL
  int tokens;
  long long vocab;
};
__device__ __forceinline__ long long target_of(const Tokens& t, int i) {
  return t.bits == 64 ? __ldg((const long long*)t.targets + i) : (long long)__ldg((const int*)t.targets + i);
}
__device__ __forceinline__ float weight_of(const Tokens& t, int i) { return t.weights ? __ldg(t.weights + i) : 1.f; }
// Which tokens count, in their order, and their weights: w = r 2^e s with s the largest weight's significand, so that
// weights that are all the same have r = 1 and lose nothing to a rounding.  One CTA, eight tokens a thread at a time.
constexpr int kPlanItems = 8;
struct Items {  // eight tokens' targets (-1 for a token that does not count) and weights
  int target[kPlanItems];
  float weight[kPlanItems];
  __device__ __forceinline__ Items(const Tokens& t, int first) {
    long long y[kPlanItems];
#pragma unroll
    for (int k = 0; k < kPlanItems; ++k) {
      const bool in = first + k < t.tokens;
      y[k] = in ? target_of(t, first + k) : -1;
      weight[k] = in ? weight_of(t, first + k) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kPlanItems; ++k) target[k] = y[k] >= 0 && y[k] < t.vocab && weight[k] != 0.f ? (int)y[k] : -1;
  }
};
__global__ void __launch_bounds__(1024) k_plan(Tokens t, int* place, int* row, int* target, float* factor, int* exponent, int* count,
                                               float* scale, float grad_scale, int shift) {
  __shared__ int sums[32];
  __shared__ float most[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kTurn = 1024 * kPlanItems;
  after_previous();
  next_may_launch();
  // the largest weight
  Items mine(t, (int)threadIdx.x * kPlanItems);
  float top = 0.f;
  const auto look = [&](const Items& x) {
#pragma unroll
    for (int k = 0; k < kPlanItems; ++k)
      if (x.target[k] >= 0 && isfinite(x.weight[k])) top = fmaxf(top, fabsf(x.weight[k]));
  };
  look(mine);
  if (t.weights)
    for (int base = kTurn; base < t.tokens; base += kTurn) look(Items(t, base + (int)threadIdx.x * kPlanItems));
  top = warp_max(top);
  if (lane == 0) most[warp] = top;
  __syncthreads();
  top = warp_max(most[lane]);
  if (top == 0.f) top = 1.f;  // no token counts, or none whose weight is finite
  const int e_top = ilogbf(top);
  const float s = scalbnf(top, -e_top);
  int before = 0;
  for (int base = 0; base < t.tokens; base += kTurn) {
    const int first = base + (int)threadIdx.x * kPlanItems;
    if (base) mine = Items(t, first);
    int n = 0;
#pragma unroll
    for (int k = 0; k < kPlanItems; ++k) n += mine.target[k] >= 0;
    const int own = n;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int up = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) n += up;
    }
    if (lane == 31) sums[warp] = n;
    __syncthreads();
    int all = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int up = __shfl_up_sync(0xffffffffu, all, o);
      if (lane >= o) all += up;
    }
    int at = before + n - own + (warp ? __shfl_sync(0xffffffffu, all, warp - 1) : 0);
    before += __shfl_sync(0xffffffffu, all, 31);
#pragma unroll
    for (int k = 0; k < kPlanItems; ++k) {
      if (first + k >= t.tokens) break;
      const bool in = mine.target[k] >= 0;
      place[first + k] = in ? at : -1;
      if (!in) continue;
      const float w = mine.weight[k];
      int e = 0;
      float r = w;
      if (w == top) {  // (the usual case: all weights are the same)
        e = e_top;
        r = 1.f;
      } else if (isfinite(w)) {
        e = ilogbf(w);
        r = scalbnf(w, -e) / s;
        if (fabsf(r) < 1.f) {
          r *= 2.f;
          --e;
        }
      }
      row[at] = first + k;
      target[at] = mine.target[k];
      factor[at] = scalbnf(r, shift);
      exponent[at] = e;
      ++at;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    count[0] = before;
    count[1] = e_top;
    scale[0] = scalbnf(grad_scale * s, e_top - shift);
    scale[1] = grad_scale * s;
  }
}

// A warp's product of two rows of 16-bit elements, of any alignment, in the order of k_losses_few.
template <typename T> __device__ __forceinline__ float warp_dot(const T* a, const T* b, int dim, bool vec) {
  const int lane = threadIdx.x & 31;
  F2 s = f2(0.f, 0.f);
#pragma unroll 4
  for (int c = lane * 8; c < dim; c += 256) {
    F2 x[4], y[4];
    if (vec) {
      to_pairs<T>(*reinterpret_cast<const uint4*>(a + c), x);
      to_pairs<T>(*reinterpret_cast<const uint4*>(b + c), y);
    } else {  // in the same order
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int u = c + 2 * i, v = u + 1;
        x[i] = f2(u < dim ? to_f(a[u]) : 0.f, v < dim ? to_f(a[v]) : 0.f);
        y[i] = f2(u < dim ? to_f(b[u]) : 0.f, v < dim ? to_f(b[v]) : 0.f);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s = fma(x[i], y[i], s);
  }
  float u, v;
  split(s, u, v);
  return warp_sum(u + v);
}

// The rows of the tokens that count, side by side, and their targets' logits, which are summed here, in rounded fp32:
// where a target is likely, its logit is by far the largest, the loss and 1 - p are the small rest, and the tensor cores'
// drift on a large sum (1e-5 of it at 1600 elements of one sign) would be more than it is.  Both passes sum it in one
// order, so that z - lse, of which 1 - p is made, has lost no more than lse's own rounding.  Backward: exp(z - lse) - 1 of it,
// and the rows times 2^(e - max e), then rows of zeros up to a whole step of the sum over tokens, and the tokens' lse.
template <typename T> struct Gather {
  const T* src;
  long long stride;
  int dim;
  const int *row, *target, *exponent, *count;
  T *h, *hs;  // hs: backward
  long long dp;
  const float* lse_of;
  float* lse;
  const T* weight;
  long long weight_stride;
  int vec_dot;
  float* at_target;  // forward: the target's logit, backward: exp(it - lse) - 1
};
// Four warps copy a row while the fifth sums its target's logit.
constexpr int kGatherThreads = 160;
template <typename T, int V> __global__ void __launch_bounds__(kGatherThreads) k_gather(Gather<T> a) {
  after_previous();
  next_may_launch();
  const int n = a.count[0], thread = threadIdx.x;
  if (thread >= 128) {
    for (int r = blockIdx.x; r < n; r += gridDim.x) {
      const float z = warp_dot(a.src + (long long)a.row[r] * a.stride, a.weight + a.target[r] * a.weight_stride, a.dim, a.vec_dot);
      if (thread == 128) a.at_target[r] = a.hs ? expm1f(z - a.lse_of[a.row[r]]) : z;
    }
    return;
  }
  const int end = a.hs ? (n + mma::kStep - 1) / mma::kStep * mma::kStep : n;
  for (int r = blockIdx.x; r < end; r += gridDim.x) {
    const bool in = r < n;
    const T* from = a.src + (in ? (long long)a.row[r] * a.stride : 0);
    const float f = in && a.hs ? scalbnf(1.f, max(a.exponent[r] - a.count[1], -200)) : 1.f;
    if (a.lse && in && thread == 0) a.lse[r] = a.lse_of[a.row[r]];
    for (int c = thread * V; c < a.dim; c += 128 * V) {
      if constexpr (V == 1) {
        const T x = in ? from[c] : from_f<T>(0.f);
        a.h[r * a.dp + c] = x;
        if (a.hs) a.hs[r * a.dp + c] = from_f<T>(to_f(x) * f);
      } else {
        const uint4 x = in ? *reinterpret_cast<const uint4*>(from + c) : make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(a.h + r * a.dp + c) = x;
        if (a.hs) {
          F2 p[V / 2];
          float v[V];
          to_pairs<T>(x, p);
#pragma unroll
          for (int i = 0; i < V / 2; ++i) split(p[i], v[2 * i], v[2 * i + 1]);
#pragma unroll
          for (int i = 0; i < V; ++i) v[i] *= f;
          store_pack<T, V>(a.hs + r * a.dp + c, v);
        }
      }
    }
  }
}

// Two entries of largest logit and sum of exponentials as one.  (An entry without a logit above -infinity has a sum of 0,
// or NaN, which stays.)
__device__ __forceinline__ float2 merge(float2 a, float2 b) {
  const float now = fmaxf(a.x, b.x);
  return make_float2(now, a.y * (a.x == -INFINITY ? 0.f : __expf(a.x - now)) + b.y * (b.x == -INFINITY ? 0.f : __expf(b.x - now)));
}
// (loss without its weight, lse) from the others' entry and the target's logit.
__device__ __forceinline__ float2 loss_of(float2 others, float z) {
  if (z >= others.x) {  // of a target that is nearly certain the loss is what the others add
    const float rest = z == INFINITY ? NAN : log1pf(others.y * __expf(others.x - z));
    return make_float2(rest, z + rest);
  }
  const float r = logf(others.y + __expf(z - others.x));
  return make_float2((others.x - z) + r, others.x + r);
}

// The forward pass of at most N tokens, in one launch and without the tensor cores: a tile's 256 rows would be idle, and
// what comes before and after a product would take half as long as it does.  A warp reads whole rows of the weight, four
// at a time (one token over 50257 x 1600 bf16: 35 us from call to call, 4.6 TB/s), and keeps its own largest logit and sum of exponentials for
// each token; the CTA that is done last adds the CTAs' entries up, always in the same order.
constexpr int kFewDim = 8192;
constexpr long long kFewTable = 1 << 25;  // elements, for more than two tokens
template <typename T, int N>
__global__ void __launch_bounds__(256, N == 1 ? 4 : 2) k_losses_few(Tokens t, const T* hidden, long long hidden_stride, const T* weight, long long stride,
                                                                    int dim, float2* part, float* at_target, int* done, float* losses, float* lses) {
  extern __shared__ __align__(16) uint4 tokens[];  // N rows of dim / 8
  __shared__ float2 all[8][N];
  __shared__ int last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, units8 = dim / 8, vocab = (int)t.vocab;
  after_previous();
  next_may_launch();
  int own[N];  // the target of a token that counts, else -1
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const long long y = i < t.tokens ? target_of(t, i) : -1;
    own[i] = y >= 0 && y < t.vocab && weight_of(t, i) != 0.f ? (int)y : -1;
    for (int c = threadIdx.x; c < dim; c += 256)
      reinterpret_cast<T*>(tokens)[i * dim + c] = own[i] >= 0 ? hidden[i * hidden_stride + c] : from_f<T>(0.f);
  }
  float2 mine[N];
#pragma unroll
  for (int i = 0; i < N; ++i) mine[i] = make_float2(-INFINITY, 0.f);
  __syncthreads();
  for (int row = (blockIdx.x * 8 + warp) * 4; row < vocab; row += gridDim.x * 32) {
    F2 acc[N][4];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[i][r] = f2(0.f, 0.f);
    const T* from[4];  // (rows behind the last: the last again)
#pragma unroll
    for (int r = 0; r < 4; ++r) from[r] = weight + min(row + r, vocab - 1) * stride;
#pragma unroll 2
    for (int u = lane; u < units8; u += 32) {
      uint4 raw[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) raw[r] = __ldg(reinterpret_cast<const uint4*>(from[r]) + u);
      F2 x[N][4];
#pragma unroll
      for (int i = 0; i < N; ++i) to_pairs<T>(tokens[i * units8 + u], x[i]);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        F2 w[4];
        to_pairs<T>(raw[r], w);
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[i][r] = fma(w[k], x[i][k], acc[i][r]);
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float z[4], most = -INFINITY;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float u, v;
        split(acc[i][r], u, v);
        z[r] = warp_sum(u + v);
        if (row + r == own[i]) {
          if (lane == 0) __stcg(at_target + i, z[r]);
          z[r] = -INFINITY;
        }
        if (row + r >= vocab) z[r] = -INFINITY;
        most = fmaxf(most, z[r]);
      }
      const float from0 = most == -INFINITY ? 0.f : most;
      mine[i] = merge(mine[i], make_float2(most, (__expf(z[0] - from0) + __expf(z[1] - from0)) + (__expf(z[2] - from0) + __expf(z[3] - from0))));
    }
  }
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) all[warp][i] = mine[i];
  __syncthreads();
  if (threadIdx.x < N) {
    float2 x = all[0][threadIdx.x];
    for (int w = 1; w < 8; ++w) x = merge(x, all[w][threadIdx.x]);
    __stcg(part + (long long)blockIdx.x * N + threadIdx.x, x);
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(done, 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float2 x = make_float2(-INFINITY, 0.f);
    for (int p = threadIdx.x; p < (int)gridDim.x; p += 256) x = merge(x, __ldcg(part + (long long)p * N + i));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float2 y = make_float2(__shfl_down_sync(0xffffffffu, x.x, o), __shfl_down_sync(0xffffffffu, x.y, o));
      x = merge(x, y);
    }
    if (lane == 0) all[warp][i] = x;
  }
  __syncthreads();
  const int i = threadIdx.x;
  if (i == 0) *done = 0;
  if (i >= t.tokens || i >= N) return;
  const long long y = target_of(t, i);
  float2 r = make_float2(0.f, 0.f);
  if (y >= 0 && y < t.vocab && weight_of(t, i) != 0.f) {
    float2 x = all[0][i];
    for (int w = 1; w < 8; ++w) x = merge(x, all[w][i]);
    r = loss_of(x, __ldcg(at_target + i));
    r.x *= weight_of(t, i);
  }
  losses[i] = r.x;
  lses[i] = r.y;
}

// Losses and log-sum-exps of 32 tokens a CTA from the tiles, whose order the warps share, and the targets' logits.
__global__ void __launch_bounds__(1024) k_losses(Tokens t, const int* place, const float2* part, long long part_rows, int parts,
                                                 const float* at_target, float* losses, float* lses) {
  __shared__ float2 all[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
  after_previous();
  next_may_launch();
  const int at = i < t.tokens ? place[i] : -1;
  float2 mine = make_float2(-INFINITY, 0.f);
  if (at >= 0)
    for (int p = warp; p < parts; p += 32 * 8) {  // eight reads under way
      float2 x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = p + 32 * k < parts ? __ldcg(part + (p + 32 * k) * part_rows + at) : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int k = 0; k < 8; ++k) mine = merge(mine, x[k]);
    }
  all[warp][lane] = mine;
  __syncthreads();
  if (warp || i >= t.tokens) return;
  float2 r = make_float2(0.f, 0.f);
  if (at >= 0) {
    for (int w = 1; w < 32; ++w) mine = merge(mine, all[w][lane]);
    r = loss_of(mine, at_target[at]);
    r.x *= weight_of(t, i);
  }
  losses[i] = r.x;
  lses[i] = r.y;
}

// dh of every token: its row of the sums times its power of two, 0 for a token that does not count.
template <typename T, int V>
__global__ void __launch_bounds__(128) k_dhidden(const float* sums, long long dp, const int* place, const int* exponent, int tokens, int dim,
                                                 const float* scale, int shift, T* dh, long long stride) {
  after_previous();
  next_may_launch();
  for (int i = blockIdx.x; i < tokens; i += gridDim.x) {
    const int at = place[i];
    const float f = at >= 0 ? scalbnf(scale[1], exponent[at] - shift) : 0.f;
    for (int c = threadIdx.x * V; c < dim; c += 128 * V) {
      float v[V];
      if constexpr (V == 1) {
        v[0] = at >= 0 ? sums[at * dp + c] * f : 0.f;
      } else {
#pragma unroll
        for (int k = 0; k < V; k += 4) {
          const float4 x = at >= 0 ? *reinterpret_cast<const float4*>(sums + at * dp + c + k) : make_float4(0.f, 0.f, 0.f, 0.f);
          v[k] = x.x * f, v[k + 1] = x.y * f, v[k + 2] = x.z * f, v[k + 3] = x.w * f;
        }
      }
      store_pack<T, V>(dh + i * stride + c, v);
    }
  }
}

int check_call(const std::string& who, const psgd_linear_ce* h, const void* hidden, int32_t dtype, int64_t hidden_stride, int64_t tokens,
               const void* weight, int64_t weight_stride, const void* targets, int32_t bits) {
  if (!h) return fail(PSGD_EINVAL, who + ": NULL handle");
  if (dtype != PSGD_F16 && dtype != PSGD_BF16) return fail(PSGD_EINVAL, who + ": hidden and weight must be float16 or bfloat16");
  if (bits != 32 && bits != 64) return fail(PSGD_EINVAL, who + ": target_bits must be 32 or 64");
  if (tokens < 0 || tokens > h->most) return fail(PSGD_EINVAL, who + ": tokens must be in [0, max_tokens]");
  if (tokens > 0 && (!hidden || !targets)) return fail(PSGD_EINVAL, who + ": NULL operand");
  if (!weight) return fail(PSGD_EINVAL, who + ": weight is NULL");
  if (!span_ok(tokens, hidden_stride) || !span_ok(h->vocab, weight_stride)) return fail(PSGD_EINVAL, who + ": bad row stride");
  return PSGD_OK;
}

// The steps that both passes share.
struct Call {
  psgd_linear_ce* h;
  const void* hidden;
  long long hidden_stride;
  const void* weight;
  long long weight_stride;
  bool bf16, in_place;  // in_place: TMA reads the weight where it is
  Tokens t;
  cudaStream_t st;
  cudaError_t e = cudaSuccess;

  Call(psgd_linear_ce* h_, const void* hidden_, int dtype, long long hs, const void* weight_, long long ws, const void* targets, int bits,
       const float* weights, long long tokens, void* stream)
      : h(h_), hidden(hidden_), hidden_stride(hs), weight(weight_), weight_stride(ws), bf16(dtype == PSGD_BF16),
        in_place(mma::in_place(weight_, ws, h_->dim)), t{targets, bits, weights, (int)tokens, h_->vocab},
        st((cudaStream_t)stream) {}

  // The tokens that count, side by side.
  void gather(bool backward, const float* lse, float grad_scale) {
    const int shift = bf16 ? 0 : kF16Shift;
    const bool vec = h->dim % 8 == 0 && aligned16(hidden) && hidden_stride % 8 == 0;
    e = launch_early(k_plan, 1, 1024, 0, 1, st, t, h->place, h->row, h->target, h->factor, h->exponent, h->count, h->scale, grad_scale, shift);
    if (e != cudaSuccess) return;
    const auto go = [&](auto* tt, auto v) {
      using T = std::remove_pointer_t<decltype(tt)>;
      constexpr int V = decltype(v)::value;
      const Gather<T> a{(const T*)hidden, hidden_stride, (int)h->dim, h->row, h->target, h->exponent, h->count, (T*)h->h,
                        backward ? (T*)h->hs : nullptr, h->dp, lse, backward ? h->lse : nullptr, (const T*)weight, weight_stride,
                        vec && in_place, h->at_target};
      e = launch_early(k_gather<T, V>, (unsigned)std::min(t.tokens + mma::kStep, 4096), kGatherThreads, 0, 1, st, a);
    };
    using One = std::integral_constant<int, 1>;
    using Eight = std::integral_constant<int, 8>;
    if (bf16) vec ? go((__nv_bfloat16*)nullptr, Eight()) : go((__nv_bfloat16*)nullptr, One());
    else vec ? go((__half*)nullptr, Eight()) : go((__half*)nullptr, One());
  }
  // The rows [v0, v0 + n) of the weight as an operand, either way around.
  void weight_map(mma::Epilogue kind, mma::Product& z, CUtensorMap* m_rows, long long v0, long long n) {
    if (e != cudaSuccess) return;
    const void* p = weight;
    long long rows = h->vocab, stride = weight_stride;
    z.b_y0 = (int)v0;
    if (!in_place) {
      e = mma::align_rows((const char*)weight + v0 * weight_stride * 2, weight_stride, n, h->dim, h->w, h->dp, st);
      p = h->w;
      rows = n;
      stride = h->dp;
      z.b_y0 = 0;
    }
    z.bn = mma::logits_columns(kind, t.tokens, n, h->pairs);
    if (e == cudaSuccess) e = mma::make_map(&z.b, p, rows, h->dim, stride, z.bn / 2, bf16);
    if (e == cudaSuccess && m_rows) e = mma::make_map(m_rows, p, rows, h->dim, stride, mma::box_rows(true), bf16);
  }
  // What a product over the logits is told: rows are tokens, columns [v0, v0 + n) of the vocabulary.
  mma::Product logits(long long v0, long long n) {
    mma::Product p{};
    p.m = t.tokens, p.n = (int)n, p.k = (int)h->dim;
    p.live = h->count, p.live_is = 1;
    p.bf16 = bf16, p.m_fast = 1, p.error = h->count + 2;
    p.column0 = (int)v0, p.vocab = (int)h->vocab;
    p.target = h->target;
    // a logit of one sign loses 1e-7 of itself for every 16 elements of a row (see chunk_of): rows of 2048 1.3e-5, as library
    // products with sums on the tensor cores do, longer ones 6e-6 and no more.  (For 1600 elements it would cost 4 %: the
    // losses of 8192 tokens of GPT-2-XL 774 -> 805 us.)
    p.chunk = h->dim > 2048 ? 16 : 0;
    if (e == cudaSuccess) e = mma::make_map(&p.a, h->h, h->cap, h->dim, h->dp, mma::box_rows(false), bf16);
    if (e == cudaSuccess) e = mma::make_map(&p.a_few, h->h, h->cap, h->dim, h->dp, mma::kFew, bf16);
    return p;
  }
};

}  // namespace
}  // namespace ops
}  // namespace psgd

using namespace psgd;
using namespace psgd::ops;

extern "C" int psgd_linear_ce_create(int64_t vocab, int64_t dim, int64_t max_tokens, int32_t device, psgd_linear_ce** out) {
  const std::string who = "psgd_linear_ce_create";
  if (!out) return fail(PSGD_EINVAL, who + ": out is NULL");
  *out = nullptr;
  if (vocab < 1 || vocab > kMostVocab) return fail(PSGD_EINVAL, who + ": vocab must be in [1, 2^24]");
  if (dim < 1 || dim > (1 << 20)) return fail(PSGD_EINVAL, who + ": dim must be in [1, 2^20]");
  if (max_tokens < 0 || max_tokens > kMostTokens) return fail(PSGD_EINVAL, who + ": max_tokens must be in [0, 2^20]");
  if (device < 0 || device >= 64) return fail(PSGD_EINVAL, who + ": device ordinal must be in [0, 63]");
  int n = 0;
  cudaError_t e = cudaGetDeviceCount(&n);
  if (e != cudaSuccess) return cuda_fail("psgd_linear_ce_create: cudaGetDeviceCount", e);
  if (device >= n) return fail(PSGD_ECUDA, who + ": no such device");
  psgd_linear_ce* h = new (std::nothrow) psgd_linear_ce;
  if (!h) return fail(PSGD_ENOMEM, who + ": out of host memory");
  DeviceScope scope(device);
  h->device = device;
  h->vocab = vocab;
  h->dim = dim;
  h->most = max_tokens;
  h->dp = mma::row_stride(dim);
  h->cap = std::max(1LL, units(max_tokens, mma::kStep)) * mma::kStep;
  // equal pieces of whole tiles
  const auto pieces_of = [](long long columns, long long fit) {
    const long long tiles = units(columns, mma::kTile);
    return units(tiles, units(tiles, std::max(1LL, fit))) * mma::kTile;
  };
  h->piece = pieces_of(vocab, kPieceBytes / (h->cap * mma::kTile * 2));
  h->gp = mma::row_stride(h->piece);
  h->copied = pieces_of(h->piece, (dim % 8 ? kOddCopyBytes : kCopyBytes) / (mma::kTile * h->dp * 2));
  e = mma::pairs_of(device, &h->pairs);
  const auto get = [&](auto** p, long long bytes) {
    if (e == cudaSuccess) e = cudaMalloc((void**)p, bytes);
    if (e == cudaSuccess) h->bytes += bytes;
    else *p = nullptr;
  };
  get(&h->h, h->cap * h->dp * 2);
  get(&h->hs, h->cap * h->dp * 2);
  get(&h->w, h->copied * h->dp * 2);
  get(&h->g, h->cap * h->gp * 2);
  get(&h->dh, h->cap * h->dp * 4);
  get(&h->slots, 2 * h->pairs * mma::kSlotFloats * 4);
  get(&h->part, (units(vocab, mma::kTile / 2) + units(vocab, h->copied)) * h->cap * 8);  // (tiles have 128 columns at least)
  for (float** p : {&h->lse, &h->factor, &h->at_target}) get(p, h->cap * 4);
  for (int** p : {&h->row, &h->target, &h->exponent, &h->place}) get(p, h->cap * 4);
  get(&h->count, 16);
  get(&h->scale, 8);
  if (e == cudaSuccess) e = cudaMemset(h->count, 0, 16);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    const int rc = cuda_fail(who.c_str(), e);
    psgd_linear_ce_destroy(h);
    return rc;
  }
  *out = h;
  return PSGD_OK;
}

extern "C" void psgd_linear_ce_destroy(psgd_linear_ce* h) {
  if (!h) return;
  {
    DeviceScope scope(h->device);
    for (void* p : {h->h, h->hs, h->w, h->g, (void*)h->dh, (void*)h->slots, (void*)h->part, (void*)h->at_target, (void*)h->lse,
                    (void*)h->factor, (void*)h->row, (void*)h->target, (void*)h->exponent, (void*)h->place, (void*)h->count,
                    (void*)h->scale})
      cudaFree(p);
  }
  delete h;
}

extern "C" size_t psgd_linear_ce_workspace_bytes(const psgd_linear_ce* h) { return h ? h->bytes : 0; }

extern "C" int psgd_linear_ce_status(psgd_linear_ce* h, void* stream) {
  if (!h) return fail(PSGD_EINVAL, "psgd_linear_ce_status: NULL handle");
  return mma::take_error("psgd_linear_ce_status", h->count + 2, h->device, stream);
}

extern "C" int psgd_linear_ce_forward(psgd_linear_ce* h, const void* hidden, psgd_dtype dtype, int64_t hidden_stride, int64_t tokens,
                                      const void* weight, int64_t weight_stride, const void* targets, int32_t target_bits,
                                      const float* weights, float* losses, float* lse, void* stream) {
  const std::string who = "psgd_linear_ce_forward";
  const int rc = check_call(who, h, hidden, dtype, hidden_stride, tokens, weight, weight_stride, targets, target_bits);
  if (rc) return rc;
  if (tokens > 0 && (!losses || !lse)) return fail(PSGD_EINVAL, who + ": losses or lse is NULL");
  const long long sb = tokens * 4;
  for (float* o : {losses, lse})
    if (overlap(o, sb, hidden, extent(tokens, h->dim, hidden_stride, dtype)) ||
        overlap(o, sb, weight, extent(h->vocab, h->dim, weight_stride, dtype)) || overlap(o, sb, targets, tokens * target_bits / 8) ||
        overlap(o, sb, weights, sb))
      return fail(PSGD_EINVAL, who + ": an output overlaps an input");
  if (overlap(losses, sb, lse, sb)) return fail(PSGD_EINVAL, who + ": the outputs overlap");
  if (tokens == 0) return PSGD_OK;
  DeviceScope scope(h->device);
  Call c(h, hidden, dtype, hidden_stride, weight, weight_stride, targets, target_bits, weights, tokens, stream);
  // Few tokens: one launch in place of a product's four.  Over 50257 x 1600 bf16 one token 35 us (47 by products), two 39 (47), three and
  // four 53 and 55 (47); over 30522 x 1024 19 (29), 19 (29), 27 and 28 (29); over 5000 x 256 7 (15), 8 (15), 12 and 13 (15): with
  // three or four tokens a row's arithmetic takes longer than its bytes, and only small tables gain.
  if (tokens <= (h->vocab * h->dim <= kFewTable ? 4 : 2) && c.in_place && h->dim % 8 == 0 && h->dim <= kFewDim) {
    const unsigned grid = (unsigned)std::min<long long>(units(h->vocab, mma::kTile / 2), h->pairs * 2 * (tokens == 1 ? 4 : 2));
    const auto go = [&](auto* tt, auto count) {
      using T = std::remove_pointer_t<decltype(tt)>;
      constexpr int N = decltype(count)::value;
      static std::atomic<unsigned long long> raised{0};
      c.e = raise_smem(k_losses_few<T, N>, raised, h->device, N * kFewDim * 2);
      if (c.e == cudaSuccess)
        c.e = launch_early(k_losses_few<T, N>, grid, 256, (size_t)N * h->dim * 2, 1, c.st, c.t, (const T*)hidden, hidden_stride, (const T*)weight,
                           weight_stride, (int)h->dim, h->part, h->at_target, h->count + 3, losses, lse);
    };
    const auto by_count = [&](auto* tt) {
      if (tokens == 1) go(tt, std::integral_constant<int, 1>());
      else if (tokens == 2) go(tt, std::integral_constant<int, 2>());
      else go(tt, std::integral_constant<int, 4>());
    };
    if (c.bf16) by_count((__nv_bfloat16*)nullptr);
    else by_count((__half*)nullptr);
    return c.e == cudaSuccess ? PSGD_OK : cuda_fail(who.c_str(), c.e);
  }
  c.gather(false, nullptr, 1.f);
  const long long step = c.in_place ? h->vocab : h->copied;
  int parts = 0;
  for (long long v0 = 0; v0 < h->vocab && c.e == cudaSuccess; v0 += step) {
    const long long n = std::min(step, h->vocab - v0);
    mma::Product p = c.logits(v0, n);
    c.weight_map(mma::kLse, p, nullptr, v0, n);
    p.part = h->part + parts * h->cap, p.part_rows = h->cap;
    parts += (int)units(n, p.bn);
    if (c.e == cudaSuccess) c.e = mma::enqueue(mma::kLse, p, h->device, h->pairs, c.st);
  }
  if (c.e == cudaSuccess)
    c.e = launch_early(k_losses, (unsigned)units(tokens, 32), 1024, 0, 1, c.st, c.t, h->place, h->part, h->cap, parts, h->at_target, losses, lse);
  return c.e == cudaSuccess ? PSGD_OK : cuda_fail(who.c_str(), c.e);
}

extern "C" int psgd_linear_ce_backward(psgd_linear_ce* h, const void* hidden, psgd_dtype dtype, int64_t hidden_stride, int64_t tokens,
                                       const void* weight, int64_t weight_stride, const void* targets, int32_t target_bits,
                                       const float* lse, const float* weights, float grad_scale, void* dhidden,
                                       int64_t dhidden_stride, void* dweight, psgd_dtype dweight_dtype, int64_t dweight_stride,
                                       int32_t accumulate, void* stream) {
  const std::string who = "psgd_linear_ce_backward";
  const int rc = check_call(who, h, hidden, dtype, hidden_stride, tokens, weight, weight_stride, targets, target_bits);
  if (rc) return rc;
  if (!dtype_ok(dweight_dtype)) return fail(PSGD_EINVAL, who + ": unknown dtype");
  if (tokens > 0 && !lse) return fail(PSGD_EINVAL, who + ": lse is NULL");
  if (dhidden && (!span_ok(tokens, dhidden_stride) || (tokens > 1 && dhidden_stride < h->dim)))
    return fail(PSGD_EINVAL, who + ": dhidden: bad row stride, or rows overlap");
  if (dweight && (!span_ok(h->vocab, dweight_stride) || (h->vocab > 1 && dweight_stride < h->dim)))
    return fail(PSGD_EINVAL, who + ": dweight: bad row stride, or rows overlap");
  const long long hb = dhidden ? extent(tokens, h->dim, dhidden_stride, dtype) : 0;
  const long long wb = dweight ? extent(h->vocab, h->dim, dweight_stride, dweight_dtype) : 0;
  const std::pair<const void*, long long> outs[] = {{dhidden, hb}, {dweight, wb}};
  for (const auto& o : outs)
    if (overlap(o.first, o.second, hidden, extent(tokens, h->dim, hidden_stride, dtype)) ||
        overlap(o.first, o.second, weight, extent(h->vocab, h->dim, weight_stride, dtype)) ||
        overlap(o.first, o.second, targets, tokens * target_bits / 8) || overlap(o.first, o.second, weights, tokens * 4) ||
        overlap(o.first, o.second, lse, tokens * 4))
      return fail(PSGD_EINVAL, who + ": an output overlaps an input");
  if (overlap(dhidden, hb, dweight, wb)) return fail(PSGD_EINVAL, who + ": the outputs overlap");
  if (!dhidden && !dweight) return PSGD_OK;
  DeviceScope scope(h->device);
  Call c(h, hidden, dtype, hidden_stride, weight, weight_stride, targets, target_bits, weights, tokens, stream);
  const int shift = c.bf16 ? 0 : kF16Shift;
  c.gather(true, lse, grad_scale);
  const long long step = c.in_place ? h->piece : h->copied;
  for (long long v0 = 0; v0 < h->vocab && c.e == cudaSuccess; v0 += step) {
    const long long n = std::min(step, h->vocab - v0);
    mma::Product z = c.logits(v0, n), dh{}, dw{};
    c.weight_map(mma::kGrad, z, &dh.b, v0, n);
    z.lse = h->lse, z.factor = h->factor, z.at_target = h->at_target;
    if (c.e == cudaSuccess) c.e = mma::make_map(&z.store, h->g, h->cap, h->piece, h->gp, 32, c.bf16);
    if (c.e == cudaSuccess && tokens > 0) c.e = mma::enqueue(mma::kGrad, z, h->device, h->pairs, c.st);
    if (dhidden && tokens > 0) {
      if (c.e == cudaSuccess) c.e = mma::make_map(&dh.a, h->g, h->cap, h->piece, h->gp, mma::box_rows(false), c.bf16);
      if (c.e == cudaSuccess) c.e = mma::make_map(&dh.a_few, h->g, h->cap, h->piece, h->gp, mma::kFew, c.bf16);
      dh.m = (int)tokens, dh.n = (int)h->dim, dh.k = (int)n;
      dh.live = h->count, dh.live_is = 1;
      dh.b_m_rows = 1, dh.b_y0 = z.b_y0;
      dh.bf16 = c.bf16, dh.error = h->count + 2;
      dh.out = h->dh, dh.ldo = h->dp, dh.dtype = PSGD_F32, dh.accumulate = v0 > 0;
      dh.slots = h->slots;
      dh.chunk = mma::chunk_of(n, dtype);  // (dhidden's type: the workspace is rounded to it)
      if (c.e == cudaSuccess) c.e = mma::enqueue(mma::kOut, dh, h->device, h->pairs, c.st);
    }
    if (dweight) {
      if (c.e == cudaSuccess) c.e = mma::make_map(&dw.a, h->g, h->cap, h->piece, h->gp, mma::box_rows(true), c.bf16);
      if (c.e == cudaSuccess) c.e = mma::make_map(&dw.b, h->hs, h->cap, h->dim, h->dp, mma::box_rows(true), c.bf16);
      dw.m = (int)n, dw.n = (int)h->dim, dw.k = (int)tokens;
      dw.live = h->count, dw.live_is = 2;
      dw.a_m_rows = dw.b_m_rows = 1;
      dw.bf16 = c.bf16, dw.error = h->count + 2;
      dw.out = (char*)dweight + v0 * dweight_stride * dtype_size(dweight_dtype), dw.ldo = dweight_stride;
      dw.dtype = dweight_dtype, dw.accumulate = accumulate != 0, dw.scale = h->scale;
      dw.slots = h->slots;
      dw.chunk = mma::chunk_of(tokens, dweight_dtype);
      if (c.e == cudaSuccess) c.e = mma::enqueue(mma::kOut, dw, h->device, h->pairs, c.st);
    }
  }
  if (c.e == cudaSuccess && dhidden && tokens > 0) {
    const unsigned grid = (unsigned)std::min<long long>(tokens, 8192);
    const auto go = [&](auto* tt) {
      using T = std::remove_pointer_t<decltype(tt)>;
      const bool vec = h->dim % 8 == 0 && aligned16(dhidden) && dhidden_stride % 8 == 0;
      c.e = launch_early(vec ? k_dhidden<T, 8> : k_dhidden<T, 1>, grid, 128, 0, 1, c.st, h->dh, h->dp, h->place, h->exponent, (int)tokens, (int)h->dim, h->scale, shift,
                         (T*)dhidden, dhidden_stride);
    };
    if (c.bf16) go((__nv_bfloat16*)nullptr);
    else go((__half*)nullptr);
  }
  return c.e == cudaSuccess ? PSGD_OK : cuda_fail(who.c_str(), c.e);
}
