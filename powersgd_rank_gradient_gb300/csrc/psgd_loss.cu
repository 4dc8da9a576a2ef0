// Softmax cross entropy of a linear output layer without its logits.
//
//   z = h W^T (tokens x vocabulary),  lse_t = log sum_v exp z_tv,  loss_t = w_t (lse_t - z_t,target)
//   G_tv = scale w_t (exp(z_tv - lse_t) - [v = target_t]),  dh = G W,  dW = [dW +] G^T h
//
// The logits are made tile by tile on the tensor cores and used where they are
// made (psgd_gemm.cu): the forward pass leaves the largest logit and the sum of
// exponentials of every 128 columns of a row, the backward pass makes them again
// and leaves G, rounded to 16 bits, for a piece of the vocabulary at a time; both
// gradients are products of that piece.  No memory grows with tokens x vocabulary
// but those pieces, which are bounded.
//
// Tokens that count (a target in the vocabulary, a weight that is not 0) are moved
// together first, so that padding costs nothing, and what its rows hold touches
// nothing.  A weight is split into its exponent and the rest, w_t = r_t 2^e_t:
// G's rows are rounded with r_t (and 2^14 for f16, whose smallest step is 6e-8),
// dh's rows are multiplied by the power of two at the end, and h's rows by
// 2^(e_t - max e) for dW, which is exact where the weights are of one size.  So G
// is rounded once, at its own size, in either type.
#include <limits.h>

#include <algorithm>
#include <new>
#include <type_traits>

#include "psgd_mma.cuh"

struct psgd_linear_ce {
  int device = 0, pairs = 0;
  long long vocab = 0, dim = 0, most = 0;
  long long dp = 0;          // row stride of h and W in the workspace: dim up to a multiple of 8
  long long cap = 0;         // rows of the workspace: max_tokens up to a multiple of 256
  long long piece = 0;       // columns of the vocabulary that G holds, a multiple of 256
  void *h = nullptr, *hs = nullptr;  // the tokens that count, and them times 2^(e - max e)
  void* w = nullptr;         // a piece of a weight that TMA cannot read in place
  void* g = nullptr;
  float* dh = nullptr;       // cap x dp
  float* slots = nullptr;
  float2* part = nullptr;    // cap for every 128 columns
  float *at_target = nullptr, *lse = nullptr, *factor = nullptr;
  int *row = nullptr, *target = nullptr, *exponent = nullptr;  // of the tokens that count
  int* place = nullptr;      // of a token among them, or -1
  int* count = nullptr;      // [0]: tokens that count, [1]: largest exponent, [2]: error
  float* scale = nullptr;    // dW's
  size_t bytes = 0;
};

namespace psgd {
namespace ops {
namespace {

constexpr long long kMostTokens = 1 << 20, kMostVocab = 1 << 24;
constexpr long long kPieceBytes = 256LL << 20;  // of G
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
__device__ __forceinline__ bool counts(const Tokens& t, int i) {
  const long long y = target_of(t, i);
  return y >= 0 && y < t.vocab && weight_of(t, i) != 0.f;
}

// Which tokens count, in their order, and the exponents of their weights.  One CTA, 1024 tokens at a time.
__global__ void __launch_bounds__(1024) k_plan(Tokens t, int* place, int* row, int* target, float* factor, int* exponent, int* count,
                                               float* scale, float grad_scale, int shift) {
  __shared__ int sums[32], most[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  after_previous();
  next_may_launch();
  int before = 0, top = INT_MIN;
  for (int base = 0; base < t.tokens; base += 1024) {
    const int i = base + (int)threadIdx.x;
    const bool in = i < t.tokens && counts(t, i);
    const unsigned votes = __ballot_sync(0xffffffffu, in);
    if (lane == 0) sums[warp] = __popc(votes);
    __syncthreads();
    int n = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int up = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) n += up;
    }
    const int all = __shfl_sync(0xffffffffu, n, 31), mine = warp ? __shfl_sync(0xffffffffu, n, warp - 1) : 0;
    const int at = before + mine + __popc(votes & ((1u << lane) - 1));
    if (i < t.tokens) place[i] = in ? at : -1;
    if (in) {
      const float w = weight_of(t, i);
      const int e = isfinite(w) ? ilogbf(w) : 0;
      row[at] = i;
      target[at] = (int)target_of(t, i);
      factor[at] = scalbnf(w, shift - e);
      exponent[at] = e;
      top = max(top, e);
    }
    before += all;
    __syncthreads();
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) most[warp] = top;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 32; ++w) top = max(top, most[w]);
    if (before == 0) top = 0;
    count[0] = before;
    count[1] = top;
    *scale = scalbnf(grad_scale, top - shift);
  }
}

// The rows of the tokens that count, side by side, then rows of zeros up to a multiple of 256 (the products'
// tiles read those).  hs (backward): the rows times 2^(e - max e); lse: theirs.
template <typename T, int V>
__global__ void __launch_bounds__(128) k_gather(const T* src, long long stride, int dim, const int* row, const int* exponent, const int* count,
                                                T* h, T* hs, long long dp, const float* lse_of, float* lse) {
  after_previous();
  next_may_launch();
  const int n = count[0], end = (n + mma::kTile - 1) / mma::kTile * mma::kTile;
  for (int r = blockIdx.x; r < end; r += gridDim.x) {
    const bool in = r < n;
    const T* from = src + (in ? (long long)row[r] * stride : 0);
    const float f = in && hs ? scalbnf(1.f, max(exponent[r] - count[1], -200)) : 1.f;
    if (lse && in && threadIdx.x == 0) lse[r] = lse_of[row[r]];
    for (int c = threadIdx.x * V; c < dim; c += 128 * V) {
      if constexpr (V == 1) {
        const T x = in ? from[c] : from_f<T>(0.f);
        h[r * dp + c] = x;
        if (hs) hs[r * dp + c] = from_f<T>(to_f(x) * f);
      } else {
        const uint4 x = in ? *reinterpret_cast<const uint4*>(from + c) : make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(h + r * dp + c) = x;
        if (hs) {
          F2 p[V / 2];
          float v[V];
          to_pairs<T>(x, p);
#pragma unroll
          for (int i = 0; i < V / 2; ++i) split(p[i], v[2 * i], v[2 * i + 1]);
#pragma unroll
          for (int i = 0; i < V; ++i) v[i] *= f;
          store_pack<T, V>(hs + r * dp + c, v);
        }
      }
    }
  }
}

// Losses and log-sum-exps of 32 tokens a CTA from the pieces of 128 columns, whose order the warps share.
__global__ void __launch_bounds__(1024) k_losses(Tokens t, const int* place, const float2* part, long long part_rows, int parts,
                                                 const float* at_target, float* losses, float* lses) {
  __shared__ float2 all[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
  after_previous();
  next_may_launch();
  const int at = i < t.tokens ? place[i] : -1;
  float top = -INFINITY, sum = 0.f;
  const auto add = [&](float2 x) {
    const float now = fmaxf(top, x.x);
    // a piece without a logit above -infinity has a sum of 0 (or NaN, which stays)
    sum = sum * (top == -INFINITY ? 0.f : __expf(top - now)) + x.y * (x.x == -INFINITY ? 0.f : __expf(x.x - now));
    top = now;
  };
  if (at >= 0)
    for (int p = warp; p < parts; p += 32) add(__ldcg(part + p * part_rows + at));
  all[warp][lane] = make_float2(top, sum);
  __syncthreads();
  if (warp || i >= t.tokens) return;
  float loss = 0.f, lse = 0.f;
  if (at >= 0) {
    for (int w = 1; w < 32; ++w) add(all[w][lane]);
    lse = top + logf(sum);
    loss = weight_of(t, i) * (lse - at_target[at]);
  }
  losses[i] = loss;
  lses[i] = lse;
}

// dh of every token: its row of the sums times its power of two, 0 for a token that does not count.
template <typename T>
__global__ void __launch_bounds__(128) k_dhidden(const float* sums, long long dp, const int* place, const int* exponent, int tokens, int dim,
                                                 float grad_scale, int shift, T* dh, long long stride) {
  after_previous();
  next_may_launch();
  for (int i = blockIdx.x; i < tokens; i += gridDim.x) {
    const int at = place[i];
    const float f = at >= 0 ? scalbnf(grad_scale, exponent[at] - shift) : 0.f;
    for (int c = threadIdx.x; c < dim; c += 128) dh[i * stride + c] = from_f<T>(at >= 0 ? sums[at * dp + c] * f : 0.f);
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
        in_place(aligned16(weight_) && ws % 8 == 0 && ws >= h_->dim), t{targets, bits, weights, (int)tokens, h_->vocab},
        st((cudaStream_t)stream) {}

  void plan(float grad_scale) {
    e = launch_early(k_plan, 1, 1024, 0, 1, st, t, h->place, h->row, h->target, h->factor, h->exponent, h->count, h->scale, grad_scale,
                     bf16 ? 0 : kF16Shift);
  }
  void gather(bool backward, const float* lse) {
    const unsigned grid = (unsigned)std::min<long long>(units(t.tokens, mma::kTile) * mma::kTile, 4096);
    if (e != cudaSuccess || grid == 0) return;
    const bool vec = h->dim % 8 == 0 && aligned16(hidden) && hidden_stride % 8 == 0;
    void* hs = backward ? h->hs : nullptr;
    const auto go = [&](auto* tt, auto v) {
      using T = std::remove_pointer_t<decltype(tt)>;
      e = launch_early(k_gather<T, decltype(v)::value>, grid, 128, 0, 1, st, (const T*)hidden, hidden_stride, (int)h->dim, h->row, h->exponent,
                       h->count, (T*)h->h, (T*)hs, h->dp, lse, backward ? h->lse : nullptr);
    };
    using One = std::integral_constant<int, 1>;
    using Eight = std::integral_constant<int, 8>;
    if (bf16) vec ? go((__nv_bfloat16*)nullptr, Eight()) : go((__nv_bfloat16*)nullptr, One());
    else vec ? go((__half*)nullptr, Eight()) : go((__half*)nullptr, One());
  }
  // The rows [v0, v0 + n) of the weight as an operand either way around, and the first row of its map that counts.
  void weight_map(CUtensorMap* k_rows, CUtensorMap* m_rows, long long v0, long long n, int* y0) {
    if (e != cudaSuccess) return;
    const void* p = weight;
    long long rows = h->vocab, stride = weight_stride;
    *y0 = (int)v0;
    if (!in_place) {
      e = mma::align_rows((const char*)weight + v0 * weight_stride * 2, weight_stride, n, h->dim, h->w, h->dp, st);
      p = h->w;
      rows = n;
      stride = h->dp;
      *y0 = 0;
    }
    if (e == cudaSuccess) e = mma::make_map(k_rows, p, rows, h->dim, stride, mma::box_rows(false), bf16);
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
    if (e == cudaSuccess) e = mma::make_map(&p.a, h->h, h->cap, h->dim, h->dp, mma::box_rows(false), bf16);
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
  h->dp = units(dim, 8) * 8;
  h->cap = std::max(1LL, units(max_tokens, mma::kTile)) * mma::kTile;
  // equal pieces of whole tiles
  const long long tiles = units(vocab, mma::kTile), fit = std::max(1LL, kPieceBytes / (h->cap * mma::kTile * 2));
  h->piece = units(tiles, units(tiles, fit)) * mma::kTile;
  e = mma::pairs_of(device, &h->pairs);
  const auto get = [&](auto** p, long long bytes) {
    if (e == cudaSuccess) e = cudaMalloc((void**)p, bytes);
    if (e == cudaSuccess) h->bytes += bytes;
    else *p = nullptr;
  };
  get(&h->h, h->cap * h->dp * 2);
  get(&h->hs, h->cap * h->dp * 2);
  get(&h->w, h->piece * h->dp * 2);
  get(&h->g, h->cap * h->piece * 2);
  get(&h->dh, h->cap * h->dp * 4);
  get(&h->slots, 2 * h->pairs * mma::kSlotFloats * 4);
  get(&h->part, tiles * 2 * h->cap * 8);
  for (float** p : {&h->at_target, &h->lse, &h->factor}) get(p, h->cap * 4);
  for (int** p : {&h->row, &h->target, &h->exponent, &h->place}) get(p, h->cap * 4);
  get(&h->count, 16);
  get(&h->scale, 4);
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
  c.plan(1.f);
  c.gather(false, nullptr);
  const long long step = c.in_place ? h->vocab : h->piece;
  for (long long v0 = 0; v0 < h->vocab && c.e == cudaSuccess; v0 += step) {
    const long long n = std::min(step, h->vocab - v0);
    mma::Product p = c.logits(v0, n);
    c.weight_map(&p.b, nullptr, v0, n, &p.b_y0);
    p.part = h->part, p.part_rows = h->cap, p.at_target = h->at_target;
    if (c.e == cudaSuccess) c.e = mma::enqueue(mma::kLse, p, h->device, h->pairs, c.st);
  }
  if (c.e == cudaSuccess)
    c.e = launch_early(k_losses, (unsigned)units(tokens, 32), 1024, 0, 1, c.st, c.t, h->place, h->part, h->cap,
                       (int)units(h->vocab, mma::kTile) * 2, h->at_target, losses, lse);
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
  c.plan(grad_scale);
  c.gather(true, lse);
  for (long long v0 = 0; v0 < h->vocab && c.e == cudaSuccess; v0 += h->piece) {
    const long long n = std::min(h->piece, h->vocab - v0);
    mma::Product z = c.logits(v0, n), dh{}, dw{};
    c.weight_map(&z.b, &dh.b, v0, n, &z.b_y0);
    z.lse = h->lse, z.factor = h->factor;
    if (c.e == cudaSuccess) c.e = mma::make_map(&z.store, h->g, h->cap, h->piece, h->piece, 32, c.bf16);
    if (c.e == cudaSuccess && tokens > 0) c.e = mma::enqueue(mma::kGrad, z, h->device, h->pairs, c.st);
    if (dhidden && tokens > 0) {
      if (c.e == cudaSuccess) c.e = mma::make_map(&dh.a, h->g, h->cap, h->piece, h->piece, mma::box_rows(false), c.bf16);
      dh.m = (int)tokens, dh.n = (int)h->dim, dh.k = (int)n;
      dh.live = h->count, dh.live_is = 1;
      dh.b_m_rows = 1, dh.b_y0 = z.b_y0;
      dh.bf16 = c.bf16, dh.error = h->count + 2;
      dh.out = h->dh, dh.ldo = h->dp, dh.dtype = PSGD_F32, dh.accumulate = v0 > 0;
      dh.slots = h->slots;
      if (c.e == cudaSuccess) c.e = mma::enqueue(mma::kOut, dh, h->device, h->pairs, c.st);
    }
    if (dweight) {
      if (c.e == cudaSuccess) c.e = mma::make_map(&dw.a, h->g, h->cap, h->piece, h->piece, mma::box_rows(true), c.bf16);
      if (c.e == cudaSuccess) c.e = mma::make_map(&dw.b, h->hs, h->cap, h->dim, h->dp, mma::box_rows(true), c.bf16);
      dw.m = (int)n, dw.n = (int)h->dim, dw.k = (int)tokens;
      dw.live = h->count, dw.live_is = 2;
      dw.a_m_rows = dw.b_m_rows = 1;
      dw.bf16 = c.bf16, dw.error = h->count + 2;
      dw.out = (char*)dweight + v0 * dweight_stride * dtype_size(dweight_dtype), dw.ldo = dweight_stride;
      dw.dtype = dweight_dtype, dw.accumulate = accumulate != 0, dw.scale = h->scale;
      dw.slots = h->slots;
      if (c.e == cudaSuccess) c.e = mma::enqueue(mma::kOut, dw, h->device, h->pairs, c.st);
    }
  }
  if (c.e == cudaSuccess && dhidden && tokens > 0) {
    const unsigned grid = (unsigned)std::min<long long>(tokens, 8192);
    const auto go = [&](auto* tt) {
      using T = std::remove_pointer_t<decltype(tt)>;
      c.e = launch_early(k_dhidden<T>, grid, 128, 0, 1, c.st, h->dh, h->dp, h->place, h->exponent, (int)tokens, (int)h->dim, grad_scale, shift,
                         (T*)dhidden, dhidden_stride);
    };
    if (c.bf16) go((__nv_bfloat16*)nullptr);
    else go((__half*)nullptr);
  }
  return c.e == cudaSuccess ? PSGD_OK : cuda_fail(who.c_str(), c.e);
}
