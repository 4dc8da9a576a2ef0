// Building blocks of a matrix product on the fifth-generation tensor cores by a
// pair of CTAs: tensor maps (TMA), barriers with bounded waits, tcgen05 with
// cta_group::2, tensor memory.
//
// A pair computes 256 x 256 results (or fewer columns), each CTA 128 rows of them in its own tensor
// memory (256 fp32 columns, of 512: one tile is drained while the next is summed).
// Of every 64 elements of the summed dimension a CTA loads its own 128 rows of A
// and 128 of the 256 columns of B, 32 KB together: with both CTAs' shared memory
// read by one instruction, a pair moves 64 KB for 8.4 MFLOP, half of what two
// single CTAs with 128 x 256 results would.
//
// Operands lie in memory either way around.  "K rows": the summed dimension is
// contiguous (tile: 128 rows of 64 elements, one TMA box, rows of 128 bytes).  "M rows": the
// result's dimension is contiguous (tile: 64 rows of the summed dimension of 128 elements, two TMA
// boxes of 64 elements, 8 KB each).  Both with the 128-byte swizzle.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "psgd_ops.cuh"

namespace psgd {
namespace mma {

constexpr int kTile = 256;     // rows and columns of a pair's tile
constexpr int kHalf = 128;     // rows of a CTA's part
constexpr int kFew = 32;
constexpr int kStep = 64;      // elements of the summed dimension per stage
constexpr int kStages = 5;     // of whole operands; of fewer rows and columns as many as their room holds
constexpr int kMostStages = 10;
constexpr int kOperand = kHalf * kStep * 2;  // bytes of one operand's part of a stage
constexpr int kStageBytes = 2 * kOperand;
constexpr int kEpilogueWarps = 16;
constexpr int kCols = 64;      // columns of a tile that an epilogue warp takes, of 32 rows
constexpr int kThreads = 32 * (kEpilogueWarps + 2);  // the last two warps: TMA and MMA
constexpr int kStaging = 4096;                       // bytes of an epilogue warp's staging
constexpr int kSmem = 1024 + kStages * kStageBytes + kEpilogueWarps * kStaging;

// A wait gives up after so many cycles (four seconds), far beyond any normal one, and after so many tries, whatever the
// clock says.
constexpr long long kWaitCycles = 8000000000ll;
constexpr int kWaitTries = 1 << 28;

__device__ __forceinline__ uint32_t saddr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The address of the same place in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t at_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}

__device__ __forceinline__ void bar_init(uint64_t* bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(bar)), "r"(count));
}
__device__ __forceinline__ bool bar_try(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  // (it may sleep 20 us: sixteen warps that ask all the time cost the tensor cores 5 % of their clock)
  asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\nselp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok)
               : "r"(saddr(bar)), "r"(parity), "r"(20000)
               : "memory");
  return ok;
}
// Waits for the phase of `parity`; false if its time ran out, or another wait of this CTA has given up.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, volatile int* dead) {
  if (bar_try(bar, parity)) return true;
  const long long began = clock64();
  for (int i = 0; i < kWaitTries; ++i) {
    if (bar_try(bar, parity)) return true;
    if ((i & 31) == 31 && (*dead || clock64() - began > kWaitCycles)) break;
  }
  *dead = 1;
  return false;
}
// The same by all lanes of a warp: false for all where it is for one.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* dead) {
  return __all_sync(0xffffffffu, bar_wait(bar, parity, dead));
}
__device__ __forceinline__ void bar_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(bar)), "r"(bytes) : "memory");
}
// One arrival at a barrier of any CTA of the cluster.  (No more than the accumulators' emptiness goes from CTA to CTA by
// barriers, which tcgen05's fences order: waits that acquire and arrivals that release at the cluster's scope cost a
// fence each, 0.5 us and more.)
__device__ __forceinline__ void bar_arrive_at(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// A box of a tensor map at (x, y) into this CTA's shared memory, completing on a barrier of either CTA of the pair.
// x times the element size is a multiple of 16 bytes.
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void store_box(const CUtensorMap* map, int x, int y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x), "r"(y), "r"(src)
               : "memory");
}
__device__ __forceinline__ void fetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle (layout type 2), version 1, of an
// operand at address `a`.  K rows: groups of 8 rows 1024 bytes apart.  M rows: groups of 8 rows of
// the summed dimension 1024 bytes apart, the two halves of 64 elements 8 KB.
__device__ __forceinline__ uint64_t describe(uint32_t a, bool m_rows) {
  const uint64_t lead = m_rows ? (uint64_t)(8192 >> 4) : 1u;
  return (uint64_t)((a >> 4) & 0x3FFFu) | (lead << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// Bytes from one 16 elements of the summed dimension to the next.
__device__ __forceinline__ uint32_t step_bytes(bool m_rows) { return m_rows ? 2048 : 32; }

// Instruction descriptor of kind::f16: fp32 sums (bits 4-5 = 1), both operands of one
// 16-bit type (bits 7-9 and 10-12: 0 f16, 1 bf16), M rows (bit 15: A, bit 16: B), N / 8 at bit 17, M / 16 at bit 24.
__device__ __forceinline__ uint32_t instruction(bool bf16, bool a_m_rows, bool b_m_rows, int n) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((a_m_rows ? 1u : 0u) << 15) | ((b_m_rows ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
}
// D += A B over 16 elements (D = A B where acc is 0), both CTAs' shared memory and tensor memory.
__device__ __forceinline__ void multiply(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
// One arrival at the same barrier of both CTAs when everything multiplied so far is done.
__device__ __forceinline__ void commit_both(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(saddr(bar)),
               "h"((uint16_t)3)
               : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 512 columns of tensor memory, by one whole warp of each CTA of the pair.
__device__ __forceinline__ void tmem_alloc(uint32_t* slot) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(saddr(slot)) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t t) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(t));
}

// 8 columns of a warp's 32 lanes; there after tmem_wait().
__device__ __forceinline__ void tmem_load8(uint32_t t, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(t));
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// ---- products ---------------------------------------------------------------------

constexpr int kMinSplit = 8;  // steps of the summed dimension that are worth a piece of a tile of their own
constexpr long long kSlotFloats = (long long)kTile * kTile;

// What a product's kernel is told.  D[m, n] = sum_k A[m, k] B[n, k].
struct Product {
  CUtensorMap a, b;
  CUtensorMap a_few;         // A with K rows: in boxes of kFew rows, for a tile that has fewer rows than a CTA's part
  CUtensorMap store;         // GRAD: the gradients' matrix, in boxes of 64 x 32
  int m, n, k;               // extents in elements
  int bn;                    // columns of a tile but the last (see width_of)
  int stages, a_bytes, stage_bytes;  // room of a stage's A and of a stage in each CTA
  const int* live;           // device: takes the place of m (live_is 1) or k (2); or NULL
  int live_is;
  int a_m_rows, b_m_rows;    // how the operands lie
  int b_y0;                  // first row of B's map
  int bf16;
  int m_fast;                // order of the tiles: neighbours share B (else A)
  int chunk;                 // steps that the tensor cores sum by themselves, 0: all (see k_product)
  int* error;                // device: set to 1 by a wait that gave up
  // OUT: out = [out +] scale * D
  void* out;
  long long ldo;
  int dtype, accumulate;
  int vec;                   // rows of out begin at multiples of 4 elements' size
  const float* scale;        // device, or NULL: 1
  float* slots;              // partial tiles, two of kSlotFloats per pair; NULL: no tile is split
  // LSE and GRAD: rows are tokens, columns the vocabulary from column0 on
  int column0, vocab;        // columns in all
  const int* target;         // per row
  float2* part;              // LSE: largest logit but the target's and sum of exp(z - it), for every tile's columns: [part][row]
  long long part_rows;       // rows between parts
  const float* lse;          // GRAD
  const float* factor;       // GRAD: multiplies a row's gradient
  const float* at_target;    // GRAD: a row's exp(z - lse) - 1 at its target
};

// How a product's tiles go to pairs of CTAs: whole tiles in turns of one for each pair; the tiles of a last turn that
// would leave pairs idle are cut along k.  Where that occupies most pairs, each into `cuts` equal pieces, the same pieces of all
// tiles at the same time, so that they share what they read (8 tiles of 477 steps: 32.9 us in runs, 31.9 so); else into equal runs of
// the steps of all of them, one for each of `workers` pairs.
struct Schedule {
  int mt, nt, kb, tiles, whole, rest, workers, cuts;
  long long steps;  // of the tiles that are cut
};
__host__ __device__ inline Schedule schedule_of(int m, int n, int bn, int k, int pairs, bool split) {
  Schedule s;
  s.mt = (int)ops::units(m, kTile);
  s.nt = (int)ops::units(n, bn);
  s.kb = (int)ops::units(k, kStep);
  s.tiles = s.mt * s.nt;
  s.whole = s.tiles;
  s.workers = s.cuts = 0;
  s.steps = 0;
  s.rest = s.tiles % pairs;
  if (!split || s.rest == 0 || s.kb < 2 * kMinSplit) return s;
  const int most = s.kb / kMinSplit, fit = pairs / s.rest, cuts = fit < most ? fit : most;
  const long long steps = (long long)s.rest * s.kb;
  if (cuts >= 2 && (cuts == most || cuts * s.rest * 8 >= pairs * 7)) {
    s.cuts = cuts;
    s.workers = cuts * s.rest;
  } else {
    const long long workers = steps / kMinSplit < pairs ? steps / kMinSplit : pairs;
    if (workers <= s.rest) return s;
    s.workers = (int)workers;
  }
  s.whole = s.tiles - s.rest;
  s.steps = steps;
  return s;
}
// Equal runs: the first step of a worker's.  Equal pieces: of a cut's.
__host__ __device__ inline long long first_step(const Schedule& s, int worker) { return worker * s.steps / s.workers; }
__host__ __device__ inline int first_of_cut(const Schedule& s, int cut) { return (int)((long long)cut * s.kb / s.cuts); }

// Columns of tile tn of n columns: `bn`, or a multiple of 32 that holds what is left.  (A tile begins at a multiple of 64
// columns of a row, so that its boxes' rows are whole lines of 128 bytes: seven tiles of 240 for 1600 columns, 0.40 us a
// step, cost more than six of 256 and one of 64, 0.36.)
__host__ __device__ inline int width_of(int n, int bn, int tn) {
  const int left = n - tn * bn;
  return left >= bn ? bn : (left + 31) / 32 * 32;
}

// Steps of the summed dimension (of k elements) that the tensor cores sum by themselves, 0: all.  They cut sums off where
// fp32 would round them: a sum of one sign with operands of 11 bits loses 1e-7 of itself for every 16 elements (16384
// rows 1e-4; gradients of both signs with 8-bit activations 8e-6).  Taken out every 1024 elements and added in
// rounded fp32 it loses 6e-6 however long it is (7e-7).  So for fp32 results always; for results of 16 bits where a sum of one
// sign could lose an eighth of half a step of theirs (2^-12 and 2^-9) otherwise: sums that are taken out cost GPT-2-XL's
// gradients 2 % (2050 -> 2100 us) and 16384 rows' bf16 weight gradient as much (263 -> 267).
inline int chunk_of(long long k, int dtype) {
  const long long fine = dtype == PSGD_F32 ? 0 : dtype == PSGD_F16 ? 4096 : 32768;
  return k > fine ? 16 : 0;
}

enum Epilogue { kLse = 0, kGrad = 1, kOut = 2 };

// ---- host side ------------------------------------------------------------------

// A map of `rows` rows of `cols` 16-bit elements, `stride` elements apart, read or written in boxes of 64 x box_rows
// with the 128-byte swizzle; what lies outside reads as zero.  The address is a multiple of 16 bytes, stride of 8
// elements.
cudaError_t make_map(CUtensorMap* map, const void* p, long long rows, long long cols, long long stride, int box_rows, bool bf16);
// Whether a map can have rows of `cols` elements, `stride` apart, as they lie (rows that overlap, a broadcast operand's, it
// cannot, nor strides of 2^40 bytes).
inline bool in_place(const void* p, long long stride, long long cols) {
  return ops::aligned16(p) && stride % 8 == 0 && stride >= cols && stride < (1LL << 39);
}
inline int box_rows(bool m_rows) { return m_rows ? kStep : kHalf; }

// Elements from row to row of a matrix of 16-bit elements in a workspace: an odd number of lines of 128 bytes, so that
// the lines that a box of many rows reads lie in all parts of L2 (GPT-2-XL's gradients 2150 -> 2121 us, the product
// over 300 tokens of BERT-large's vocabulary 46 -> 41).
inline long long row_stride(long long cols) { return (ops::units(cols, 64) | 1) * 64; }
// Pairs of CTAs that a device holds at once.
cudaError_t pairs_of(int device, int* pairs);
// Columns of the tiles of an LSE or GRAD product over n columns; B's boxes have half as many rows.
int logits_columns(Epilogue kind, long long rows, long long n, int pairs);
// Enqueues a product, and for split tiles the sum of their parts.
cudaError_t enqueue(Epilogue kind, Product p, int device, int pairs, cudaStream_t st);
// Rows of 16-bit elements of any stride and alignment into rows `to` elements apart.
cudaError_t align_rows(const void* src, long long stride, long long rows, long long cols, void* dst, long long to, cudaStream_t st);
// Reads and clears a handle's error word; synchronises the stream.
int take_error(const char* who, int* error, int device, void* stream);

}  // namespace mma
}  // namespace psgd
