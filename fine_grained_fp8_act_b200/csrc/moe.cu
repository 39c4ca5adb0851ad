// moe.cu -- a whole mixture-of-experts layer for few tokens (sm_100a):
//
//   y[t] = sum over the token's slots j of weights[t, j] * W2[e] . h[t, j],   e = ids[t, j]
//   h    = silu(gate) * up,   gate = W13[e][:I] . x[t],   up = W13[e][I:] . x[t]
//
// x and h are quantized per token in groups of 1 x 128 as the dense layers'
// activations are (x inside the first kernel, or for many tokens an expert by
// a launch in front of it, with the same codes); gate, up, h and the down products stay in float32 until
// that quantization and until y's one rounding to bf16.
//
// With few tokens the layer is bound by reading the reached experts' e4m3
// weights once (3 H I bytes an expert), so both kernels are weight streams:
// moe_kernel<UP> computes h (codes and scales, to the workspace),
// moe_kernel<DOWN> the down products and y.  Both run one CTA per SM.
//
// Work: the routed pairs (token, slot) are grouped by expert in chunks of at
// most 32; chunk and 256-row weight tile (128 gate and the matching 128 up
// rows, or 256 rows of W2) make a unit of Kb K-blocks of 128.  All units in a
// row (tile by tile, the chunks innermost, so that an expert's second chunk
// finds the tile in L2) are dealt out in consecutive runs, one per CTA: whole
// units where that is even enough, else equal runs of K-blocks, so that every
// SM streams the same number of bytes whatever the routing is.  A unit that a
// cut divides is added up in CTA order by whichever of its CTAs finishes
// last, so the result does not depend on which one that is.
//
// Roles (512 threads):
//   warp 0      producer: per K-block, two TMA boxes of 128 x 128 weights
//   warp 1      MMA issuer: weights are the tensor core's M side (2 x 128
//               rows), the chunk's tokens its N side (16 or 32 columns)
//   warps 2-7   activations: each K-block's token rows gathered by pair into
//               the MMA's B operand (128-byte swizzle), quantized on the way
//               if x is bf16, with their scales and the tile's weight scales.
//               A ring of its own, deeper than the weights', takes their
//               latency off the stream; loads go out before a slot is free.
//   warps 8-15  epilogue: thread = weight row, four warps per box.  Each
//               K-block's partial products land in a TMEM buffer of their own
//               (8 of them, which cover the epilogue's end-of-unit work) and
//               are promoted, acc += P * (sx * sw), then finished per unit:
//               silu(gate) * up, the 128-row group's amax, scale and codes
//               (UP); the pairs' products, and by the last CTA of a row tile
//               the weighted sums over the slots (DOWN).
//
// DOWN is launched to overlap UP's end: its first weight tiles, one ring of
// them, are on their way while UP's last units finish.  Then every role waits
// for UP before its first bounded wait and before it touches the workspace: how
// long UP still takes must not count against DOWN's limit, and the partial
// sums and counters are UP's until then.
// (Having UP's producers bring DOWN's first 5, 8 or 12 K-blocks per CTA into
// L2 at their end changed nothing: 70.4 to 71.0 us against 70.4 for one token
// over 8 experts of 7168 x 2048.)
//
// Every wait is bounded; on expiry the kernel records FG8_ERR_TIMEOUT in the
// status word, drains its copies and tensor-core ops, frees TMEM and returns.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <atomic>

#include "fg8_internal.h"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace fg8 {
namespace {

using namespace qm;

constexpr uint32_t kTimeoutStatus = 6u;     // FG8_ERR_TIMEOUT
constexpr uint32_t kInvalidArgStatus = 1u;  // FG8_ERR_INVALID_ARG
constexpr uint64_t kDrainNs = 1000000000ull;

constexpr int kMaxGrid = 160;   // split-unit counters and partials are sized for this many CTAs
constexpr int kRowTile = 256;   // weight rows of a unit: two MMAs of 128
constexpr int kChunk = 32;      // tokens of a unit
constexpr int kMinRun = 2;      // K-blocks per CTA below which fewer CTAs share the work
constexpr int kSortRow = 16;    // bytes of an expert's row of per-warp counts, kSortWarps of them in use
constexpr int kSortWarps = 14;  // warps 2-15
constexpr int kFewPairs = 96;   // placed by one warp
constexpr int kMaxJobs = kMoeMaxExperts + kMoeMaxPairs / kChunk;
constexpr size_t kPartFloats = static_cast<size_t>(kRowTile) * kChunk;
static_assert(kMaxGrid + kMoeMaxHidden / kRowTile <= kHeaderCounters, "counters in the workspace header");

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// [header | h codes [P, I] | h scales float32 [P, ceil(I/128)] | partial
// sums of split units, two per CTA | down products float32 [P, H] | with
// quantize_first: x's codes and scales]
struct MoeWs {
  size_t hq, hs, split, part, xq, xs, total;
};

// Whether bf16 x is quantized by a launch of its own: every CTA that runs a
// token's expert quantizes the token again, which from some 8 tokens an
// expert on takes longer than the launch.  us, one / the other: 64 tokens,
// top-8 of 64, 7168 x 2048 463 / 461; 64, top-2 of 8, 4096 x 14336 268 / 258;
// 100, top-4 of 8, 4096 x 2048 110 / 100.
bool quantize_first(int64_t T, int64_t k, int64_t E) { return T * k >= 8 * E; }

MoeWs moe_ws_layout(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
  MoeWs w;
  const int64_t P = T * k, Ib = (I + 127) / 128;
  w.hq = kWorkspaceHeaderBytes;
  w.hs = align256(w.hq + P * I);
  w.split = align256(w.hs + P * Ib * 4);
  w.part = align256(w.split + 2 * kMaxGrid * kPartFloats * 4);
  w.xq = align256(w.part + P * H * 4);
  w.xs = align256(w.xq + (quantize_first(T, k, E) ? T * H : 0));
  w.total = align256(w.xs + (quantize_first(T, k, E) ? T * ((H + 127) / 128) * 4 : 0));
  return w;
}

struct MoeParams {
  const void* x;        // UP: bf16 [T, H] (row stride ld_x) or e4m3 codes [T, H]
  int64_t ld_x;
  const void* x_scale;  // UP on codes: [T, Hb]
  const int32_t* ids;
  const float* weights;
  const void* w_scale;  // this kernel's weight scales [E][Nb][Kb]
  int T, k, E, H, I;
  int K, Kb, Nb;        // products' length and its blocks; scale rows per expert
  int tiles;            // row tiles per expert
  uint8_t* hq;
  float* hs;
  float* split;
  float* part;
  void* y;
  int64_t ld_y;
  uint32_t* status;
  uint32_t* counters;
  uint64_t wait_limit_ns;
  int test_stall, test_late;
};

enum Phase : int { UP = 0, DOWN = 1 };

template <int PHASE_, int FMT_, bool CODES_>
struct MoeCfg {
  static constexpr int PHASE = PHASE_, FMT = FMT_;
  static constexpr bool CODES = CODES_;  // the activations come as codes and scales
  static constexpr int kStage = 2 * 128 * 128, STAGES = 5;  // weight ring
  // slot i of the activation ring, its scales and TMEM buffer i serve the
  // same K-block, and the epilogue hands all three back together
  static constexpr int kSlots = 8, kX = kChunk * 128, kSlotFloats = kChunk + 8, kAccCols = 2 * kChunk;
  static constexpr int kFillWarp0 = 2, kFillWarps = 6, kEpiWarp0 = 8, kEpiThreads = 256;
  static constexpr int kThreads = kEpiWarp0 * 32 + kEpiThreads;
  static constexpr int kOffX = STAGES * kStage;
  static constexpr int kOffSc = kOffX + kSlots * kX;
  static constexpr int kStagePairs = 16;
  static constexpr int kOffStage = kOffSc + kSlots * kSlotFloats * 4;     // [2][kStagePairs][128] float32
  static constexpr int kOffList = kOffStage + 2 * kStagePairs * 128 * 4;  // pairs by expert
  static constexpr int kOffOff = kOffList + kMoeMaxPairs * 2;             // first pair of each expert
  static constexpr int kOffJob = kOffOff + kMoeMaxExperts * 2;            // its first chunk
  static constexpr int kOffJobE = kOffJob + kMoeMaxExperts * 2;           // expert of each chunk
  static constexpr int kOffCnt = (kOffJobE + kMaxJobs * 2 + 15) / 16 * 16;  // pairs per expert
  static constexpr int kOffBar = kOffCnt + kMoeMaxExperts * 2;
  // while the pairs are sorted, before anything is staged
  static constexpr int kOffCount = kOffX, kOffIds = kOffCount + kMoeMaxExperts * 4;
  static constexpr int kOffBlock = kOffIds + kMoeMaxPairs * 2;
  static_assert(kOffBlock % 16 == 0 && kOffBlock + kMoeMaxExperts * kSortRow <= kOffSc, "sort scratch");
  static constexpr int kSmem = 1024 + kOffBar + 512;
  static_assert(kSmem <= 232448, "shared memory budget");
  static_assert(kStage % 1024 == 0 && kX % 1024 == 0, "swizzled operands start on 1024-byte boundaries");
  static_assert((2 * STAGES + 3 * kSlots + 2) * 8 + 32 <= 512, "barrier area");
  // M = 128 weight rows, K-major e4m3 operands, f32 accumulate; N is added per unit
  static_assert(kSlots * kAccCols == 512, "TMEM columns");
  // An activation warp that comes to K-block i last waited for i - kFillWarps
  // - kSlots to be consumed, which with kFillWarps <= kSlots puts i - 2 kSlots
  // behind it: the slot's barrier is at most one phase back, and the parity
  // that the warp waits for is not that of an earlier phase.  (The one MMA
  // issuer and the epilogue see every K-block.)
  static_assert(kFillWarps <= kSlots, "phases told apart by their parity");
  static_assert(kFillWarp0 == 2 && kThreads == 64 + kSortWarps * 32 && kSortWarps <= kSortRow, "warps that place the pairs");
  static constexpr uint32_t kIdesc = (1u << 4) | (uint32_t(128 >> 4) << 24);
};

template <int FMT>
__device__ __forceinline__ float scale_value(const void* s, int64_t i) {
  if (FMT == 0) return __ldg(static_cast<const float*>(s) + i);
  const uint32_t b = __ldg(static_cast<const uint8_t*>(s) + i);
  return __uint_as_float(b == 0u ? 0x00400000u : b << 23);  // 2^(b - 127)
}

// The routing as every CTA holds it: pairs sorted by expert (stable), and
// the expert of each chunk of kChunk pairs.
struct Routing {
  uint16_t *list, *cnt, *off, *job, *job_e;
  uint32_t* count;  // scratch of the sort, as ids and block
  uint16_t* ids;
  uint8_t* block;   // [expert][warp]: pairs in the 32 that the warp holds
};

// Counting sort of the P ids by expert.  Every thread counts its ids (integer
// atomics: the counts do not depend on their order), one warp makes the
// prefix sums, which is all that the weights' producer and the MMA issuer
// wait for; then warps 2-15 place the pairs, 32 each at a time: a warp match
// ranks equal ids within the 32, the counts of the warps in front add to it.
// Up to kFewPairs pairs one warp places them all before the others set out:
// it takes some 0.15 us for each 32, and less code comes first.  us, one warp
// / all: 400 pairs 99.5 / 97.3, 2048 pairs 747 / 725.
__device__ __forceinline__ void clear_counts(const MoeParams& p, const Routing& r) {
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
    r.count[e] = 0u;
    if (p.T * p.k > kFewPairs) *reinterpret_cast<uint4*>(r.block + e * kSortRow) = make_uint4(0u, 0u, 0u, 0u);
  }
}

// UP reports an expert out of range (once: DOWN has the same ids), and never
// over a timeout, after which y is unspecified as a whole.
template <int PHASE>
__device__ __forceinline__ void count_pairs(const MoeParams& p, const Routing& r) {
  const int P = p.T * p.k;
  for (int i = threadIdx.x; i < P; i += blockDim.x) {
    const int id = __ldg(p.ids + i);
    const bool on = id >= 0 && id < p.E;
    if (p.weights != nullptr) prefetch_l1(p.weights + i);  // for the sums at the end
    r.ids[i] = on ? static_cast<uint16_t>(id) : static_cast<uint16_t>(0xFFFFu);
    if (on) atomicAdd(r.count + id, 1u);
    else if (PHASE == UP && id >= 0 && blockIdx.x == 0) atomicCAS(p.status, 0u, kInvalidArgStatus);
  }
}

// One warp; returns the number of chunks.
__device__ __forceinline__ int place_experts(const MoeParams& p, const Routing& r) {
  const int lane = threadIdx.x & 31;
  const int per = (p.E + 31) / 32, e0 = lane * per, e1 = e0 + per < p.E ? e0 + per : p.E;
  int pairs = 0, jobs = 0;  // of this lane's experts
  for (int e = e0; e < e1; ++e) {
    const int c = static_cast<int>(r.count[e]);
    pairs += c;
    jobs += (c + kChunk - 1) / kChunk;
  }
  int sp = pairs, sj = jobs;  // inclusive sums over the lanes
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int a = __shfl_up_sync(0xFFFFFFFFu, sp, d), b = __shfl_up_sync(0xFFFFFFFFu, sj, d);
    if (lane >= d) sp += a, sj += b;
  }
  const int all = __shfl_sync(0xFFFFFFFFu, sj, 31);
  int at = sp - pairs, job = sj - jobs;
  for (int e = e0; e < e1; ++e) {
    const int c = static_cast<int>(r.count[e]);
    r.cnt[e] = static_cast<uint16_t>(c);
    r.off[e] = static_cast<uint16_t>(at);
    r.job[e] = static_cast<uint16_t>(job);
    r.count[e] = static_cast<uint32_t>(at);  // from here on: where the expert's next pair goes
    at += c;
    for (int n = (c + kChunk - 1) / kChunk; n > 0; --n) r.job_e[job++] = static_cast<uint16_t>(e);
  }
  return all;
}

// Sum of the first n bytes of 16.
__device__ __forceinline__ uint32_t byte_sum(const uint4& v, int n) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t s = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int left = n - 4 * i;
    const uint32_t ones = left >= 4 ? 0x01010101u : left <= 0 ? 0u : 0x01010101u >> (32 - 8 * left);
    s = __dp4a(w[i], ones, s);
  }
  return s;
}

// One warp, behind place_experts: 32 pairs at a time, lanes with equal ids
// finding each other with a warp match.
__device__ __forceinline__ void place_few(const MoeParams& p, const Routing& r) {
  const int lane = threadIdx.x & 31, P = p.T * p.k;
  __syncwarp();
#pragma unroll 1
  for (int p0 = 0; p0 < P; p0 += 32) {
    const int id = p0 + lane < P ? r.ids[p0 + lane] : 0xFFFF;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, id);
    const uint32_t below = same & ((1u << lane) - 1u);
    const uint32_t first = id != 0xFFFF ? r.count[id] : 0u;
    __syncwarp();
    if (id != 0xFFFF) {
      r.list[first + __popc(below)] = static_cast<uint16_t>(p0 + lane);
      if (below == 0u) r.count[id] = first + __popc(same);
    }
    __syncwarp();
  }
}

// Warps 2-15, behind place_experts.
__device__ __noinline__ void place_many(int P, int E, const uint16_t* ids, uint32_t* next, uint8_t* block,
                                        uint16_t* list) {
  constexpr int kThreads = kSortWarps * 32;
  const int t = static_cast<int>(threadIdx.x) - 64, warp = t >> 5, lane = t & 31;
  for (int p0 = 0;; p0 += kThreads) {
    const int pair = p0 + t;
    const int id = pair < P ? ids[pair] : 0xFFFF;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, id);
    const uint32_t below = same & ((1u << lane) - 1u);
    uint8_t* row = block + id * kSortRow;
    if (id != 0xFFFF && below == 0u) row[warp] = static_cast<uint8_t>(__popc(same));
    named_barrier_sync(2, kThreads);
    if (id != 0xFFFF)
      list[next[id] + byte_sum(*reinterpret_cast<const uint4*>(row), warp) + __popc(below)] =
          static_cast<uint16_t>(pair);
    named_barrier_sync(2, kThreads);
    if (p0 + kThreads >= P) return;
    for (int e = t; e < E; e += kThreads) {
      uint4* v = reinterpret_cast<uint4*>(block + e * kSortRow);
      next[e] += byte_sum(*v, 16);
      *v = make_uint4(0u, 0u, 0u, 0u);
    }
    named_barrier_sync(2, kThreads);
  }
}

// This CTA's run of K-blocks, cut into units: unit u = tile * jobs + job.
// (total <= kMaxJobs * kMoeMaxInner K-blocks: 32 bits hold it)
struct Walk {
  int left, total, run;  // K-blocks to go, of all CTAs; run: K-blocks per CTA where units stay whole, else 0
  int ctas, jobs, Kb;
  // the current unit
  int job, e, tile, start, m, k0, k1;
  int begin;  // first K-block of the next unit

  __device__ __forceinline__ Walk(int tiles, int blocks, int njobs) {
    jobs = njobs;
    Kb = blocks;
    const int grid = gridDim.x, units = jobs * tiles;
    total = units * Kb;
    // Whole units: the longest run has n of them, and the CTAs beside it
    // leave it more of the bandwidth (one CTA alone streams a K-block in 0.60
    // us, all 148 together in 0.73).  Equal runs: total / grid, and putting
    // the cut units together, 2 to 3 us or 4 K-blocks.  us, whole / cut, H x I
    // of the experts reached: 8 of 7168 x 2048 70.3 / 72.3, 8 of 4096 x 14336
    // 221 / 225, 49 of 2064 x 1424 89.6 / 94.0; 41 of 2048 x 1408 79.5 / 76.0,
    // 3 of 2048 x 768 23.1 / 17.4, 2 of 1024 x 512 17.0 / 15.6.
    const int n = (units + grid - 1) / grid;
    run = static_cast<int64_t>(n) * Kb * 5 <= (static_cast<int64_t>(total / grid) + 4) * 6 ? n * Kb : 0;
    if (run > 0) {
      ctas = (units + n - 1) / n;
    } else {
      const int most = (total + kMinRun - 1) / kMinRun;
      ctas = most < grid ? most : grid;
    }
    left = 0;
    if (static_cast<int>(blockIdx.x) < ctas) {
      const int w = begin_of(blockIdx.x);
      left = begin_of(blockIdx.x + 1) - w;
      const int u = w / Kb;  // the unit before the first, for next() to step from
      begin = w - u * Kb;
      tile = u / jobs;
      job = u - tile * jobs - 1;
    }
  }
  __device__ __forceinline__ int begin_of(int cta) const {
    if (run > 0) return cta * run < total ? cta * run : total;  // (ctas - 1) * run < total: no overflow
    return static_cast<int>(static_cast<int64_t>(cta) * total / ctas);
  }
  // the CTA whose run holds K-block x: of equal runs the b with b total / ctas < x + 1 <= (b + 1) total / ctas
  __device__ __forceinline__ int cta_of(int x) const {
    return run > 0 ? x / run : static_cast<int>((static_cast<int64_t>(x + 1) * ctas - 1) / total);
  }
  __device__ __forceinline__ int first_block() const { return (tile * jobs + job) * Kb; }

  __device__ __forceinline__ bool next(const Routing& r) {
    if (left <= 0) return false;
    k0 = begin;
    begin = 0;
    k1 = left < Kb - k0 ? k0 + left : Kb;
    left -= k1 - k0;
    if (++job == jobs) {
      job = 0;
      ++tile;
    }
    e = r.job_e[job];
    const int q = job - r.job[e], c = r.cnt[e];
    start = r.off[e] + q * kChunk;
    m = c - q * kChunk < kChunk ? c - q * kChunk : kChunk;
    return true;
  }
  // after the current unit: this CTA's run leaves the unit's row tile
  __device__ __forceinline__ bool leaves_tile() const { return left <= 0 || job + 1 == jobs; }
};

struct Bars {
  uint64_t *full, *empty, *xfull, *tfull, *tempty, *teardown, *stall;
  volatile int *abort_flag, *epi_flag;
};

__device__ __forceinline__ void moe_raise(const MoeParams& p, const Bars& b) {
  *b.abort_flag = 1;
  atomicExch(p.status, kTimeoutStatus);
}

// First weight rows of a unit's two boxes in the [E * rows, K] matrix.
template <class C>
__device__ __forceinline__ int box_row(const MoeParams& p, int e, int tile, int half) {
  if (C::PHASE == UP) return e * 2 * p.I + half * p.I + tile * 128;
  return e * p.H + tile * kRowTile + half * 128;
}

// DOWN's last tile may end inside its first box: the second is not loaded
// then, and what the MMA makes of the stage's old bytes is never stored.
template <class C>
__device__ __forceinline__ bool has_second(const MoeParams& p, int tile) {
  return C::PHASE == UP || tile * kRowTile + 128 < p.H;
}

template <class C>
__device__ __forceinline__ void moe_producer(const CUtensorMap* tmW, const MoeParams& p, const Routing& r, uint8_t* smem,
                                             const Bars& b, Walk walk) {
  int64_t it = 0;
  bool ok = true;
  while (ok && walk.next(r)) {
    const int row0 = box_row<C>(p, walk.e, walk.tile, 0), row1 = box_row<C>(p, walk.e, walk.tile, 1);
    const bool second = has_second<C>(p, walk.tile);
    for (int kb = walk.k0; kb < walk.k1; ++kb, ++it) {
      const int slot = static_cast<int>(it % C::STAGES);
      if (C::PHASE == DOWN && it == C::STAGES) grid_wait_prerequisites();  // the ring is full
      if (!mbar_wait(b.empty + slot, static_cast<uint32_t>((it / C::STAGES) & 1) ^ 1u, p.wait_limit_ns, b.abort_flag)) {
        moe_raise(p, b);
        ok = false;
        break;
      }
      uint8_t* stage = smem + slot * C::kStage;
      mbar_arrive_expect_tx(b.full + slot, second ? C::kStage : C::kStage / 2);
      tma_load_2d(stage, tmW, b.full + slot, kb * 128, row0);
      if (second) tma_load_2d(stage + 16384, tmW, b.full + slot, kb * 128, row1);
    }
  }
  // every issued copy lands before shared memory goes away
  for (int64_t i = it > C::STAGES ? it - C::STAGES : 0; i < it; ++i)
    (void)mbar_wait(b.full + i % C::STAGES, static_cast<uint32_t>((i / C::STAGES) & 1), kDrainNs, nullptr);
}

template <class C>
__device__ __forceinline__ void moe_mma(const MoeParams& p, const Routing& r, uint8_t* smem, uint32_t tmem,
                                        const Bars& b, Walk walk) {
  bool ok = true;
  if (C::PHASE == DOWN) grid_wait_prerequisites();
  // test hook: a barrier nothing arrives on, so the bounded wait runs out
  if (p.test_stall && !mbar_wait(b.stall, 0, p.wait_limit_ns, b.abort_flag)) {
    moe_raise(p, b);
    ok = false;
  }
  uint32_t it = 0;
  while (ok && walk.next(r)) {
    const uint32_t idesc = C::kIdesc | (uint32_t(walk.m <= 16 ? 2 : 4) << 17);
    for (int kb = walk.k0; kb < walk.k1; ++kb, ++it) {
      const uint32_t slot = it % C::STAGES, phase = (it / C::STAGES) & 1u;
      // (xfull: its warp waited for the slot's TMEM buffer as well)
      const uint32_t ab = it % C::kSlots, aphase = (it / C::kSlots) & 1u;
      if (!mbar_wait(b.xfull + ab, aphase, p.wait_limit_ns, b.abort_flag) ||
          !mbar_wait(b.full + slot, phase, p.wait_limit_ns, b.abort_flag)) {
        moe_raise(p, b);
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t a = smem_u32(smem + slot * C::kStage), x = smem_u32(smem + C::kOffX + ab * C::kX);
      const uint32_t d = tmem + ab * C::kAccCols;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint64_t bd = smem_desc(x + k * 32, 16, 1024, 2);
        mma_f8f6f4(d, smem_desc(a + k * 32, 16, 1024, 2), bd, idesc, k > 0 ? 1u : 0u);
        mma_f8f6f4(d + kChunk, smem_desc(a + 16384 + k * 32, 16, 1024, 2), bd, idesc, k > 0 ? 1u : 0u);
      }
      tc_commit(b.empty + slot);
      tc_commit(b.tfull + ab);
    }
  }
  tc_commit(b.teardown);  // all tensor-core ops done before TMEM is released
  (void)mbar_wait(b.teardown, 0, kDrainNs, nullptr);
}

// Warp f of the activation warps takes K-blocks f, f + kFillWarps, ... of the run.
// Eight lanes own one token's 128 channels, four tokens a pass.
template <class C>
__device__ __forceinline__ void moe_fill(const MoeParams& p, const Routing& r, uint8_t* smem, const Bars& b, Walk walk) {
  if (C::PHASE == DOWN) grid_wait_prerequisites();  // h comes from the kernel in front
  const int fw = (static_cast<int>(threadIdx.x) >> 5) - C::kFillWarp0;
  const int lane = threadIdx.x & 31, l = lane & 7, r_in = lane >> 3;
  // pair / k as a product: pair < 2^12 and k <= 2^5 leave an error below 2^-8
  const uint32_t inv_k = ((1u << 20) + p.k - 1) / p.k;
  uint32_t it = 0;
  while (walk.next(r)) {
    for (int kb = walk.k0; kb < walk.k1; ++kb, ++it) {
      if (static_cast<int>(it % C::kFillWarps) != fw) continue;
      const uint32_t ss = it % C::kSlots, sphase = ((it / C::kSlots) & 1u) ^ 1u;
      uint8_t* xs = smem + C::kOffX + ss * C::kX;
      float* sc = reinterpret_cast<float*>(smem + C::kOffSc) + ss * C::kSlotFloats;
      // weight scales: lane 0 the first box's, lanes 1 and 2 the second's (its rows may lie in two blocks)
      float sw = 0.0f;
      if (lane < 3) {
        int nb;
        if (C::PHASE == UP) nb = lane == 0 ? walk.tile : (p.I + walk.tile * 128) / 128 + (lane - 1);
        else nb = 2 * walk.tile + (lane == 0 ? 0 : 1);
        if (nb > p.Nb - 1) nb = p.Nb - 1;  // rows past the matrix: never used
        sw = scale_value<C::FMT>(p.w_scale, (static_cast<int64_t>(walk.e) * p.Nb + nb) * p.Kb + kb);
      }
      const int ch = kb * 128 + l * 16;
      bool waited = false, ok = true;
      // passes whose loads are in flight together; x in bf16 comes with few
      // tokens an expert, where less code counts for more (1 / 4 of them: one
      // token over 8 experts of 7168 x 2048 69.0 / 70.9 us, codes the same)
      constexpr int kBatch = C::PHASE == UP && !C::CODES ? 1 : 4;
      for (int c0 = 0; ok && c0 < walk.m; c0 += 4 * kBatch) {
        uint4 v[kBatch][2];
        float vs[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int c = c0 + 4 * i + r_in;
          v[i][0] = v[i][1] = make_uint4(0u, 0u, 0u, 0u);
          vs[i] = 1.0f;
          if (c < walk.m) {
            const int pair = r.list[walk.start + c];
            if (C::PHASE == DOWN) {
              if (ch < p.K) v[i][0] = __ldcg(reinterpret_cast<const uint4*>(p.hq + static_cast<int64_t>(pair) * p.I + ch));
              if (l == 0) vs[i] = __ldcg(p.hs + static_cast<int64_t>(pair) * p.Kb + kb);
            } else if (C::CODES) {
              const int t = static_cast<int>((static_cast<uint32_t>(pair) * inv_k) >> 20);
              if (ch < p.K)
                v[i][0] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.x) + static_cast<int64_t>(t) * p.H + ch);
              if (l == 0) vs[i] = scale_value<C::FMT>(p.x_scale, static_cast<int64_t>(t) * p.Kb + kb);
            } else if (ch < p.K) {
              const int t = static_cast<int>((static_cast<uint32_t>(pair) * inv_k) >> 20);
              const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) +
                                                                static_cast<int64_t>(t) * p.ld_x + ch);
              v[i][0] = src[0];
              v[i][1] = src[1];
            }
          }
        }
        if (!waited) {
          waited = true;
          if (!mbar_wait_warp(b.tempty + ss, sphase, p.wait_limit_ns, b.abort_flag)) {
            ok = false;
            break;
          }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          if (c0 + 4 * i >= walk.m) break;
          const int c = c0 + 4 * i + r_in;
          uint4 q = v[i][0];
          float s = vs[i];
          if (C::PHASE == UP && !C::CODES) {
            float f[16];
            {
              float f0[8], f1[8];
              unpack_bf16x8(v[i][0], f0);
              unpack_bf16x8(v[i][1], f1);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                f[j] = f0[j];
                f[8 + j] = f1[j];
              }
            }
            float amax = 0.0f;
#pragma unroll
            for (int j = 0; j < 16; ++j) amax = fmaxf(amax, fabsf(f[j]));
            amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
            amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 4));
            s = group_scale(amax);
            const uint32_t sb = C::FMT == 1 ? e8m0_ceil_byte(s) : 0u;
            q = quantize16<C::FMT>(f, s, sb);
            if (C::FMT == 1) s = __uint_as_float(sb << 23);
          }
          if (c < walk.m) {
            *reinterpret_cast<uint4*>(xs + (c >> 3) * 1024 + (c & 7) * 128 + ((l ^ (c & 7)) << 4)) = q;
            if (l == 0) sc[c] = s;
          }
        }
      }
      if (!ok) {
        if (lane == 0) moe_raise(p, b);
        return;
      }
      if (lane < 3) sc[kChunk + lane] = sw;
      fence_proxy_async_smem();  // the tensor core reads what these threads wrote
      __syncwarp();
      if (lane == 0) mbar_arrive(b.xfull + ss);
    }
  }
}

// acc[c] += P[c] * (sx[c] * sw) for one K-block's W columns of a box.
template <int W>
__device__ __forceinline__ void promote(uint32_t taddr, const float* sc, float sw, float (&acc)[kChunk]) {
  uint32_t r[W];
  if constexpr (W == 16) {
    tmem_ld_32x32b_x16(taddr, r);
    tmem_wait_ld();
    tmem_reg_fence16(r);
  } else {
    tmem_ld_32x32b_x32(taddr, r);
    tmem_wait_ld();
    tmem_reg_fence(r);
  }
#pragma unroll
  for (int j = 0; j < W; j += 4) {
    const float4 sx = *reinterpret_cast<const float4*>(sc + j);
    acc[j] = __fmaf_rn(__uint_as_float(r[j]), sx.x * sw, acc[j]);
    acc[j + 1] = __fmaf_rn(__uint_as_float(r[j + 1]), sx.y * sw, acc[j + 1]);
    acc[j + 2] = __fmaf_rn(__uint_as_float(r[j + 2]), sx.z * sw, acc[j + 2]);
    acc[j + 3] = __fmaf_rn(__uint_as_float(r[j + 3]), sx.w * sw, acc[j + 3]);
  }
}

// Sum of a cut unit's partials at (column, row of the thread), in CTA order.
struct CutUnit {
  int first, last;  // its CTAs
  __device__ __forceinline__ const float* part(const MoeParams& p, int cta) const {
    return p.split + (2 * cta + (cta == first ? 1 : 0)) * kPartFloats;
  }
  // columns c .. c + 3; 16 loads in flight
  __device__ __forceinline__ float4 sum4(const MoeParams& p, int c, int m, int et) const {
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int cta = first; cta <= last; cta += 4) {
      float v[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[i][j] = cta + i <= last && c + j < m ? __ldcg(part(p, cta + i) + (c + j) * kRowTile + et) : 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] += v[i][j];
    }
    return make_float4(s[0], s[1], s[2], s[3]);
  }
};

// UP: silu(gate) * up of a unit's 128 rows, one group per pair: both halves
// through shared memory ([box][pair][row], 16 pairs at a time), then one warp
// per pair for the products, amax, scale and codes.  Only the stores from the
// accumulators are unrolled: this code runs once per unit, and unrolled as a
// whole it spent more time on instruction fetches than on work (a unit's end
// took 4 to 6 us).
template <class C>
__device__ __forceinline__ void finish_up(const MoeParams& p, const Routing& r, const Walk& w, float* stage, int et,
                                          const float (&acc)[kChunk], bool cut, const CutUnit& cu) {
  float* mine = stage + (et >> 7) * (C::kStagePairs * 128) + (et & 127);
  const int lane = et & 31, i = w.tile * 128 + lane * 4;
#pragma unroll
  for (int c0 = 0; c0 < kChunk; c0 += C::kStagePairs) {
    if (c0 >= w.m) break;
    const int n = w.m - c0 < C::kStagePairs ? w.m - c0 : C::kStagePairs;
    named_barrier_sync(1, C::kEpiThreads);  // the stage's last readers are done
    if (cut) {
#pragma unroll 1
      for (int c = 0; c < n; c += 4) {
        const float4 v = cu.sum4(p, c0 + c, w.m, et);
        mine[c * 128] = v.x;
        mine[(c + 1) * 128] = v.y;
        mine[(c + 2) * 128] = v.z;
        mine[(c + 3) * 128] = v.w;
      }
    } else {
#pragma unroll
      for (int c = 0; c < C::kStagePairs; ++c)
        if (c < n) mine[c * 128] = acc[c0 + c];
    }
    named_barrier_sync(1, C::kEpiThreads);
#pragma unroll 1
    for (int c = et >> 5; c < n; c += C::kEpiThreads / 32) {
      const float4 g = *reinterpret_cast<const float4*>(stage + c * 128 + lane * 4);
      const float4 u = *reinterpret_cast<const float4*>(stage + (C::kStagePairs + c) * 128 + lane * 4);
      const float2 f01 = silu_mul2(make_float2(g.x, g.y), make_float2(u.x, u.y));
      const float2 f23 = silu_mul2(make_float2(g.z, g.w), make_float2(u.z, u.w));
      float f[4] = {f01.x, f01.y, f23.x, f23.y};
      float amax = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (i >= p.I) f[j] = 0.0f;  // I % 16 == 0: four channels are wholly inside or outside
        amax = fmaxf(amax, fabsf(f[j]));
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, off));
      float s = group_scale(amax);
      if (C::FMT == 1) s = __uint_as_float(e8m0_ceil_byte(s) << 23);
      const int64_t pair = r.list[w.start + c0 + c];
      if (i < p.I)
        *reinterpret_cast<uint32_t*>(p.hq + pair * p.I + i) =
            pack_e4m3x4(__fdiv_rn(f[0], s), __fdiv_rn(f[1], s), __fdiv_rn(f[2], s), __fdiv_rn(f[3], s));
      if (lane == 0) p.hs[pair * ((p.I + 127) / 128) + w.tile] = s;
    }
  }
}

// The weighted sums over the slots for one row tile, all tokens: one warp per
// token, eight channels per lane, the slots in order.
template <class C>
__device__ __forceinline__ void combine(const MoeParams& p, int tile, int et) {
  const int n = tile * kRowTile + (et & 31) * 8;
  if (n >= p.H) return;  // H % 16 == 0
  for (int t = et >> 5; t < p.T; t += C::kEpiThreads / 32) {
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
    for (int j0 = 0; j0 < p.k; j0 += 8) {
      float4 v[8][2];
      float wt[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int pair = t * p.k + j0 + j;
        const int id = j0 + j < p.k ? __ldg(p.ids + pair) : -1;
        wt[j] = 0.0f;
        v[j][0] = v[j][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (id >= 0 && id < p.E) {
          const float4* src = reinterpret_cast<const float4*>(p.part + static_cast<int64_t>(pair) * p.H + n);
          wt[j] = __ldg(p.weights + pair);
          v[j][0] = __ldcg(src);
          v[j][1] = __ldcg(src + 1);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        acc[0] = fmaf(wt[j], v[j][0].x, acc[0]);
        acc[1] = fmaf(wt[j], v[j][0].y, acc[1]);
        acc[2] = fmaf(wt[j], v[j][0].z, acc[2]);
        acc[3] = fmaf(wt[j], v[j][0].w, acc[3]);
        acc[4] = fmaf(wt[j], v[j][1].x, acc[4]);
        acc[5] = fmaf(wt[j], v[j][1].y, acc[5]);
        acc[6] = fmaf(wt[j], v[j][1].z, acc[6]);
        acc[7] = fmaf(wt[j], v[j][1].w, acc[7]);
      }
    }
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(acc[2 * i]))) |
             (static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(acc[2 * i + 1]))) << 16);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.y) + static_cast<int64_t>(t) * p.ld_y + n) =
        make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// Counts an arrival on *counter after this CTA's epilogue stores; true for
// every epilogue thread of the CTA that brings it to `want` (which zeroes it
// for the next call).  The barriers put the threads' stores in front of the
// one thread's atomic and their loads behind it; it releases and acquires.
template <class C>
__device__ __forceinline__ bool arrive_last(uint32_t* counter, uint32_t want, int et, volatile int* flag) {
  if (want == 1u) {
    named_barrier_sync(1, C::kEpiThreads);
    return true;
  }
  named_barrier_sync(1, C::kEpiThreads);
  if (et == 0) {
    const uint32_t done = atomic_add_acq_rel(counter, 1u) + 1u;
    *flag = done == want ? 1 : 0;
    if (done == want) *counter = 0u;
  }
  named_barrier_sync(1, C::kEpiThreads);
  return *flag != 0;
}

template <class C>
__device__ __forceinline__ void moe_epilogue(const MoeParams& p, const Routing& r, uint8_t* smem, uint32_t tmem,
                                             const Bars& b, Walk walk) {
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = threadIdx.x & 31;
  const int q = warp & 3;                           // TMEM lane quadrant
  const int half = (warp - C::kEpiWarp0) >> 2;      // box
  const int row = q * 32 + lane;                    // weight row inside the box
  const int et = half * 128 + row;
  const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
  // the box's weight scale: the second box of UP may lie in two scale blocks
  const int at = kChunk + (half == 0 ? 0 : (C::PHASE == UP && row >= 128 - p.I % 128) ? 2 : 1);
  float* stage = reinterpret_cast<float*>(smem + C::kOffStage);
  if (C::PHASE == DOWN) grid_wait_prerequisites();
  uint32_t it = 0;
  bool ok = true;
  while (walk.next(r)) {
    float acc[kChunk];
#pragma unroll
    for (int c = 0; c < kChunk; ++c) acc[c] = 0.0f;
    for (int kb = walk.k0; ok && kb < walk.k1; ++kb, ++it) {
      const uint32_t ss = it % C::kSlots, phase = (it / C::kSlots) & 1u;
      if (!mbar_wait_warp(b.xfull + ss, phase, p.wait_limit_ns, b.abort_flag) ||
          !mbar_wait_warp(b.tfull + ss, phase, p.wait_limit_ns, b.abort_flag)) {
        // from here on this warp only keeps its barriers (every warp's next
        // wait fails likewise); what it stores is unspecified, in bounds
        if (lane == 0) moe_raise(p, b);
        ok = false;
        break;
      }
      tc_fence_after();
      const float* sc = reinterpret_cast<const float*>(smem + C::kOffSc) + ss * C::kSlotFloats;
      const uint32_t taddr = tmem + lane_base + ss * C::kAccCols + half * kChunk;
      if (walk.m <= 16) promote<16>(taddr, sc, sc[at], acc);
      else promote<32>(taddr, sc, sc[at], acc);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b.tempty + ss);
    }
    const bool cut = walk.k0 != 0 || walk.k1 != p.Kb;
    bool whole = true;
    CutUnit cu{0, 0};
    if (cut) {  // partial sums, added up by the last of the unit's CTAs
      const int b0 = walk.first_block();
      cu.first = walk.cta_of(b0);
      cu.last = walk.cta_of(b0 + p.Kb - 1);
      float* mine = p.split + (2 * blockIdx.x + (static_cast<int>(blockIdx.x) == cu.first ? 1 : 0)) * kPartFloats;
#pragma unroll
      for (int c = 0; c < kChunk; ++c)
        if (c < walk.m) __stcg(mine + c * kRowTile + et, acc[c]);
      whole = arrive_last<C>(p.counters + cu.first, static_cast<uint32_t>(cu.last - cu.first + 1), et, b.epi_flag);
    }
    if (C::PHASE == UP) {
      if (whole) finish_up<C>(p, r, walk, stage, et, acc, cut, cu);
      continue;
    }
    const int n = walk.tile * kRowTile + et;
    if (whole && n < p.H) {
      float* out = p.part + n;
      const uint16_t* pairs = r.list + walk.start;
      if (cut) {
#pragma unroll 1
        for (int c = 0; c < walk.m; c += 4) {
          const float4 v = cu.sum4(p, c, walk.m, et);
          __stcg(out + static_cast<int64_t>(pairs[c]) * p.H, v.x);
          if (c + 1 < walk.m) __stcg(out + static_cast<int64_t>(pairs[c + 1]) * p.H, v.y);
          if (c + 2 < walk.m) __stcg(out + static_cast<int64_t>(pairs[c + 2]) * p.H, v.z);
          if (c + 3 < walk.m) __stcg(out + static_cast<int64_t>(pairs[c + 3]) * p.H, v.w);
        }
      } else {
#pragma unroll
        for (int c = 0; c < kChunk; ++c)
          if (c < walk.m) __stcg(out + static_cast<int64_t>(pairs[c]) * p.H, acc[c]);
      }
    }
    if (walk.leaves_tile()) {  // one arrival per CTA and row tile
      const int per_tile = walk.jobs * p.Kb;
      const int first = walk.cta_of(walk.tile * per_tile), last = walk.cta_of((walk.tile + 1) * per_tile - 1);
      if (arrive_last<C>(p.counters + kMaxGrid + walk.tile, static_cast<uint32_t>(last - first + 1), et, b.epi_flag))
        combine<C>(p, walk.tile, et);
    }
  }
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1)
    moe_kernel(const __grid_constant__ CUtensorMap tmW, const MoeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Routing r;
  r.list = reinterpret_cast<uint16_t*>(smem + C::kOffList);
  r.cnt = reinterpret_cast<uint16_t*>(smem + C::kOffCnt);
  r.count = reinterpret_cast<uint32_t*>(smem + C::kOffCount);
  r.ids = reinterpret_cast<uint16_t*>(smem + C::kOffIds);
  r.block = smem + C::kOffBlock;
  r.off = reinterpret_cast<uint16_t*>(smem + C::kOffOff);
  r.job = reinterpret_cast<uint16_t*>(smem + C::kOffJob);
  r.job_e = reinterpret_cast<uint16_t*>(smem + C::kOffJobE);
  Bars b;
  b.full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  b.empty = b.full + C::STAGES;
  b.xfull = b.empty + C::STAGES;
  b.tfull = b.xfull + C::kSlots;
  b.tempty = b.tfull + C::kSlots;
  b.teardown = b.tempty + C::kSlots;
  b.stall = b.teardown + 1;
  int* words = reinterpret_cast<int*>(b.stall + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(words);
  b.abort_flag = words + 1;
  b.epi_flag = words + 2;
  int* jobs_slot = words + 3;

  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = threadIdx.x & 31;
  clear_counts(p, r);
  if (threadIdx.x == 0) {
    prefetch_tmap(&tmW);
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(b.full + s, 1);
      mbar_init(b.empty + s, 1);
    }
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(b.xfull + s, 1);
      mbar_init(b.tfull + s, 1);
      mbar_init(b.tempty + s, C::kEpiThreads / 32);
    }
    mbar_init(b.teardown, 1);
    mbar_init(b.stall, 1);
    *b.abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  __syncthreads();
  // UP: everything it reads may come from the kernel in front.  DOWN: that is
  // UP, which waited itself; only h is new.
  if (C::PHASE == UP) grid_wait_prerequisites();
  grid_launch_dependents();
  if (p.test_late == C::PHASE + 1 && blockIdx.x == 0)  // test hook
    for (const uint64_t t0 = global_timer_ns(); global_timer_ns() - t0 < 3 * p.wait_limit_ns;) __nanosleep(100000);
  count_pairs<C::PHASE>(p, r);
  __syncthreads();
  if (warp == C::kFillWarp0) {
    const int jobs = place_experts(p, r);
    if (lane == 0) *jobs_slot = jobs;
    if (p.T * p.k <= kFewPairs) place_few(p, r);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int jobs = *jobs_slot;
  if (jobs > 0) {
    const Walk walk(p.tiles, p.Kb, jobs);
    if (warp == 0) {
      if (lane == 0) moe_producer<C>(&tmW, p, r, smem, b, walk);
    } else if (warp == 1) {
      if (lane == 0) moe_mma<C>(p, r, smem, tmem, b, walk);
    } else {
      if (p.T * p.k > kFewPairs) place_many(p.T * p.k, p.E, r.ids, r.count, r.block, r.list);
      if (warp < C::kEpiWarp0) moe_fill<C>(p, r, smem, b, walk);
      else moe_epilogue<C>(p, r, smem, tmem, b, walk);
    }
  } else if (C::PHASE == DOWN && warp >= C::kEpiWarp0) {  // no valid slot at all: zeros
    grid_wait_prerequisites();
    for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x)
      combine<C>(p, tile, static_cast<int>(threadIdx.x) - C::kEpiWarp0 * 32);
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

typedef CUresult (*EncodeTiledFnMoe)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                     const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                     CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFnMoe encode_fn_moe() {
  // looked up once per process (thread-safe static initialisation)
  static const EncodeTiledFnMoe fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<EncodeTiledFnMoe>(ptr);
    return static_cast<EncodeTiledFnMoe>(nullptr);
  }();
  return fn;
}

// Every expert's rows as one e4m3 matrix [rows, K]: 128 x 128 boxes, 128-byte swizzle.
cudaError_t weight_map(CUtensorMap* map, const uint8_t* w, int64_t rows, int K) {
  const EncodeTiledFnMoe fn = encode_fn_moe();
  if (fn == nullptr) return cudaErrorInvalidValue;
  const cuuint32_t estr[2] = {1, 1}, box[2] = {128, 128};
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K)};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(w), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

template <class C>
cudaError_t launch_phase(const MoeParams& p, const uint8_t* w, int64_t rows, int num_sms, cudaStream_t s) {
  CUtensorMap tmW;
  if (const cudaError_t e = weight_map(&tmW, w, rows, p.K); e != cudaSuccess) return e;
  auto kern = moe_kernel<C>;
  // the shared-memory opt-in, once per device
  static std::atomic<uint64_t> configured{0};
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = 1ull << (dev & 63);
  if ((configured.load(std::memory_order_acquire) & bit) == 0) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(num_sms < kMaxGrid ? num_sms : kMaxGrid));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tmW, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

template <int FMT>
cudaError_t launch_fmt(const MoeArgs& a, const MoeParams& up, const MoeParams& down, int num_sms, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(a.E) * 2 * a.I;
  const cudaError_t e = a.x_scale != nullptr ? launch_phase<MoeCfg<UP, FMT, true>>(up, a.w13, rows, num_sms, s)
                                             : launch_phase<MoeCfg<UP, FMT, false>>(up, a.w13, rows, num_sms, s);
  if (e != cudaSuccess) return e;
  return launch_phase<MoeCfg<DOWN, FMT, true>>(down, a.w2, static_cast<int64_t>(a.E) * a.H, num_sms, s);
}

}  // namespace

size_t moe_workspace_need(int T, int k, int E, int H, int I, int fmt) { return moe_ws_layout(T, k, E, H, I).total; }

cudaError_t launch_moe_mlp(const MoeArgs& a, int fmt, int num_sms, cudaStream_t s) {
  const MoeWs L = moe_ws_layout(a.T, a.k, a.E, a.H, a.I);
  const int Hb = (a.H + 127) / 128, Ib = (a.I + 127) / 128;
  if (a.x_scale == nullptr && quantize_first(a.T, a.k, a.E)) {
    ActQuantArgs q{};
    q.x = a.x;
    q.ld_x = a.ld_x;
    q.M = a.T;
    q.K = a.H;
    q.Kb = Hb;
    q.xq = a.ws + L.xq;
    q.xs = a.ws + L.xs;
    q.layout = kScaleRowMajor;
    if (const cudaError_t e = launch_act_quant(q, fmt, num_sms, s); e != cudaSuccess) return e;
    MoeArgs b = a;
    b.x = q.xq;
    b.ld_x = a.H;
    b.x_scale = q.xs;
    return launch_moe_mlp(b, fmt, num_sms, s);
  }
  MoeParams p{};
  p.x = a.x;
  p.ld_x = a.ld_x;
  p.x_scale = a.x_scale;
  p.ids = a.ids;
  p.weights = a.weights;
  p.T = a.T;
  p.k = a.k;
  p.E = a.E;
  p.H = a.H;
  p.I = a.I;
  p.hq = a.ws + L.hq;
  p.hs = reinterpret_cast<float*>(a.ws + L.hs);
  p.split = reinterpret_cast<float*>(a.ws + L.split);
  p.part = reinterpret_cast<float*>(a.ws + L.part);
  p.y = a.y;
  p.ld_y = a.ld_y;
  p.status = reinterpret_cast<uint32_t*>(a.ws);
  p.counters = reinterpret_cast<uint32_t*>(a.ws + kHeaderCounterOffset);
  p.wait_limit_ns = a.wait_limit_ns;
  p.test_stall = a.test_stall;
  p.test_late = a.test_late;
  MoeParams up = p, down = p;
  up.w_scale = a.s13;
  up.K = a.H;
  up.Kb = Hb;
  up.Nb = (2 * a.I + 127) / 128;
  up.tiles = Ib;
  down.w_scale = a.s2;
  down.K = a.I;
  down.Kb = Ib;
  down.Nb = Hb;
  down.tiles = (a.H + kRowTile - 1) / kRowTile;
  up.weights = nullptr;  // only DOWN sums
  if (a.test_stall == 3) down.test_stall = 0;
  return fmt == 0 ? launch_fmt<0>(a, up, down, num_sms, s) : launch_fmt<1>(a, up, down, num_sms, s);
}

}  // namespace fg8
