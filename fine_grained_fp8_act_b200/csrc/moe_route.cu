// moe_route.cu -- the router of a mixture-of-experts layer: softmax over a
// token's expert logits, its k largest, their weights (sm_100a).
//
// One warp per token, the logits in registers as unsigned keys that order as
// the floats do, 0 for NaN and -inf (never chosen).  The k-th largest of the
// 32 lanes' largest keys bounds the choice from below: k warp reductions on
// one value per lane.  The keys at or above it, few more than k, are gathered
// in index order and each counts those in front of it, larger keys and equal
// ones of lower index: its place.  So equal logits (frequent in bf16) go to
// the lowest index, whatever the lanes' order.  A token with more than 32
// such keys (many equal logits, k near 32) is chosen from one round at a time.
//
// 16384 tokens of 256 experts read 17 MB (2.6 us) and take 8.7 us, bound by
// instructions: 453 a token are 6.4 us of all issue slots, which are 78% busy
// while warps run.  Choosing every token by k rounds over all keys took 16 us.
//
// exp(l - l_max) of the k chosen ones (or, without renormalization, of all)
// is summed in float32 in a fixed order.

#include <cuda_bf16.h>

#include "fg8_internal.h"
#include "ptx.cuh"

namespace fg8 {
namespace {

// Larger float <=> larger key; NaN and -inf: 0.
__device__ __forceinline__ uint32_t order_key(float f) {
  const float g = f + 0.0f;  // -0 and +0 are one value
  const uint32_t b = __float_as_uint(g);
  const uint32_t key = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
  return g > __int_as_float(0xff800000) ? key : 0u;
}

__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

// exp(v - top): 1 where both are the same value, infinities included.
__device__ __forceinline__ float exp_below(float v, float top) { return v == top ? 1.0f : expf(v - top); }

// V values per lane: expert e = lane + 32 i.
template <int V, class T>
__global__ void __launch_bounds__(128) moe_route_kernel(const RouteArgs a) {
  __shared__ __align__(16) uint32_t cand_keys[4][32];
  __shared__ uint16_t cand_es[4][32];
  grid_wait_prerequisites();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  uint32_t* cand_key = cand_keys[threadIdx.x >> 5];
  uint16_t* cand_e = cand_es[threadIdx.x >> 5];
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (t >= a.T) return;
  // all loads first (with a test around each one they came one after the
  // other: one token of 256 experts 3.0 us, together 2.0); experts past the
  // last one read as -inf
  const T* row = static_cast<const T*>(a.logits) + t * a.ld;
  float f[V];
  if (a.E == 32 * V) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = static_cast<float>(row[lane + 32 * i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = static_cast<float>(row[min(lane + 32 * i, a.E - 1)]);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = lane + 32 * i < a.E ? f[i] : __int_as_float(0xff800000);
  }
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = order_key(f[i]);
  // the sum over all experts, before the selection clears the chosen keys
  float all = 0.0f;
  if (!a.renormalize) {
    uint32_t best = 0u;
#pragma unroll
    for (int i = 0; i < V; ++i) best = key[i] > best ? key[i] : best;
    const float top = key_value(__reduce_max_sync(0xFFFFFFFFu, best));
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] != 0u) all += exp_below(key_value(key[i]), top);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, off);
  }
  uint32_t mine = 0u;  // lane j: the key and expert of the j-th choice
  int mine_e = -1;
  uint32_t most = 0u;
#pragma unroll
  for (int i = 0; i < V; ++i) most = key[i] > most ? key[i] : most;
  cand_key[lane] = 0u;
  uint32_t bound = 0u;
  for (int j = 0; j < a.k; ++j) {
    bound = __reduce_max_sync(0xFFFFFFFFu, most);
    if (most == bound) most = 0u;
  }
  bound = bound > 0u ? bound : 1u;  // fewer than k lanes hold a logit: every one there is
  __syncwarp();
  int found = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const bool in = key[i] >= bound;
    const uint32_t who = __ballot_sync(0xFFFFFFFFu, in);
    const int at = found + __popc(who & ((1u << lane) - 1u));
    if (in && at < 32) {
      cand_key[at] = key[i];
      cand_e[at] = static_cast<uint16_t>(lane + 32 * i);
    }
    found += __popc(who);
  }
  __syncwarp();
  if (found <= 32) {
    const uint32_t c = cand_key[lane];
    const uint16_t e = cand_e[lane];
    // o in front of c: o > c, or equal and of lower index, as one comparison
    // (a key is at most that of inf, 0xFF800000; the zeros past the last one
    // are behind every candidate)
    int place = 0;
    for (int j = 0; j < found; j += 4) {
      const uint4 o = *reinterpret_cast<const uint4*>(cand_key + j);
      place += o.x + (j < lane ? 1u : 0u) > c;
      place += o.y + (j + 1 < lane ? 1u : 0u) > c;
      place += o.z + (j + 2 < lane ? 1u : 0u) > c;
      place += o.w + (j + 3 < lane ? 1u : 0u) > c;
    }
    __syncwarp();  // every lane holds its candidate
    if (lane < found && place < a.k) {
      cand_key[place] = c;
      cand_e[place] = e;
    }
    __syncwarp();
    if (lane < a.k && lane < found) mine = cand_key[lane], mine_e = cand_e[lane];
  } else {
    for (int j = 0; j < a.k; ++j) {
      uint32_t best = 0u;
      int at = 0;
#pragma unroll
      for (int i = V - 1; i >= 0; --i)
        if (key[i] >= best) best = key[i], at = i;
      const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
      if (top == 0u) break;  // nothing left to choose
      const int e = static_cast<int>(
          __reduce_min_sync(0xFFFFFFFFu, best == top ? static_cast<uint32_t>(lane + 32 * at) : 0xFFFFFFFFu));
      if (lane == j) mine = top, mine_e = e;
      if ((e & 31) == lane) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i == e >> 5) key[i] = 0u;
      }
    }
  }
  const float first = key_value(__shfl_sync(0xFFFFFFFFu, mine, 0));
  float w = mine != 0u ? exp_below(key_value(mine), first) : 0.0f;
  float sum = w;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
  if (!a.renormalize) sum = all;
  if (mine != 0u) w = __fdiv_rn(w, sum) * a.scale;
  if (lane < a.k) {
    a.ids[t * a.k + lane] = mine_e;
    a.weights[t * a.k + lane] = w;
  }
}

template <int V>
cudaError_t launch(const cudaLaunchConfig_t& cfg, const RouteArgs& a) {
  return a.bf16 ? cudaLaunchKernelEx(&cfg, moe_route_kernel<V, __nv_bfloat16>, a)
                : cudaLaunchKernelEx(&cfg, moe_route_kernel<V, float>, a);
}

}  // namespace

cudaError_t launch_moe_route(const RouteArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(a.T) + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  // (halfway sizes too: 16384 tokens of 384 experts, 12 / 16 values a lane, 10.3 / 15.0 us)
  if (a.E <= 32) e = launch<1>(cfg, a);
  else if (a.E <= 64) e = launch<2>(cfg, a);
  else if (a.E <= 96) e = launch<3>(cfg, a);
  else if (a.E <= 128) e = launch<4>(cfg, a);
  else if (a.E <= 192) e = launch<6>(cfg, a);
  else if (a.E <= 256) e = launch<8>(cfg, a);
  else if (a.E <= 384) e = launch<12>(cfg, a);
  else if (a.E <= 512) e = launch<16>(cfg, a);
  else if (a.E <= 768) e = launch<24>(cfg, a);
  else if (a.E <= kRouteMaxExperts) e = launch<32>(cfg, a);
  else return cudaErrorInvalidValue;
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace fg8
