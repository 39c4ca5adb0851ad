// moe_route.cu -- the router of a mixture-of-experts layer: softmax over a
// token's expert logits, its k largest, their weights (sm_100a).
//
// One warp per token, the logits in registers.  A logit becomes an unsigned
// key that orders as the float does, 0 for NaN and -inf (never chosen), so a
// round of the selection is two warp reductions on integers: the largest
// key, then the lowest index that holds it.  Equal logits (frequent in bf16)
// therefore go to the lowest index, whatever the order of the lanes.
// exp(l - l_max) of the k chosen ones (or, without renormalization, of all)
// is summed in float32 in a fixed order.

#include <cuda_bf16.h>

#include "fg8_internal.h"
#include "ptx.cuh"

namespace fg8 {
namespace {

// Larger float <=> larger key; NaN and -inf: 0.
__device__ __forceinline__ uint32_t order_key(float f) {
  if (!(f > __int_as_float(0xff800000))) return 0u;
  const uint32_t b = __float_as_uint(f == 0.0f ? 0.0f : f);  // -0 and +0 are one value
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

// exp(v - top): 1 where both are the same value, infinities included.
__device__ __forceinline__ float exp_below(float v, float top) { return v == top ? 1.0f : expf(v - top); }

// V values per lane: expert e = lane + 32 i.
template <int V>
__global__ void __launch_bounds__(128) moe_route_kernel(const RouteArgs a) {
  grid_wait_prerequisites();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (t >= a.T) return;
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 32 * i;
    key[i] = 0u;
    if (e < a.E) {
      const float f = a.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[t * a.ld + e])
                             : static_cast<const float*>(a.logits)[t * a.ld + e];
      key[i] = order_key(f);
    }
  }
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
  if (a.E <= 32) e = cudaLaunchKernelEx(&cfg, moe_route_kernel<1>, a);
  else if (a.E <= 64) e = cudaLaunchKernelEx(&cfg, moe_route_kernel<2>, a);
  else if (a.E <= 128) e = cudaLaunchKernelEx(&cfg, moe_route_kernel<4>, a);
  else if (a.E <= 256) e = cudaLaunchKernelEx(&cfg, moe_route_kernel<8>, a);
  else if (a.E <= 512) e = cudaLaunchKernelEx(&cfg, moe_route_kernel<16>, a);
  else if (a.E <= kRouteMaxExperts) e = cudaLaunchKernelEx(&cfg, moe_route_kernel<32>, a);
  else return cudaErrorInvalidValue;
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace fg8
