// moe.cu -- a whole mixture-of-experts layer for few tokens (sm_100a):
//
//   y[t] = sum over the token's slots j of weights[t, j] * W2[e] . h[t, j],   e = ids[t, j]
//   h    = silu(gate) * up,   gate = W13[e][:I] . x[t],   up = W13[e][I:] . x[t]
//
// x and h are quantized per token in groups of 1 x 128 as the dense layers'
// activations are; gate, up, h and the down products stay in float32 until
// that quantization and until y's one rounding to bf16.
//
// With few tokens the layer is bound by reading the reached experts' e4m3
// weights once (3 H I bytes an expert).
//
// First form: one warp per weight row and routed pair, plain loads.

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "fg8_internal.h"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace fg8 {
namespace {

using namespace qm;

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

struct MoeWs {
  size_t xq, xs, hq, hs, part, total;
};

MoeWs moe_ws_layout(int64_t T, int64_t k, int64_t H, int64_t I) {
  MoeWs w;
  const int64_t P = T * k, Hb = (H + 127) / 128, Ib = (I + 127) / 128;
  w.xq = kWorkspaceHeaderBytes;
  w.xs = align256(w.xq + T * H);
  w.hq = align256(w.xs + T * Hb * 4);
  w.hs = align256(w.hq + P * I);
  w.part = align256(w.hs + P * Ib * 4);
  w.total = align256(w.part + P * H * 4);
  return w;
}

template <int FMT>
__device__ __forceinline__ float scale_value(const void* s, int64_t i) {
  if (FMT == 0) return static_cast<const float*>(s)[i];
  const uint32_t b = static_cast<const uint8_t*>(s)[i];
  return __uint_as_float(b == 0u ? 0x00400000u : b << 23);  // 2^(b - 127)
}

__device__ __forceinline__ float dot16(const uint4& a, const uint4& b) {
  const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      __nv_fp8_e4m3 p, q;
      p.__x = static_cast<__nv_fp8_storage_t>(aw[i] >> (8 * j));
      q.__x = static_cast<__nv_fp8_storage_t>(bw[i] >> (8 * j));
      s = fmaf(static_cast<float>(p), static_cast<float>(q), s);
    }
  return s;
}

// One weight row times one quantized activation row, by a warp.
template <int FMT>
__device__ float row_dot(const uint8_t* w, const void* ws, int64_t ws_row, const uint8_t* xq, const float* xs, int K) {
  const int lane = threadIdx.x & 31;
  float acc = 0.0f;
  for (int k = lane * 16; k < K; k += 512) {
    const float p = dot16(*reinterpret_cast<const uint4*>(w + k), *reinterpret_cast<const uint4*>(xq + k));
    acc = fmaf(p, xs[k / 128] * scale_value<FMT>(ws, ws_row + k / 128), acc);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, off);
  return acc;
}

// gate, up, silu, quantization: CTA = (128 rows of I, routed pair).
template <int FMT>
__global__ void __launch_bounds__(256) moe_up_kernel(const MoeArgs a, const uint8_t* xq, const void* xs_in,
                                                     uint8_t* hq, float* hs) {
  __shared__ float v[128], red[8], xs[kMoeMaxHidden / 128];
  const int p = blockIdx.y, t = p / a.k, e = a.ids[p];
  if (e >= a.E && blockIdx.x == 0 && threadIdx.x == 0) atomicExch(reinterpret_cast<uint32_t*>(a.ws), 1u);
  if (e < 0 || e >= a.E) return;
  const int Hb = (a.H + 127) / 128, N13b = (2 * a.I + 127) / 128;
  for (int i = threadIdx.x; i < Hb; i += 256) xs[i] = scale_value<FMT>(xs_in, static_cast<int64_t>(t) * Hb + i);
  if (threadIdx.x < 128) v[threadIdx.x] = 0.0f;
  __syncthreads();
  const int warp = threadIdx.x >> 5;
  for (int r = warp; r < 128; r += 8) {
    const int i = blockIdx.x * 128 + r;
    if (i >= a.I) break;
    const uint8_t* w = a.w13 + static_cast<int64_t>(e) * 2 * a.I * a.H;
    const uint8_t* x = xq + static_cast<int64_t>(t) * a.H;
    const float g = row_dot<FMT>(w + static_cast<int64_t>(i) * a.H, a.s13,
                                 (static_cast<int64_t>(e) * N13b + i / 128) * Hb, x, xs, a.H);
    const float u = row_dot<FMT>(w + static_cast<int64_t>(a.I + i) * a.H, a.s13,
                                 (static_cast<int64_t>(e) * N13b + (a.I + i) / 128) * Hb, x, xs, a.H);
    if ((threadIdx.x & 31) == 0) v[r] = silu_mul(g, u);
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    float f[4], amax = 0.0f;
    for (int j = 0; j < 4; ++j) f[j] = v[threadIdx.x * 4 + j], amax = fmaxf(amax, fabsf(f[j]));
    for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, off));
    float s = group_scale(amax);
    if (FMT == 1) s = __uint_as_float(e8m0_ceil_byte(s) << 23);
    const int i = blockIdx.x * 128 + threadIdx.x * 4;
    if (i < a.I)
      *reinterpret_cast<uint32_t*>(hq + static_cast<int64_t>(p) * a.I + i) =
          pack_e4m3x4(__fdiv_rn(f[0], s), __fdiv_rn(f[1], s), __fdiv_rn(f[2], s), __fdiv_rn(f[3], s));
    if (threadIdx.x == 0) hs[static_cast<int64_t>(p) * ((a.I + 127) / 128) + blockIdx.x] = s;
  }
}

// down products of one pair: CTA = (128 rows of H, routed pair).
template <int FMT>
__global__ void __launch_bounds__(256) moe_down_kernel(const MoeArgs a, const uint8_t* hq, const float* hs,
                                                       float* part) {
  const int p = blockIdx.y, e = a.ids[p];
  if (e < 0 || e >= a.E) return;
  const int Hb = (a.H + 127) / 128, Ib = (a.I + 127) / 128;
  for (int r = threadIdx.x >> 5; r < 128; r += 8) {
    const int n = blockIdx.x * 128 + r;
    if (n >= a.H) break;
    const float o = row_dot<FMT>(a.w2 + (static_cast<int64_t>(e) * a.H + n) * a.I, a.s2,
                                 (static_cast<int64_t>(e) * Hb + n / 128) * Ib, hq + static_cast<int64_t>(p) * a.I,
                                 hs + static_cast<int64_t>(p) * Ib, a.I);
    if ((threadIdx.x & 31) == 0) part[static_cast<int64_t>(p) * a.H + n] = o;
  }
}

__global__ void __launch_bounds__(256) moe_combine_kernel(const MoeArgs a, const float* part) {
  const int t = blockIdx.y, n = blockIdx.x * 256 + threadIdx.x;
  if (n >= a.H) return;
  float acc = 0.0f;
  for (int j = 0; j < a.k; ++j) {
    const int e = a.ids[t * a.k + j];
    if (e >= 0 && e < a.E)
      acc = fmaf(a.weights[t * a.k + j], part[(static_cast<int64_t>(t) * a.k + j) * a.H + n], acc);
  }
  static_cast<__nv_bfloat16*>(a.y)[static_cast<int64_t>(t) * a.ld_y + n] = __float2bfloat16_rn(acc);
}

}  // namespace

size_t moe_workspace_need(int T, int k, int E, int H, int I, int fmt) { return moe_ws_layout(T, k, H, I).total; }

cudaError_t launch_moe_mlp(const MoeArgs& a, int fmt, int num_sms, cudaStream_t s) {
  const MoeWs L = moe_ws_layout(a.T, a.k, a.H, a.I);
  const uint8_t* xq = static_cast<const uint8_t*>(a.x);
  const void* xs = a.x_scale;
  if (xs == nullptr) {
    ActQuantArgs q{};
    q.x = a.x;
    q.ld_x = a.ld_x;
    q.M = a.T;
    q.K = a.H;
    q.Kb = (a.H + 127) / 128;
    q.xq = a.ws + L.xq;
    q.xs = a.ws + L.xs;
    q.layout = kScaleRowMajor;
    if (const cudaError_t e = launch_act_quant(q, fmt, num_sms, s); e != cudaSuccess) return e;
    xq = a.ws + L.xq;
    xs = a.ws + L.xs;
  }
  uint8_t* hq = a.ws + L.hq;
  float* hs = reinterpret_cast<float*>(a.ws + L.hs);
  float* part = reinterpret_cast<float*>(a.ws + L.part);
  const dim3 up((a.I + 127) / 128, a.T * a.k), down((a.H + 127) / 128, a.T * a.k), comb((a.H + 255) / 256, a.T);
  if (fmt == 0) {
    moe_up_kernel<0><<<up, 256, 0, s>>>(a, xq, xs, hq, hs);
    moe_down_kernel<0><<<down, 256, 0, s>>>(a, hq, hs, part);
  } else {
    moe_up_kernel<1><<<up, 256, 0, s>>>(a, xq, xs, hq, hs);
    moe_down_kernel<1><<<down, 256, 0, s>>>(a, hq, hs, part);
  }
  moe_combine_kernel<<<comb, 256, 0, s>>>(a, part);
  return cudaGetLastError();
}

}  // namespace fg8
