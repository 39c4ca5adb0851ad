// norm_act.cu -- what stands in front of the FP8 linears of a transformer
// block, fused with the activation quantization: RMS norm with the
// residual's addition, and silu(gate) * up (sm_100a).
//
//   rmsnorm:  z = x + residual;  v = z * (1 / sqrt(mean(z^2) + eps)) * weight
//   silu_mul: v = gate / (1 + exp(-gate)) * up
//
// then, per token and group of 128 (64, 32) channels, the scale and codes of
// quant_math.cuh.  All of it is float32 and v is never rounded to bf16 on
// its way to the codes: a bf16 step in between would move a group's amax, and
// with it every code of the group, by up to 2^-9.  bf16 outputs (the new
// residual z, v itself) are rounded once.
//
// Both are streams bound by HBM: 16-byte loads and stores, 16 channels per
// thread and step, everything between in registers.

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "fg8_internal.h"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace fg8 {
namespace {

using namespace qm;

__device__ __forceinline__ void load16(const uint16_t* p, float (&f)[16]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + 8);
  float lo[8], hi[8];
  unpack_bf16x8(a, lo);
  unpack_bf16x8(b, hi);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[i] = lo[i];
    f[8 + i] = hi[i];
  }
}

__device__ __forceinline__ void store16(uint16_t* p, const float (&f)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w[i] = static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(f[2 * i]))) |
           (static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(f[2 * i + 1]))) << 16);
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(p + 8) = make_uint4(w[4], w[5], w[6], w[7]);
}

// One thread's 16 channels of a group owned by GL neighbouring lanes: the
// group's amax over the lanes, scale, codes.  Every lane of the warp calls
// it (lanes without channels pass zeros and `real` false).
template <int FMT, int GL>
__device__ __forceinline__ void quantize_group(const NormActArgs& a, const float (&v)[16], int64_t m, int k, int l,
                                               bool real) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
  for (int off = GL / 2; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, off));
  const float s = group_scale(amax);
  const uint32_t sbyte = FMT == 1 ? e8m0_ceil_byte(s) : 0u;
  const uint4 q = quantize16<FMT>(v, s, sbyte);
  if (!real) return;
  *reinterpret_cast<uint4*>(a.xq + m * a.K + k) = q;
  if (a.y != nullptr) store16(static_cast<uint16_t*>(a.y) + m * a.ld_y + k, v);
  if (l == 0) {
    const int64_t g = m * a.Kb + k / (16 * GL);
    if (FMT == 0) static_cast<float*>(a.xs)[g] = s;
    else static_cast<uint8_t*>(a.xs)[g] = static_cast<uint8_t>(sbyte);
  }
}

// ------------------------------------------------------------- rms norm ----
// One CTA of THREADS threads per token; thread t owns channels 16 (t + i
// THREADS) .. + 15, kept in registers between the sum of squares and the
// quantization (up to CH steps; longer rows are read twice).
template <int FMT, int GL, int THREADS, int CH>
__global__ void __launch_bounds__(THREADS) rmsnorm_quant_kernel(const NormActArgs a) {
  __shared__ float red[THREADS / 32];
  grid_wait_prerequisites();
  grid_launch_dependents();
  const int t = threadIdx.x, l = t % GL;
  const int64_t m = blockIdx.x;
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + m * a.ld_x;
  const uint16_t* r = a.x2 != nullptr ? static_cast<const uint16_t*>(a.x2) + m * a.ld_x2 : nullptr;
  const uint16_t* w = static_cast<const uint16_t*>(a.weight);
  const int steps = (a.K + 16 * THREADS - 1) / (16 * THREADS);

  auto load = [&](int i, float (&z)[16]) {
    const int k = 16 * (t + i * THREADS);
    if (k < a.K) {
      load16(x + k, z);
      if (r != nullptr) {
        float f[16];
        load16(r + k, f);
#pragma unroll
        for (int j = 0; j < 16; ++j) z[j] += f[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) z[j] = 0.0f;
    }
  };

  float z[CH][16];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < CH; ++i) load(i, z[i]);
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) ss = fmaf(z[i][j], z[i][j], ss);
  for (int i = CH; i < steps; ++i) {
    float e[16];
    load(i, e);
#pragma unroll
    for (int j = 0; j < 16; ++j) ss = fmaf(e[j], e[j], ss);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, off);
  if (THREADS > 32) {
    if ((t & 31) == 0) red[t >> 5] = ss;
    __syncthreads();
    ss = 0.0f;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) ss += red[i];
  }
  const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(ss, static_cast<float>(a.K)) + a.eps));

  auto finish = [&](int i, float (&e)[16]) {
    const int k = 16 * (t + i * THREADS);
    const bool real = k < a.K;
    if (real) {
      if (a.x2_out != nullptr) store16(static_cast<uint16_t*>(a.x2_out) + m * a.ld_x2_out + k, e);
      float g[16];
      load16(w + k, g);
#pragma unroll
      for (int j = 0; j < 16; ++j) e[j] = e[j] * rstd * g[j];
    }
    quantize_group<FMT, GL>(a, e, m, k, l, real);
  };
#pragma unroll
  for (int i = 0; i < CH; ++i)
    if (i < steps) finish(i, z[i]);
  for (int i = CH; i < steps; ++i) {
    float e[16];
    load(i, e);
    finish(i, e);
  }
}

// ------------------------------------------------------------- silu_mul ----
// Groups of 16 GL channels, GL neighbouring lanes each; a grid-stride loop
// over all groups (the group of a lane: (m, kb) = (g / Kb, g % Kb)).
template <int FMT, int GL>
__global__ void __launch_bounds__(256) silu_mul_quant_kernel(const NormActArgs a, const int64_t total) {
  grid_wait_prerequisites();
  grid_launch_dependents();
  constexpr int kGpw = 32 / GL;
  const int lane = threadIdx.x & 31, oct = lane / GL, l = lane % GL;
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t nwarps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
  for (int64_t base = warp * kGpw; base < total; base += nwarps * kGpw) {
    const int64_t g = base + oct;
    const int64_t m = g / a.Kb;
    const int k = static_cast<int>(g - m * a.Kb) * (16 * GL) + l * 16;
    const bool real = g < total && k < a.K;
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.0f;
    if (real) {
      float u[16];
      load16(static_cast<const uint16_t*>(a.x) + m * a.ld_x + k, v);
      load16(static_cast<const uint16_t*>(a.x2) + m * a.ld_x2 + k, u);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = silu_mul(v[i], u[i]);
    }
    quantize_group<FMT, GL>(a, v, m, k, l, real);
  }
}

template <int FMT, int GL>
cudaError_t launch_rms(const NormActArgs& a, cudaLaunchConfig_t& cfg) {
  const int n16 = (a.K + 15) / 16;
  cfg.gridDim = dim3(static_cast<unsigned>(a.M));
#define FG8_RMS(T, C) \
  { cfg.blockDim = dim3(T); return cudaLaunchKernelEx(&cfg, rmsnorm_quant_kernel<FMT, GL, T, C>, a); }
  if (n16 <= 32) FG8_RMS(32, 1)
  if (n16 <= 64) FG8_RMS(64, 1)
  if (n16 <= 128) FG8_RMS(128, 1)
  if (n16 <= 256) FG8_RMS(256, 1)
  if (n16 <= 512) FG8_RMS(256, 2)
  if (n16 <= 768) FG8_RMS(256, 3)
  FG8_RMS(512, 3)
#undef FG8_RMS
}

}  // namespace

cudaError_t launch_rmsnorm_quant(const NormActArgs& a, int fmt, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaErrorInvalidValue;
  if (a.group == 128) e = fmt == 0 ? launch_rms<0, 8>(a, cfg) : launch_rms<1, 8>(a, cfg);
  else if (a.group == 64) e = fmt == 0 ? launch_rms<0, 4>(a, cfg) : launch_rms<1, 4>(a, cfg);
  else if (a.group == 32) e = fmt == 0 ? launch_rms<0, 2>(a, cfg) : launch_rms<1, 2>(a, cfg);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t launch_silu_mul_quant(const NormActArgs& a, int fmt, int num_sms, cudaStream_t s) {
  const int64_t total = static_cast<int64_t>(a.M) * a.Kb;
  const int64_t per_block = 8 * (32 / (a.group / 16));
  int64_t blocks = (total + per_block - 1) / per_block;
  const int64_t cap = static_cast<int64_t>(num_sms) * 8;
  if (blocks > cap) blocks = cap;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaErrorInvalidValue;
#define FG8_SM(F, GL) cudaLaunchKernelEx(&cfg, silu_mul_quant_kernel<F, GL>, a, total)
  if (a.group == 128) e = fmt == 0 ? FG8_SM(0, 8) : FG8_SM(1, 8);
  else if (a.group == 64) e = fmt == 0 ? FG8_SM(0, 4) : FG8_SM(1, 4);
  else if (a.group == 32) e = fmt == 0 ? FG8_SM(0, 2) : FG8_SM(1, 2);
#undef FG8_SM
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace fg8
