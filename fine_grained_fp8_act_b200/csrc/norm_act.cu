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
// with it every code of the group, by up to 2^-8.  bf16 outputs (the new
// residual z, v itself) are rounded once.
//
// Both are streams bound by HBM.  A lane owns 8 neighbouring channels (16
// bytes of bf16), so a group is 16, 8 or 4 lanes.

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <atomic>

#include "fg8_internal.h"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace fg8 {
namespace {

using namespace qm;

constexpr float kInf = __builtin_huge_valf();

__device__ __forceinline__ void unpack8(const uint4& v, float2 (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

__device__ __forceinline__ uint4 pack8(const float2 (&f)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __float22bfloat162_rn(f[i]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint4 flip_signs(const uint4& v) {  // of 8 packed bf16
  return make_uint4(v.x ^ 0x80008000u, v.y ^ 0x80008000u, v.z ^ 0x80008000u, v.w ^ 0x80008000u);
}

__device__ __forceinline__ uint4 ldg16(const void* p, int64_t at) {
  return *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
}

// The scale of token m's group g: row-major, or where the GEMM reads it, which
// then needs no pass of its own over the scales.  In a scale-factor tile the
// slots past the last group are set to 2^0 together with it.
// ROW: known to be row-major (the stream kernels have no register to spare).
template <int FMT, bool ROW>
__device__ __forceinline__ void store_scale(const NormActArgs& a, int64_t m, int g, float s, uint32_t sbyte) {
  if (ROW || a.layout == kScaleRowMajor) {
    if (FMT == 0) static_cast<float*>(a.xs)[m * a.Kb + g] = s;
    else static_cast<uint8_t*>(a.xs)[m * a.Kb + g] = static_cast<uint8_t>(sbyte);
  } else if (FMT == 0) {
    static_cast<float*>(a.xs)[g * a.ld_s + m] = s;
  } else {
    uint8_t* t = static_cast<uint8_t*>(a.xs) + sf_tile_offset(m, g, a.Kq);
    *t = static_cast<uint8_t>(sbyte);
    if (g == a.Kb - 1)
      for (int j = g + 1; (j & 3) != 0; ++j) *++t = 127u;
  }
}

// Rows past the last token of a scale-factor tile: 2^0 in every slot.
__device__ __forceinline__ void pad_scales(const NormActArgs& a, int64_t m, int from, int step) {
  for (int q = from; q < a.Kq; q += step)
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.xs) + sf_tile_offset(m, 4 * q, a.Kq)) = 0x7F7F7F7Fu;
}

// A lane's 8 channels k .. k + 7 of token m, as n = -v (quantize_negated):
// the group's amax over its lanes (a.group / 8 neighbours), scale, codes, and
// v in bf16 on request.  Every lane of the warp calls it (lanes without
// channels: zeros, `real` false).
template <int FMT>
__device__ __forceinline__ void quantize_lane(const NormActArgs& a, const float2 (&n)[4], int64_t m, int k, bool real) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) amax = fmaxf(amax, fmaxf(fabsf(n[i].x), fabsf(n[i].y)));
  amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
  if (a.group >= 64) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 4));
  if (a.group >= 128) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 8));
  const float s = group_scale_fast(amax);
  const uint32_t sbyte = FMT == 1 ? e8m0_ceil_byte(s) : 0u;
  uint32_t q[2];
  quantize_negated<FMT, 4>(n, s, sbyte, q);
  if (!real) return;
  *reinterpret_cast<uint2*>(a.xq + m * a.K + k) = make_uint2(q[0], q[1]);
  if (a.y != nullptr) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + m * a.ld_y + k) = flip_signs(pack8(n));
  if ((k & (a.group - 1)) == 0) store_scale<FMT, false>(a, m, k >> a.group_shift, s, sbyte);
}

__device__ __forceinline__ float square_sum(const float2 (&z)[4], float ss) {
  float2 t = make_float2(ss, 0.0f);
#pragma unroll
  for (int i = 0; i < 4; ++i) t = __ffma2_rn(z[i], z[i], t);
  return t.x + t.y;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
  return v;
}

__device__ __forceinline__ float row_mean(const NormActArgs& a, float ss) { return fmaf(ss, a.inv_k, a.eps); }

// 1 / sqrt(m) of a finite m: the hardware's approximation (2^-22.9) and one
// Newton step, y + y/2 (1 - m y y), good to an ulp or so.
__device__ __forceinline__ float rstd_of(float m) {
  const float y = rsqrtf(m);
  return fmaf(0.5f * y, fmaf(-m * y, y, 1.0f), y);
}

// Rows of finite z whose m does not fit float32 (|z| from some 2^64 / sqrt(K)
// on, or a large eps) take the squares of z 2^-80: at most 2^96, K of them
// 2^126, while what underflows (|z| < 2^6) is nothing beside 2^128 / K.  Above
// an rms of 2^126 the result is subnormal: 4 U off in place of a rounding's U.
// (An infinite z: 0, so that finite elements become zeros and it NaN.)
// Up to 3% slower than without, where there is no residual: 16384 x 12288 134
// us against 131, one token of 2048 1.63 against 1.57.
constexpr float kDown = 8.27180612553027674871e-25f;  // 2^-80
__device__ __forceinline__ float rstd_of_down(const NormActArgs& a, float ss_down) {
  const float m = fmaf(ss_down, a.inv_k, a.eps * kDown * kDown);
  return m < kInf ? rstd_of(m) * kDown : 0.0f;
}

__device__ __forceinline__ float square_sum_down(const float2 (&z)[4], float ss) {
  float2 d[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] = __fmul2_rn(z[i], make_float2(kDown, kDown));
  return square_sum(d, ss);
}

// z of a lane's 8 channels, once the row's 1 / rms is known: the new
// residual, v = z rstd weight, codes.
template <int FMT>
__device__ __forceinline__ void finish_norm(const NormActArgs& a, float2 (&z)[4], const uint4& w, float rstd, int64_t m,
                                            int k, bool real) {
  if (real && a.x2_out != nullptr)
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.x2_out) + m * a.ld_x2_out + k) = pack8(z);
  float2 g[4];
  unpack8(w, g);
#pragma unroll
  for (int i = 0; i < 4; ++i) z[i] = __fmul2_rn(__fmul2_rn(z[i], make_float2(-rstd, -rstd)), g[i]);
  quantize_lane<FMT>(a, z, m, k, real);
}

// ---------------------------------------------------- rms norm, one row ----
// Few tokens (or rows past the stream kernel's length): one CTA per token,
// channels 8 (t + i THREADS) .. + 7 in thread t, plain loads, all of them in
// flight at once; rows longer than 8 THREADS CH are read twice.
template <int FMT, int THREADS, int CH>
__global__ void __launch_bounds__(THREADS) rmsnorm_row_kernel(const NormActArgs a) {
  __shared__ float red[2][THREADS / 32];
  grid_wait_prerequisites();
  grid_launch_dependents();
  const int t = threadIdx.x;
  const int64_t m = blockIdx.x;
  if (m >= a.M) return pad_scales(a, m, t, THREADS);
  const int steps = (a.K + 8 * THREADS - 1) / (8 * THREADS);
  auto load = [&](int i, float2 (&z)[4]) {
    const int k = 8 * (t + i * THREADS);
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (k < a.K) v = ldg16(a.x, m * a.ld_x + k);
    unpack8(v, z);
    if (a.x2 != nullptr && k < a.K) {
      float2 f[4];
      unpack8(ldg16(a.x2, m * a.ld_x2 + k), f);
#pragma unroll
      for (int j = 0; j < 4; ++j) z[j] = __fadd2_rn(z[j], f[j]);
    }
  };
  auto weight = [&](int i) {
    const int k = 8 * (t + i * THREADS);
    return k < a.K ? ldg16(a.weight, k) : make_uint4(0u, 0u, 0u, 0u);
  };
  float2 z[CH][4];
  uint4 w[CH];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    load(i, z[i]);
    w[i] = weight(i);
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) ss = square_sum(z[i], ss);
  for (int i = CH; i < steps; ++i) {
    float2 e[4];
    load(i, e);
    ss = square_sum(e, ss);
  }
  auto row_sum = [&](float v, int set) {
    v = warp_sum(v);
    if (THREADS > 32) {
      if ((t & 31) == 0) red[set][t >> 5] = v;
      __syncthreads();
      v = warp_sum((t & 31) < THREADS / 32 ? red[set][t & 31] : 0.0f);
    }
    return v;
  };
  const float mean = row_mean(a, row_sum(ss, 0));
  float rstd = rstd_of(mean);
  if (mean == kInf) {  // the same in every thread
    ss = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i) ss = square_sum_down(z[i], ss);
    for (int i = CH; i < steps; ++i) {
      float2 e[4];
      load(i, e);
      ss = square_sum_down(e, ss);
    }
    rstd = rstd_of_down(a, row_sum(ss, 1));
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int k = 8 * (t + i * THREADS);
    finish_norm<FMT>(a, z[i], w[i], rstd, m, k, k < a.K);
  }
  for (int i = CH; i < steps; ++i) {
    const int k = 8 * (t + i * THREADS);
    float2 e[4];
    load(i, e);
    finish_norm<FMT>(a, e, weight(i), rstd, m, k, k < a.K);
  }
}

// ------------------------------------------------------------ streaming ----
// Many tokens: one CTA per SM, all warps streaming.  A warp copies what it
// will read (cp.async, 16 bytes a lane) NBUF items ahead through a ring of
// its own in shared memory, so that up to 190 KB per SM are in flight without
// a register spent on them and without a barrier between warps.  An item is S
// steps of 512 channels; a lane owns 16 neighbouring channels of a step,
// which halves the per-group work (scale, reciprocal, amax steps) against 8.
// The copies are made in address order, piece p of 16 bytes by lane p % 32,
// and stored at piece p ^ (p / 8 % 2): a lane's two pieces, 2 l and 2 l + 1,
// are then read without bank conflicts.
constexpr int kStreamSmem = 192 * 1024;

struct LanePieces {
  int put[2], get[2];  // byte offsets in a step's 1 KB: where this lane's copies go, where its channels are
  __device__ __forceinline__ explicit LanePieces(int lane) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int p = lane + 32 * h, g = 2 * lane + h;
      put[h] = (p ^ ((p >> 3) & 1)) * 16;
      get[h] = (g ^ ((g >> 3) & 1)) * 16;
    }
  }
};

__device__ __forceinline__ void lds_channels(const uint8_t* src, const LanePieces& lp, bool real, float2 (&f)[8]) {
  uint4 v[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  if (real) {
    v[0] = *reinterpret_cast<const uint4*>(src + lp.get[0]);
    v[1] = *reinterpret_cast<const uint4*>(src + lp.get[1]);
  }
  float2 lo[4], hi[4];
  unpack8(v[0], lo);
  unpack8(v[1], hi);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = lo[i], f[4 + i] = hi[i];
}

// 16 values to global memory as bf16.
template <bool FLIP>
__device__ __forceinline__ void store_channels(uint16_t* p, const float2 (&f)[8]) {
  const float2 lo[4] = {f[0], f[1], f[2], f[3]}, hi[4] = {f[4], f[5], f[6], f[7]};
  const uint4 a = pack8(lo), b = pack8(hi);
  *reinterpret_cast<uint4*>(p) = FLIP ? flip_signs(a) : a;
  *reinterpret_cast<uint4*>(p + 8) = FLIP ? flip_signs(b) : b;
}

// quantize_lane for 16 channels (a group is 8, 4 or 2 lanes); `lead`: the
// lane stores its group's scale.
template <int FMT, bool ROW>
__device__ __forceinline__ void quantize_channels(const NormActArgs& a, const float2 (&n)[8], int64_t m, int k,
                                                  bool lead, bool real) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fmaxf(fabsf(n[i].x), fabsf(n[i].y)));
  amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
  if (a.group >= 64) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
  if (a.group >= 128) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 4));
  const float s = group_scale_fast(amax);
  const uint32_t sbyte = FMT == 1 ? e8m0_ceil_byte(s) : 0u;
  uint32_t q[4];
  quantize_negated<FMT, 8>(n, s, sbyte, q);
  if (!real) return;
  *reinterpret_cast<uint4*>(a.xq + m * a.K + k) = make_uint4(q[0], q[1], q[2], q[3]);
  if (a.y != nullptr) store_channels<true>(static_cast<uint16_t*>(a.y) + m * a.ld_y + k, n);
  if (lead) store_scale<FMT, ROW>(a, m, k >> a.group_shift, s, sbyte);
}

// RMS norm: a team of W warps per token (up to 32 / W tokens at a time); the
// team's sum of squares meets in shared memory at the team's own barrier.
// warps of a CTA at most: rings of four two-operand items leave room for 24
constexpr int rms_warps(int S, int OPS, int NBUF) { return S == 2 || OPS * NBUF == 8 ? 24 : 32; }

template <int FMT, int S, int OPS, int NBUF, bool ROW>
__global__ void __launch_bounds__(rms_warps(S, OPS, NBUF) * 32, 1) rmsnorm_stream_kernel(const NormActArgs a, const int W) {
  constexpr int kItem = S * OPS * 1024;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[2][32];
  grid_wait_prerequisites();
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int teams = static_cast<int>(blockDim.x >> 5) / W, team = warp / W, wt = warp - team * W;
  const LanePieces lp(lane);
  uint8_t* mine = ring + warp * NBUF * kItem;
  const int base = wt * S * 512;  // the warp's channels: S steps of 512
  const int k0 = base + lane * 16;
  // the weight of one step stays in registers; of two it would spill (48 to 92
  // bytes: 16384 x 12288 with a residual 229 us), and comes out of L1 for
  // every token (216)
  uint4 held[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  if (S == 1 && k0 < a.K) held[0] = ldg16(a.weight, k0), held[1] = ldg16(a.weight, k0 + 8);
  // (M < 2^31 and the stride is at most 148 x 32: 32 unsigned bits hold both)
  const uint32_t stride = gridDim.x * teams, first = blockIdx.x * teams + team, M = a.M;
  uint32_t mi = first;  // the next token to copy
  const uint16_t* px = static_cast<const uint16_t*>(a.x) + first * a.ld_x + base + lane * 8;
  const uint16_t* pr = static_cast<const uint16_t*>(a.x2) + first * a.ld_x2 + base + lane * 8;
  auto issue = [&](int buf) {
    if (mi < M) {
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (base + s * 512 + h * 256 + lane * 8 < a.K) {
            uint8_t* dst = mine + buf * kItem + s * OPS * 1024 + lp.put[h];
            cp_async16(dst, px + s * 512 + h * 256);
            if (OPS == 2) cp_async16(dst + 1024, pr + s * 512 + h * 256);
          }
      mi += stride;
      px += stride * a.ld_x;
      if (OPS == 2) pr += stride * a.ld_x2;
    }
    cp_async_commit();  // empty past the end: the count of groups stays that of the items
  };
#pragma unroll
  for (int n = 0; n < NBUF - 1; ++n) issue(n);
  const bool lead = (k0 & (a.group - 1)) == 0;
  int buf = 0, ahead = NBUF - 1, flip = 0;
  for (uint32_t m = first; m < M; m += stride) {
    __syncwarp();  // every lane has read the buffer that is filled now
    issue(ahead);
    cp_async_wait_group<NBUF - 1>();
    __syncwarp();
    float2 z[S][8];
    float2 ss = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const uint8_t* src = mine + buf * kItem + s * OPS * 1024;
      const bool real = k0 + s * 512 < a.K;
      lds_channels(src, lp, real, z[s]);
      if (OPS == 2) {
        float2 f[8];
        lds_channels(src + 1024, lp, real, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[s][j] = __fadd2_rn(z[s][j], f[j]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = __ffma2_rn(z[s][j], z[s][j], ss);
    }
    auto team_sum = [&](float v) {
      v = warp_sum(v);
      if (W > 1) {
        // two sets in turn: a warp ahead by one sum writes the other one
        if (lane == 0) red[flip][warp] = v;
        named_barrier_sync(team, W * 32);  // at most 16 teams, 16 barriers: the CTA's own (0) is not used here
        v = warp_sum(lane < W ? red[flip][team * W + lane] : 0.0f);
        flip ^= 1;
      }
      return v;
    };
    const float mean = row_mean(a, team_sum(ss.x + ss.y));
    float rstd = rstd_of(mean);
    if (mean == kInf) {  // the same in the whole team
      ss = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 d = __fmul2_rn(z[s][j], make_float2(kDown, kDown));
          ss = __ffma2_rn(d, d, ss);
        }
      rstd = rstd_of_down(a, team_sum(ss.x + ss.y));
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const bool real = k0 + s * 512 < a.K;
      const int k = k0 + s * 512;
      if (OPS == 2 && real) store_channels<false>(static_cast<uint16_t*>(a.x2_out) + m * a.ld_x2_out + k, z[s]);
      uint4 w[2] = {held[0], held[1]};
      if (S > 1 && real) w[0] = ldg16(a.weight, k), w[1] = ldg16(a.weight, k + 8);
      float2 lo[4], hi[4];
      unpack8(w[0], lo);
      unpack8(w[1], hi);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        z[s][j] = __fmul2_rn(__fmul2_rn(z[s][j], make_float2(-rstd, -rstd)), j < 4 ? lo[j & 3] : hi[j & 3]);
      quantize_channels<FMT, ROW>(a, z[s], m, k, lead, real);
    }
    buf = buf + 1 == NBUF ? 0 : buf + 1;
    ahead = ahead + 1 == NBUF ? 0 : ahead + 1;
  }
  if (!ROW && a.layout == kScaleSfTiles)
    for (int m = a.M + blockIdx.x; m < a.M_pad; m += gridDim.x) pad_scales(a, m, threadIdx.x, blockDim.x);
}

// silu(gate) * up: an item is 512 channels of a token (the last of a token
// may be shorter).
constexpr int kSiluWarps = 32, kSiluBuffers = 3;

template <int FMT, bool ROW>
__global__ void __launch_bounds__(kSiluWarps * 32, 1) silu_mul_stream_kernel(const NormActArgs a, const int per_row,
                                                                             const int64_t items) {
  constexpr int kItem = 2048, NBUF = kSiluBuffers;
  static_assert(kSiluWarps * NBUF * kItem <= kStreamSmem, "ring");
  extern __shared__ __align__(16) uint8_t ring[];
  grid_wait_prerequisites();
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const LanePieces lp(lane);
  uint8_t* mine = ring + warp * NBUF * kItem;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kSiluWarps;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kSiluWarps + warp;
  // (token, item of it) of the next copy and of the next result; both step by
  // stride items, the token's share of which is divided once
  const int64_t dm = stride / per_row;
  const int dj = static_cast<int>(stride - dm * per_row);
  int64_t mi = first / per_row, mo = mi;
  int ji = static_cast<int>(first - mi * per_row), jo = ji;
  auto step = [&](int64_t& m, int& j) {
    m += dm;
    j += dj;
    if (j >= per_row) {
      j -= per_row;
      ++m;
    }
  };
  auto issue = [&](int buf) {
    if (mi < a.M) {
      const int k = ji * 512 + lane * 8;
      const uint16_t* g = static_cast<const uint16_t*>(a.x) + mi * a.ld_x + k;
      const uint16_t* u = static_cast<const uint16_t*>(a.x2) + mi * a.ld_x2 + k;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (k + h * 256 < a.K) {
          uint8_t* dst = mine + buf * kItem + lp.put[h];
          cp_async16(dst, g + h * 256);
          cp_async16(dst + 1024, u + h * 256);
        }
      step(mi, ji);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int n = 0; n < NBUF - 1; ++n) issue(n);
  const bool lead = (lane * 16 & (a.group - 1)) == 0;
  int buf = 0, ahead = NBUF - 1;
  for (int64_t i = first; i < items; i += stride) {
    __syncwarp();
    issue(ahead);
    cp_async_wait_group<NBUF - 1>();
    __syncwarp();
    const int k = jo * 512 + lane * 16;
    const bool real = k < a.K;
    const uint8_t* src = mine + buf * kItem;
    float2 v[8], u[8];
    lds_channels(src, lp, real, v);
    lds_channels(src + 1024, lp, real, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = silu_mul2<true>(v[j], u[j]);
    quantize_channels<FMT, ROW>(a, v, mo, k, lead, real);
    step(mo, jo);
    buf = buf + 1 == NBUF ? 0 : buf + 1;
    ahead = ahead + 1 == NBUF ? 0 : ahead + 1;
  }
  if (!ROW && a.layout == kScaleSfTiles)
    for (int m = a.M + blockIdx.x; m < a.M_pad; m += gridDim.x) pad_scales(a, m, threadIdx.x, blockDim.x);
}

template <int FMT>
__device__ __forceinline__ void finish_silu(const NormActArgs& a, const uint4& g, const uint4& u, int64_t m, int k,
                                            bool real) {
  float2 v[4], f[4];
  unpack8(g, v);
  unpack8(u, f);
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = silu_mul2<true>(v[j], f[j]);
  quantize_lane<FMT>(a, v, m, k, real);
}

// Few tokens: a warp per 256 channels, plain loads.
template <int FMT>
__global__ void __launch_bounds__(128) silu_mul_row_kernel(const NormActArgs a, const int per_row, const int64_t items) {
  grid_wait_prerequisites();
  grid_launch_dependents();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int64_t m = i / per_row;
  if (a.layout == kScaleSfTiles && m >= a.M) {  // items past the tokens' own: one per padding row and 256 channels
    if (m < a.M_pad) pad_scales(a, m, static_cast<int>(i - m * per_row) * 32 + (threadIdx.x & 31), per_row * 32);
    return;
  }
  if (i >= items) return;
  const int k = static_cast<int>(i - m * per_row) * 256 + (threadIdx.x & 31) * 8;
  const bool real = k < a.K;
  uint4 g = make_uint4(0u, 0u, 0u, 0u), u = g;
  if (real) {
    g = ldg16(a.x, m * a.ld_x + k);
    u = ldg16(a.x2, m * a.ld_x2 + k);
  }
  finish_silu<FMT>(a, g, u, m, k, real);
}

// Launch with the stream's dynamic shared memory (opted in once per device).
template <class... P, class... A>
cudaError_t launch_stream(void (*kern)(P...), std::atomic<uint64_t>& configured, int warps, cudaLaunchConfig_t& cfg,
                          A... args) {
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = 1ull << (dev & 63);
  if ((configured.load(std::memory_order_acquire) & bit) == 0) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamSmem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_release);
  }
  cfg.blockDim = dim3(static_cast<unsigned>(warps * 32));
  cfg.dynamicSmemBytes = kStreamSmem;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int FMT, int S, int OPS, int NBUF>
cudaError_t rms_stream(const NormActArgs& a, int W, int warps, cudaLaunchConfig_t& cfg) {
  static std::atomic<uint64_t> configured[2];
  if (warps * NBUF * S * OPS * 1024 > kStreamSmem) return cudaErrorInvalidValue;
  if (a.layout == kScaleRowMajor)
    return launch_stream(rmsnorm_stream_kernel<FMT, S, OPS, NBUF, true>, configured[0], warps, cfg, a, W);
  return launch_stream(rmsnorm_stream_kernel<FMT, S, OPS, NBUF, false>, configured[1], warps, cfg, a, W);
}

template <int FMT>
cudaError_t launch_rms(const NormActArgs& a, int num_sms, cudaLaunchConfig_t& cfg) {
  const int n = (a.K + 511) / 512;  // steps of 512 channels in a row
  // Two steps a warp: fewer shuffles and barriers a channel.  Up to eight
  // steps it makes no difference, and for 25 to 32 there would be one team of
  // 16 warps at most.  us, two steps / one, float scales, 16384 tokens with a
  // residual and without: x 12288 216 / 234, 134 / 148; x 8192 146 / 157,
  // 91 / 93; x 5632 104 / 105, 68 / 73; but x 6144 121 / 116, 69 / 75.
  const int S = n <= 8 || (n > 24 && n <= 32) ? 1 : 2, W = (n + S - 1) / S;
  const int most = S == 1 ? 32 : 24;
  if (W <= most) {
    const int teams = most / W, warps = teams * W;  // (16 teams at most where W > 1: 16 hardware barriers)
    // The rings pay from a few tokens on; below that the one-row kernel has
    // more loads in flight.  Times of row kernel / stream, without and with a
    // residual: two steps a warp (by tokens an SM) 300 x 7168 (2) 1.39, 1.12;
    // 450 x 7168 (3) 1.20, 0.95; 300 x 12288 (2) 1.16, 0.89; 450 x 12288 (3)
    // 1.43, 1.10; one step (by tokens a team) 900 x 4096 (1.5) 1.17, 0.84; 2400
    // x 4096 (4) 1.39, 0.98; 3600 x 4096 (6) 1.52, 1.35; 2400 x 2048 (2) 0.99,
    // 0.73; and 16384 x 512 with one (3) 1.6.
    const int halves = S == 2 ? (a.x2 == nullptr ? 4 : 6) : (n == 1 ? 4 : a.x2 == nullptr ? 3 : 8) * teams;
    if (2 * static_cast<int64_t>(a.M) >= static_cast<int64_t>(halves) * num_sms) {
      cfg.gridDim = dim3(static_cast<unsigned>(num_sms));
      if (a.x2 == nullptr)
        return S == 1 ? rms_stream<FMT, 1, 1, 4>(a, W, warps, cfg) : rms_stream<FMT, 2, 1, 4>(a, W, warps, cfg);
      if (S == 2) return rms_stream<FMT, 2, 2, 2>(a, W, warps, cfg);
      return warps <= 24 ? rms_stream<FMT, 1, 2, 4>(a, W, warps, cfg) : rms_stream<FMT, 1, 2, 3>(a, W, warps, cfg);
    }
  }
  cfg.gridDim = dim3(static_cast<unsigned>(a.layout == kScaleSfTiles ? a.M_pad : a.M));
#define FG8_RMS(T, C) \
  { cfg.blockDim = dim3(T); return cudaLaunchKernelEx(&cfg, rmsnorm_row_kernel<FMT, T, C>, a); }
  if (a.K <= 256) FG8_RMS(32, 1)
  if (a.K <= 512) FG8_RMS(64, 1)
  if (a.K <= 1024) FG8_RMS(128, 1)
  if (a.K <= 2048) FG8_RMS(256, 1)
  if (a.K <= 4096) FG8_RMS(512, 1)
  if (a.K <= 8192) FG8_RMS(1024, 1)
  if (a.K <= 12288) FG8_RMS(768, 2)
  FG8_RMS(1024, 2)
#undef FG8_RMS
}

template <int FMT>
cudaError_t launch_silu(const NormActArgs& a, int num_sms, cudaLaunchConfig_t& cfg) {
  const int per_row = (a.K + 511) / 512;
  // us, stream / row kernel, float scales: 512 x 14336 (3 items a warp) 10.4 /
  // 9.2, 1024 x 14336 (6) 16.6 / 16.8, 8192 x 2048 (7) 16.9 / 19.0
  if (static_cast<int64_t>(a.M) * per_row >= static_cast<int64_t>(6) * num_sms * kSiluWarps) {
    static std::atomic<uint64_t> configured[2];
    const int64_t items = static_cast<int64_t>(a.M) * per_row;
    cfg.gridDim = dim3(static_cast<unsigned>(num_sms));
    if (a.layout == kScaleRowMajor)
      return launch_stream(silu_mul_stream_kernel<FMT, true>, configured[0], kSiluWarps, cfg, a, per_row, items);
    return launch_stream(silu_mul_stream_kernel<FMT, false>, configured[1], kSiluWarps, cfg, a, per_row, items);
  }
  const int row = (a.K + 255) / 256;
  const int64_t items = static_cast<int64_t>(a.M) * row;
  const int64_t warps = a.layout == kScaleSfTiles ? static_cast<int64_t>(a.M_pad) * row : items;
  cfg.gridDim = dim3(static_cast<unsigned>((warps + 3) / 4));
  cfg.blockDim = dim3(128);
  return cudaLaunchKernelEx(&cfg, silu_mul_row_kernel<FMT>, a, row, items);
}

cudaLaunchConfig_t overlapped(cudaLaunchAttribute (&attr)[1], cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

}  // namespace

cudaError_t launch_rmsnorm_quant(const NormActArgs& a, int fmt, int num_sms, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = overlapped(attr, s);
  const cudaError_t e = fmt == 0 ? launch_rms<0>(a, num_sms, cfg) : launch_rms<1>(a, num_sms, cfg);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t launch_silu_mul_quant(const NormActArgs& a, int fmt, int num_sms, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = overlapped(attr, s);
  const cudaError_t e = fmt == 0 ? launch_silu<0>(a, num_sms, cfg) : launch_silu<1>(a, num_sms, cfg);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace fg8
