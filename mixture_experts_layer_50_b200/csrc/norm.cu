// Residual RMS norm with an optional 8-bit output: the row that a layer's router and experts
// read.
//
//   s = x + residual                         (fp32; residual_out = s rounded to the row type)
//   y = s * rsqrt(mean(s^2) + eps) * weight  (fp32; y rounded once to the row type)
//   c = amax(|y| over a group) / 448,  y8 = e4m3(y / c)   (from the fp32 y, times fp32's 1 / c)
//
// The norm takes the unrounded fp32 sum: only what is stored is rounded.  The reductions run in
// fp32 over a fixed tree, so the result does not depend on the launch's timing.
//
// Bound: HBM, for batches.  A row is read once into registers (16-byte vectors), reduced, and
// written once: 16384 rows of 5120 in bf16 with the residual and the 8-bit output take 115 us,
// 6.6 TB/s, as fast as a copy of as many bytes, at half the threads an SM can hold; 3001 rows of
// 1408 in fp32 take 8.9 us (their 38 MB stay in the L2 cache from call to call).  One row of 7168
// takes 2.3 us in a captured graph, hardly more than an empty launch: a load, two reductions and a
// store, in a row.
//
// The sum of squares needs the whole row before its first output, so a row stays with one team of
// threads that can hold it: a warp up to 128 vectors (eight rows in a block, no barrier), a block
// beyond.  Two vectors a thread up to 512 of them and four beyond keep several blocks on an SM
// (59 registers), whose loads cover one another's reductions; a few rows cannot fill the GPU and
// take a vector a thread instead, which is the shortest way through a row.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <typename T>
struct Vec;  // 16 bytes of a row
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};

template <int kN>
__device__ __forceinline__ void store_e4m3(uint8_t* dst, const float (&f)[kN], float inv) {
  uint32_t w[kN / 4];
#pragma unroll
  for (int i = 0; i < kN / 4; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i] * inv, f[4 * i + 1] * inv),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(
        make_float2(f[4 * i + 2] * inv, f[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  if constexpr (kN == 8)
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(dst) = w[0];
}

// The scale of a group with largest magnitude amax, and its reciprocal for the quotients.  A
// group of zeros has scale 0 (and zero codes); a scale below the smallest normal number is
// raised to it, so that its reciprocal stays finite.  A NaN stays a NaN.
__device__ __forceinline__ void e4m3_scale(float amax, float& scale, float& inv) {
  scale = amax == 0.f ? 0.f : max_nan(amax * (1.0f / 448.0f), 1.17549435e-38f);
  inv = amax == 0.f ? 0.f : 1.0f / scale;
}

struct NormArgs {
  const void* x;
  const void* residual;
  const void* weight;
  void* y;
  void* residual_out;
  uint8_t* y8;
  float* y8_scale;
  int64_t N;
  int d;
  float eps;
  float low;  // a sum of squares below it is taken again, scaled (0: none is)
  int group;  // 128, or 0: one scale for a row
};

// kTeam threads own a row: 32 (a warp, several rows per block) or 0 (the whole block).  Thread
// i of the team holds vectors i, i + team, ...; kVpt of them.
template <typename T, int kVpt, int kTeam>
__global__ void __launch_bounds__(kTeam == 32 ? 256 : 1024) rms_norm_kernel(const NormArgs a) {
  using V = Vec<T>;
  constexpr int kN = V::kN;
  constexpr int kGroupLanes = 128 / kN;  // lanes that hold one group of 128 columns
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = kTeam == 32 ? 32 : (int)blockDim.x;
  const int ti = kTeam == 32 ? lane : (int)threadIdx.x;
  const int64_t row = kTeam == 32 ? (int64_t)blockIdx.x * (blockDim.x >> 5) + warp : blockIdx.x;
  if (kTeam == 32 && row >= a.N) return;
  const int nvec = a.d / kN;
  const size_t base = (size_t)row * a.d;
  const uint4* px = reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + base);
  const uint4* pr = a.residual == nullptr
                        ? nullptr
                        : reinterpret_cast<const uint4*>(static_cast<const T*>(a.residual) + base);
  const uint4* pw = static_cast<const uint4*>(a.weight);

  uint4 vx[kVpt], vr[kVpt];
#pragma unroll
  for (int i = 0; i < kVpt; ++i)
    if (ti + i * team < nvec) vx[i] = px[ti + i * team];
  if (pr != nullptr) {
#pragma unroll
    for (int i = 0; i < kVpt; ++i)
      if (ti + i * team < nvec) vr[i] = pr[ti + i * team];
  }
  float s[kVpt][kN];
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < kVpt; ++i) {
    const int v = ti + i * team;
    if (v < nvec) {
      V::unpack(vx[i], s[i]);
      if (pr != nullptr) {
        float r[kN];
        V::unpack(vr[i], r);
#pragma unroll
        for (int j = 0; j < kN; ++j) s[i][j] += r[j];
        if (a.residual_out != nullptr)
          reinterpret_cast<uint4*>(static_cast<T*>(a.residual_out) + base)[v] = V::pack(s[i]);
      }
#pragma unroll
      for (int j = 0; j < kN; ++j) sq = fmaf(s[i][j], s[i][j], sq);
    } else {
#pragma unroll
      for (int j = 0; j < kN; ++j) s[i][j] = 0.f;
    }
  }
  __shared__ float s_part[32];
  auto team_sum = [&](float v) {
    v = warp_sum(v);
    if (kTeam != 32) {
      if (lane == 0) s_part[warp] = v;
      __syncthreads();
      const int nw = blockDim.x >> 5;
      v = warp_sum(lane < nw ? s_part[lane] : 0.f);
    }
    return v;
  };
  sq = team_sum(sq);
  float eps = a.eps;
  // A row whose squares overflow, or vanish beside an eps that does too, is scaled by a power of
  // two first: y stays the same.  2^-75 brings the largest sum (2^15 squares of 2^128) to 2^121,
  // 2^100 the smallest number's square to 2^-98.
  if (__builtin_expect(sq == INFINITY || sq < a.low, 0)) {
    const float by = sq == INFINITY ? 0x1p-75f : 0x1p100f;
    sq = 0.f;
#pragma unroll
    for (int i = 0; i < kVpt; ++i)
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        s[i][j] *= by;
        sq = fmaf(s[i][j], s[i][j], sq);
      }
    eps = eps * by * by;
    if (kTeam != 32) __syncthreads();  // the first sum's parts have been read
    sq = team_sum(sq);
  }
  const float r = rsqrtf(sq / (float)a.d + eps);
  float rowmax = 0.f;
#pragma unroll
  for (int i = 0; i < kVpt; ++i) {
    const int v = ti + i * team;
    const bool in = v < nvec;
    float w[kN];
    if (in && pw != nullptr) {
      V::unpack(__ldg(pw + v), w);
    } else {
#pragma unroll
      for (int j = 0; j < kN; ++j) w[j] = 1.f;
    }
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      s[i][j] = in ? s[i][j] * r * w[j] : 0.f;
      m = max_nan(m, fabsf(s[i][j]));
    }
    if (in && a.y != nullptr)
      reinterpret_cast<uint4*>(static_cast<T*>(a.y) + base)[v] = V::pack(s[i]);
    if (a.y8 == nullptr) continue;
    if (a.group == 0) {
      rowmax = max_nan(rowmax, m);
      continue;
    }
#pragma unroll
    for (int o = kGroupLanes / 2; o > 0; o >>= 1)
      m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    float scale, inv;
    e4m3_scale(m, scale, inv);
    if (in) {
      store_e4m3<kN>(a.y8 + base + (size_t)v * kN, s[i], inv);
      if (v % kGroupLanes == 0)
        a.y8_scale[(size_t)row * ((a.d + 127) / 128) + v / kGroupLanes] = scale;
    }
  }
  if (a.y8 != nullptr && a.group == 0) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) rowmax = max_nan(rowmax, __shfl_xor_sync(0xffffffffu, rowmax, o));
    if (kTeam != 32) {
      __shared__ float s_max[32];
      if (lane == 0) s_max[warp] = rowmax;
      __syncthreads();
      const int nw = blockDim.x >> 5;
      rowmax = lane < nw ? s_max[lane] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        rowmax = max_nan(rowmax, __shfl_xor_sync(0xffffffffu, rowmax, o));
    }
    float scale, inv;
    e4m3_scale(rowmax, scale, inv);
#pragma unroll
    for (int i = 0; i < kVpt; ++i) {
      const int v = ti + i * team;
      if (v < nvec) store_e4m3<kN>(a.y8 + base + (size_t)v * kN, s[i], inv);
    }
    if (ti == 0) a.y8_scale[row] = scale;
  }
}

template <typename T>
cudaError_t launch(const NormArgs& a, cudaStream_t stream) {
  const int nvec = a.d / Vec<T>::kN;
  if (nvec <= 128) {
    const dim3 grid((unsigned)((a.N + 7) / 8));
    if (nvec <= 32) return launch_pdl(rms_norm_kernel<T, 1, 32>, grid, 256, 0, stream, a);
    if (nvec <= 64) return launch_pdl(rms_norm_kernel<T, 2, 32>, grid, 256, 0, stream, a);
    return launch_pdl(rms_norm_kernel<T, 4, 32>, grid, 256, 0, stream, a);
  }
  const dim3 grid((unsigned)a.N);
  auto threads = [&](int vpt) { return (nvec + 32 * vpt - 1) / (32 * vpt) * 32; };
  // few rows: a vector a thread, for the shortest way through; else as few threads as hold the
  // row (at most 4096 vectors, checked by the caller: 1024 threads of up to 64 registers)
  if (a.N < 512 && nvec <= 1024)
    return launch_pdl(rms_norm_kernel<T, 1, 0>, grid, threads(1), 0, stream, a);
  if (nvec <= 512) return launch_pdl(rms_norm_kernel<T, 2, 0>, grid, threads(2), 0, stream, a);
  return launch_pdl(rms_norm_kernel<T, 4, 0>, grid, threads(4), 0, stream, a);
}

}  // namespace

cudaError_t launch_rms_norm(int64_t N, int d, bool f32, const void* x, const void* residual,
                            const void* weight, float eps, void* y, void* residual_out, void* y8,
                            float* y8_scale, int group, cudaStream_t stream, int* launches) {
  if (N == 0) return cudaSuccess;
  const NormArgs a{x, residual, weight, y, residual_out, static_cast<uint8_t*>(y8), y8_scale,
                   N, d, eps, eps < 0x1p-80f ? 0x1p-100f : 0.f, group};
  ++*launches;
  return f32 ? launch<float>(a, stream) : launch<__nv_bfloat16>(a, stream);
}

}  // namespace moe
