// Device helpers shared by the kernels that work on rows (the joint between
// blocks, the operators on logits): 16-byte vectors of either element type and
// sums over the threads that share a row.
#pragma once

#include <atomic>

#include "poet_internal.cuh"

namespace poet {

// Lets a kernel use all the dynamic shared memory that its static part leaves
// of a block's on the current device, where a launch asks for `bytes` of it.
// Asked of the runtime once per kernel and device.
template <auto KERN>
poet_status allow_smem(size_t bytes) {
  static std::atomic<uint64_t> done{0};
  if (bytes <= 32 * 1024) return POET_OK;  // with the static part below the default of 48 KB
  int dev = 0;
  POET_CUDA_TRY(cudaGetDevice(&dev));
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return POET_OK;
  int most = 0;
  cudaFuncAttributes f;
  POET_CUDA_TRY(cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev));
  POET_CUDA_TRY(cudaFuncGetAttributes(&f, KERN));
  POET_CUDA_TRY(cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, most - int(f.sharedSizeBytes)));
  done.fetch_or(bit, std::memory_order_release);
  return POET_OK;
}

// VW consecutive elements of a row: 16 bytes where rows are aligned, one
// element where they are not.
template <typename T, int VW>
struct RowVec;
template <>
struct RowVec<bf16, 8> {
  uint4 r;
  __device__ __forceinline__ void load(const bf16 *p) { r = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
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
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ void store(bf16 *p, const float (&f)[8]) { *reinterpret_cast<uint4 *>(p) = pack(f); }
};
template <>
struct RowVec<float, 4> {
  float4 r;
  __device__ __forceinline__ void load(const float *p) { r = *reinterpret_cast<const float4 *>(p); }
  __device__ __forceinline__ void get(float (&f)[4]) const { f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w; }
  static __device__ __forceinline__ void store(float *p, const float (&f)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <>
struct RowVec<bf16, 1> {
  bf16 r;
  __device__ __forceinline__ void load(const bf16 *p) { r = *p; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = __bfloat162float(r); }
  static __device__ __forceinline__ void store(bf16 *p, const float (&f)[1]) { *p = __float2bfloat16_rn(f[0]); }
};
template <>
struct RowVec<float, 1> {
  float r;
  __device__ __forceinline__ void load(const float *p) { r = *p; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = r; }
  static __device__ __forceinline__ void store(float *p, const float (&f)[1]) { *p = f[0]; }
};

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float<bf16>(bf16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_float<float>(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ bf16 from_float<bf16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }

// Two floats at a time: one instruction for both.
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// 1 / sqrt(x) for x > 0: CUDA's approximation and one Newton step (0 for x = inf).
__device__ __forceinline__ float inv_sqrt(float x) {
  const float y = rsqrtf(x);
  return y > 0.f ? fmaf(0.5f * y, fmaf(-x * y, y, 1.f), y) : y;
}

// Sums two values over the `warps` warps that share a row; every thread gets the
// totals, added in one fixed order.  Within a warp one butterfly sums both: its
// first step exchanges one value for the other, which takes six shuffles for
// both.  One barrier: `slot` (2 * 32 floats, 16-byte aligned, zero behind the
// last warp) alternates between two buffers, and a buffer is written again only
// after the barrier of the other one, which no thread passes before all have
// read the first.
__device__ __forceinline__ void row_sum_2(float (&v)[2], float *slot, int warps, int warp, int bar, int threads) {
  const int lane = threadIdx.x & 31;
  const bool hi = lane & 16;
  float t = (hi ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[1], 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  if (warps == 1) {
    v[0] = __shfl_sync(0xffffffffu, t, 0);
    v[1] = __shfl_sync(0xffffffffu, t, 16);
    return;
  }
  if (lane % 16 == 0) slot[warp * 2 + lane / 16] = t;
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(threads) : "memory");
  const float4 *s4 = reinterpret_cast<const float4 *>(slot);
  float2 a = both(0.f), b = both(0.f);
  const int quads = (warps + 1) / 2;
#pragma unroll 2
  for (int i = 0; i < quads; ++i) {
    const float4 f = s4[i];
    a = add2(a, make_float2(f.x, f.y));
    b = add2(b, make_float2(f.z, f.w));
  }
  v[0] = a.x + b.x;
  v[1] = a.y + b.y;
}

// The same for four values and, where `fifth` is true, one more.  slot: 5 * 32
// floats, the fifth values behind the others.
__device__ __forceinline__ void row_sum_5(float (&v)[5], bool fifth, float *slot, int warps, int warp, int bar,
                                          int threads) {
  const int lane = threadIdx.x & 31;
  const bool hi = lane & 16, up = lane & 8;
  const float a = (hi ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], 16);
  const float b = (hi ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, hi ? v[1] : v[3], 16);
  float t = (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, 8);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  if (fifth) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[4] += __shfl_xor_sync(0xffffffffu, v[4], o);
  }
  if (warps == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(0xffffffffu, t, i * 8);
    return;
  }
  if (lane % 8 == 0) slot[warp * 4 + lane / 8] = t;
  if (fifth && lane == 0) slot[128 + warp] = v[4];
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(threads) : "memory");
  const float4 *s4 = reinterpret_cast<const float4 *>(slot);
  float2 lo = both(0.f), up2 = both(0.f);
#pragma unroll 2
  for (int i = 0; i < warps; ++i) {
    const float4 f = s4[i];
    lo = add2(lo, make_float2(f.x, f.y));
    up2 = add2(up2, make_float2(f.z, f.w));
  }
  v[0] = lo.x; v[1] = lo.y; v[2] = up2.x; v[3] = up2.y;
  if (fifth) {
    v[4] = 0.f;
    for (int i = 0; i < warps; ++i) v[4] += slot[128 + i];
  }
}

}  // namespace poet
