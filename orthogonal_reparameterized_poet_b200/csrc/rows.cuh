// Device helpers shared by the kernels that work on rows (the joint between
// blocks, the operators on logits): 16-byte vectors of either element type and
// sums over the threads that share a row.
#pragma once

#include "poet_internal.cuh"

namespace poet {

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

// Sums v[0..N) over the `warps` warps that share a row; every thread gets the
// totals, added in one fixed order.  One barrier: `slot` alternates between
// two buffers, and a buffer is written again only after the barrier of the
// other one, which no thread passes before all have read the first.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float *slot, int warps, int warp, int bar, int threads) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (warps == 1) return;
  const int lane = threadIdx.x & 31;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) slot[i * 32 + warp] = v[i];
  asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(threads) : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = lane < warps ? slot[i * 32 + lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  }
}

}  // namespace poet
