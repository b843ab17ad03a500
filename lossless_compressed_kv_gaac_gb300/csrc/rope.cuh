// Shared pieces of the kernels that turn heads by their positions: vectors of the model's types, the angle, and the
// check of output strides.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace gaac {

template <typename T, int V>
struct alignas(sizeof(T) * V) RopeVec {
  T v[V];
};

__device__ __forceinline__ float2 rope_pair(__nv_bfloat162 w) { return __bfloat1622float2(w); }
__device__ __forceinline__ float2 rope_pair(__half2 w) { return __half22float2(w); }
template <typename T>
struct RopePair;
template <>
struct RopePair<__nv_bfloat16> {
  using type = __nv_bfloat162;
  static __device__ __forceinline__ type pack(float a, float b) { return __floats2bfloat162_rn(a, b); }
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct RopePair<__half> {
  using type = __half2;
  static __device__ __forceinline__ type pack(float a, float b) { return __floats2half2_rn(a, b); }
  static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
};

template <typename T, int V>
__device__ __forceinline__ void rope_unpack(const RopeVec<T, V>& x, float* f) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = x.v[i];
  } else if constexpr (V == 1) {
    f[0] = RopePair<T>::get(x.v[0]);
  } else {
    const auto* w = reinterpret_cast<const typename RopePair<T>::type*>(x.v);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 p = rope_pair(w[i]);
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
}
template <typename T, int V>
__device__ __forceinline__ void rope_pack(RopeVec<T, V>& x, const float* f) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) x.v[i] = f[i];
  } else if constexpr (V == 1) {
    x.v[0] = RopePair<T>::put(f[0]);
  } else {
    auto* w = reinterpret_cast<typename RopePair<T>::type*>(x.v);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = RopePair<T>::pack(f[2 * i], f[2 * i + 1]);
  }
}

__device__ __forceinline__ uint64_t rope_position(const void* pos, int pos64, int64_t i) {
  return pos64 ? static_cast<uint64_t>(static_cast<const int64_t*>(pos)[i])
               : static_cast<uint64_t>(static_cast<int64_t>(static_cast<const int32_t*>(pos)[i]));
}

// Sine and cosine, times mscale, of a fraction of a turn in 64-bit fixed point, for results of type T.
template <typename T>
__device__ __forceinline__ void rope_sincos(uint64_t turn, float mscale, float& s, float& c) {
  turn += 1ull << 31;
  const float half_turns = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
  // A 16-bit result is rounded at 2^-12 or coarser, so the hardware's sine and cosine (2^-21.2 off at most in
  // [-pi, pi]) serve it; they take a tenth of the instructions, which bound the kernels otherwise.
  if constexpr (sizeof(T) == 2)
    __sincosf(half_turns * 3.14159265358979f, &s, &c);
  else
    sincospif(half_turns, &s, &c);
  s *= mscale;
  c *= mscale;
}

// Elements (seq, tok, head) of the output are distinct: taken from the smallest stride up, each dimension
// steps over everything below it.  Dimensions of size 1 do not count.
inline bool distinct(int64_t dim, int64_t n[3], int64_t s[3]) {
  int64_t extent = dim;
  bool used[3] = {n[0] <= 1, n[1] <= 1, n[2] <= 1};
  for (int k = 0; k < 3; ++k) {
    int at = -1;
    for (int i = 0; i < 3; ++i)
      if (!used[i] && (at < 0 || s[i] < s[at])) at = i;
    if (at < 0) return true;
    if (s[at] < extent) return false;
    extent = s[at] * (n[at] - 1) + extent;
    used[at] = true;
  }
  return true;
}

}  // namespace gaac
