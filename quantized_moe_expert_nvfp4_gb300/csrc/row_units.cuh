// Units of eight consecutive row elements (bf16: 16 bytes, fp32: 32 bytes) as fp32 values.
#pragma once

#include "internal.cuh"

namespace moe {

template <typename V>
struct Unit8;

template <>
struct Unit8<uint16_t> {
  uint4 q;
  __device__ __forceinline__ void load(const void* base, int64_t unit) { q = __ldg(static_cast<const uint4*>(base) + unit); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    q = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void store(void* base, int64_t unit) const { static_cast<uint4*>(base)[unit] = q; }
};

template <>
struct Unit8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* base, int64_t unit) {
    a = __ldg(static_cast<const float4*>(base) + 2 * unit);
    b = __ldg(static_cast<const float4*>(base) + 2 * unit + 1);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
  __device__ __forceinline__ void store(void* base, int64_t unit) const {
    static_cast<float4*>(base)[2 * unit] = a;
    static_cast<float4*>(base)[2 * unit + 1] = b;
  }
};

}  // namespace moe
