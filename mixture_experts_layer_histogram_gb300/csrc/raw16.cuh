// Sixteen consecutive values of a row in one thread's registers, as the quantising passes (MXFP4, 8 bits) take them.
#pragma once

#include "common.cuh"

namespace moe {

__device__ __forceinline__ void store32(void *p, const uint4 &a, const uint4 &b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
               "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// Sixteen consecutive values of a row as they lie in memory.
template <typename T> struct Raw16;
template <> struct Raw16<__nv_bfloat16> {
  uint4 q[2];
  __device__ __forceinline__ void zero() { q[0] = q[1] = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    q[0] = __ldg(reinterpret_cast<const uint4 *>(p));
    q[1] = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
  }
  __device__ __forceinline__ void unpack(float *v) const {
    unpack_bf16x8(q[0], v);
    unpack_bf16x8(q[1], v + 8);
  }
  // Largest magnitude as fp32 bits. bf16 magnitudes order as 16-bit integers, two at a time (NaN above infinity).
  __device__ __forceinline__ uint32_t amax() const {
    const uint32_t w[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
    uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    return max(m << 16, m & 0xffff0000u);
  }
  // wide: 32-byte aligned, one store
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float *v, bool wide) {
    const uint4 a = pack_bf16x8(v), b = pack_bf16x8(v + 8);
    if (wide) {
      store32(p, a, b);
    } else {
      reinterpret_cast<uint4 *>(p)[0] = a;
      reinterpret_cast<uint4 *>(p)[1] = b;
    }
  }
};
template <> struct Raw16<float> {
  float4 q[4];
  __device__ __forceinline__ void zero() { q[0] = q[1] = q[2] = q[3] = make_float4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const float *p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = __ldg(reinterpret_cast<const float4 *>(p) + i);
  }
  __device__ __forceinline__ void unpack(float *v) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[4 * i] = q[i].x; v[4 * i + 1] = q[i].y; v[4 * i + 2] = q[i].z; v[4 * i + 3] = q[i].w;
    }
  }
  __device__ __forceinline__ uint32_t amax() const {
    float v[16];
    unpack(v);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
  }
  static __device__ __forceinline__ void store(float *p, const float *v, bool wide) {
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                        __float_as_uint(v[4 * i + 3]));
    if (wide) {
      store32(p, w[0], w[1]);
      store32(p + 8, w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) reinterpret_cast<uint4 *>(p)[i] = w[i];
    }
  }
};

}  // namespace moe
