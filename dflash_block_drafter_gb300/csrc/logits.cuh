// Values of a row of logits (FP32, BF16 or FP16), in 16-byte pieces and one by one.
#pragma once

#include "common.cuh"

namespace dflash {

template <int TYPE>
struct Elem {
  static constexpr int BYTES = TYPE == DFLASH_T_FP32 ? 4 : 2;
  static constexpr int VEC = 16 / BYTES;
  static __device__ __forceinline__ void widen(uint4 v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (TYPE == DFLASH_T_FP32) {
        x[i] = __uint_as_float(w[i]);
      } else if constexpr (TYPE == DFLASH_T_BF16) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
  }
  // the larger of two 32-bit words' values, value by value; the larger value of a word
  static __device__ __forceinline__ uint32_t max_words(uint32_t a, uint32_t b) {
    if constexpr (TYPE == DFLASH_T_FP32) {
      return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    } else if constexpr (TYPE == DFLASH_T_BF16) {
      const __nv_bfloat162 m = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
      return *reinterpret_cast<const uint32_t*>(&m);
    } else {
      const __half2 m = __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
      return *reinterpret_cast<const uint32_t*>(&m);
    }
  }
  static __device__ __forceinline__ float max_of(uint32_t w) {
    if constexpr (TYPE == DFLASH_T_FP32) return __uint_as_float(w);
    if constexpr (TYPE == DFLASH_T_BF16) return fmaxf(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return fmaxf(f.x, f.y);
  }
  // a word whose values are -infinity
  static constexpr uint32_t NOTHING = TYPE == DFLASH_T_FP32 ? 0xff800000u : TYPE == DFLASH_T_BF16 ? 0xff80ff80u : 0xfc00fc00u;
  // the word of two (one for FP32) values of a row
  static __device__ __forceinline__ uint32_t raw(const uint8_t* row, long long i, long long n) {
    if constexpr (TYPE == DFLASH_T_FP32) {
      return i >= 0 && i < n ? __ldg(reinterpret_cast<const uint32_t*>(row) + i) : NOTHING;
    } else {
      const uint32_t lo = i >= 0 && i < n ? __ldg(reinterpret_cast<const uint16_t*>(row) + i) : NOTHING & 0xffffu;
      const uint32_t hi = i + 1 >= 0 && i + 1 < n ? __ldg(reinterpret_cast<const uint16_t*>(row) + i + 1) : NOTHING & 0xffffu;
      return lo | hi << 16;
    }
  }
  // value i of a lane's pieces
  static __device__ __forceinline__ float shown(const uint4* p, int i) {
    if constexpr (TYPE == DFLASH_T_FP32) return reinterpret_cast<const float*>(p)[i];
    const uint16_t h = reinterpret_cast<const uint16_t*>(p)[i];
    if constexpr (TYPE == DFLASH_T_BF16) return __uint_as_float(static_cast<uint32_t>(h) << 16);
    return __half2float(__ushort_as_half(h));
  }
  static __device__ __forceinline__ float one(const uint8_t* row, int i) {
    if constexpr (TYPE == DFLASH_T_FP32) return __ldg(reinterpret_cast<const float*>(row) + i);
    const uint16_t h = __ldg(reinterpret_cast<const uint16_t*>(row) + i);
    if constexpr (TYPE == DFLASH_T_BF16) return __uint_as_float(static_cast<uint32_t>(h) << 16);
    return __half2float(__ushort_as_half(h));
  }
};

}  // namespace dflash
