// rows.h -- 8-element chunks of BF16 / FP32 rows, used by the kernels around
// the expert products: loads and stores of a whole chunk (16 or 32 bytes,
// 16-byte aligned) and of one element.
#pragma once
#include <stdint.h>

#include "../launch.h"
#include "codec.h"

namespace mxk {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// two FP32 values rounded to BF16 (nearest even; NaN stays NaN), one v_cvt_pk
__device__ inline uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}

template <int DT>
__device__ inline float load1(const void* p, int64_t off) {
  if constexpr (DT == DT_BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[off]);
  else return static_cast<const float*>(p)[off];
}

template <int DT>
__device__ inline void store1(void* p, int64_t off, float v) {
  if constexpr (DT == DT_BF16) static_cast<uint16_t*>(p)[off] = (uint16_t)pack_bf16(v, v);
  else static_cast<float*>(p)[off] = v;
}

template <int DT>
__device__ inline void load8(const void* __restrict__ p, int64_t off, float (&v)[8]) {
  if constexpr (DT == DT_BF16) {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + off);
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = u2f(ww[i] << 16);
      v[2 * i + 1] = u2f(ww[i] & 0xFFFF0000u);
    }
  } else {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + off);
    const float4 a = q[0], b = q[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

template <int DT>
__device__ inline void store8(void* __restrict__ p, int64_t off, const float (&v)[8]) {
  if constexpr (DT == DT_BF16) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + off) =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  } else {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + off);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

}  // namespace mxk
