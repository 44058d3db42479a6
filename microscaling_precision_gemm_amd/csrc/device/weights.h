// weights.h -- 32 consecutive elements of a block-scaled weight row (one MX
// block, two NVFP4 blocks) decoded to BF16 matrix-instruction operands.
//   8-bit MX types   decode8.h
//   MXFP4            gfx950's scaled conversion, code * 2^(sc - 127) to BF16
//   NVFP4            e2m1 * e4m3 has at most 6 significant bits: formed in FP32
//                    and packed to BF16, both exact; the tensor scale is left to
//                    the sum
#pragma once
#include <stdint.h>

#include "decode8.h"

namespace mxk {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t word4 __attribute__((ext_vector_type(4)));

template <int FMT>
constexpr bool kFourBit = FMT == FMT_MXFP4 || FMT == FMT_NVFP4;

// code bytes of 32 elements
template <int FMT>
constexpr int kBlockBytes = kFourBit<FMT> ? 16 : 32;

// The scale bytes of one block of 32 (NVFP4: two, the lower first).
template <int FMT>
__device__ inline uint32_t load_scale(const uint8_t* __restrict__ scales, int64_t block) {
  if constexpr (FMT == FMT_NVFP4) return reinterpret_cast<const uint16_t*>(scales)[block];
  else return scales[block];
}

// Elements 8 J .. 8 J + 7 of the block with code words w[] and scale bytes sc.
template <int FMT, int J>
__device__ inline bf16x8 decode_eighth(const uint32_t* w, uint32_t sc) {
  uint32_t p[4];
  if constexpr (FMT == FMT_MXFP4) {
    const float x = u2f(sc << 23);
    p[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[J], x, 0));
    p[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[J], x, 1));
    p[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[J], x, 2));
    p[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[J], x, 3));
  } else if constexpr (FMT == FMT_NVFP4) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    const float x = J < 2 ? __builtin_amdgcn_cvt_f32_fp8(sc, 0) : __builtin_amdgcn_cvt_f32_fp8(sc, 1);
    const f2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[J], 1.0f, 0);
    const f2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[J], 1.0f, 1);
    const f2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[J], 1.0f, 2);
    const f2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[J], 1.0f, 3);
    p[0] = pack_bf16(a[0] * x, a[1] * x);
    p[1] = pack_bf16(b[0] * x, b[1] * x);
    p[2] = pack_bf16(c[0] * x, c[1] * x);
    p[3] = pack_bf16(d[0] * x, d[1] * x);
  } else {
    const float x = scale8<FMT>(sc);
    p[0] = decode2_bf16<FMT, 0>(w[2 * J], x);
    p[1] = decode2_bf16<FMT, 1>(w[2 * J], x);
    p[2] = decode2_bf16<FMT, 0>(w[2 * J + 1], x);
    p[3] = decode2_bf16<FMT, 1>(w[2 * J + 1], x);
  }
  return __builtin_bit_cast(bf16x8, word4{p[0], p[1], p[2], p[3]});
}

}  // namespace mxk
