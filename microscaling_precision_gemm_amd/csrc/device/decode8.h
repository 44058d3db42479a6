// decode8.h -- the 8-bit MX element types (E4M3, E5M2, INT8) times their block
// scale, as FP32 (exact) and as BF16.  gfx950's scaled conversions give the
// BF16 value of code * 2^(sc - 127) for every code and every scale code
// 0..254, rounded to nearest even where BF16 cannot hold it (checked on the
// device over all pairs: E4M3 is exact for scale codes 3..254, E5M2 for
// 10..254).  Scale code 255 makes the block NaN.
#pragma once
#include <stdint.h>

#include "codec.h"
#include "rows.h"

namespace mxk {

// 2^(sc - 127) as FP32: code 0 is the subnormal 2^-127, 255 is NaN
__device__ inline float e8m0_value(uint32_t sc) {
  return sc == 0xFFu ? __builtin_nanf("") : (sc == 0u ? u2f(0x00400000u) : u2f(sc << 23));
}

// 4 codes of w times 2^(sc - 127), exactly, as FP32.  The FP8 conversions give
// NaN for scale code 255 and the NaN codes (checked on the device over all
// codes and scale codes, FP32 subnormal results among them).
template <int FMT>
__device__ inline void decode4_f32(uint32_t w, uint32_t sc, float* v) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  if constexpr (FMT == FMT_MXINT8) {
    const float X = e8m0_value(sc);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = int8_value((w >> (8 * i)) & 0xFFu) * X;
  } else {
    const float X = u2f(sc << 23);
    f2 a, b;
    if constexpr (FMT == FMT_MXFP8) {
      a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, X, false);
      b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, X, true);
    } else {
      a = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(w, X, false);
      b = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(w, X, true);
    }
    v[0] = a[0];
    v[1] = a[1];
    v[2] = b[0];
    v[3] = b[1];
  }
}

// Codes 2 H and 2 H + 1 of w times a block scale, as a BF16 pair.  x holds the
// scale as scale8<FMT>() or scale8_word<FMT>() gives it.  The FP8 conversions
// look at the exponent field of x alone and give NaN for 255 whatever the code
// (checked on the device over all codes and scale codes).
template <int FMT, int H>
__device__ inline uint32_t decode2_bf16(uint32_t w, float x) {
  if constexpr (FMT == FMT_MXINT8) {
    // (opaque: of a word whose every use is a byte the compiler would keep the
    // bytes, and take them apart as soon as the word is loaded)
    asm("" : "+v"(w));
    return pack_bf16((float)(int8_t)(uint8_t)(w >> (16 * H)) * x, (float)(int8_t)(uint8_t)(w >> (16 * H + 8)) * x);
  } else if constexpr (FMT == FMT_MXFP8) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, x, H != 0));
  } else {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, x, H != 0));
  }
}
template <int FMT>
__device__ inline float scale8(uint32_t sc) {
  if constexpr (FMT == FMT_MXINT8) {
    const float x = __builtin_amdgcn_ldexpf(0.015625f, (int)sc - 127);
    return sc == 0xFFu ? __builtin_nanf("") : x;
  }
  else return u2f(sc << 23);
}
// the same from byte `shift` / 8 of a word: for FP8 one rotation puts it into
// the exponent field, and what comes beside it is not looked at
template <int FMT>
__device__ inline float scale8_word(uint32_t w, uint32_t shift) {
  if constexpr (FMT == FMT_MXINT8) return scale8<FMT>((w >> shift) & 0xFFu);
  else return u2f(__builtin_amdgcn_alignbit(w, w, shift + 9u));
}

}  // namespace mxk
