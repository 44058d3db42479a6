// linear_epilogue.h -- what follows the sum of a product (Epilogue of
// launch_dense.h) on 8 consecutive columns of one row:
//   z = sum + bias,  out = residual + drop(act(z))
// in FP32; z and out are rounded once each.
#pragma once
#include <type_traits>

#include "act.h"
#include "chunk8.h"

namespace mxk {

// which of the matrices have 16-byte aligned rows (bias: its start)
struct EpilogueVec {
  bool bias, z, residual, out;
};
inline EpilogueVec epilogue_vec(const Epilogue& e) {
  return {(reinterpret_cast<uintptr_t>(e.bias) & 15u) == 0, rows_aligned16(e.z, e.ld_z, e.dt),
          rows_aligned16(e.residual, e.ld_r, e.dt), rows_aligned16(e.out, e.ld_o, e.dt)};
}

// bias of columns col .. col + 7 (a multiple of 8), of which n exist
__device__ inline void load_bias(const Epilogue& e, const EpilogueVec& vec, int64_t col, int n, float (&b)[8]) {
  if (!e.bias) {
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = 0.0f;
  } else if (e.bias_dt == DT_BF16) load_chunk<DT_BF16>(e.bias, col, n, vec.bias, b);
  else load_chunk<DT_F32>(e.bias, col, n, vec.bias, b);
}

// v: the sums of columns col .. col + 7, of which n exist; res: the residual
// there, if there is one.  Results larger than the L2s go by streaming stores
// (16384 x 14336 BF16 and z: 1628 -> 1588 us).
template <int DT, bool STREAM>
__device__ inline void epilogue_chunk(const Epilogue& e, const EpilogueVec& vec, int64_t row, int64_t col, int64_t N,
                                      int n, const float (&b)[8], const RawChunk& res, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] += b[i];
  if (e.z) store_chunk<DT, STREAM>(e.z, row * e.ld_z + col, n, vec.z, v);
  with_act(e.act, [&](auto kind) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act<decltype(kind)::value>(v[i]);
  });
  if (e.drop.threshold) drop_chunk(e.drop, (uint64_t)(row * ((N + 7) / 8) + col / 8), v);
  if (e.residual) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = raw_value<DT>(res, i) + v[i];
  }
  store_chunk<DT, STREAM>(e.out, row * e.ld_o + col, n, vec.out, v);
}

}  // namespace mxk
