// chunk8.h -- 8 consecutive columns of a BF16 or FP32 row as FP32 values, whole or
// the first n of them, by 16-byte accesses where the matrix allows them, and the
// dropout of such a chunk.
#pragma once
#include "../launch_dense.h"
#include "codec.h"
#include "rows.h"

namespace mxk {

// Whether rows of a matrix are 16-byte aligned, so that chunks at multiples of 8
// columns are.
inline bool rows_aligned16(const void* p, int64_t ld, int dt) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * (dt == DT_F32 ? 4 : 2)) % 16 == 0;
}

// (the columns past n read as 0)
template <int DT>
__device__ inline void load_chunk(const void* p, int64_t off, int n, bool vec, float (&v)[8]) {
  if (n >= 8 && vec) return load8<DT>(p, off, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < n ? load1<DT>(p, off + i) : 0.0f;
}
template <int DT>
__device__ inline void store_chunk(void* p, int64_t off, int n, bool vec, const float (&v)[8]) {
  if (n >= 8 && vec) return store8<DT>(p, off, v);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) store1<DT>(p, off + i, v[i]);
}

// Chunk q of the stream (row * ceil(cols / 8) + column / 8): element i takes the
// 16 bits that the quantizers' stochastic rounding would.
__device__ inline void drop_chunk(const Drop& d, uint64_t q, float (&v)[8]) {
  uint32_t r[8];
  rand16x8(d.seed, d.counter, q, r);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = r[i] < d.threshold ? 0.0f : v[i] * d.factor;
}

}  // namespace mxk
