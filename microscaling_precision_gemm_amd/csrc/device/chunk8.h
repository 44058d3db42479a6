// chunk8.h -- 8 consecutive columns of a BF16 or FP32 row as FP32 values, whole or
// the first n of them, by 16-byte accesses where the matrix allows them, and the
// dropout of such a chunk.
#pragma once
#include "../launch_dense.h"
#include "codec.h"
#include "rows.h"
#include "wave.h"

namespace mxk {

// Whether rows of a matrix are 16-byte aligned, so that chunks at multiples of 8
// columns are.
inline bool rows_aligned16(const void* p, int64_t ld, int dt) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * (dt == DT_F32 ? 4 : 2)) % 16 == 0;
}

// a chunk as it lies in memory (BF16: a alone)
typedef uint32_t raw16 __attribute__((ext_vector_type(4)));
struct RawChunk {
  raw16 a, b;
};
template <int DT>
__device__ inline RawChunk load_raw8(const void* p, int64_t off, int n, bool vec) {
  RawChunk r = {};
  if (n >= 8 && vec) {
    const raw16* q = reinterpret_cast<const raw16*>(static_cast<const char*>(p) + off * (DT == DT_BF16 ? 2 : 4));
    r.a = q[0];
    if constexpr (DT == DT_F32) r.b = q[1];
    return r;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) {
      if constexpr (DT == DT_BF16) r.a[i / 2] |= (uint32_t)static_cast<const uint16_t*>(p)[off + i] << (16 * (i & 1));
      else (i < 4 ? r.a : r.b)[i & 3] = static_cast<const uint32_t*>(p)[off + i];
    }
  return r;
}
template <int DT>
__device__ inline float raw_value(const RawChunk& r, int i) {
  if constexpr (DT == DT_BF16) return u2f(i & 1 ? r.a[i / 2] & 0xFFFF0000u : r.a[i / 2] << 16);
  else return u2f(i < 4 ? r.a[i & 3] : r.b[i & 3]);
}

// (the columns past n read as 0)
template <int DT>
__device__ inline void load_chunk(const void* p, int64_t off, int n, bool vec, float (&v)[8]) {
  if (n >= 8 && vec) return load8<DT>(p, off, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < n ? load1<DT>(p, off + i) : 0.0f;
}
// Streaming: a matrix that nothing here reads back at once, larger than the L2s.
template <int DT, bool STREAM = false>
__device__ inline void store_chunk(void* p, int64_t off, int n, bool vec, const float (&v)[8]) {
  if (n >= 8 && vec) {
    if constexpr (!STREAM) return store8<DT>(p, off, v);
    if constexpr (DT == DT_BF16) {
      store_nt(static_cast<uint16_t*>(p) + off, pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
               pack_bf16(v[6], v[7]));
    } else {
      store_nt(static_cast<float*>(p) + off, f2u(v[0]), f2u(v[1]), f2u(v[2]), f2u(v[3]));
      store_nt(static_cast<float*>(p) + off + 4, f2u(v[4]), f2u(v[5]), f2u(v[6]), f2u(v[7]));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) store1<DT>(p, off + i, v[i]);
}

// A unit is 16 bytes of a row: 8 BF16 or 4 FP32 values.  Passes that HBM bounds go by
// units, so that lanes' accesses lie next to each other in both types.
template <int DT>
constexpr int kUnit = DT == DT_BF16 ? 8 : 4;
template <int DT>
__device__ inline raw16 load_unit(const void* p, int64_t off, int n, bool vec) {
  if (n >= kUnit<DT> && vec)
    return *reinterpret_cast<const raw16*>(static_cast<const char*>(p) + off * (DT == DT_BF16 ? 2 : 4));
  return load_raw8<DT>(p, off, n < kUnit<DT> ? n : kUnit<DT>, false).a;
}
template <int DT>
__device__ inline float unit_value(const raw16& r, int i) {
  return raw_value<DT>(RawChunk{r, r}, i);
}
// v: kUnit values, the first n of which are stored, streaming
template <int DT>
__device__ inline void store_unit(void* p, int64_t off, int n, bool vec, const float* v) {
  if (n >= kUnit<DT> && vec) {
    char* q = static_cast<char*>(p) + off * (DT == DT_BF16 ? 2 : 4);
    raw16 r;
    if constexpr (DT == DT_BF16)
      r = raw16{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
    else r = raw16{f2u(v[0]), f2u(v[1]), f2u(v[2]), f2u(v[3])};
    store_nt(q, r[0], r[1], r[2], r[3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < kUnit<DT>; ++i)
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

// The same for FP32 units: lanes 2 j and 2 j + 1 hold the halves of chunk qa in v[0 ..
// 3] and those of chunk qb in v[4 .. 7].  Each lane draws one of them and gives the
// other the half that is its.
__device__ inline void drop_halves(const Drop& d, uint64_t qa, uint64_t qb, float (&v)[8]) {
  const bool odd = threadIdx.x & 1;
  const u32x4 w = rand_words(d.seed, d.counter, odd ? qb : qa);
  const uint32_t g0 = dpp_xor1(odd ? w.x : w.z), g1 = dpp_xor1(odd ? w.y : w.w);
  const uint32_t r[4] = {odd ? g0 : w.x, odd ? g1 : w.y, odd ? w.z : g0, odd ? w.w : g1};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = (i & 1 ? r[i / 2] >> 16 : r[i / 2] & 0xFFFFu) < d.threshold ? 0.0f : v[i] * d.factor;
}

}  // namespace mxk
