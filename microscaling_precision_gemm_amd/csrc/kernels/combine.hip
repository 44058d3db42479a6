// combine.hip -- bringing the rows of a mixture-of-experts product back to
// their tokens, and the gradients of that step.
//   out[t, :]     = sum_j w[t, j] * Y[slot_row[t, j], :]
//   dY[row, :]    = w[t, j] * d_out[t, :]            (row = slot_row[t, j])
//   d_w[t, j]     = sum_c d_out[t, c] * Y[row, c]
// A slot without a row (slot_row < 0, or past Y) adds nothing.  Sums are FP32
// in slot order (out) or in a fixed tree (d_w), so results repeat bit for bit.
// dY is stored, not added to: the rows that slots name are distinct where it is
// wanted.
//
// Both are bound by HBM: Y (or dY) is k times the size of the token matrix, is
// read (written) once and does not fit a cache, so it goes by streaming
// accesses.  Measured: 4096 tokens x 8 rows x 7168 BF16 89 us (5.9 TB/s), with
// 16-byte accesses and a wave for every 16 bytes x 64 of a row; the backward
// pass of 4001 tokens 177 us (5.5 TB/s, half of it writes); one token 6.7 us, of
// which the kernel is 3.4.
#include "../device/rows.h"
#include "../device/wave.h"
#include "../launch_moe.h"

namespace mxk {

namespace {

// 16 bytes of a row, and their values
typedef uint32_t raw4 __attribute__((ext_vector_type(4)));
template <int DT>
constexpr int per_chunk() { return DT == DT_BF16 ? 8 : 4; }

template <int DT>
__device__ inline const char* address(const void* p, int64_t off) {
  return static_cast<const char*>(p) + off * (DT == DT_BF16 ? 2 : 4);
}
// the first n elements of a chunk (the others read as 0: a row may end at its
// last column); `stream`: it is read once
template <int DT, bool STREAM>
__device__ inline raw4 load_raw(const void* p, int64_t off, int n) {
  constexpr int E = per_chunk<DT>();
  if (n == E) {
    const raw4* q = reinterpret_cast<const raw4*>(address<DT>(p, off));
    if constexpr (STREAM) return __builtin_nontemporal_load(q);
    else return *q;
  }
  raw4 r = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (i < n) {
      if constexpr (DT == DT_BF16) r[i / 2] |= (uint32_t)static_cast<const uint16_t*>(p)[off + i] << (16 * (i & 1));
      else r[i] = static_cast<const uint32_t*>(p)[off + i];
    }
  return r;
}
template <int DT>
__device__ inline void widen(const raw4& r, float (&v)[per_chunk<DT>()]) {
  if constexpr (DT == DT_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = u2f(r[i] << 16);
      v[2 * i + 1] = u2f(r[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = u2f(r[i]);
  }
}
// E values to n elements of a row of type ODT; `whole`: all E, 16-byte aligned rows
template <int ODT, int E>
__device__ inline void store_values(void* p, int64_t off, int n, bool whole, const float (&v)[E]) {
  if (whole) {
    if constexpr (ODT == DT_BF16) {
      uint32_t w[E / 2];
#pragma unroll
      for (int i = 0; i < E / 2; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
      char* q = static_cast<char*>(p) + off * 2;
      if constexpr (E == 8) store_nt(q, w[0], w[1], w[2], w[3]);
      else store_nt(q, w[0], w[1]);
    } else {
      char* q = static_cast<char*>(p) + off * 4;
#pragma unroll
      for (int i = 0; i < E; i += 4) store_nt(q + 4 * i, f2u(v[i]), f2u(v[i + 1]), f2u(v[i + 2]), f2u(v[i + 3]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (i < n) store1<ODT>(p, off + i, v[i]);
  }
}

__device__ inline int64_t slot_row_of(const int32_t* slot_row, int64_t slot, int64_t rows) {
  const int64_t r = slot_row[slot];
  return r < rows ? r : -1;
}

// A wave owns 64 consecutive 16-byte chunks of one token's row, so the token's
// row numbers and weights are the same for the whole wave (scalar loads), and
// keeps the loads of up to 8 slots in flight.
constexpr int kThreads = 256;
template <int DT, int ODT>
__global__ __launch_bounds__(kThreads) void k_combine(const void* __restrict__ y, int64_t ld_y, int64_t rows,
                                                      const int32_t* __restrict__ slot_row,
                                                      const float* __restrict__ weights, int64_t tokens, int topk,
                                                      int64_t cols, uint32_t segs, void* __restrict__ out,
                                                      int64_t ld_out, bool vec_out) {
  constexpr int E = per_chunk<DT>();
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t units = tokens * segs;
  for (int64_t unit = (int64_t)blockIdx.x * (kThreads / 64) + wave; unit < units;
       unit += (int64_t)gridDim.x * (kThreads / 64)) {
    const int64_t t = unit <= UINT32_MAX ? (int64_t)((uint32_t)unit / segs) : unit / segs;
    const int64_t c = ((unit - t * segs) * 64 + (threadIdx.x & 63u)) * E;
    if (c >= cols) continue;
    const int n = cols - c < E ? (int)(cols - c) : E;
    float acc[E] = {};
    for (int j0 = 0; j0 < topk; j0 += 8) {
      raw4 v[8];
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        w[j] = 0.0f;
        v[j] = raw4{0, 0, 0, 0};
        const int64_t r = j0 + j < topk ? slot_row_of(slot_row, t * topk + j0 + j, rows) : -1;
        if (r >= 0) {
          w[j] = weights ? weights[t * topk + j0 + j] : 1.0f;
          v[j] = load_raw<DT, true>(y, r * ld_y + c, n);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float f[E];
        widen<DT>(v[j], f);
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = fmaf(w[j], f[i], acc[i]);
      }
    }
    store_values<ODT, E>(out, t * ld_out + c, n, vec_out && n == E, acc);
  }
}

// Sums of 8 values over the wave, by exchanging halves: of two values a lane
// keeps one and gives the other to its neighbour, so three steps leave one
// value a lane and three more add up; lane l ends with the sum of value l % 8.
__device__ inline float wave_sums8(const float (&v)[8], uint32_t lane) {
  float a[4], b[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool o = lane & 1u;
    a[i] = (o ? v[2 * i + 1] : v[2 * i]) + dpp_xor1f(o ? v[2 * i] : v[2 * i + 1]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool o = lane & 2u;
    b[i] = (o ? a[2 * i + 1] : a[2 * i]) + u2f(dpp_xor2(f2u(o ? a[2 * i] : a[2 * i + 1])));
  }
  const bool o = lane & 4u;
  float s = (o ? b[1] : b[0]) + __shfl_xor(o ? b[0] : b[1], 4);
  s += u2f((uint32_t)__builtin_amdgcn_update_dpp(0, (int)f2u(s), 0x128, 0xF, 0xF, false));  // lane ^ 8
  s += __shfl_xor(s, 16);
  s += __shfl_xor(s, 32);
  return s;
}

// One workgroup per token; its waves share the row's segments of 64 chunks.
template <int DT>
__global__ __launch_bounds__(1024) void k_combine_bwd(const void* __restrict__ d_out, int64_t ld_do,
                                                      const void* __restrict__ y, int64_t ld_y, int64_t rows,
                                                      const int32_t* __restrict__ slot_row,
                                                      const float* __restrict__ weights, int64_t tokens, int topk,
                                                      int64_t cols, void* __restrict__ dy, int64_t ld_dy,
                                                      float* __restrict__ d_weights) {
  constexpr int E = per_chunk<DT>();
  __shared__ float red[16][8];
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
    for (int j0 = 0; j0 < topk; j0 += 8) {
      float dot[8] = {};
      for (int64_t c = ((int64_t)wave * 64 + lane) * E; c < cols; c += (int64_t)waves * 64 * E) {
        const int n = cols - c < E ? (int)(cols - c) : E;
        const raw4 graw = load_raw<DT, false>(d_out, t * ld_do + c, n);
        raw4 v[8];
        if (d_weights) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            v[j] = raw4{0, 0, 0, 0};
            const int64_t r = j0 + j < topk ? slot_row_of(slot_row, t * topk + j0 + j, rows) : -1;
            if (r >= 0) v[j] = load_raw<DT, true>(y, r * ld_y + c, n);
          }
        }
        float g[E];
        widen<DT>(graw, g);
        if (dy) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int64_t r = j0 + j < topk ? slot_row_of(slot_row, t * topk + j0 + j, rows) : -1;
            if (r < 0) continue;
            const float w = weights ? weights[t * topk + j0 + j] : 1.0f;
            float o[E];
#pragma unroll
            for (int i = 0; i < E; ++i) o[i] = w * g[i];
            store_values<DT, E>(dy, r * ld_dy + c, n, n == E, o);
          }
        }
        if (d_weights) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float f[E];
            widen<DT>(v[j], f);
#pragma unroll
            for (int i = 0; i < E; ++i) dot[j] = fmaf(g[i], f[i], dot[j]);
          }
        }
      }
      if (d_weights) {
        const float s = wave_sums8(dot, lane);
        if (waves == 1) {
          if (lane < 8 && j0 + (int)lane < topk)
            d_weights[t * topk + j0 + lane] =
                slot_row_of(slot_row, t * topk + j0 + lane, rows) >= 0 ? s : 0.0f;
          continue;
        }
        if (lane < 8) red[wave][lane] = s;
        __syncthreads();
        if (threadIdx.x < 8 && j0 + (int)threadIdx.x < topk) {
          float sum = red[0][threadIdx.x];
          for (uint32_t w = 1; w < waves; ++w) sum += red[w][threadIdx.x];
          // (0, not 0 times what d_out holds, for a slot without a row)
          d_weights[t * topk + j0 + threadIdx.x] =
              slot_row_of(slot_row, t * topk + j0 + threadIdx.x, rows) >= 0 ? sum : 0.0f;
        }
        __syncthreads();
      }
    }
  }
}

}  // namespace

hipError_t launch_combine(const void* y, int ydt, int64_t ld_y, int64_t rows, const int32_t* slot_row,
                          const float* weights, int64_t tokens, int topk, int64_t cols, void* out, int odt,
                          int64_t ld_out, hipStream_t s) {
  const uint32_t segs = (uint32_t)((cols + (ydt == DT_BF16 ? 511 : 255)) / (ydt == DT_BF16 ? 512 : 256));
  const int64_t need = (tokens * segs + kThreads / 64 - 1) / (kThreads / 64);
  const uint32_t blocks = (uint32_t)(need < (1 << 20) ? need : (1 << 20));
  const int64_t eb = odt == DT_F32 ? 4 : 2;
  const bool vec = (reinterpret_cast<uintptr_t>(out) & 15u) == 0 && (ld_out * eb) % 16 == 0;
#define MXK_CB(D, O)                                                                                             \
  hipLaunchKernelGGL((k_combine<D, O>), dim3(blocks), dim3(kThreads), 0, s, y, ld_y, rows, slot_row, \
                     weights, tokens, topk, cols, segs, out, ld_out, vec)
  if (ydt == DT_BF16) {
    if (odt == DT_BF16) MXK_CB(DT_BF16, DT_BF16);
    else MXK_CB(DT_BF16, DT_F32);
  } else {
    if (odt == DT_BF16) MXK_CB(DT_F32, DT_BF16);
    else MXK_CB(DT_F32, DT_F32);
  }
#undef MXK_CB
  return hipGetLastError();
}

hipError_t launch_combine_bwd(const void* d_out, int dt, int64_t ld_do, const void* y, int64_t ld_y, int64_t rows,
                              const int32_t* slot_row, const float* weights, int64_t tokens, int topk,
                              int64_t cols, void* dy, int64_t ld_dy, float* d_weights, hipStream_t s) {
  const int g = (int)(tokens < (1 << 20) ? tokens : (1 << 20));
  // Waves: the row's segments in equal shares, 8 waves at most while the
  // tokens fill the CUs, else 16.
  const int64_t segs = (cols + (dt == DT_BF16 ? 511 : 255)) / (dt == DT_BF16 ? 512 : 256);
  const int64_t most = tokens < 512 ? 16 : 8;
  const int64_t rounds = (segs + most - 1) / most;
  const int threads = segs ? (int)((segs + rounds - 1) / rounds) * 64 : 64;
  if (dt == DT_BF16)
    hipLaunchKernelGGL(k_combine_bwd<DT_BF16>, dim3(g), dim3(threads), 0, s, d_out, ld_do, y, ld_y, rows, slot_row,
                       weights, tokens, topk, cols, dy, ld_dy, d_weights);
  else
    hipLaunchKernelGGL(k_combine_bwd<DT_F32>, dim3(g), dim3(threads), 0, s, d_out, ld_do, y, ld_y, rows, slot_row,
                       weights, tokens, topk, cols, dy, ld_dy, d_weights);
  return hipGetLastError();
}

}  // namespace mxk
