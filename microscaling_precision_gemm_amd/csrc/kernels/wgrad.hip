// wgrad.hip -- the weight gradients of a grouped product from saved 8-bit
// activations:
//   dW_e[n, k] = sum over the rows r of group e of dY[r, n] * X[src(r), k]
// with dY in BF16, X an 8-bit block-scaled checkpoint (E4M3, E5M2 or INT8,
// blocks along k) read through an optional row index.  The checkpoint's
// blocks lie along k and the sum runs over rows, so no block scale is common
// to a sum: elements are decoded to BF16 (exact for scale codes 10 .. 254) on
// the way into LDS and contracted on the BF16 matrix instruction, whose
// products are exact in the FP32 sums.  Both operands have the summed index as
// their rows, so the fragments are read transposed out of LDS
// (ds_read_b64_tr_b16: 16 lanes turn 4 rows x 16 columns into 4 row values of
// one column each).
#include <type_traits>

#include "../device/decode8.h"
#include "../device/gemm_common.h"
#include "../launch.h"

namespace mxk {

namespace {

typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s* lds_v4s;

constexpr int kTileN = 128, kTileK = 128, kStep = 32;
constexpr int kPitch = 128 + 8;  // BF16 elements of one LDS row

struct WgradParams {
  const uint16_t* dy;
  int64_t ld_dy, R, N;
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t x_rows, K;
  const int32_t* row_index;
  const int64_t* offsets;  // nullptr: one group of all rows
  int32_t groups;
  void* dw;
  int64_t ld_dw;
  uint32_t tn, tk;
};

// an operand fragment of 32 columns x 16 rows at (row, col) of an LDS tile:
// lane l holds column l % 32, rows 8 (l / 32) .. + 7
__device__ inline v8b frag(const uint16_t* tile, int row, int col, uint32_t lane) {
  const uint32_t s = lane & 15u, g = lane >> 4;
  const uint16_t* p = tile + (row + 8 * (g >> 1) + (s >> 2)) * kPitch + col + 16 * (g & 1) + 4 * (s & 3);
  union {
    v4s h[2];
    v8b v;
  } u;
  u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)p);
  u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(p + 4 * kPitch));
  return u.v;
}

template <int FMT, int WDT, bool ACC>
__global__ __launch_bounds__(256) void k_wgrad(WgradParams p) {
  __shared__ __attribute__((aligned(16))) uint16_t A[kStep * kPitch], B[kStep * kPitch];
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wid = tid >> 6;
  const int wn = (wid >> 1) * 64, wk = (wid & 1) * 64;
  const int64_t total = (int64_t)p.tn * p.tk * p.groups;
  for (int64_t id = blockIdx.x; id < total; id += gridDim.x) {
    const int32_t e = (int32_t)(id / ((int64_t)p.tn * p.tk));
    const uint32_t in = (uint32_t)(id - (int64_t)e * p.tn * p.tk);
    const int64_t n0 = (int64_t)(in / p.tk) * kTileN, k0 = (int64_t)(in % p.tk) * kTileK;
    int64_t lo = 0, hi = p.R;
    if (p.offsets) {  // clamped into [0, R]
      lo = p.offsets[e];
      hi = p.offsets[e + 1];
      lo = lo < 0 ? 0 : (lo > p.R ? p.R : lo);
      hi = hi < lo ? lo : (hi > p.R ? p.R : hi);
    }
    v16f acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
    for (int64_t r0 = lo; r0 < hi; r0 += kStep) {
      // dY: 32 rows x 16 chunks of 8 columns
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t q = tid + 256 * h;
        const int row = q >> 4, c = (q & 15) * 8;
        const int64_t r = r0 + row, n = n0 + c;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (r < hi) {
          if (n + 8 <= p.N) {
            w = *reinterpret_cast<const uint4*>(p.dy + r * p.ld_dy + n);
          } else {
            uint32_t* ww = reinterpret_cast<uint32_t*>(&w);
            for (int i = 0; i < 8; ++i)
              if (n + i < p.N) ww[i >> 1] |= (uint32_t)p.dy[r * p.ld_dy + n + i] << (16 * (i & 1));
          }
        }
        *reinterpret_cast<uint4*>(A + row * kPitch + c) = w;
      }
      // X: 32 rows x 8 chunks of 16 codes
      {
        const int row = tid >> 3, c = (tid & 7) * 16;
        const int64_t r = r0 + row, k = k0 + c;
        uint32_t o[8] = {};
        if (r < hi && k < p.K) {
          int64_t src = r;
          if (p.row_index) {
            src = p.row_index[r];
            src = src < 0 ? 0 : (src < p.x_rows ? src : p.x_rows - 1);
          }
          const uint4 w = *reinterpret_cast<const uint4*>(p.codes + src * p.K + k);
          const uint32_t sc = p.scales[src * (p.K / 32) + k / 32];
          decode4_bf16<FMT>(w.x, sc, o);
          decode4_bf16<FMT>(w.y, sc, o + 2);
          decode4_bf16<FMT>(w.z, sc, o + 4);
          decode4_bf16<FMT>(w.w, sc, o + 6);
        }
        *reinterpret_cast<uint4*>(B + row * kPitch + c) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(B + row * kPitch + c + 8) = make_uint4(o[4], o[5], o[6], o[7]);
      }
      __syncthreads();
#pragma unroll
      for (int s = 0; s < kStep; s += 16) {
        v8b a[2], b[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          a[i] = frag(A, s, wn + 32 * i, lane);
          b[i] = frag(B, s, wk + 32 * i, lane);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int64_t n = n0 + wn + 32 * i + 8 * (v / 4) + 4 * (lane >> 5) + (v % 4);
          const int64_t k = k0 + wk + 32 * j + (lane & 31u);
          if (n < p.N && k < p.K) {
            const int64_t off = ((int64_t)e * p.N + n) * p.ld_dw + k;
            float o = acc[i][j][v];
            if constexpr (ACC) o += load1<WDT>(p.dw, off);
            store1<WDT>(p.dw, off, o);
          }
        }
  }
}

}  // namespace

hipError_t launch_wgrad_grouped(const WgradArgs& a, hipStream_t s) {
  WgradParams p = {a.dy, a.ld_dy, a.R, a.N, a.codes, a.scales, a.x_rows, a.K, a.row_index, a.offsets, a.groups,
                   a.dw, a.ld_dw, (uint32_t)((a.N + kTileN - 1) / kTileN), (uint32_t)((a.K + kTileK - 1) / kTileK)};
  const int64_t total = (int64_t)p.tn * p.tk * p.groups;
  const uint32_t g = (uint32_t)(total < (1 << 20) ? total : (1 << 20));
  auto go = [&](auto fmt) {
    constexpr int F = decltype(fmt)::value;
    if (a.dwdt == DT_F32) {
      if (a.accumulate) hipLaunchKernelGGL((k_wgrad<F, DT_F32, true>), dim3(g), dim3(256), 0, s, p);
      else hipLaunchKernelGGL((k_wgrad<F, DT_F32, false>), dim3(g), dim3(256), 0, s, p);
    } else {
      if (a.accumulate) hipLaunchKernelGGL((k_wgrad<F, DT_BF16, true>), dim3(g), dim3(256), 0, s, p);
      else hipLaunchKernelGGL((k_wgrad<F, DT_BF16, false>), dim3(g), dim3(256), 0, s, p);
    }
  };
  if (a.fmt == FMT_MXFP8) go(std::integral_constant<int, FMT_MXFP8>());
  else if (a.fmt == FMT_MXFP8_E5M2) go(std::integral_constant<int, FMT_MXFP8_E5M2>());
  else go(std::integral_constant<int, FMT_MXINT8>());
  return hipGetLastError();
}

}  // namespace mxk
