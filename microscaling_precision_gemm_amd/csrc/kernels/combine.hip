// combine.hip -- bringing the rows of a mixture-of-experts product back to
// their tokens, and the gradients of that step.
//   out[t, :]     = sum_j w[t, j] * Y[slot_row[t, j], :]
//   dY[row, :]    = w[t, j] * d_out[t, :]            (row = slot_row[t, j])
//   d_w[t, j]     = sum_c d_out[t, c] * Y[row, c]
// A slot without a row (slot_row < 0, or past Y) adds nothing.  Sums are FP32
// in slot order (out) or in a fixed tree (d_w), so results repeat bit for bit.
//
// Both are bound by HBM: Y (or dY) is k times the size of the token matrix.
#include "../device/rows.h"
#include "../launch.h"

namespace mxk {

namespace {

constexpr int kThreads = 256;

// A wave owns 64 consecutive 8-element chunks of one token's row, so the
// token's row numbers and weights are the same for the whole wave, and keeps
// the loads of up to 8 slots in flight.
template <int DT, int ODT>
__global__ __launch_bounds__(kThreads) void k_combine(const void* __restrict__ y, int64_t ld_y, int64_t rows,
                                                      const int32_t* __restrict__ slot_row,
                                                      const float* __restrict__ weights, int64_t tokens, int topk,
                                                      int64_t cols, uint32_t segs, void* __restrict__ out,
                                                      int64_t ld_out, bool vec_out) {
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t units = tokens * segs;
  for (int64_t unit = (int64_t)blockIdx.x * (kThreads / 64) + wave; unit < units;
       unit += (int64_t)gridDim.x * (kThreads / 64)) {
    const int64_t t = unit / segs;
    const int64_t c = ((unit - t * segs) * 64 + (threadIdx.x & 63u)) * 8;
    if (c >= cols) continue;
    const int n = cols - c < 8 ? (int)(cols - c) : 8;
    float acc[8] = {};
    for (int j0 = 0; j0 < topk; j0 += 8) {
      float v[8][8];
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        w[j] = 0.0f;
        const int64_t r = j0 + j < topk ? slot_row[t * topk + j0 + j] : -1;
        if (r >= 0 && r < rows) {
          w[j] = weights ? weights[t * topk + j0 + j] : 1.0f;
          load_n<DT>(y, r * ld_y + c, n, n == 8, v[j]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(w[j], v[j][i], acc[i]);
    }
    store_n<ODT>(out, t * ld_out + c, n, vec_out && n == 8, acc);
  }
}

// One workgroup per token; its waves share the row's segments of 64 chunks
// and reduce the products of up to 8 slots at a time.
template <int DT>
__global__ __launch_bounds__(kThreads) void k_combine_bwd(const void* __restrict__ d_out, int64_t ld_do,
                                                          const void* __restrict__ y, int64_t ld_y, int64_t rows,
                                                          const int32_t* __restrict__ slot_row,
                                                          const float* __restrict__ weights, int64_t tokens,
                                                          int topk, int64_t cols, void* __restrict__ dy,
                                                          int64_t ld_dy, float* __restrict__ d_weights) {
  __shared__ float red[kThreads / 64][8];
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
    for (int j0 = 0; j0 < topk; j0 += 8) {
      float dot[8] = {};
      for (int64_t c = (wave * 64 + lane) * 8; c < cols; c += kThreads * 8) {
        const int n = cols - c < 8 ? (int)(cols - c) : 8;
        float g[8];
        load_n<DT>(d_out, t * ld_do + c, n, n == 8, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int64_t r = j0 + j < topk ? slot_row[t * topk + j0 + j] : -1;
          if (r < 0 || r >= rows) continue;
          if (d_weights) {
            float v[8];
            load_n<DT>(y, r * ld_y + c, n, n == 8, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot[j] = fmaf(g[i], v[i], dot[j]);
          }
          if (dy) {
            const float w = weights ? weights[t * topk + j0 + j] : 1.0f;
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = w * g[i];
            store_n<DT>(dy, r * ld_dy + c, n, n == 8, o);
          }
        }
      }
      if (d_weights) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          for (int off = 32; off >= 1; off >>= 1) dot[j] += __shfl_xor(dot[j], off);
        if (lane == 0) {
#pragma unroll
          for (int j = 0; j < 8; ++j) red[wave][j] = dot[j];
        }
        __syncthreads();
        if (threadIdx.x < 8 && j0 + (int)threadIdx.x < topk) {
          float s = red[0][threadIdx.x];
          for (int w = 1; w < kThreads / 64; ++w) s += red[w][threadIdx.x];
          d_weights[t * topk + j0 + threadIdx.x] = s;
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
  const uint32_t segs = (uint32_t)((cols + 511) / 512);
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
  if (dt == DT_BF16)
    hipLaunchKernelGGL(k_combine_bwd<DT_BF16>, dim3(g), dim3(kThreads), 0, s, d_out, ld_do, y, ld_y, rows, slot_row,
                       weights, tokens, topk, cols, dy, ld_dy, d_weights);
  else
    hipLaunchKernelGGL(k_combine_bwd<DT_F32>, dim3(g), dim3(kThreads), 0, s, d_out, ld_do, y, ld_y, rows, slot_row,
                       weights, tokens, topk, cols, dy, ld_dy, d_weights);
  return hipGetLastError();
}

}  // namespace mxk
