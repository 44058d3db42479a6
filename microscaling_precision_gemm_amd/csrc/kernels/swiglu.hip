// swiglu.hip -- the gated activation between the two products of an expert,
// its 8-bit checkpoint and its backward pass from that checkpoint.
//   h = [gate | up],  s = 1 / (1 + exp(-gate)),  y = gate * s * up
//   saved = Q8(h): h block-scaled to 8 bits along its rows, exactly the codes
//   and scales the quantizer gives ("Thinking Machines ... Inkling 2 Small",
//   section "A precision choice for each stage": saved forward tensors are
//   kept quantized and decoded again for the backward pass)
//   from h' = dec(saved):  d_gate = dy * up' * s' * (1 + gate' * (1 - s'))
//                          d_up   = dy * gate' * s'
// All steps are FP32; y, dh are rounded once.
//
// Bound by HBM.  A lane takes 8 consecutive gate elements and the 8 up
// elements beside them, a lane quad one 32-element block of each half, so the
// block maxima need two DPP steps and h is read once for both results.
// Measured, 32768 x 2048 BF16: forward 71 us (5.7 TB/s), with an MXFP8
// checkpoint 105 us (5.1 TB/s) and max |y| 116 us (4.6 TB/s: few workgroups, see
// kMaxGrid), backward 99 us (5.5 TB/s), and with the operand of the next weight
// gradient 114 us (5.3 TB/s).  Of these 2 to 6 us are the sigmoid's corrections:
// a wave of the backward pass issues 250 vector instructions for 8 elements a
// lane (200 without them), about two thirds of its time.
#include "../device/codec.h"
#include "../device/cvt.h"
#include "../device/decode8.h"
#include "../device/exp.h"
#include "../device/mxenc.h"
#include "../device/rows.h"
#include "../device/wave.h"
#include "../launch_moe.h"

namespace mxk {

namespace {

constexpr int kThreads = 256;
// With max |y| a workgroup that has a new one does an atomic on one word, and
// these serialize, so there are few, large workgroups that walk over the tensor
// and look at the word just before (32768 x 2048 BF16 with an MXFP8
// checkpoint: 110 us; 122 with a workgroup per 1024 chunks that looked at its
// start, 206 with one per 512 that did not look; 4099 x 4096 FP32: 47 us, 56
// with a workgroup per 1024 chunks; all with a sigmoid that took 6 us less).
constexpr int kMaxThreads = 1024, kMaxGrid = 256;
constexpr int64_t kOneChunks = 4096;  // tensors up to this go to one workgroup

__global__ void k_clear(float* p) { *p = 0.0f; }

// row and 8-column chunk of chunk q of a matrix with cpr chunks a row
__device__ inline void locate(int64_t q, int64_t cpr, int64_t* r, int64_t* c) {
  if (q <= UINT32_MAX && cpr <= UINT32_MAX) *r = (uint32_t)q / (uint32_t)cpr;
  else *r = q / cpr;
  *c = q - *r * cpr;
}

// largest of the workgroup's bit patterns (FP32 bits of non-negative values
// order as integers; the order of the maxima is no matter), in thread 0
__device__ inline uint32_t block_max(uint32_t m) {
  __shared__ uint32_t red[kMaxThreads / 64];
  m = wave_max_u32(m);
  if ((threadIdx.x & 63u) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x == 0)
    for (uint32_t w = 1; w < blockDim.x / 64; ++w) m = red[w] > m ? red[w] : m;
  return m;
}

// FMT 0: nothing is saved.  Q chunks of 8 columns, cpr of them in a row, one a
// thread: HBM was fullest with as many small waves as there are chunks (at
// 32768 x 2048 BF16 without a checkpoint 5.8 TB/s, against 5.6 with two chunks
// a thread and 5.4 with workgroups that walk over the tensor, all with a shorter
// sigmoid).  AMAX 0: not
// wanted; 1: the workgroup is alone, so *amax needs no clearing before and no
// atomic; 2: *amax is cleared before.
template <int DT, int FMT, bool SR, int AMAX>
__global__ __launch_bounds__(AMAX ? kMaxThreads : kThreads) void k_swiglu(
    const void* __restrict__ h, int64_t ld_h, int64_t cpr, int64_t Q, void* __restrict__ y, int64_t ld_y,
    uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, MxEnc enc, float* __restrict__ amax) {
  constexpr int T = AMAX ? kMaxThreads : kThreads;
  const int64_t cols = 8 * cpr;
  uint32_t* const top = reinterpret_cast<uint32_t*>(amax);
  uint32_t m = 0;
  // (lane quads stand or fall together: Q and a workgroup's chunks are multiples of 4)
  for (int64_t q = (int64_t)blockIdx.x * T + threadIdx.x; q < Q; q += (int64_t)gridDim.x * T) {
    int64_t r, c;
    locate(q, cpr, &r, &c);
    float g[8], u[8], v[8];
    load8<DT>(h, r * ld_h + 8 * c, g);
    load8<DT>(h, r * ld_h + cols + 8 * c, u);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = g[k] * sigmoid(g[k]) * u[k];
    store8<DT>(y, r * ld_y + 8 * c, v);
    if constexpr (AMAX != 0) {
      if constexpr (DT == DT_BF16) {  // of the values as stored
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = u2f(pack_bf16(v[k], v[k]) << 16);
      }
      const uint32_t o = max_abs_bits(v);
      m = o > m ? o : m;
    }
    if constexpr (FMT != 0) {
      const int64_t qg = r * 2 * cpr + c, qu = qg + cpr;  // chunks of the saved [rows, 2 cols] tensor
      Enc<FMT> eg, eu;
      encode_mx<FMT, SR>(enc, qg, g, eg);
      encode_mx<FMT, SR>(enc, qu, u, eu);
      *reinterpret_cast<uint2*>(codes + 8 * qg) = make_uint2(eg.w[0], eg.w[1]);
      *reinterpret_cast<uint2*>(codes + 8 * qu) = make_uint2(eu.w[0], eu.w[1]);
      if ((c & 3) == 0) {
        scales[qg >> 2] = (uint8_t)eg.sc;
        scales[qu >> 2] = (uint8_t)eu.sc;
      }
    }
  }
  if constexpr (AMAX != 0) {
    m = block_max(m);
    if (threadIdx.x == 0) {
      if constexpr (AMAX == 1) *top = m;
      else if (m > __hip_atomic_load(top, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) atomicMax(top, m);
    }
  }
}

// 8 elements of an 8-bit MX format times their block scale, exactly
template <int FMT>
__device__ inline void decode8(uint2 w, uint32_t sc, float (&v)[8]) {
  decode4_f32<FMT>(w.x, sc, v);
  decode4_f32<FMT>(w.y, sc, v + 4);
}

template <int DT, int FMT, int YFMT>
__global__ __launch_bounds__(kThreads) void k_swiglu_bwd(const uint8_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales, int64_t cpr, int64_t Q,
                                                         const void* __restrict__ dy, int64_t ld_dy,
                                                         void* __restrict__ dh, int64_t ld_dh,
                                                         uint8_t* __restrict__ y_codes,
                                                         uint8_t* __restrict__ y_scales) {
  const int64_t cols = 8 * cpr;
  for (int64_t q = (int64_t)blockIdx.x * kThreads + threadIdx.x; q < Q; q += (int64_t)gridDim.x * kThreads) {
    int64_t r, c;
    locate(q, cpr, &r, &c);
    const int64_t qg = r * 2 * cpr + c, qu = qg + cpr;
    float g[8], u[8], d[8], y[8];
    decode8<FMT>(*reinterpret_cast<const uint2*>(codes + 8 * qg), scales[qg >> 2], g);
    decode8<FMT>(*reinterpret_cast<const uint2*>(codes + 8 * qu), scales[qu >> 2], u);
    load8<DT>(dy, r * ld_dy + 8 * c, d);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float s = sigmoid(g[k]), gs = g[k] * s;
      const float dg = d[k] * u[k] * (s * fmaf(g[k], 1.0f - s, 1.0f));
      const float du = d[k] * gs;
      y[k] = gs * u[k];
      g[k] = dg;
      u[k] = du;
    }
    store8<DT>(dh, r * ld_dh + 8 * c, g);
    store8<DT>(dh, r * ld_dh + cols + 8 * c, u);
    if constexpr (YFMT != 0) {
      Enc<YFMT> e;
      encode_mx<YFMT, false>(MxEnc{false, 0, 0}, q, y, e);
      *reinterpret_cast<uint2*>(y_codes + 8 * q) = make_uint2(e.w[0], e.w[1]);
      if ((c & 3) == 0) y_scales[q >> 2] = (uint8_t)e.sc;
    }
  }
}

// a thread per chunk, up to the largest grid
int grid_of(int64_t Q, int threads, int64_t most = 1 << 21) {
  const int64_t g = (Q + threads - 1) / threads;
  return (int)(g < most ? g : most);
}

template <int DT, int FMT>
void swiglu_f(const SwigluArgs& a, int64_t Q, hipStream_t s) {
  const MxEnc enc{false, a.seed, a.counter};
#define MXK_SG(SR, AMAX, GRID, T)                                                                              \
  hipLaunchKernelGGL((k_swiglu<DT, FMT, SR, AMAX>), dim3(GRID), dim3(T), 0, s, a.h, a.ld_h, a.cols / 8, Q, a.y, \
                     a.ld_y, a.codes, a.scales, enc, a.amax)
#define MXK_SGA(SR)                                                               \
  if (!a.amax) MXK_SG(SR, 0, grid_of(Q, kThreads), kThreads);                     \
  else if (Q <= kOneChunks) MXK_SG(SR, 1, 1, kMaxThreads);                        \
  else MXK_SG(SR, 2, grid_of(Q, kMaxThreads, kMaxGrid), kMaxThreads)
  if (FMT != 0 && a.sr) {
    MXK_SGA((FMT != 0));
  } else {
    MXK_SGA(false);
  }
#undef MXK_SGA
#undef MXK_SG
}

template <int DT>
void swiglu_d(const SwigluArgs& a, int64_t Q, hipStream_t s) {
  switch (a.fmt) {
    case FMT_MXFP8: return swiglu_f<DT, FMT_MXFP8>(a, Q, s);
    case FMT_MXFP8_E5M2: return swiglu_f<DT, FMT_MXFP8_E5M2>(a, Q, s);
    case FMT_MXINT8: return swiglu_f<DT, FMT_MXINT8>(a, Q, s);
    default: return swiglu_f<DT, 0>(a, Q, s);
  }
}

template <int DT, int FMT>
void bwd_f(const SwigluBwdArgs& a, int64_t Q, hipStream_t s) {
#define MXK_SB(Y)                                                                                                  \
  hipLaunchKernelGGL((k_swiglu_bwd<DT, FMT, Y>), dim3(grid_of(Q, kThreads)), dim3(kThreads), 0, s, a.codes, a.scales,     \
                     a.cols / 8, Q, a.dy, a.ld_dy, a.dh, a.ld_dh, a.y_codes, a.y_scales)
  switch (a.y_fmt) {
    case FMT_MXFP8: MXK_SB(FMT_MXFP8); break;
    case FMT_MXFP8_E5M2: MXK_SB(FMT_MXFP8_E5M2); break;
    case FMT_MXINT8: MXK_SB(FMT_MXINT8); break;
    default: MXK_SB(0); break;
  }
#undef MXK_SB
}

template <int DT>
void bwd_d(const SwigluBwdArgs& a, int64_t Q, hipStream_t s) {
  switch (a.fmt) {
    case FMT_MXFP8: return bwd_f<DT, FMT_MXFP8>(a, Q, s);
    case FMT_MXFP8_E5M2: return bwd_f<DT, FMT_MXFP8_E5M2>(a, Q, s);
    default: return bwd_f<DT, FMT_MXINT8>(a, Q, s);
  }
}

}  // namespace

hipError_t launch_swiglu(const SwigluArgs& a, hipStream_t s) {
  const int64_t Q = a.rows * (a.cols / 8);
  if (a.amax && (Q == 0 || Q > kOneChunks)) hipLaunchKernelGGL(k_clear, dim3(1), dim3(1), 0, s, a.amax);
  if (Q > 0) {
    if (a.dt == DT_BF16) swiglu_d<DT_BF16>(a, Q, s);
    else swiglu_d<DT_F32>(a, Q, s);
  }
  return hipGetLastError();
}

hipError_t launch_swiglu_bwd(const SwigluBwdArgs& a, hipStream_t s) {
  const int64_t Q = a.rows * (a.cols / 8);
  if (a.dt == DT_BF16) bwd_d<DT_BF16>(a, Q, s);
  else bwd_d<DT_F32>(a, Q, s);
  return hipGetLastError();
}

}  // namespace mxk
