// linear.hip -- the product of BF16 activations with block-scaled weights, and the
// epilogue behind it:
//   z = X W^T + bias,   out = residual + drop(act(z))
// X [M, K] BF16, W [N, K] in an MX format or NVFP4, decoded to BF16 on its way to
// the matrix instruction (v_mfma_f32_16x16x32_bf16: exact products, FP32 sums).
//
// The weights are the first operand of the instruction and the tokens the second,
// so a lane holds 4 neighbouring columns of one token's row.  The order of the 32
// elements of K within an instruction is free as long as both operands agree: a
// lane takes the 32 consecutive elements that share its block scale (one 16-byte
// load of 4-bit codes), and instruction j of four takes elements 8 j .. 8 j + 7
// of every lane.
#include <atomic>

#include "../device/linear_epilogue.h"
#include "../device/weights.h"

namespace mxk {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

// ---- operands straight from memory -----------------------------------------
// A workgroup of NW waves takes a tile of 16 TM tokens x 16 TN columns; its waves
// share out the steps of K and add their sums through LDS, in order.  A step is
// 128 bytes of a weight row (256 4-bit or 128 8-bit elements): lane group g of
// four takes 32 bytes of them.
template <int FMT, int TM, int TN, int NW>
__global__ __launch_bounds__(NW * 64) void k_linear_direct(LinearArgs a, EpilogueVec vec, uint32_t tiles_m) {
  constexpr int B = kFourBit<FMT> ? 2 : 1;  // blocks of 32 a lane and step
  constexpr int kPitch = TN * 16 + 4;       // floats of a token's row in LDS
  extern __shared__ __attribute__((aligned(16))) float red[];
  const uint32_t lane = threadIdx.x & 63u, wid = threadIdx.x >> 6, l = lane & 15u, g = lane >> 4;
  const int64_t m0 = (int64_t)(blockIdx.x % tiles_m) * (16 * TM), n0 = (int64_t)(blockIdx.x / tiles_m) * (16 * TN);
  const int64_t row_bytes = a.K / 32 * kBlockBytes<FMT>, blocks = a.K / 32;

  const uint8_t* w[TN];
  int64_t first[TN];  // block number of the row's first block
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    int64_t n = n0 + 16 * j + l;
    n = n < a.N ? n : a.N - 1;  // (columns past N are not stored)
    w[j] = a.codes + n * row_bytes;
    first[j] = n * blocks;
  }
  const uint16_t* x[TM];
  bool there[TM];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int64_t m = m0 + 16 * i + l;
    there[i] = m < a.M;
    x[i] = a.x + (there[i] ? m : 0) * a.ld_x;
  }

  v4f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0, 0, 0, 0};

  const int64_t steps = (blocks + 4 * B - 1) / (4 * B);
  for (int64_t st = wid; st < steps; st += NW) {
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int64_t blk = st * 4 * B + g * B + b;
      const bool in = blk < blocks;
      word4 cw[TN][2];
      uint32_t sc[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        sc[j] = 0;
        cw[j][0] = cw[j][1] = word4{0, 0, 0, 0};
        if (in) {
          const word4* p = reinterpret_cast<const word4*>(w[j] + blk * kBlockBytes<FMT>);
          cw[j][0] = p[0];
          if constexpr (!kFourBit<FMT>) cw[j][1] = p[1];
          sc[j] = load_scale<FMT>(a.scales, first[j] + blk);
        }
      }
      word4 xv[TM][4];
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          xv[i][e] = word4{0, 0, 0, 0};
          if (in && there[i]) xv[i][e] = *reinterpret_cast<const word4*>(x[i] + blk * 32 + e * 8);
        }
      auto eighth = [&](auto num) {
        constexpr int J = decltype(num)::value;
        bf16x8 wb[TN];
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          uint32_t u[8];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            u[q] = cw[j][0][q];
            u[4 + q] = cw[j][1][q];
          }
          wb[j] = decode_eighth<FMT, J>(u, sc[j]);
        }
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j], __builtin_bit_cast(bf16x8, xv[i][J]),
                                                                acc[i][j], 0, 0, 0);
      };
      eighth(std::integral_constant<int, 0>());
      eighth(std::integral_constant<int, 1>());
      eighth(std::integral_constant<int, 2>());
      eighth(std::integral_constant<int, 3>());
    }
  }

  float* mine = red + (size_t)wid * (16 * TM * kPitch);
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
      *reinterpret_cast<v4f*>(mine + (16 * i + l) * kPitch + 16 * j + 4 * g) = acc[i][j];
  __syncthreads();

  const float ts = FMT == FMT_NVFP4 ? *a.tensor_scale : 1.0f;
  for (uint32_t q = threadIdx.x; q < 32u * TM * TN; q += NW * 64) {
    const uint32_t t = q / (2 * TN), c = (q % (2 * TN)) * 8;
    const int64_t row = m0 + t, col = n0 + c;
    if (row >= a.M || col >= a.N) continue;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const float* p = red + (size_t)k * (16 * TM * kPitch) + t * kPitch + c;
      const v4f lo = *reinterpret_cast<const v4f*>(p), hi = *reinterpret_cast<const v4f*>(p + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] += lo[i];
        v[4 + i] += hi[i];
      }
    }
    if constexpr (FMT == FMT_NVFP4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= ts;
    }
    const int n = (int)(a.N - col < 8 ? a.N - col : 8);
    if (a.ep.dt == DT_BF16) epilogue_chunk<DT_BF16>(a.ep, vec, row, col, a.N, n, v);
    else epilogue_chunk<DT_F32>(a.ep, vec, row, col, a.N, n, v);
  }
}

// Raise a kernel's dynamic LDS limit once per device, so that later launches
// (also inside HIP graphs) make no call beyond the launch itself.
hipError_t allow_lds(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (!bit || !(done.load(std::memory_order_acquire) & bit)) {
    e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    done.fetch_or(bit, std::memory_order_acq_rel);
  }
  return hipSuccess;
}

template <int FMT, int TM, int TN, int NW>
hipError_t launch_direct(const LinearArgs& a, hipStream_t s) {
  constexpr int kLds = NW * 16 * TM * (TN * 16 + 4) * 4;
  static_assert(kLds <= 160 * 1024, "LDS of a workgroup");
  auto kernel = k_linear_direct<FMT, TM, TN, NW>;
  static std::atomic<uint64_t> done{0};
  const hipError_t e = allow_lds((const void*)kernel, kLds, done);
  if (e != hipSuccess) return e;
  const int64_t tm = (a.M + 16 * TM - 1) / (16 * TM), tn = (a.N + 16 * TN - 1) / (16 * TN);
  hipLaunchKernelGGL(kernel, dim3((uint32_t)(tm * tn)), dim3(NW * 64), kLds, s, a, epilogue_vec(a.ep), (uint32_t)tm);
  return hipGetLastError();
}

template <int FMT>
hipError_t launch_fmt(const LinearArgs& a, hipStream_t s) {
  if (a.M <= 16) return launch_direct<FMT, 1, 1, 8>(a, s);
  if (a.M <= 32) return launch_direct<FMT, 2, 2, 8>(a, s);
  return launch_direct<FMT, 4, 4, 4>(a, s);
}

}  // namespace

hipError_t launch_linear(const LinearArgs& a, hipStream_t s) {
  switch (a.fmt) {
    case FMT_MXFP8: return launch_fmt<FMT_MXFP8>(a, s);
    case FMT_MXFP8_E5M2: return launch_fmt<FMT_MXFP8_E5M2>(a, s);
    case FMT_MXINT8: return launch_fmt<FMT_MXINT8>(a, s);
    case FMT_NVFP4: return launch_fmt<FMT_NVFP4>(a, s);
    default: return launch_fmt<FMT_MXFP4>(a, s);
  }
}

}  // namespace mxk
