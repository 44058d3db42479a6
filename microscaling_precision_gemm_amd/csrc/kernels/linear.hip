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

// ---- operands through LDS ---------------------------------------------------
// A workgroup takes a tile of BM tokens x BN columns, each wave WM x WN of it
// (v_mfma_f32_32x32x16_bf16).  A stage holds 64 elements of K of every row:
// 128 bytes of X, 32 or 64 bytes of codes, copied to LDS by 16-byte
// global-to-LDS loads, three stages in a ring, so that one barrier a stage is
// enough: behind it the stage has landed for all waves and the one before it is
// no longer read.  Lane half h takes elements 32 h .. 32 h + 31 of a stage
// (one block), 8 of them for each of four instructions; W is decoded from the
// codes as it leaves LDS.  The 16-byte chunks of a row are exchanged by row
// number on their way in, so that 16 neighbouring rows' chunks lie in all banks.
typedef float v16f __attribute__((ext_vector_type(16)));

template <int FMT, int BM, int BN>
struct Stage {
  static constexpr int kXBytes = BM * 128;
  static constexpr int kRow = 2 * kBlockBytes<FMT>;  // code bytes of a row
  static constexpr int kBytes = kXBytes + BN * kRow;
  static constexpr int kCount = 3;
};

// slot of chunk c among the chunks of row r
__device__ inline uint32_t x_slot(uint32_t r, uint32_t c) { return r * 8 + (c ^ ((r >> 1) & 7u)); }
template <int FMT>
__device__ inline uint32_t w_slot(uint32_t r, uint32_t c) {
  if constexpr (kFourBit<FMT>) return r * 2 + (c ^ ((r >> 3) & 1u));
  else return r * 4 + (c ^ ((r >> 2) & 3u));
}

// Tile of workgroup `id`: the ids of one XCD (id mod 8) take neighbouring tiles,
// in groups of 4 tiles of tokens.
__device__ inline void tile_at(uint32_t id, uint32_t tm, uint32_t tn, uint32_t* m, uint32_t* n) {
  const uint32_t total = tm * tn, per = total >> 3, more = total & 7u, x = id & 7u;
  const uint32_t lin = x * per + (x < more ? x : more) + (id >> 3);
  const uint32_t group = lin / (4 * tn), first = group * 4;
  const uint32_t size = tm - first < 4 ? tm - first : 4, in = lin - group * 4 * tn;
  *m = first + in % size;
  *n = in / size;
}

typedef __attribute__((address_space(3))) void* lds_ptr;
typedef const __attribute__((address_space(1))) void* global_ptr;

template <int N>
__device__ inline void wait_loads() {  // all but the last N vector-memory operations have landed
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
// Every wave is here and has read what it wanted of LDS; copies in flight are not
// waited for.
__device__ inline void stage_barrier() {
  __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4) | (0 << 8));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <int FMT, int BM, int BN, int WAVES_M, int WAVES_N>
__global__ __launch_bounds__(WAVES_M * WAVES_N * 64, 2) void k_linear_tile(LinearArgs a, EpilogueVec vec,
                                                                          uint32_t tiles_m, uint32_t tiles_n) {
  using S = Stage<FMT, BM, BN>;
  constexpr int NW = WAVES_M * WAVES_N, TM = BM / WAVES_M / 32, TN = BN / WAVES_N / 32;
  constexpr int kXCopies = BM * 8 / 64 / NW, kWCopies = BN * S::kRow / 1024 / NW;  // of 1 KB, a wave
  constexpr int kCopies = kXCopies + kWCopies;
  static_assert(BM * 8 % (64 * NW) == 0 && BN * S::kRow % (1024 * NW) == 0, "copies of a stage");
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  uint32_t ti, tj;
  tile_at(blockIdx.x, tiles_m, tiles_n, &ti, &tj);
  const int64_t m0 = (int64_t)ti * BM, n0 = (int64_t)tj * BN;
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t wm = wid / WAVES_N * (BM / WAVES_M), wn = wid % WAVES_N * (BN / WAVES_N);
  const uint32_t l = lane & 31u, h = lane >> 5;
  const int64_t row_bytes = a.K / 32 * kBlockBytes<FMT>;
  const uint32_t steps = (uint32_t)(a.K / 64);

  // this lane's source of each of the wave's copies: slot 64 i + lane of a
  // stage's X (or codes) holds the chunk that x_slot (w_slot) puts there; rows
  // past the last are the last one (their results are not stored)
  const uint8_t* src[kCopies];
#pragma unroll
  for (int i = 0; i < kXCopies; ++i) {
    const uint32_t slot = (wid * kXCopies + i) * 64 + lane, r = slot / 8, c = slot % 8 ^ ((r >> 1) & 7u);
    const int64_t m = m0 + r < a.M ? m0 + r : a.M - 1;
    src[i] = reinterpret_cast<const uint8_t*>(a.x + m * a.ld_x) + c * 16;
  }
#pragma unroll
  for (int i = 0; i < kWCopies; ++i) {
    constexpr uint32_t kPer = S::kRow / 16;
    const uint32_t slot = (wid * kWCopies + i) * 64 + lane, r = slot / kPer;
    const uint32_t c = slot % kPer ^ (kFourBit<FMT> ? (r >> 3) & 1u : (r >> 2) & 3u);
    const int64_t n = n0 + r < a.N ? n0 + r : a.N - 1;
    src[kXCopies + i] = a.codes + n * row_bytes + c * 16;
  }
  // stage `step` into its place in the ring; past the last one the last again,
  // into a place that is not read
  auto copy_stage = [&](uint32_t step) {
    uint8_t* to = smem + (step % S::kCount) * S::kBytes;
    const uint32_t from = step < steps ? step : steps - 1;
#pragma unroll
    for (int i = 0; i < kXCopies; ++i)
      __builtin_amdgcn_global_load_lds((global_ptr)(src[i] + from * 128u), (lds_ptr)(to + (wid * kXCopies + i) * 1024),
                                       16, 0, 0);
#pragma unroll
    for (int i = 0; i < kWCopies; ++i)
      __builtin_amdgcn_global_load_lds((global_ptr)(src[kXCopies + i] + from * (uint32_t)S::kRow),
                                       (lds_ptr)(to + S::kXBytes + (wid * kWCopies + i) * 1024), 16, 0, 0);
  };

  // scale bytes of this lane's weight rows: a word holds 4 blocks of 32 (two
  // stages), or NVFP4's 4 blocks of 16 (one)
  constexpr uint32_t kPerWord = FMT == FMT_NVFP4 ? 1 : 2;
  const uint8_t* srow[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    int64_t n = n0 + wn + 32 * j + l;
    n = n < a.N ? n : a.N - 1;
    srow[j] = a.scales + n * (a.K / (FMT == FMT_NVFP4 ? 16 : 32));
  }
  uint32_t sc[TN], next[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j) next[j] = *reinterpret_cast<const uint32_t*>(srow[j]);

  v16f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

  copy_stage(0);
  copy_stage(1);
  for (uint32_t st = 0; st < steps; ++st) {
    wait_loads<kCopies>();  // all but the next stage's copies
    stage_barrier();
    if (st % kPerWord == 0) {
      const uint32_t w = st / kPerWord + 1 < steps / kPerWord ? st / kPerWord + 1 : st / kPerWord;
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        sc[j] = next[j];
        next[j] = *reinterpret_cast<const uint32_t*>(srow[j] + w * 4);
      }
    }
    copy_stage(st + 2);
    const uint8_t* xs = smem + (st % S::kCount) * S::kBytes;
    const uint8_t* ws = xs + S::kXBytes;
    uint32_t cw[TN][8], s[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const uint32_t r = wn + 32 * j + l;
      if constexpr (kFourBit<FMT>) {
        const word4 c = *reinterpret_cast<const word4*>(ws + w_slot<FMT>(r, h) * 16);
#pragma unroll
        for (int q = 0; q < 4; ++q) cw[j][q] = c[q];
      } else {
        const word4 c = *reinterpret_cast<const word4*>(ws + w_slot<FMT>(r, 2 * h) * 16);
        const word4 d = *reinterpret_cast<const word4*>(ws + w_slot<FMT>(r, 2 * h + 1) * 16);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          cw[j][q] = c[q];
          cw[j][4 + q] = d[q];
        }
      }
      if constexpr (FMT == FMT_NVFP4) s[j] = h ? sc[j] >> 16 : sc[j];
      else s[j] = (sc[j] >> ((st % 2) * 16 + h * 8)) & 0xFFu;
    }
    auto eighth = [&](auto num) {
      constexpr int J = decltype(num)::value;
      bf16x8 xf[TM], wf[TN];
#pragma unroll
      for (int i = 0; i < TM; ++i)
        xf[i] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const word4*>(xs + x_slot(wm + 32 * i + l, 4 * h + J) * 16));
#pragma unroll
      for (int j = 0; j < TN; ++j) wf[j] = decode_eighth<FMT, J>(cw[j], s[j]);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wf[j], xf[i], acc[i][j], 0, 0, 0);
    };
    eighth(std::integral_constant<int, 0>());
    eighth(std::integral_constant<int, 1>());
    eighth(std::integral_constant<int, 2>());
    eighth(std::integral_constant<int, 3>());
  }
  wait_loads<0>();  // the repeated copies too: LDS is used again
  stage_barrier();

  // 32 tokens at a time through the wave's own part of LDS, so that a lane gets 8
  // neighbouring columns of a row
  constexpr int kCols = 32 * TN, kPitch = kCols + 4, kPer = kCols / 8, kRows = 64 / kPer;
  static_assert(NW * 32 * kPitch * 4 <= S::kCount * S::kBytes, "epilogue in the stages' LDS");
  float* mine = reinterpret_cast<float*>(smem) + wid * (32 * kPitch);
  const float ts = FMT == FMT_NVFP4 ? *a.tensor_scale : 1.0f;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<v4f*>(mine + l * kPitch + 32 * j + 8 * q + 4 * h) =
            v4f{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    __builtin_amdgcn_wave_barrier();
#pragma unroll 1
    for (int p = 0; p < 32 / kRows; ++p) {
      const uint32_t t = p * kRows + lane / kPer, c = lane % kPer * 8;
      const int64_t row = m0 + wm + 32 * i + t, col = n0 + wn + c;
      if (row >= a.M || col >= a.N) continue;
      const v4f lo = *reinterpret_cast<const v4f*>(mine + t * kPitch + c);
      const v4f hi = *reinterpret_cast<const v4f*>(mine + t * kPitch + c + 4);
      float v[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = lo[e] * ts;
        v[4 + e] = hi[e] * ts;
      }
      const int n = (int)(a.N - col < 8 ? a.N - col : 8);
      if (a.ep.dt == DT_BF16) epilogue_chunk<DT_BF16>(a.ep, vec, row, col, a.N, n, v);
      else epilogue_chunk<DT_F32>(a.ep, vec, row, col, a.N, n, v);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <int FMT, int BM, int BN, int WAVES_M, int WAVES_N>
hipError_t launch_tile(const LinearArgs& a, hipStream_t s) {
  using S = Stage<FMT, BM, BN>;
  constexpr int kLds = S::kCount * S::kBytes;
  static_assert(kLds <= 160 * 1024, "LDS of a workgroup");
  auto kernel = k_linear_tile<FMT, BM, BN, WAVES_M, WAVES_N>;
  static std::atomic<uint64_t> done{0};
  const hipError_t e = allow_lds((const void*)kernel, kLds, done);
  if (e != hipSuccess) return e;
  const uint32_t tm = (uint32_t)((a.M + BM - 1) / BM), tn = (uint32_t)((a.N + BN - 1) / BN);
  hipLaunchKernelGGL(kernel, dim3(tm * tn), dim3(WAVES_M * WAVES_N * 64), kLds, s, a, epilogue_vec(a.ep), tm, tn);
  return hipGetLastError();
}

template <int FMT>
hipError_t launch_fmt(const LinearArgs& a, hipStream_t s) {
  if (a.M <= 16) return launch_direct<FMT, 1, 1, 8>(a, s);
  if (a.M <= 32) return launch_direct<FMT, 2, 2, 8>(a, s);
  // (stages are whole at multiples of 64, scale words at multiples of 128)
  if (a.M > 64 && a.K % 128 == 0 && a.K > 0) {
    const int64_t large = ((a.M + 255) / 256) * ((a.N + 255) / 256);
    return large >= 256 ? launch_tile<FMT, 256, 256, 2, 4>(a, s) : launch_tile<FMT, 128, 128, 2, 2>(a, s);
  }
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
