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
#include "../linear_plan.h"

namespace mxk {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

// The sums of NW waves over one tile of BM tokens x BN columns, rows of BN + 4
// floats in LDS, added in order; then the epilogue.
template <int FMT, int DT, int BM, int BN, int NW>
__device__ inline void join_waves(const LinearArgs& a, const EpilogueVec& vec, const float* red, int64_t m0,
                                  int64_t n0) {
  constexpr int kPitch = BN + 4;
  const float ts = FMT == FMT_NVFP4 ? *a.tensor_scale : 1.0f;
  for (uint32_t q = threadIdx.x; q < BM * BN / 8; q += NW * 64) {
    const uint32_t t = q / (BN / 8), c = q % (BN / 8) * 8;
    const int64_t row = m0 + t, col = n0 + c;
    if (row >= a.M || col >= a.N) continue;
    const int n = (int)(a.N - col < 8 ? a.N - col : 8);
    RawChunk res = {};
    if (a.ep.residual) res = load_raw8<DT>(a.ep.residual, row * a.ep.ld_r + col, n, vec.residual);
    float b[8];
    load_bias(a.ep, vec, col, n, b);
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const float* p = red + k * (BM * kPitch) + t * kPitch + c;
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
    epilogue_chunk<DT, false>(a.ep, vec, row, col, a.N, n, b, res, v);
  }
}

// ---- operands straight from memory -----------------------------------------
// A workgroup of NW waves takes all tokens, at most 16, x 16 columns; its waves share out
// the steps of K and add their sums through LDS, in order.  A step is 128 bytes of a
// weight row (256 4-bit or 128 8-bit elements): lane group g of four takes 32 bytes of
// them.  Each wave has neighbouring steps, and tiles start at different ones: rows of a
// power of two of bytes would otherwise all be read at the same offset at a time, from
// a part of the memory channels.  The next step's operands are loaded while this one's
// are multiplied.
// A call is bound by latency: 1 x 7168 x 2048 NVFP4 with residual takes 5.7 us for
// 8.3 MB, an empty kernel 1.5 to 2; a wave has one step, so load, decoding and the
// sum over the waves follow one another.
template <int FMT>
struct DirectStep {
  static constexpr int B = kFourBit<FMT> ? 2 : 1;  // blocks of 32 a lane
  word4 codes[2];
  uint32_t scales[B];
  word4 x[B][4];
};

template <int FMT, int DT, int NW>
__global__ __launch_bounds__(NW * 64) void k_linear_direct(LinearArgs a, EpilogueVec vec) {
  using Step = DirectStep<FMT>;
  constexpr int B = Step::B;
  constexpr int kPitch = 16 + 4;  // floats of a token's row in LDS
  __shared__ __attribute__((aligned(16))) float red[NW * 16 * kPitch];
  const uint32_t lane = threadIdx.x & 63u, l = lane & 15u, g = lane >> 4;
  const uint32_t wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t tile = blockIdx.x;
  const int64_t n0 = (int64_t)tile * 16;
  const int64_t row_bytes = a.K / 32 * kBlockBytes<FMT>, blocks = a.K / 32;

  // rows past the last are the last one (their results are not stored)
  const int64_t n = n0 + l < a.N ? n0 + l : a.N - 1, m = l < a.M ? l : a.M - 1;
  const uint8_t* const w = a.codes + n * row_bytes;
  const int64_t first = n * blocks;  // block number of the row's first block
  const uint16_t* const x = a.x + m * a.ld_x;

  v4f acc = {0, 0, 0, 0};

  // the lane's blocks start at `blk`
  auto load = [&](Step& s, int64_t blk) {
    const word4* p = reinterpret_cast<const word4*>(w + blk * kBlockBytes<FMT>);
    s.codes[0] = p[0];
    s.codes[1] = p[1];
#pragma unroll
    for (int b = 0; b < B; ++b) s.scales[b] = load_scale<FMT>(a.scales, first + blk + b);
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) s.x[b][e] = *reinterpret_cast<const word4*>(x + (blk + b) * 32 + e * 8);
  };
  auto eighth = [&](const Step& s, auto block, auto num) {
    constexpr int b = decltype(block)::value, J = decltype(num)::value;
    uint32_t u[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      u[q] = s.codes[kFourBit<FMT> ? b : 0][q];
      u[4 + q] = s.codes[1][q];
    }
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(decode_eighth<FMT, J>(u, s.scales[b]),
                                                  __builtin_bit_cast(bf16x8, s.x[b][J]), acc, 0, 0, 0);
  };
  auto multiply = [&](const Step& s) {
    auto block = [&](auto b) {
      eighth(s, b, std::integral_constant<int, 0>());
      eighth(s, b, std::integral_constant<int, 1>());
      eighth(s, b, std::integral_constant<int, 2>());
      eighth(s, b, std::integral_constant<int, 3>());
    };
    block(std::integral_constant<int, 0>());
    if constexpr (B == 2) block(std::integral_constant<int, 1>());
  };

  const uint32_t steps = (uint32_t)(blocks / (4 * B));  // whole ones
  const uint32_t per = (steps + NW - 1) / NW, lo = wid * per < steps ? wid * per : steps;
  const uint32_t count = steps - lo < per ? steps - lo : per;
  if (count > 0) {
    const uint32_t turn = tile % count;
    auto at = [&](uint32_t i) {  // the lane's blocks of the i-th step taken
      const uint32_t st = turn + i < count ? turn + i : turn + i - count;
      return (int64_t)(lo + st) * (4 * B) + g * B;
    };
    Step p, q;
    load(p, at(0));
    for (uint32_t i = 0; i < count; i += 2) {
      load(q, at(i + 1 < count ? i + 1 : i));
      multiply(p);
      if (i + 1 == count) break;
      load(p, at(i + 2 < count ? i + 2 : i));
      multiply(q);
    }
  }
  // what is left of K, fewer blocks than a step has: lanes past it take zeros
  if (wid == NW - 1 && steps * (4 * B) < blocks) {
    Step s = {};
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int64_t blk = (int64_t)steps * (4 * B) + g * B + b;
      if (blk < blocks) {
        const word4* p = reinterpret_cast<const word4*>(w + blk * kBlockBytes<FMT>);
        s.codes[b] = p[0];
        if constexpr (!kFourBit<FMT>) s.codes[1] = p[1];
        s.scales[b] = load_scale<FMT>(a.scales, first + blk);
#pragma unroll
        for (int e = 0; e < 4; ++e) s.x[b][e] = *reinterpret_cast<const word4*>(x + blk * 32 + e * 8);
      }
    }
    multiply(s);
  }

  *reinterpret_cast<v4f*>(red + wid * (16 * kPitch) + l * kPitch + 4 * g) = acc;
  __syncthreads();

  join_waves<FMT, DT, 16, 16, NW>(a, vec, red, 0, n0);
}

template <int FMT, int DT, int NW>
hipError_t launch_direct(const LinearArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((k_linear_direct<FMT, DT, NW>), dim3((uint32_t)((a.N + 15) / 16)), dim3(NW * 64), 0, s, a,
                     epilogue_vec(a.ep));
  return hipGetLastError();
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

// ---- operands through LDS ---------------------------------------------------
// A workgroup takes a tile of BM tokens x BN columns, each wave a part of it
// (v_mfma_f32_32x32x16_bf16).  A step is 64 elements of K: 128 bytes of every row
// of X, and 64 bytes of every weight row for one step (8-bit codes) or two
// (4-bit).  Both come by 16-byte global-to-LDS copies, three steps (or units of
// codes) in a ring, so that one barrier a step is enough: behind it the next step
// has landed for all waves and this one is no longer read.  Lane half h takes
// elements 32 h .. 32 h + 31 of a step (one block), 8 of them for each of four
// instructions; W is decoded from the codes as it leaves LDS.
//
// One copy instruction fills 1 KB of LDS in lane order: 8 rows of X or 16 of
// codes, each of them whole and in order, since lanes out of order cost the L1
// twice the requests (974 requests a step and 65% of the cycles with products;
// a permutation of chunks and 32-byte pieces of codes did that).  The rows of one
// copy are BM / 8 (BN / 16) apart and the copies 1040 bytes, so that 16
// neighbouring rows, which are read together, lie in all banks.
//
// The matrix unit at the card's power limit is what bounds a large product: 16384
// x 14336 x 4096 MXFP4 is 1405 us (1370 TFLOP/s), the instructions busy 71% of the
// time at 1.7 GHz, where a library's product of BF16 weights is busy 85% at 1.6
// GHz (1307 us).  Decoding W costs about 10% of that (both waves of a column
// decode it; from LDS as BF16 its reads would fill the LDS).  Nothing runs beside a
// tile's end: gelu and a kept z make it 1550 us, gelu's 32 vector instructions a
// result alone 1510.  4096 x 7168 x 2048 NVFP4 with dropout and residual is 123 us
// (977 TFLOP/s): 448 tiles are 1.75 rounds of 256, and NVFP4 takes 16 vector
// instructions for 8 weights, MXFP4 4.
// No faster: four steps in the ring, 256 x 128 tiles two a CU, wave tiles of 128 x
// 128, workgroups that start at different steps.
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr uint32_t kCopyPitch = 1040;

template <int BM, int BN>
struct Ring {
  static constexpr uint32_t kXBytes = BM / 8 * kCopyPitch, kWBytes = BN / 16 * kCopyPitch;
  static constexpr uint32_t kCount = 3, kBytes = kCount * (kXBytes + kWBytes);
  // byte offsets of chunk c (16 bytes) of row r
  static __device__ uint32_t x(uint32_t r, uint32_t c) {
    return r % (BM / 8) * kCopyPitch + r / (BM / 8) * 128 + c * 16;
  }
  static __device__ uint32_t w(uint32_t r, uint32_t c) {
    return r % (BN / 16) * kCopyPitch + r / (BN / 16) * 64 + c * 16;
  }
};

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

// Order a region as MF matrix instructions with D LDS reads behind the first
// ones, and M vector-memory and V vector instructions spread between them.
__device__ inline void region() { __builtin_amdgcn_sched_barrier(0); }
template <int MF, int D, int M, int V, int I = 0>
__device__ inline void spread() {
  if constexpr (I < MF) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    constexpr int d = I < MF / 2 ? ((I + 1) * D + MF / 2 - 1) / (MF / 2) - (I * D + MF / 2 - 1) / (MF / 2) : 0;
    constexpr int m = ((I + 1) * M + MF - 1) / MF - (I * M + MF - 1) / MF;
    constexpr int v = ((I + 1) * V + MF - 1) / MF - (I * V + MF - 1) / MF;
    if constexpr (d > 0) __builtin_amdgcn_sched_group_barrier(0x100, d, 0);
    if constexpr (m > 0) __builtin_amdgcn_sched_group_barrier(0x010, m, 0);
    if constexpr (v > 0) __builtin_amdgcn_sched_group_barrier(0x002, v, 0);
    spread<MF, D, M, V, I + 1>();
  }
}

// What a copy takes past the end of a row.
__device__ const word4 kZeros = {0, 0, 0, 0};

// The scale bytes of a pair of steps: four blocks of 32, or NVFP4's eight of 16.
// (A row of scales starts at any byte where K % 128 != 0.)
template <int FMT>
using ScaleWord = std::conditional_t<FMT == FMT_NVFP4, uint64_t, uint32_t>;
template <int FMT>
__device__ inline ScaleWord<FMT> load_pair_scales(const uint8_t* p) {
  ScaleWord<FMT> w;
  __builtin_memcpy(&w, p, sizeof(w));
  return w;
}
// those of the last 1 .. 3 blocks of a row, and 1 behind them
template <int FMT>
__device__ inline ScaleWord<FMT> load_rest_scales(const uint8_t* p, uint32_t blocks) {
  constexpr int kBytes = FMT == FMT_NVFP4 ? 2 : 1;
  constexpr ScaleWord<FMT> kOne = FMT == FMT_NVFP4 ? 0x38 : 127;
  ScaleWord<FMT> w = 0;
#pragma unroll
  for (uint32_t i = 0; i < sizeof(w); ++i)
    w |= (i < blocks * kBytes ? (ScaleWord<FMT>)p[i] : kOne) << (8 * i);
  return w;
}

template <int FMT, int DT, int BM, int BN, int WAVES_M, int WAVES_N>
__global__ __launch_bounds__(WAVES_M * WAVES_N * 64, 2) void k_linear_tile(LinearArgs a, EpilogueVec vec,
                                                                          uint32_t tiles_m, uint32_t tiles_n) {
  using R = Ring<BM, BN>;
  constexpr int NW = WAVES_M * WAVES_N, TM = BM / WAVES_M / 32, TN = BN / WAVES_N / 32;
  constexpr int kWCopies = BN / 16 / NW;  // of a unit, a wave
  constexpr bool kTwoSteps = kFourBit<FMT>;  // a unit of codes is two steps
  static_assert(BM / 8 == 4 * NW && BN / 16 == kWCopies * NW && kWCopies == 2, "copies of a wave");
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  uint8_t* const wring = smem + R::kCount * R::kXBytes;
  uint32_t ti, tj;
  tile_at(blockIdx.x, tiles_m, tiles_n, &ti, &tj);
  const int64_t m0 = (int64_t)ti * BM, n0 = (int64_t)tj * BN;
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t wm = wid / WAVES_N * (BM / WAVES_M), wn = wid % WAVES_N * (BN / WAVES_N);
  const uint32_t l = lane & 31u, h = lane >> 5;
  const int64_t row_bytes = a.K / 32 * kBlockBytes<FMT>;
  const uint32_t pairs = (uint32_t)(a.K / 128);  // of steps
  const uint32_t units = kTwoSteps ? pairs : 2 * pairs;
  const uint32_t rest = (uint32_t)(a.K / 32 % 4);  // blocks behind them

  // this lane's source of each of the wave's copies; rows past the last are the
  // last one (their results are not stored)
  const uint8_t* xsrc[4];
  const uint8_t* wsrc[kWCopies];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + (wid * 4 + i) + lane / 8 * (BM / 8);
    xsrc[i] = reinterpret_cast<const uint8_t*>(a.x + (m < a.M ? m : a.M - 1) * a.ld_x) + lane % 8 * 16;
  }
#pragma unroll
  for (int i = 0; i < kWCopies; ++i) {
    const int64_t n = n0 + (wid * kWCopies + i) + lane / 4 * (BN / 16);
    wsrc[i] = a.codes + (n < a.N ? n : a.N - 1) * row_bytes + lane % 4 * 16;
  }
  // one copy of a step's X, or of a unit's codes, into their places in the ring;
  // past the last the last one again, which is then not used
  auto copy_x = [&](uint32_t step, auto num) {
    constexpr int i = decltype(num)::value;
    const uint32_t from = step < 2 * pairs ? step : 2 * pairs - 1;
    __builtin_amdgcn_global_load_lds(
        (global_ptr)(xsrc[i] + from * 128u),
        (lds_ptr)(smem + step % R::kCount * R::kXBytes + (wid * 4 + i) * kCopyPitch), 16, 0, 0);
  };
  auto copy_w = [&](uint32_t unit, auto num) {
    constexpr int i = decltype(num)::value;
    const uint32_t from = unit < units ? unit : units - 1;
    __builtin_amdgcn_global_load_lds(
        (global_ptr)(wsrc[i] + from * 64u),
        (lds_ptr)(wring + unit % R::kCount * R::kWBytes + (wid * kWCopies + i) * kCopyPitch), 16, 0, 0);
  };
  constexpr std::integral_constant<int, 0> s0;
  constexpr std::integral_constant<int, 1> s1;
  constexpr std::integral_constant<int, 2> s2;
  constexpr std::integral_constant<int, 3> s3;

  const uint8_t* srow[TN];  // scales of this lane's weight rows
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int64_t n = n0 + wn + 32 * j + l;
    srow[j] = a.scales + (n < a.N ? n : a.N - 1) * (a.K / (FMT == FMT_NVFP4 ? 16 : 32));
  }

  v16f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

  // What follows is one slice (16 elements of K, 8 a lane half) ahead of the
  // products: its X fragments and decoded weights are in registers when its
  // instructions start, also across the barrier.
  uint32_t cw[TN][8], sc[TN];
  ScaleWord<FMT> scales[TN];  // of a pair of steps
  bf16x8 xf[2][TM], wf[2][TN];
  auto read_codes = [&](uint32_t st) {
    const uint8_t* ws = wring + (kTwoSteps ? st / 2 : st) % R::kCount * R::kWBytes;
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int b = 0; b < (kTwoSteps ? 1 : 2); ++b) {
        const word4 c =
            *reinterpret_cast<const word4*>(ws + R::w(wn + 32 * j + l, kTwoSteps ? st % 2 * 2 + h : 2 * h + b));
#pragma unroll
        for (int q = 0; q < 4; ++q) cw[j][4 * b + q] = c[q];
      }
  };
  auto read_x = [&](uint32_t st, auto num) {
    constexpr int J = decltype(num)::value;
    const uint8_t* xs = smem + st % R::kCount * R::kXBytes;
#pragma unroll
    for (int i = 0; i < TM; ++i)
      xf[J % 2][i] =
          __builtin_bit_cast(bf16x8, *reinterpret_cast<const word4*>(xs + R::x(wm + 32 * i + l, 4 * h + J)));
  };
  auto decode = [&](auto num) {
    constexpr int J = decltype(num)::value;
#pragma unroll
    for (int j = 0; j < TN; ++j) wf[J % 2][j] = decode_eighth<FMT, J>(cw[j], sc[j]);
  };
  auto products = [&](auto num) {
    constexpr int J = decltype(num)::value;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wf[J % 2][j], xf[J % 2][i], acc[i][j], 0, 0, 0);
  };
  auto step_scales = [&](auto num) {
    constexpr int P = decltype(num)::value;
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      if constexpr (FMT == FMT_NVFP4) sc[j] = (uint32_t)(scales[j] >> (32 * P)) >> (16 * h);
      else sc[j] = (scales[j] >> (16 * P + 8 * h)) & 0xFFu;
    }
  };
  auto load_scales = [&](uint32_t pair) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
      scales[j] = load_pair_scales<FMT>(srow[j] + (pair < pairs ? pair : pairs - 1) * sizeof(ScaleWord<FMT>));
  };

  // vector instructions of a slice's decoding, about
  constexpr int kDecode = TN * (FMT == FMT_NVFP4 ? 17 : FMT == FMT_MXINT8 ? 20 : 4) + 2;
  constexpr int kReads = TN * (kTwoSteps ? 1 : 2);
  auto step = [&](uint32_t st, auto parity) {
    constexpr int P = decltype(parity)::value;
    constexpr bool kCodes = !kTwoSteps || P == 0;  // a unit of codes is copied
    const uint32_t unit = (kTwoSteps ? st / 2 : st) + 2;
    region();
    read_x(st, s1);
    copy_x(st + 2, s1);
    if constexpr (kCodes) copy_w(unit, s0);
    products(s0);
    decode(s1);
    spread<TM * TN, TM, 1 + kCodes, kDecode>();
    region();
    read_x(st, s2);
    copy_x(st + 2, s2);
    if constexpr (kCodes) copy_w(unit, s1);
    products(s1);
    decode(s2);
    spread<TM * TN, TM, 1 + kCodes, kDecode>();
    region();
    read_x(st, s3);
    copy_x(st + 2, s3);
    products(s2);
    decode(s3);
    spread<TM * TN, TM, 1, kDecode>();
    region();
    // this step has been read (its last slice is in registers); the next one has
    // landed: what was issued behind its last copy is not waited for
    wait_loads<4 + (kCodes ? kWCopies : 0)>();
    stage_barrier();
    region();
    step_scales(std::integral_constant<int, 1 - P>());
    region();
    if constexpr (P == 0) load_scales(st / 2 + 1);  // (wanted a step from now)
    region();
    copy_x(st + 3, s0);
    read_codes(st + 1);
    read_x(st + 1, s0);
    products(s3);
    decode(s0);
    spread<TM * TN, TM + kReads, 1, kDecode + 10>();
    region();
  };
  if (pairs > 0) {
    load_scales(0);
    auto copy_step = [&](uint32_t st) {
      copy_w(st, s0);
      copy_w(st, s1);
      copy_x(st, s0);
      copy_x(st, s1);
      copy_x(st, s2);
      copy_x(st, s3);
    };
    copy_step(0);
    copy_step(1);
    wait_loads<4 + kWCopies>();
    stage_barrier();
    copy_x(2, s0);
    step_scales(s0);
    read_codes(0);
    read_x(0, s0);
    decode(s0);
    for (uint32_t pair = 0; pair < pairs; ++pair) {
      step(2 * pair, s0);
      step(2 * pair + 1, s1);
    }
    wait_loads<0>();  // the repeated copies too: LDS is used again
    stage_barrier();
  }
  if (rest) {  // what is left of K, as a pair that ends in zeros; nothing runs ahead
    auto copy_rest_x = [&](uint32_t st, auto num) {
      constexpr int i = decltype(num)::value;
      const bool in = st * 64 + lane % 8 * 8 < rest * 32;
      const uint8_t* from = in ? xsrc[i] + (2 * pairs + st) * 128u : reinterpret_cast<const uint8_t*>(&kZeros);
      __builtin_amdgcn_global_load_lds((global_ptr)from,
                                       (lds_ptr)(smem + st * R::kXBytes + (wid * 4 + i) * kCopyPitch), 16, 0, 0);
    };
    auto copy_rest_w = [&](uint32_t unit, auto num) {
      constexpr int i = decltype(num)::value;
      const bool in = unit * 64 + lane % 4 * 16 < rest * kBlockBytes<FMT>;
      const uint8_t* from = in ? wsrc[i] + (units + unit) * 64u : reinterpret_cast<const uint8_t*>(&kZeros);
      __builtin_amdgcn_global_load_lds(
          (global_ptr)from, (lds_ptr)(wring + unit * R::kWBytes + (wid * kWCopies + i) * kCopyPitch), 16, 0, 0);
    };
    auto copy_rest = [&](uint32_t st) {
      copy_rest_x(st, s0);
      copy_rest_x(st, s1);
      copy_rest_x(st, s2);
      copy_rest_x(st, s3);
      if (kTwoSteps && st == 1) return;
      copy_rest_w(st, s0);
      copy_rest_w(st, s1);
    };
    copy_rest(0);
    copy_rest(1);
#pragma unroll
    for (int j = 0; j < TN; ++j) scales[j] = load_rest_scales<FMT>(srow[j] + pairs * sizeof(ScaleWord<FMT>), rest);
    wait_loads<0>();
    stage_barrier();
    auto rest_step = [&](auto parity) {
      constexpr uint32_t P = decltype(parity)::value;
      step_scales(parity);
      read_codes(P);
      auto slice = [&](auto num) {
        read_x(P, num);
        decode(num);
        products(num);
      };
      slice(s0);
      slice(s1);
      slice(s2);
      slice(s3);
    };
    rest_step(s0);
    if (rest > 2) rest_step(s1);
    stage_barrier();
  }

  // 32 tokens at a time through the wave's own part of LDS, so that a lane gets 8
  // neighbouring columns of a row; a pass takes kRows of them.  The residual of the
  // next 32 tokens is on its way meanwhile (16384 x 14336 x 4096 with residual 1475
  // us; that of the next pass alone 1548).  Two passes are unrolled (one: 1490);
  // all of them do not fit the instruction cache beside the loop above (3 times
  // slower as a whole).
  constexpr int kCols = 32 * TN, kPitch = kCols + 4, kPer = kCols / 8, kRows = 64 / kPer, kPasses = 32 / kRows;
  static_assert(NW * 32 * kPitch * 4 <= R::kBytes, "epilogue in the ring's LDS");
  float* mine = reinterpret_cast<float*>(smem) + wid * (32 * kPitch);
  const float ts = FMT == FMT_NVFP4 ? *a.tensor_scale : 1.0f;
  const uint32_t t0 = lane / kPer, c = lane % kPer * 8;
  const int64_t row0 = m0 + wm + t0, col = n0 + wn + c;
  const int n = (int)(col >= a.N ? 0 : a.N - col < 8 ? a.N - col : 8);
  float b[8];
  load_bias(a.ep, vec, col, n, b);
  auto residual_of = [&](int pass) {
    const int64_t row = row0 + pass * kRows;
    return a.ep.residual && row < a.M ? load_raw8<DT>(a.ep.residual, row * a.ep.ld_r + col, n, vec.residual)
                                      : RawChunk{};
  };
  RawChunk ahead[kPasses];
  auto load_ahead = [&](int first) {
#pragma unroll
    for (int p = 0; p < kPasses; ++p) ahead[p] = residual_of(first + p);
  };
  load_ahead(0);
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<v4f*>(mine + l * kPitch + 32 * j + 8 * q + 4 * h) =
            v4f{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    __builtin_amdgcn_wave_barrier();
    RawChunk now[kPasses];
#pragma unroll
    for (int p = 0; p < kPasses; ++p) now[p] = ahead[p];
    if (i + 1 < TM) load_ahead((i + 1) * kPasses);
#pragma unroll 2
    for (int pass = i * kPasses; pass < (i + 1) * kPasses; ++pass) {
      RawChunk res = now[0];
#pragma unroll
      for (int p = 1; p < kPasses; ++p)
        if (pass == i * kPasses + p) res = now[p];
      const int64_t row = row0 + pass * kRows;
      if (row >= a.M || n == 0) continue;
      const float* p = mine + (pass % kPasses * kRows + t0) * kPitch + c;
      const v4f lo = *reinterpret_cast<const v4f*>(p), hi = *reinterpret_cast<const v4f*>(p + 4);
      float v[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = FMT == FMT_NVFP4 ? lo[e] * ts : lo[e];
        v[4 + e] = FMT == FMT_NVFP4 ? hi[e] * ts : hi[e];
      }
      epilogue_chunk<DT, true>(a.ep, vec, row, col, a.N, n, b, res, v);
    }
  }
}

template <int FMT, int DT, int BM, int BN, int WAVES_M, int WAVES_N>
hipError_t launch_tile(const LinearArgs& a, hipStream_t s) {
  constexpr int kLds = Ring<BM, BN>::kBytes;
  static_assert(kLds <= 160 * 1024, "LDS of a workgroup");
  auto kernel = k_linear_tile<FMT, DT, BM, BN, WAVES_M, WAVES_N>;
  static std::atomic<uint64_t> done{0};
  const hipError_t e = allow_lds((const void*)kernel, kLds, done);
  if (e != hipSuccess) return e;
  const uint32_t tm = (uint32_t)((a.M + BM - 1) / BM), tn = (uint32_t)((a.N + BN - 1) / BN);
  hipLaunchKernelGGL(kernel, dim3(tm * tn), dim3(WAVES_M * WAVES_N * 64), kLds, s, a, epilogue_vec(a.ep), tm, tn);
  return hipGetLastError();
}

// ---- K shared out among the waves of a tile ---------------------------------
// Between the two: batches whose large tiles would leave most of the card idle.
// Each wave of a workgroup takes the whole BM x BN tile over its own part of K
// (neighbouring pairs of steps), from a ring of LDS that is its own: no barriers,
// three steps of copies in flight for each of NW waves.  The waves' sums are added
// through LDS in order.  On a full card no unit fills its time (256 x 4096 x 4096 MXFP4
// 15 us, 573 TFLOP/s): of the 35000 cycles that a wave lives, its matrix instructions
// take 8200 and the vector ones 6700; the L1 serves 17000 accesses in them (four
// waves' 10 KB a step are 10000 at 64 bytes); a third goes by in waits for copies,
// since three steps in flight are less than the memory's latency when the card is
// busy, and a third in waits to issue.  With few tokens every tile reads all rows of X
// (37 x 14336 x 4096 with silu: 117 MB through the L1s beside the weights, MXFP8 18.2 us
// from the last-level cache and 23.2 from HBM, MXFP4 14.3 and 17.1; of 24 tokens 58 MB,
// MXFP8 15.4 and 19.5, MXFP4 10.4 and 13.2; rows of X that are not 128-byte aligned
// cost 5% more).  Copies that leave the rows past the last out were 10% slower by their
// branches.
template <int FMT, int BM, int BN>
struct SplitRing {
  static constexpr bool kTwoSteps = kFourBit<FMT>;
  static constexpr uint32_t kXBytes = BM / 8 * kCopyPitch, kWBytes = BN / 16 * kCopyPitch;
  static constexpr uint32_t kXSlots = 3, kWSlots = kTwoSteps ? 2 : 3;
  static constexpr uint32_t kBytes = kXSlots * kXBytes + kWSlots * kWBytes;
};

template <int FMT, int DT, int BM, int BN, int NW>
__global__ __launch_bounds__(NW * 64) void k_linear_split(LinearArgs a, EpilogueVec vec, uint32_t tiles_m,
                                                          uint32_t tiles_n) {
  using R = Ring<BM, BN>;
  using S = SplitRing<FMT, BM, BN>;
  constexpr int TM = BM / 32, TN = BN / 32, kXCopies = BM / 8, kWCopies = BN / 16;
  constexpr bool kTwoSteps = S::kTwoSteps;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  uint32_t ti, tj;
  tile_at(blockIdx.x, tiles_m, tiles_n, &ti, &tj);
  const int64_t m0 = (int64_t)ti * BM, n0 = (int64_t)tj * BN;
  const uint32_t lane = threadIdx.x & 63u, l = lane & 31u, h = lane >> 5;
  const uint32_t wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint8_t* const xring = smem + wid * S::kBytes;
  uint8_t* const wring = xring + S::kXSlots * S::kXBytes;
  const int64_t row_bytes = a.K / 32 * kBlockBytes<FMT>;
  const uint32_t all = (uint32_t)(a.K / 128);  // pairs of steps
  const uint32_t per = (all + NW - 1) / NW, lo = wid * per < all ? wid * per : all;
  const uint32_t pairs = all - lo < per ? all - lo : per;
  const uint32_t rest = wid == NW - 1 ? (uint32_t)(a.K / 32 % 4) : 0;  // blocks behind them

  v16f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

  // sources of the copies; rows past the last are the last one
  const uint8_t* xsrc[kXCopies];
  const uint8_t* wsrc[kWCopies];
#pragma unroll
  for (int i = 0; i < kXCopies; ++i) {
    const int64_t m = m0 + i + lane / 8 * (BM / 8);
    xsrc[i] = reinterpret_cast<const uint8_t*>(a.x + (m < a.M ? m : a.M - 1) * a.ld_x) + lane % 8 * 16;
  }
#pragma unroll
  for (int i = 0; i < kWCopies; ++i) {
    const int64_t n = n0 + i + lane / 4 * (BN / 16);
    wsrc[i] = a.codes + (n < a.N ? n : a.N - 1) * row_bytes + lane % 4 * 16;
  }
  const uint8_t* srow[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int64_t n = n0 + 32 * j + l;
    srow[j] = a.scales + (n < a.N ? n : a.N - 1) * (a.K / (FMT == FMT_NVFP4 ? 16 : 32));
  }
  ScaleWord<FMT> scales[TN];
  uint32_t sc[2][TN], cw[TN][8];
  bf16x8 xf[4][TM];
  // a step's operands out of the ring, and its products
  auto read = [&](uint32_t st, auto parity) {
    constexpr int P = decltype(parity)::value;
    const uint8_t* xs = xring + st % S::kXSlots * S::kXBytes;
    const uint8_t* ws = wring + (kTwoSteps ? st / 2 : st) % S::kWSlots * S::kWBytes;
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int b = 0; b < (kTwoSteps ? 1 : 2); ++b) {
        const word4 c = *reinterpret_cast<const word4*>(ws + R::w(32 * j + l, kTwoSteps ? P * 2 + h : 2 * h + b));
#pragma unroll
        for (int q = 0; q < 4; ++q) cw[j][4 * b + q] = c[q];
      }
#pragma unroll
    for (int J = 0; J < 4; ++J)
#pragma unroll
      for (int i = 0; i < TM; ++i)
        xf[J][i] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const word4*>(xs + R::x(32 * i + l, 4 * h + J)));
  };
  auto split_scales = [&] {
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        if constexpr (FMT == FMT_NVFP4) sc[p][j] = (uint32_t)(scales[j] >> (32 * p)) >> (16 * h);
        else sc[p][j] = (scales[j] >> (16 * p + 8 * h)) & 0xFFu;
      }
  };
  auto products = [&](auto parity) {
    constexpr int P = decltype(parity)::value;
    auto slice = [&](auto num) {
      constexpr int J = decltype(num)::value;
      bf16x8 wf[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j) wf[j] = decode_eighth<FMT, J>(cw[j], sc[P][j]);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wf[j], xf[J][i], acc[i][j], 0, 0, 0);
    };
    slice(std::integral_constant<int, 0>());
    slice(std::integral_constant<int, 1>());
    slice(std::integral_constant<int, 2>());
    slice(std::integral_constant<int, 3>());
  };
  constexpr std::integral_constant<int, 0> even;
  constexpr std::integral_constant<int, 1> odd;

  if (pairs > 0) {
    // the wave's pairs, from another one on for each tile; past the last one it
    // again, which is then not used
    const uint32_t turn = (ti + tj) % pairs;
    auto pair_at = [&](uint32_t i) {
      i = i < pairs ? i : pairs - 1;
      return lo + (turn + i < pairs ? turn + i : turn + i - pairs);
    };
    auto copy_x = [&](uint32_t st) {
      const uint32_t from = (pair_at(st / 2) * 2 + st % 2) * 128u;
#pragma unroll
      for (int i = 0; i < kXCopies; ++i)
        __builtin_amdgcn_global_load_lds((global_ptr)(xsrc[i] + from),
                                         (lds_ptr)(xring + st % S::kXSlots * S::kXBytes + i * kCopyPitch), 16, 0, 0);
    };
    auto copy_w = [&](uint32_t unit) {  // a pair's codes, or a step's
      const uint32_t from = (kTwoSteps ? pair_at(unit) : pair_at(unit / 2) * 2 + unit % 2) * 64u;
#pragma unroll
      for (int i = 0; i < kWCopies; ++i)
        __builtin_amdgcn_global_load_lds((global_ptr)(wsrc[i] + from),
                                         (lds_ptr)(wring + unit % S::kWSlots * S::kWBytes + i * kCopyPitch), 16, 0, 0);
    };
    auto load_scales = [&](uint32_t i) {
#pragma unroll
      for (int j = 0; j < TN; ++j)
        scales[j] = load_pair_scales<FMT>(srow[j] + pair_at(i) * sizeof(ScaleWord<FMT>));
    };
    // three steps of copies in flight; kBehind of them may be younger than what a
    // step waits for (its own X and codes)
    constexpr int kBehind = 2 * kXCopies + (kTwoSteps ? 1 : 2) * kWCopies;
    load_scales(0);
    copy_w(0);
    copy_x(0);
    if constexpr (!kTwoSteps) copy_w(1);
    copy_x(1);
    copy_w(kTwoSteps ? 1 : 2);
    copy_x(2);
    auto step = [&](uint32_t st, auto parity) {
      constexpr int P = decltype(parity)::value;
      wait_loads<kBehind>();
      asm volatile("" ::: "memory");
      read(st, parity);
      if constexpr (P == 0) split_scales();
      // everything has left the ring: the step three behind takes its place
      __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4) | (0 << 8));
      asm volatile("" ::: "memory");
      if constexpr (P == 0) load_scales(st / 2 + 1);
      if constexpr (!kTwoSteps) copy_w(st + 3);
      else if constexpr (P == 1) copy_w(st / 2 + 2);
      copy_x(st + 3);
      products(parity);
    };
    for (uint32_t i = 0; i < pairs; ++i) {
      step(2 * i, even);
      step(2 * i + 1, odd);
    }
    wait_loads<0>();  // the repeated copies too: LDS is used again
    asm volatile("" ::: "memory");
  }
  if (rest) {  // what is left of K, as a pair that ends in zeros
    for (uint32_t st = 0; st < 2; ++st) {
      const bool in = st * 64 + lane % 8 * 8 < rest * 32;
#pragma unroll
      for (int i = 0; i < kXCopies; ++i)
        __builtin_amdgcn_global_load_lds(
            (global_ptr)(in ? xsrc[i] + (2 * all + st) * 128u : reinterpret_cast<const uint8_t*>(&kZeros)),
            (lds_ptr)(xring + st * S::kXBytes + i * kCopyPitch), 16, 0, 0);
    }
    for (uint32_t unit = 0; unit < (kTwoSteps ? 1 : 2); ++unit) {
      const bool in = unit * 64 + lane % 4 * 16 < rest * kBlockBytes<FMT>;
#pragma unroll
      for (int i = 0; i < kWCopies; ++i)
        __builtin_amdgcn_global_load_lds((global_ptr)(in ? wsrc[i] + ((kTwoSteps ? all : 2 * all) + unit) * 64u
                                                         : reinterpret_cast<const uint8_t*>(&kZeros)),
                                         (lds_ptr)(wring + unit * S::kWBytes + i * kCopyPitch), 16, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) scales[j] = load_rest_scales<FMT>(srow[j] + all * sizeof(ScaleWord<FMT>), rest);
    split_scales();
    wait_loads<0>();
    asm volatile("" ::: "memory");
    read(0, even);
    products(even);
    if (rest > 2) {
      read(1, odd);
      products(odd);
    }
  }
  __syncthreads();

  constexpr int kPitch = BN + 4;
  static_assert(BM * kPitch * 4 <= S::kBytes, "sums in the rings' LDS");
  float* red = reinterpret_cast<float*>(smem);
  float* mine = red + wid * (BM * kPitch);
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<v4f*>(mine + (32 * i + l) * kPitch + 32 * j + 8 * q + 4 * h) =
            v4f{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
  __syncthreads();
  join_waves<FMT, DT, BM, BN, NW>(a, vec, red, m0, n0);
}

template <int FMT, int DT, int BM, int BN, int NW>
hipError_t launch_split(const LinearArgs& a, hipStream_t s) {
  constexpr int kLds = NW * SplitRing<FMT, BM, BN>::kBytes;
  static_assert(kLds <= 160 * 1024, "LDS of a workgroup");
  auto kernel = k_linear_split<FMT, DT, BM, BN, NW>;
  static std::atomic<uint64_t> done{0};
  const hipError_t e = allow_lds((const void*)kernel, kLds, done);
  if (e != hipSuccess) return e;
  const uint32_t tm = (uint32_t)((a.M + BM - 1) / BM), tn = (uint32_t)((a.N + BN - 1) / BN);
  hipLaunchKernelGGL(kernel, dim3(tm * tn), dim3(NW * 64), kLds, s, a, epilogue_vec(a.ep), tm, tn);
  return hipGetLastError();
}

template <int FMT, int DT>
hipError_t launch_as(const LinearArgs& a, hipStream_t s) {
  switch (linear_kernel(a.M, a.N)) {
    case LinearKernel::kDirect: return launch_direct<FMT, DT, 8>(a, s);
    case LinearKernel::kSplit32x32: return launch_split<FMT, DT, 32, 32, 8>(a, s);
    case LinearKernel::kSplit32x64: return launch_split<FMT, DT, 32, 64, 4>(a, s);
    case LinearKernel::kSplit64x32: return launch_split<FMT, DT, 64, 32, 4>(a, s);
    case LinearKernel::kSplit64x64: return launch_split<FMT, DT, 64, 64, 4>(a, s);
    case LinearKernel::kTile128: return launch_tile<FMT, DT, 128, 128, 2, 2>(a, s);
    default: return launch_tile<FMT, DT, 256, 256, 2, 4>(a, s);
  }
}

template <int FMT>
hipError_t launch_fmt(const LinearArgs& a, hipStream_t s) {
  return a.ep.dt == DT_BF16 ? launch_as<FMT, DT_BF16>(a, s) : launch_as<FMT, DT_F32>(a, s);
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
