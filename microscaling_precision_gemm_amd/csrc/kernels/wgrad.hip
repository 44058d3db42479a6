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
#include <atomic>

#include "../device/decode8.h"
#include "../device/gemm_common.h"
#include "../launch.h"

namespace mxk {

namespace {

typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s* lds_v4s;

constexpr int kStep = 64;  // rows of one stage

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
  int32_t e0;  // first group of this launch
  bool f32, accumulate;
};

// A stage holds kStep rows of T BF16 columns of each operand.  16-byte chunk c
// of row r lies at chunk place(r, c) of its row: a transposed read touches 4
// rows x 64 bytes (and the 4 rows 8 below), which without the exchange of bits
// 1..3 fall on the same banks; bit 0 does the same for the writes of decoded
// codes, where neighbouring lanes are two chunks apart.
__device__ inline uint32_t swz(uint32_t r) { return ((r & 3u) << 2) | ((r >> 2) & 2u); }
template <int T>
__device__ inline uint32_t place(uint32_t r, uint32_t c) {
  return c ^ swz(r) ^ (T == 256 ? (c >> 4) & 1u : r & 1u);
}

__device__ inline void stage_barrier() {
  __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4) | (0 << 8));  // lgkmcnt(0): own LDS accesses done
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// What one thread copies of a stage: DC chunks of 8 dY columns and XC chunks
// of 16 codes, and which stage row and column they are.
template <int FMT, int WT, bool GATHER>
struct Copy {
  static constexpr int T = 2 * WT;               // tile edge
  static constexpr int DC = kStep * T / 8 / 256;  // dY chunks
  static constexpr int XC = kStep * T / 16 / 256; // code chunks
  static constexpr int PITCH = 2 * T;            // bytes of a stage row
  static constexpr int HALF = kStep * PITCH;     // bytes of an operand's stage

  uint4 d[DC], x[XC];
  uint32_t sc[XC];
  int32_t src[XC];  // rows of X the next loads take

  // stage row / column (elements) of chunk i
  static __device__ uint32_t drow(uint32_t tid, int i) { return (tid + 256u * i) / (T / 8); }
  static __device__ uint32_t dcol(uint32_t tid) { return tid % (T / 8) * 8; }
  static __device__ uint32_t xrow(uint32_t tid, int i) { return (tid + 256u * i) / (T / 16); }
  static __device__ uint32_t xcol(uint32_t tid) { return tid % (T / 16) * 16; }
};

struct Group {
  int64_t lo;       // first row
  int32_t cnt;      // rows
  int32_t steps;    // stages
};

// Row `row` of stage `st`, clamped into the group, relative to the stage's
// first row; stages past the last repeat it (their copies are never used).
// WHOLE: the stage is known to lie inside the group.
template <bool WHOLE>
__device__ inline int32_t clamp_stage(const Group& g, int32_t st) {
  return WHOLE || st < g.steps ? st : g.steps - 1;
}
template <bool WHOLE>
__device__ inline int32_t clamp_row(const Group& g, int32_t st, uint32_t row) {
  const int32_t rem = g.cnt - st * kStep - 1;
  return WHOLE || (int32_t)row < rem ? (int32_t)row : rem;
}

template <bool WHOLE, int FMT, int WT, bool GATHER>
__device__ inline void load_src(const WgradParams& p, const Group& g, int32_t st, uint32_t tid, int i,
                                Copy<FMT, WT, GATHER>& c) {
  st = clamp_stage<WHOLE>(g, st);
  const int64_t base = g.lo + (int64_t)st * kStep;
  const int32_t r = clamp_row<WHOLE>(g, st, Copy<FMT, WT, GATHER>::xrow(tid, i));
  if constexpr (GATHER) c.src[i] = p.row_index[base + r];
  else c.src[i] = (int32_t)base + r;
}

template <bool WHOLE, bool ODD, int FMT, int WT, bool GATHER>
__device__ inline void load_d(const WgradParams& p, const Group& g, int32_t st, uint32_t tid, int64_t n0, int i,
                              Copy<FMT, WT, GATHER>& c) {
  typedef Copy<FMT, WT, GATHER> C;
  st = clamp_stage<WHOLE>(g, st);
  const uint32_t col = C::dcol(tid);
  if constexpr (ODD) {  // rows may end inside a chunk
    const int32_t r = clamp_row<WHOLE>(g, st, C::drow(tid, i));
    const uint16_t* at = p.dy + (g.lo + (int64_t)st * kStep + r) * p.ld_dy + n0 + col;
    uint32_t w[4] = {};
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (n0 + col + e < p.N) w[e >> 1] |= (uint32_t)at[e] << (16 * (e & 1));
    c.d[i] = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    // a uniform base and a 32-bit lane offset (64 rows of a pitch below 2^24)
    const uint16_t* base = p.dy + (g.lo + (int64_t)st * kStep) * p.ld_dy + n0;
    const uint32_t cc = n0 + col < p.N ? col : 0;  // columns past N are computed and not stored
    uint32_t off;
    if constexpr (WHOLE) {
      base += (int64_t)(256 / (C::T / 8) * i) * p.ld_dy;
      off = (C::drow(tid, 0) * (uint32_t)p.ld_dy + cc) * 2u;
    } else {
      off = ((uint32_t)clamp_row<WHOLE>(g, st, C::drow(tid, i)) * (uint32_t)p.ld_dy + cc) * 2u;
    }
    c.d[i] = *reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(base) + off);
  }
}

template <int FMT, int WT, bool GATHER>
__device__ inline void load_x(const WgradParams& p, uint32_t tid, int64_t k0, int i, Copy<FMT, WT, GATHER>& c) {
  typedef Copy<FMT, WT, GATHER> C;
  int32_t src = c.src[i];
  src = min(max(src, 0), (int32_t)p.x_rows - 1);
  uint32_t k = C::xcol(tid);
  k = k0 + k < p.K ? k : 0;  // columns past K are computed and not stored
  c.x[i] = *reinterpret_cast<const uint4*>(p.codes + k0 + ((uint64_t)(uint32_t)src * (uint32_t)p.K + k));
  c.sc[i] = p.scales[k0 / 32 + ((uint64_t)(uint32_t)src * (uint32_t)(p.K / 32) + k / 32)];
}

// the thread's dY chunk i of stage st into LDS; rows past the group are 0
template <bool WHOLE, int FMT, int WT, bool GATHER>
__device__ inline void put_d(const Group& g, int32_t st, uint32_t tid, int i, const Copy<FMT, WT, GATHER>& c, uint8_t* stage) {
  typedef Copy<FMT, WT, GATHER> C;
  const uint32_t r = C::drow(tid, i);
  uint4 w = c.d[i];
  if constexpr (!WHOLE) {
    const bool in = st * kStep + (int32_t)r < g.cnt;
    w.x = in ? w.x : 0;
    w.y = in ? w.y : 0;
    w.z = in ? w.z : 0;
    w.w = in ? w.w : 0;
  }
  *reinterpret_cast<uint4*>(stage + r * C::PITCH + 16u * place<C::T>(r, C::dcol(tid) / 8)) = w;
}

// the thread's code chunk i, decoded
template <bool WHOLE, int FMT, int WT, bool GATHER>
__device__ inline void put_x(const Group& g, int32_t st, uint32_t tid, int i, const Copy<FMT, WT, GATHER>& c, uint8_t* stage) {
  typedef Copy<FMT, WT, GATHER> C;
  const uint32_t r = C::xrow(tid, i);
  uint32_t o[8];
  decode4_bf16<FMT>(c.x[i].x, c.sc[i], o);
  decode4_bf16<FMT>(c.x[i].y, c.sc[i], o + 2);
  decode4_bf16<FMT>(c.x[i].z, c.sc[i], o + 4);
  decode4_bf16<FMT>(c.x[i].w, c.sc[i], o + 6);
  if constexpr (!WHOLE) {
    const bool in = st * kStep + (int32_t)r < g.cnt;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = in ? o[e] : 0;
  }
  const uint32_t ch = C::xcol(tid) / 8;
  uint8_t* row = stage + C::HALF + r * C::PITCH;
  *reinterpret_cast<uint4*>(row + 16u * place<C::T>(r, ch)) = make_uint4(o[0], o[1], o[2], o[3]);
  *reinterpret_cast<uint4*>(row + 16u * place<C::T>(r, ch + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
}

template <int F>
struct Frags {
  v8b a[F], b[F];
};

// the fragments of rows 16 q .. 16 q + 15: lane l holds column l % 32, rows
// 8 (l / 32) .. + 7 of each 32-column block; off[i]: this lane's byte offset
// of block i in a stage row group
template <int WT>
__device__ inline void read_frags(const uint8_t* stage, int q, const uint32_t (&aoff)[WT / 32],
                                  const uint32_t (&boff)[WT / 32], Frags<WT / 32>& f) {
  constexpr int PITCH = 4 * WT, HALF = kStep * PITCH;
  union {
    v4s h[2];
    v8b v;
  } u;
#pragma unroll
  for (int i = 0; i < WT / 32; ++i) {
    const uint8_t* pa = stage + aoff[i] + q * (16 * PITCH);
    u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)pa);
    u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(pa + 4 * PITCH));
    f.a[i] = u.v;
    const uint8_t* pb = stage + HALF + boff[i] + q * (16 * PITCH);
    u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)pb);
    u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(pb + 4 * PITCH));
    f.b[i] = u.v;
  }
}

template <int F>
__device__ inline void mma(const Frags<F>& f, v16f (&acc)[F][F]) {
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
}

// Writes the share W (0..3) of stage st's copy into its buffer and issues the
// loads of the same share of stage st + 1 into the freed registers.  WHOLE:
// stages st .. st + 2 lie inside the group.
template <int W, bool WHOLE, bool ODD, int FMT, int WT, bool GATHER>
__device__ inline void copy_share(const WgradParams& p, const Group& g, int32_t st, uint32_t tid, int64_t n0,
                                  int64_t k0, Copy<FMT, WT, GATHER>& c, uint8_t* smem) {
  typedef Copy<FMT, WT, GATHER> C;
  uint8_t* stage = smem + (st & 1) * (2 * C::HALF);
#pragma unroll
  for (int i = W * C::DC / 4; i < (W + 1) * C::DC / 4; ++i) {
    put_d<WHOLE>(g, st, tid, i, c, stage);
    load_d<WHOLE, ODD>(p, g, st + 1, tid, n0, i, c);
  }
#pragma unroll
  for (int i = W * C::XC / 4; i < (W + 1) * C::XC / 4; ++i) {
    put_x<WHOLE>(g, st, tid, i, c, stage);
    load_x(p, tid, k0, i, c);
    load_src<WHOLE>(p, g, st + 2, tid, i, c);
  }
}

// Spreads a window's other work over its 16 products: the next fragments
// first, so that they have landed when the window ends, then the stage writes
// and the loads.
template <int I = 0>
__device__ inline void spread_window() {
  if constexpr (I < 16) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                          // matrix
    if constexpr (I < 8) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);     // LDS read
    __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);                          // VALU
    if constexpr (I >= 8 && I % 2) __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);  // LDS write
    if constexpr (I >= 8 && I < 13) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // load
    spread_window<I + 1>();
  }
}
template <int WT>
__device__ inline void window_end() {
  if constexpr (WT == 128) spread_window();
  __builtin_amdgcn_sched_barrier(0);
}

// One stage: windows of 16 rows.  While a window's products run, the next
// window's fragments are read and a quarter of the next stage is written.  The
// barrier comes before the last window, when its fragments are in registers:
// behind it the stage is free to be overwritten and the next one is complete.
template <bool WHOLE, bool ODD, int FMT, int WT, bool GATHER>
__device__ inline void stage_products(const WgradParams& p, const Group& g, int32_t st, uint32_t tid, int64_t n0,
                                      int64_t k0, Copy<FMT, WT, GATHER>& c, uint8_t* smem, const uint32_t (&aoff)[WT / 32],
                                      const uint32_t (&boff)[WT / 32], Frags<WT / 32> (&f)[2],
                                      v16f (&acc)[WT / 32][WT / 32]) {
  typedef Copy<FMT, WT, GATHER> C;
  const uint8_t* cur = smem + (st & 1) * (2 * C::HALF);
  const uint8_t* nxt = smem + ((st + 1) & 1) * (2 * C::HALF);
  read_frags<WT>(cur, 1, aoff, boff, f[1]);
  copy_share<0, WHOLE, ODD>(p, g, st + 1, tid, n0, k0, c, smem);
  mma(f[0], acc);
  window_end<WT>();
  read_frags<WT>(cur, 2, aoff, boff, f[0]);
  copy_share<1, WHOLE, ODD>(p, g, st + 1, tid, n0, k0, c, smem);
  mma(f[1], acc);
  window_end<WT>();
  read_frags<WT>(cur, 3, aoff, boff, f[1]);
  copy_share<2, WHOLE, ODD>(p, g, st + 1, tid, n0, k0, c, smem);
  mma(f[0], acc);
  window_end<WT>();
  stage_barrier();
  read_frags<WT>(nxt, 0, aoff, boff, f[0]);
  copy_share<3, WHOLE, ODD>(p, g, st + 2, tid, n0, k0, c, smem);
  mma(f[1], acc);
  window_end<WT>();
}

// the wave's products: lanes 0..31 and 32..63 each store 32 adjacent columns
template <int WDT, bool ACC, int F>
__device__ inline void store_products(const WgradParams& p, int64_t row0, int64_t n1, int64_t k1, uint32_t lane,
                                      const v16f (&acc)[F][F]) {
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int64_t n = n1 + 32 * i + 8 * (v / 4) + 4 * (lane >> 5) + (v % 4);
      if (n >= p.N) continue;
#pragma unroll
      for (int j = 0; j < F; ++j) {
        const int64_t k = k1 + 32 * j + (lane & 31u);
        if (k >= p.K) continue;
        const int64_t off = (row0 + n) * p.ld_dw + k;
        float o = acc[i][j][v];
        if constexpr (ACC) o += load1<WDT>(p.dw, off);
        store1<WDT>(p.dw, off, o);
      }
    }
}

template <int FMT, int WT, bool ODD, bool GATHER>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(WT == 128 ? 1 : 2, WT == 128 ? 1 : 2))) void
k_wgrad(WgradParams p) {
  typedef Copy<FMT, WT, GATHER> C;
  constexpr int F = WT / 32, T = C::T;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t wn = (wid >> 1) * WT, wk = (wid & 1u) * WT;
  // The tiles of a group are dealt to the 8 XCDs (workgroup id mod 8) in
  // runs, n fastest: the workgroups of an XCD share the rows of dY.
  const uint32_t per = (p.tn * p.tk + 7) / 8;  // tiles of a group on one XCD
  const uint32_t slot = blockIdx.x >> 3;
  const int32_t e = p.e0 + (int32_t)(slot / per);
  const uint32_t in = (blockIdx.x & 7u) * per + slot % per;
  if (in >= p.tn * p.tk) return;
  const int64_t n0 = (int64_t)(in % p.tn) * T, k0 = (int64_t)(in / p.tn) * T;
  Group g = {0, 0, 0};
  {
    int64_t lo = 0, hi = p.R;
    if (p.offsets) {  // clamped into [0, R]
      lo = p.offsets[e];
      hi = p.offsets[e + 1];
      lo = lo < 0 ? 0 : (lo > p.R ? p.R : lo);
      hi = hi < lo ? lo : (hi > p.R ? p.R : hi);
    }
    g.lo = lo;
    g.cnt = (int32_t)(hi - lo);
    g.steps = (g.cnt + kStep - 1) / kStep;
  }
  v16f acc[F][F];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

  if (g.steps > 0) {
    // fragment addresses: 16 lanes read 4 rows x 16 columns
    uint32_t aoff[F], boff[F];
    {
      const uint32_t s = lane & 15u, gr = lane >> 4;
      const uint32_t row = 8 * (gr >> 1) + (s >> 2);
#pragma unroll
      for (int i = 0; i < F; ++i) {
        const uint32_t col = 32 * i + 16 * (gr & 1) + 4 * (s & 3);
        aoff[i] = row * C::PITCH + 16u * place<T>(row, (wn + col) / 8) + 8 * (s & 1);
        boff[i] = row * C::PITCH + 16u * place<T>(row, (wk + col) / 8) + 8 * (s & 1);
      }
    }
    C c;
#pragma unroll
    for (int i = 0; i < C::XC; ++i) load_src<false>(p, g, 0, tid, i, c);
#pragma unroll
    for (int i = 0; i < C::DC; ++i) load_d<false, ODD>(p, g, 0, tid, n0, i, c);
#pragma unroll
    for (int i = 0; i < C::XC; ++i) load_x(p, tid, k0, i, c);
#pragma unroll
    for (int i = 0; i < C::XC; ++i) load_src<false>(p, g, 1, tid, i, c);
    copy_share<0, false, ODD>(p, g, 0, tid, n0, k0, c, smem);
    copy_share<1, false, ODD>(p, g, 0, tid, n0, k0, c, smem);
    copy_share<2, false, ODD>(p, g, 0, tid, n0, k0, c, smem);
    copy_share<3, false, ODD>(p, g, 0, tid, n0, k0, c, smem);
    stage_barrier();
    Frags<F> f[2];
    read_frags<WT>(smem, 0, aoff, boff, f[0]);
    copy_share<3, false, ODD>(p, g, 1, tid, n0, k0, c, smem);
    int32_t st = 0;
    for (; (st + 5) * kStep <= g.cnt; ++st)  // stages up to st + 4 whole
      stage_products<true, ODD>(p, g, st, tid, n0, k0, c, smem, aoff, boff, f, acc);
    for (; st < g.steps; ++st) stage_products<false, ODD>(p, g, st, tid, n0, k0, c, smem, aoff, boff, f, acc);
  }
  const int64_t row0 = (int64_t)e * p.N, n1 = n0 + wn, k1 = k0 + wk;
  if (p.f32) {
    if (p.accumulate) store_products<DT_F32, true>(p, row0, n1, k1, lane, acc);
    else store_products<DT_F32, false>(p, row0, n1, k1, lane, acc);
  } else {
    if (p.accumulate) store_products<DT_BF16, true>(p, row0, n1, k1, lane, acc);
    else store_products<DT_BF16, false>(p, row0, n1, k1, lane, acc);
  }
}

template <int FMT, int WT, bool ODD, bool GATHER>
hipError_t launch_t(const WgradArgs& a, hipStream_t s) {
  typedef Copy<FMT, WT, GATHER> C;
  WgradParams p = {a.dy, a.ld_dy, a.R, a.N, a.codes, a.scales, a.x_rows, a.K, a.row_index, a.offsets, a.groups,
                   a.dw, a.ld_dw, (uint32_t)((a.N + C::T - 1) / C::T), (uint32_t)((a.K + C::T - 1) / C::T), 0,
                   a.dwdt == DT_F32, a.accumulate};
  constexpr int smem = 4 * C::HALF;
  auto kern = k_wgrad<FMT, WT, ODD, GATHER>;
  // the dynamic LDS limit is raised once per device
  static std::atomic<uint64_t> attr_done{0};
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (!bit || !(attr_done.load(std::memory_order_acquire) & bit)) {
    e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != hipSuccess) return e;
    attr_done.fetch_or(bit, std::memory_order_acq_rel);
  }
  // (a grid holds fewer than 2^24 workgroups of 256)
  const int64_t each = ((int64_t)p.tn * p.tk + 7) / 8 * 8;
  const int64_t most = each < (1 << 23) ? (1 << 23) / each : 1;
  for (int64_t e0 = 0; e0 < a.groups; e0 += most) {
    p.e0 = (int32_t)e0;
    const int64_t n = a.groups - e0 < most ? a.groups - e0 : most;
    hipLaunchKernelGGL(kern, dim3((uint32_t)(n * each)), dim3(256), smem, s, p);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int FMT, bool GATHER>
hipError_t launch_g(const WgradArgs& a, hipStream_t s) {
  // dY rows that end inside a 16-byte chunk (or of a pitch past 32-bit
  // offsets) are loaded element by element
  if (a.N % 8 || a.ld_dy >= (1 << 24)) return launch_t<FMT, 64, true, GATHER>(a, s);
  // 256 x 256 tiles when they fill the CUs, else 128 x 128
  const int64_t big = ((a.N + 255) / 256) * ((a.K + 255) / 256) * a.groups;
  return big >= 256 ? launch_t<FMT, 128, false, GATHER>(a, s) : launch_t<FMT, 64, false, GATHER>(a, s);
}

template <int FMT>
hipError_t launch_f(const WgradArgs& a, hipStream_t s) {
  return a.row_index ? launch_g<FMT, true>(a, s) : launch_g<FMT, false>(a, s);
}

}  // namespace

hipError_t launch_wgrad_grouped(const WgradArgs& a, hipStream_t s) {
  if (a.fmt == FMT_MXFP8) return launch_f<FMT_MXFP8>(a, s);
  if (a.fmt == FMT_MXFP8_E5M2) return launch_f<FMT_MXFP8_E5M2>(a, s);
  return launch_f<FMT_MXINT8>(a, s);
}

}  // namespace mxk
