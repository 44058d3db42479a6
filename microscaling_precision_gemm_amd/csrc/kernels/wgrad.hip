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
#include <type_traits>

#include "../device/decode8.h"
#include "../device/gemm_common.h"
#include "../launch.h"

namespace mxk {

namespace {

typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s* lds_v4s;
typedef __attribute__((address_space(3))) u4* lds_u4;

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
  uint32_t tn, tk;  // tiles along N and K
  uint32_t units;   // tiles of all groups, rounded up for the deal to the XCDs
  bool f32, accumulate, vec;
};

// A stage holds kStep rows of T BF16 columns of each operand.  16-byte chunk c
// of row r lies at chunk place(r, c) of its row: a transposed read touches 4
// rows x 64 bytes (and the 4 rows 8 below), which without the exchange of bits
// 1..3 fall on the same banks; bit 0 does the same for the writes of decoded
// codes, where neighbouring lanes are two chunks apart.
__device__ __forceinline__ uint32_t swz(uint32_t r) { return ((r & 3u) << 2) | ((r >> 2) & 2u); }
template <int T>
__device__ __forceinline__ uint32_t place(uint32_t r, uint32_t c) {
  return c ^ swz(r) ^ (T == 256 ? (c >> 4) & 1u : r & 1u);
}

__device__ __forceinline__ void stage_barrier() {
  __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4) | (0 << 8));  // lgkmcnt(0): own LDS accesses done
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The variants.  WT: columns of a wave's tile (a workgroup's is T = 2 WT
// square).  ANY: any N, K, pitch and size of X, otherwise dY in whole 16-byte
// chunks, K a multiple of 128 (a scale code is then loaded as the aligned word
// around it) and offsets within 32 bits.  GATHER: X's rows by the row index.
template <int FMT_, int WT_, bool ANY_, bool GATHER_>
struct Variant {
  static constexpr int FMT = FMT_, WT = WT_;
  static constexpr bool ANY = ANY_, GATHER = GATHER_;
  static constexpr int F = WT / 32, T = 2 * WT;
  static constexpr int DC = kStep * T / 8 / 256;   // a thread's chunks of 8 dY columns in a stage,
  static constexpr int DR = 256 / (T / 8);         // and the rows between them
  static constexpr int XC = kStep * T / 16 / 256;  // the same for chunks of 16 codes
  static constexpr int XR = 256 / (T / 16);
  static constexpr int PITCH = 2 * T;              // bytes of a stage row
  static constexpr int HALF = kStep * PITCH;       // bytes of an operand's stage
  static constexpr int SCRATCH = 64 * WT;          // bytes a wave needs to turn its products into rows
  static constexpr int LDS = 4 * HALF + 4 * SCRATCH;
};

// One tile and its rows (the same in all lanes).
struct Unit {
  uint32_t n0, k0;
  int32_t e;         // group; -1: there is none
  int32_t row, cnt;  // its rows, at least one
  // Stages: at least 3, so that the copies, which run ahead of the products,
  // never reach past the tile after this one.
  __device__ __forceinline__ int32_t stages() const { return max((cnt + kStep - 1) / kStep, 3); }
};

template <class V>
__device__ __forceinline__ void clear_tile(const WgradParams& p, uint32_t e, uint32_t n0, uint32_t k0) {
  for (uint32_t q = threadIdx.x; q < V::T * V::T; q += 256) {
    const int64_t n = (int64_t)n0 + q / V::T, k = (int64_t)k0 + q % V::T;
    if (n < p.N && k < p.K) {
      const int64_t off = (e * p.N + n) * p.ld_dw + k;
      if (p.f32) static_cast<float*>(p.dw)[off] = 0.0f;
      else static_cast<uint16_t*>(p.dw)[off] = 0;
    }
  }
}

// Unit `id` or the next one of this workgroup that has rows.  The tiles of a
// group are dealt to the 8 XCDs (workgroup id mod 8) in runs, n fastest, so
// that the workgroups of an XCD share rows of dY and X in its L2.  A group
// without rows is passed over; its tiles of dW are cleared on the way.
template <class V>
__device__ __forceinline__ Unit seek(const WgradParams& p, uint32_t& id) {
  const uint32_t tiles = p.tn * p.tk, per = (tiles + 7) / 8;
  for (; id < p.units; id += gridDim.x) {
    const uint32_t slot = id >> 3, e = slot / per;
    const uint32_t in = (id & 7u) * per + (slot - e * per);
    if (in >= tiles) continue;
    int64_t lo = 0, hi = p.R;
    if (p.offsets) {  // clamped into [0, R]
      lo = p.offsets[e];
      hi = p.offsets[e + 1];
      lo = lo < 0 ? 0 : (lo > p.R ? p.R : lo);
      hi = hi < lo ? lo : (hi > p.R ? p.R : hi);
    }
    const uint32_t tk = in / p.tn, n0 = (in - tk * p.tn) * V::T, k0 = tk * V::T;
    if (hi > lo) return {n0, k0, (int32_t)e, (int32_t)lo, (int32_t)(hi - lo)};
    if (!p.accumulate) clear_tile<V>(p, e, n0, k0);
  }
  return {0, 0, -1, 0, 1};
}

// A position in the stream of stages.
struct Cursor {
  int32_t row, rem;  // first row of the stage, rows of the group from there on
  int32_t left;      // stages of the tile from this one on
  __device__ __forceinline__ void start(const Unit& u) {
    row = u.row;
    rem = u.cnt;
    left = u.stages();
  }
  // To the next stage; true when that begins `next` (the last tile's last
  // stage is repeated for ever).  A tile's stages beyond its rows repeat the
  // last one with rows.
  __device__ __forceinline__ bool step(const Unit& next) {
    if (--left == 0) {
      if (next.e >= 0) {
        start(next);
        return true;
      }
      left = INT32_MAX;
    }
    if (rem > kStep) {
      row += kStep;
      rem -= kStep;
    }
    return false;
  }
};

// What one thread copies.
template <class V>
struct Copy {
  typedef typename std::conditional<V::ANY, uint64_t, uint32_t>::type Off;
  u4 d[V::DC], x[V::XC];
  uint32_t sc[V::XC];
  // where the next loads take it from: byte offsets from uniform bases
  const char* dbase;
  const uint8_t* xbase;
  uint32_t doff[V::DC];
  Off xoff[V::XC];
  int32_t ridx;  // GATHER: lane r of the wave holds the row of X of row r of the stage after that
  uint32_t kk;   // first of the thread's columns of X in the tile, 0 past K
  // constants: the thread's columns, first rows, and LDS addresses of its
  // chunk 0 in the buffer that is written (the other chunks lie whole rows
  // below; for dY of 256-wide tiles bit 1 of the chunk number changes in turn)
  uint32_t dcol, xcol, drow, xrow;
  uint32_t dput, dput1, xput, sc_shift;

  __device__ __forceinline__ void init(uint32_t tid) {
    dcol = tid % (V::T / 8) * 8;
    xcol = tid % (V::T / 16) * 16;
    drow = tid / (V::T / 8);
    xrow = tid / (V::T / 16);
    dput = drow * V::PITCH + 16u * place<V::T>(drow, dcol / 8);
    dput1 = V::DR == 8 ? dput ^ 32u : dput;
    xput = V::HALF + xrow * V::PITCH + 16u * place<V::T>(xrow, xcol / 16 * 2);
    sc_shift = xcol / 32 % 4 * 8;
  }
  __device__ __forceinline__ void flip() {  // to the other buffer
    dput ^= 2 * V::HALF;
    dput1 ^= 2 * V::HALF;
    xput ^= 2 * V::HALF;
  }
  __device__ __forceinline__ uint32_t dput_of(int i) const {
    return ((i & 1) ? dput1 : dput) + (uint32_t)(i * V::DR * V::PITCH);
  }
};

// Row numbers of X for the stage at `at` (rows past the group repeat the last;
// drop_rows() clears them in LDS).
template <class V>
__device__ __forceinline__ void load_rows(const WgradParams& p, const Cursor& at, uint32_t lane, Copy<V>& c) {
  if constexpr (V::GATHER)
    c.ridx = *reinterpret_cast<const int32_t*>(reinterpret_cast<const char*>(p.row_index + at.row) +
                                               4u * (uint32_t)min((int32_t)lane, at.rem - 1));
}

// Aims the loads at the stage at `at` of tile u.  `fresh`: the tile, or the
// number of rows, is another than before; the lane offsets of full stages of
// one tile are the same.
template <class V>
__device__ __forceinline__ void aim(const WgradParams& p, const Unit& u, const Cursor& at, bool fresh, Copy<V>& c) {
  c.dbase = reinterpret_cast<const char*>(p.dy + (int64_t)at.row * p.ld_dy + u.n0);
  if (fresh || at.rem < kStep) {
    // columns past N and K are computed from others and not stored
    const uint32_t cc = u.n0 + c.dcol < (uint32_t)p.N ? 2u * c.dcol : 0u;
    c.kk = u.k0 + c.xcol < (uint32_t)p.K ? c.xcol : 0u;
    const uint32_t last = (uint32_t)min(at.rem, kStep) - 1u;
#pragma unroll
    for (int i = 0; i < V::DC; ++i) {
      const uint32_t r = min(c.drow + i * V::DR, last);
      c.doff[i] = V::ANY ? r : r * 2u * (uint32_t)p.ld_dy + cc;
    }
    if constexpr (!V::GATHER) {
#pragma unroll
      for (int i = 0; i < V::XC; ++i)
        c.xoff[i] = (typename Copy<V>::Off)min(c.xrow + i * V::XR, last) * (uint32_t)p.K + c.kk;
    }
  }
  if constexpr (V::GATHER) {
    c.xbase = p.codes + u.k0;
    const uint32_t r = (uint32_t)min(max(c.ridx, 0), (int32_t)p.x_rows - 1);
    if constexpr (V::ANY) {
#pragma unroll
      for (int i = 0; i < V::XC; ++i)
        c.xoff[i] = (uint64_t)lane_read(r, c.xrow + i * V::XR) * (uint32_t)p.K + c.kk;
    } else {
      const uint32_t o = r * (uint32_t)p.K;
#pragma unroll
      for (int i = 0; i < V::XC; ++i) c.xoff[i] = lane_read(o, c.xrow + i * V::XR) + c.kk;
    }
  } else {
    c.xbase = p.codes + (int64_t)at.row * p.K + u.k0;
  }
}

template <class V>
__device__ __forceinline__ void load_d(const WgradParams& p, uint32_t n0, int i, Copy<V>& c) {
  if constexpr (V::ANY) {  // rows may end inside a chunk, or have a large pitch
    const uint16_t* at = reinterpret_cast<const uint16_t*>(c.dbase) + (int64_t)c.doff[i] * p.ld_dy + c.dcol;
    uint32_t w[4] = {};
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (n0 + c.dcol + e < (uint32_t)p.N) w[e >> 1] |= (uint32_t)at[e] << (16 * (e & 1));
    c.d[i] = u4{w[0], w[1], w[2], w[3]};
  } else {
    c.d[i] = *reinterpret_cast<const u4*>(c.dbase + c.doff[i]);
  }
}

template <class V>
__device__ __forceinline__ void load_x(int i, Copy<V>& c) {
  c.x[i] = *reinterpret_cast<const u4*>(c.xbase + c.xoff[i]);
}
// Scale codes: one for 32 codes, so at 1/32 of the code offset from the start
// (sbase: of the scales at the uniform part of it).
template <class V>
__device__ __forceinline__ void load_sc(const WgradParams& p, int i, Copy<V>& c) {
  const uint8_t* sbase = p.scales + (uint64_t)(c.xbase - p.codes) / 32;
  if constexpr (V::ANY) c.sc[i] = sbase[c.xoff[i] / 32];
  else c.sc[i] = *reinterpret_cast<const uint32_t*>(sbase + ((c.xoff[i] >> 5) & ~3u));
}

// the thread's dY chunk i into LDS
template <class V>
__device__ __forceinline__ void put_d(int i, const Copy<V>& c) {
  *(lds_u4)c.dput_of(i) = c.d[i];
}
// Its code chunk i on the way: scale, pair by pair, into LDS by halves.
struct Decoded {
  float x;
  uint32_t o[8];
};
template <class V>
__device__ __forceinline__ void decode_scale(int i, const Copy<V>& c, Decoded& d) {
  if constexpr (V::ANY) d.x = scale8<V::FMT>(c.sc[i]);
  else d.x = scale8_word<V::FMT>(c.sc[i], c.sc_shift);
}
template <int P, class V>
__device__ __forceinline__ void decode_pair(int i, const Copy<V>& c, Decoded& d) {
  d.o[P] = decode2_bf16<V::FMT, P & 1>(c.x[i][P / 2], d.x);
}
template <int H, class V>
__device__ __forceinline__ void put_x(int i, const Copy<V>& c, const Decoded& d) {
  *(lds_u4)((c.xput ^ (16u * H)) + i * V::XR * V::PITCH) = u4{d.o[4 * H], d.o[4 * H + 1], d.o[4 * H + 2], d.o[4 * H + 3]};
}

// Clears the rows from `rem` on of the stage that was just written, in both
// operands (a row that is not of the group may hold NaN).  Each thread clears
// what it wrote itself, and a wave's LDS accesses keep their order, so no
// barrier is needed between.
template <class V>
__device__ __forceinline__ void drop_rows(int32_t rem, const Copy<V>& c) {
  const u4 z = u4{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < V::DC; ++i)
    if ((int32_t)c.drow + i * V::DR >= rem) *(lds_u4)c.dput_of(i) = z;
#pragma unroll
  for (int i = 0; i < V::XC; ++i)
    if ((int32_t)c.xrow + i * V::XR >= rem) {
      const uint32_t at = i * V::XR * V::PITCH;
      *(lds_u4)(c.xput + at) = z;
      *(lds_u4)((c.xput ^ 16u) + at) = z;
    }
}

template <int F>
struct Frags {
  v8b k[F], n[F];  // columns of X, of dY
};

// half H (4 of its rows) of a fragment of rows 16 q .. 16 q + 15: lane l holds
// column l % 32, rows 8 (l / 32) .. + 7 of a 32-column block; off: this lane's
// LDS address of the block in the first rows
template <int H, int WT>
__device__ __forceinline__ void read_half(int q, uint32_t off, v8b& f) {
  constexpr int PITCH = 4 * WT;
  typedef short v8s __attribute__((ext_vector_type(8)));
  v8s v = __builtin_bit_cast(v8s, f);
  const v4s h = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(off + (q * 16 + 4 * H) * PITCH));
#pragma unroll
  for (int e = 0; e < 4; ++e) v[4 * H + e] = h[e];
  f = __builtin_bit_cast(v8b, v);
}
// half-fragment R (0 .. 4 F - 1) of a window, in the order of their use
template <int R, int WT>
__device__ __forceinline__ void read_nth(int q, const uint32_t (&noff)[WT / 32], const uint32_t (&koff)[WT / 32],
                                         Frags<WT / 32>& f) {
  constexpr int F = WT / 32, I = R / 2;
  if constexpr (I == 0) read_half<R & 1, WT>(q, koff[0], f.k[0]);
  else if constexpr (I <= F) read_half<R & 1, WT>(q, noff[I - 1], f.n[I - 1]);
  else read_half<R & 1, WT>(q, koff[I - F], f.k[I - F]);
}
template <int WT, int R = 0>
__device__ __forceinline__ void read_frags(int q, const uint32_t (&noff)[WT / 32], const uint32_t (&koff)[WT / 32],
                                           Frags<WT / 32>& f) {
  if constexpr (R < 4 * (WT / 32)) {
    read_nth<R, WT>(q, noff, koff, f);
    read_frags<WT, R + 1>(q, noff, koff, f);
  }
}

// Writes the share W (0..3) of a stage into its buffer and issues the loads of
// the same share of the stage after it.
template <int W, class V>
__device__ __forceinline__ void copy_share(const WgradParams& p, uint32_t n0, Copy<V>& c) {
#pragma unroll
  for (int i = W * V::DC / 4; i < (W + 1) * V::DC / 4; ++i) {
    put_d(i, c);
    load_d(p, n0, i, c);
  }
#pragma unroll
  for (int i = W * V::XC / 4; i < (W + 1) * V::XC / 4; ++i) {
    Decoded d;
    decode_scale(i, c, d);
    decode_pair<0>(i, c, d);
    decode_pair<1>(i, c, d);
    decode_pair<2>(i, c, d);
    decode_pair<3>(i, c, d);
    put_x<0>(i, c, d);
    decode_pair<4>(i, c, d);
    decode_pair<5>(i, c, d);
    decode_pair<6>(i, c, d);
    decode_pair<7>(i, c, d);
    put_x<1>(i, c, d);
    load_x(i, c);
    load_sc(p, i, c);
  }
}

// One window of 16 rows: the products of `f`, and between them the reads of
// the next window's fragments (rows 16 q of the buffer at noff / koff) and the
// share W of the copies.  With one wave on a SIMD the order is the schedule:
// each product (32 cycles of the matrix unit) is followed by what fits beside
// it, and nothing moves over it.
template <int W, class V, int M = 0>
__device__ __forceinline__ void window(const WgradParams& p, uint32_t n0, Copy<V>& c, int q,
                                       const uint32_t (&noff)[V::F], const uint32_t (&koff)[V::F],
                                       const Frags<V::F>& f, Frags<V::F>& next, v16f (&acc)[V::F][V::F], Decoded& d) {
  constexpr int F = V::F;
  if constexpr (F == 2) {  // two waves on a SIMD: they fill each other's gaps
    read_frags<V::WT>(q, noff, koff, next);
    copy_share<W>(p, n0, c);
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < F; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.k[i], f.n[j], acc[i][j], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  } else if constexpr (M < F * F) {
    static_assert(V::DC == 8 && V::XC == 4, "shares of two dY chunks and one code chunk");
    acc[M / F][M % F] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.k[M / F], f.n[M % F], acc[M / F][M % F], 0, 0, 0);
    read_nth<M, V::WT>(q, noff, koff, next);
    if constexpr (M == 0) decode_scale(W, c, d);
    if constexpr (M >= 1 && M <= 8) decode_pair<(M - 1) & 7>(W, c, d);
    if constexpr (M == 5) put_x<0>(W, c, d);
    if constexpr (M == 9) put_x<1>(W, c, d);
    if constexpr (M == 10) put_d(2 * W, c);
    if constexpr (M == 11) put_d(2 * W + 1, c);
    if constexpr (M == 12) load_x(W, c);
    if constexpr (M == 13) load_sc(p, W, c);
    if constexpr (M == 14) load_d(p, n0, 2 * W, c);
    if constexpr (M == 15) load_d(p, n0, 2 * W + 1, c);
    __builtin_amdgcn_sched_barrier(0);
    window<W, V, M + 1>(p, n0, c, q, noff, koff, f, next, acc, d);
  }
}

// A wave's tile of products, 32 columns of N at a time and PC of K, through
// 128 PC bytes of LDS of its own into rows of dW.  Chunk c of 4 columns of row
// r lies at chunk c ^ (r mod chunks): writes of 16 rows and reads of one row
// are free of conflicts.  PLAIN: the tile lies inside dW, whose rows are
// 16-byte aligned, and is not added to; otherwise chunk by chunk with checks.
template <int WDT, bool PLAIN, class V>
__device__ __forceinline__ void store_tile(const WgradParams& p, const Unit& u, uint32_t wn, uint32_t wk, uint32_t lane,
                                           const v16f (&acc)[V::F][V::F], uint32_t scratch) {
  constexpr int PC = V::WT / 2;                // columns of a pass
  constexpr int CH = PC / 4;                   // 16-byte chunks of a scratch row
  constexpr int CPL = WDT == DT_F32 ? 1 : 2;   // chunks a lane stores
  constexpr int EB = WDT == DT_F32 ? 4 : 2;
  constexpr int RPI = 64 / (CH / CPL);         // rows stored at once
  typedef __attribute__((address_space(3))) f4* lds_f4;
  // (opaque, so that the addresses below are not kept over the main loop)
  asm volatile("" : "+v"(lane));
  const uint32_t lr = lane & 31u, lg = lane >> 5;
  const uint32_t rr = lane / (CH / CPL), cc = lane % (CH / CPL) * CPL;
  const uint32_t wbase = scratch + lr * (PC * 4), wx = lg ^ (lr & (CH - 1));
  uint8_t* base = static_cast<uint8_t*>(p.dw) +
                  (((int64_t)u.e * p.N + u.n0 + wn) * p.ld_dw + u.k0 + wk) * EB;  // uniform
  const int64_t loff = ((int64_t)rr * p.ld_dw + 4 * cc) * EB;
#pragma unroll
  for (int j = 0; j < V::F; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i2 = 0; i2 < PC / 32; ++i2)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const v16f& a = acc[h * (PC / 32) + i2][j];
          *(lds_f4)(wbase + 16u * (wx ^ (uint32_t)(8 * i2 + 2 * v))) = f4{a[4 * v], a[4 * v + 1], a[4 * v + 2], a[4 * v + 3]};
        }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int t = 0; t < 32 / RPI; ++t) {
        const uint32_t r = t * RPI + rr;
        float o[4 * CPL];
#pragma unroll
        for (int k = 0; k < CPL; ++k) {
          const f4 x = *(lds_f4)(scratch + r * (PC * 4) + 16u * ((cc + k) ^ (r & (CH - 1))));
#pragma unroll
          for (int e = 0; e < 4; ++e) o[4 * k + e] = x[e];
        }
        uint8_t* at = base + ((int64_t)(32 * j + t * RPI) * p.ld_dw + PC * h) * EB + loff;
        if constexpr (PLAIN) {
          if constexpr (WDT == DT_F32) *reinterpret_cast<f4*>(at) = f4{o[0], o[1], o[2], o[3]};
          else *reinterpret_cast<u4*>(at) = u4{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]),
                                              pack_bf16(o[6], o[7])};
        } else {
          // (K is a multiple of 32: a lane's columns are all inside or outside)
          const bool in = (int64_t)u.n0 + wn + 32 * j + r < p.N && (int64_t)u.k0 + wk + PC * h + 4 * cc < p.K;
          if (in) {
#pragma unroll
            for (int e = 0; e < 4 * CPL; ++e) {
              if (p.accumulate) o[e] += load1<WDT>(at, e);
              store1<WDT>(at, e, o[e]);
            }
          }
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
}

// Stages flow through the pipeline without a break between tiles: while a
// tile's last products run, the next tile's first stages are being copied.
// The workgroup's LDS is addressed by plain offsets from its start (there is no
// static allocation), so that changing buffers is one exclusive or.
template <class V>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(V::WT == 128 ? 1 : 2, V::WT == 128 ? 1 : 2))) void
k_wgrad(WgradParams p) {
  constexpr int F = V::F, T = V::T;
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t wn = (wid >> 1) * V::WT, wk = (wid & 1u) * V::WT;

  // fragment addresses: 16 lanes read 4 rows x 16 columns
  uint32_t noff[F], koff[F];
  {
    const uint32_t s = lane & 15u, gr = lane >> 4;
    const uint32_t row = 8 * (gr >> 1) + (s >> 2);
#pragma unroll
    for (int i = 0; i < F; ++i) {
      const uint32_t col = 32 * i + 16 * (gr & 1) + 4 * (s & 3);
      noff[i] = row * V::PITCH + 16u * place<T>(row, (wn + col) / 8) + 8 * (s & 1);
      koff[i] = V::HALF + row * V::PITCH + 16u * place<T>(row, (wk + col) / 8) + 8 * (s & 1);
    }
  }

  uint32_t id = blockIdx.x;
  Unit tile = seek<V>(p, id);  // whose products run
  if (tile.e < 0) return;
  Unit next = {0, 0, -1, 0, 1};  // the one after it, once the row cursor has come to it
  Cursor rows, load, put;        // the stages whose row numbers are loaded, that are loaded, that are written
  rows.start(tile);
  load.start(tile);
  put.start(tile);
  int32_t left = put.left;
  uint32_t n0 = tile.n0;  // of the tile that is loaded

  Copy<V> c;
  c.init(tid);
  load_rows(p, rows, lane, c);
  aim(p, tile, load, true, c);
#pragma unroll
  for (int i = 0; i < V::DC; ++i) load_d(p, n0, i, c);
#pragma unroll
  for (int i = 0; i < V::XC; ++i) {
    load_x(i, c);
    load_sc(p, i, c);
  }
  // (a tile has at least 3 stages: no cursor leaves it here)
  rows.step(next);
  load_rows(p, rows, lane, c);
  load.step(next);
  aim(p, tile, load, false, c);
  copy_share<0>(p, n0, c);
  copy_share<1>(p, n0, c);
  copy_share<2>(p, n0, c);
  copy_share<3>(p, n0, c);
  if (put.rem < kStep) drop_rows(put.rem, c);
  int32_t put_rem = put.rem - kStep;  // rows of the stage that is written; none in stages beyond the rows
  --put.left;
  rows.step(next);
  load_rows(p, rows, lane, c);
  load.step(next);
  aim(p, tile, load, false, c);
  stage_barrier();
  Frags<F> f[2];
  read_frags<V::WT>(0, noff, koff, f[0]);
  c.flip();
  copy_share<3>(p, n0, c);

  for (;;) {  // tiles
    v16f acc[F][F];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < F; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
    // Windows of 16 rows.  While a window's products run, the next window's
    // fragments are read and a quarter of a later stage is written.  The
    // barrier comes before the last window, when its fragments are in
    // registers: behind it the stage is free to be overwritten and the next
    // one is complete.
    Decoded d;
    do {
      if (rows.left == 1) {  // the row cursor leaves its tile
        id += gridDim.x;
        next = seek<V>(p, id);
      }
      rows.step(next);
      load_rows(p, rows, lane, c);
      window<0>(p, n0, c, 1, noff, koff, f[0], f[1], acc, d);
      window<1>(p, n0, c, 2, noff, koff, f[1], f[0], acc, d);
      window<2>(p, n0, c, 3, noff, koff, f[0], f[1], acc, d);
      if (put_rem < kStep) drop_rows(put_rem, c);
      put_rem -= kStep;
      if (--put.left == 0) {
        put_rem = next.cnt;
        put.left = next.e >= 0 ? next.stages() : INT32_MAX;
      }
      const bool fresh = load.step(next);
      if (fresh) n0 = next.n0;
      aim(p, fresh ? next : tile, load, fresh, c);
      c.flip();  // the other buffer is read from here on, and this one written
#pragma unroll
      for (int i = 0; i < F; ++i) {
        noff[i] ^= 2 * V::HALF;
        koff[i] ^= 2 * V::HALF;
      }
      stage_barrier();
      window<3>(p, n0, c, 0, noff, koff, f[1], f[0], acc, d);
    } while (--left != 0);
    const bool inside = p.vec && !p.accumulate && (int64_t)tile.n0 + T <= p.N && (int64_t)tile.k0 + T <= p.K;
    const uint32_t scratch = 4 * V::HALF + wid * V::SCRATCH;
    if (p.f32) {
      if (inside) store_tile<DT_F32, true, V>(p, tile, wn, wk, lane, acc, scratch);
      else store_tile<DT_F32, false, V>(p, tile, wn, wk, lane, acc, scratch);
    } else {
      if (inside) store_tile<DT_BF16, true, V>(p, tile, wn, wk, lane, acc, scratch);
      else store_tile<DT_BF16, false, V>(p, tile, wn, wk, lane, acc, scratch);
    }
    if (next.e < 0) break;
    tile = next;
    left = tile.stages();
  }
}

template <class V>
hipError_t launch_v(const WgradArgs& a, hipStream_t s) {
  WgradParams p = {};
  p.dy = a.dy;
  p.ld_dy = a.ld_dy;
  p.R = a.R;
  p.N = a.N;
  p.codes = a.codes;
  p.scales = a.scales;
  p.x_rows = a.x_rows;
  p.K = a.K;
  p.row_index = a.row_index;
  p.offsets = a.offsets;
  p.groups = a.groups;
  p.dw = a.dw;
  p.ld_dw = a.ld_dw;
  p.tn = (uint32_t)((a.N + V::T - 1) / V::T);
  p.tk = (uint32_t)((a.K + V::T - 1) / V::T);
  p.f32 = a.dwdt == DT_F32;
  p.accumulate = a.accumulate;
  p.vec = (reinterpret_cast<uintptr_t>(a.dw) & 15u) == 0 && (a.ld_dw * (p.f32 ? 4 : 2)) % 16 == 0;
  const int64_t units = ((int64_t)p.tn * p.tk + 7) / 8 * 8 * a.groups;
  if (units > UINT32_MAX / 2) return hipErrorInvalidValue;
  p.units = (uint32_t)units;
  auto kern = k_wgrad<V>;
  // the dynamic LDS limit is raised once per device
  static std::atomic<uint64_t> attr_done{0};
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (!bit || !(attr_done.load(std::memory_order_acquire) & bit)) {
    e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, V::LDS);
    if (e != hipSuccess) return e;
    attr_done.fetch_or(bit, std::memory_order_acq_rel);
  }
  // as many workgroups as the 256 CUs hold at once
  const uint32_t most = V::WT == 128 ? 256 : 512;
  hipLaunchKernelGGL(kern, dim3(p.units < most ? p.units : most), dim3(256), V::LDS, s, p);
  return hipGetLastError();
}

template <int FMT, bool GATHER>
hipError_t launch_g(const WgradArgs& a, hipStream_t s) {
  if (a.N % 8 || a.ld_dy >= (1 << 24) || a.K % 128 || a.x_rows * a.K >= (int64_t)UINT32_MAX)
    return launch_v<Variant<FMT, 64, true, GATHER>>(a, s);
  // 256 x 256 tiles when they fill the CUs, else 128 x 128
  const int64_t big = ((a.N + 255) / 256) * ((a.K + 255) / 256) * a.groups;
  return big >= 256 ? launch_v<Variant<FMT, 128, false, GATHER>>(a, s)
                    : launch_v<Variant<FMT, 64, false, GATHER>>(a, s);
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
