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

// What one thread copies of a stage: DC chunks of 8 dY columns and XC chunks
// of 16 codes, and which stage row and column they are.
template <int FMT, int WT, bool GATHER>
struct Copy {
  static constexpr int T = 2 * WT;               // tile edge
  static constexpr int DC = kStep * T / 8 / 256;  // dY chunks
  static constexpr int XC = kStep * T / 16 / 256; // code chunks
  static constexpr int PITCH = 2 * T;            // bytes of a stage row
  static constexpr int HALF = kStep * PITCH;     // bytes of an operand's stage

  static constexpr int DR = 256 / (T / 8);       // rows between a thread's dY chunks
  static constexpr int XR = 256 / (T / 16);      // and between its code chunks

  u4 d[DC], x[XC];
  // scale codes: the aligned word that holds one (K a multiple of 128), whose
  // load needs no widening, or the byte
  static constexpr bool WORDS = WT == 128;
  uint32_t sc[XC];
  int32_t src[XC];  // rows of X the next loads take
  // LDS offsets of chunk 0 in the buffer that is written (the other chunks
  // are whole rows below, for dY of 256-wide tiles with bit 1 of the chunk
  // number exchanged in turn), and the thread's columns
  uint32_t dput, xput, dcol, xcol, sc_shift;

  __device__ __forceinline__ void init(uint32_t tid) {
    dcol = tid % (T / 8) * 8;
    xcol = tid % (T / 16) * 16;
    sc_shift = WORDS ? xcol / 32 % 4 * 8 : 0;
    const uint32_t dr = tid / (T / 8), xr = tid / (T / 16);
    dput = dr * PITCH + 16u * place<T>(dr, dcol / 8);
    xput = HALF + xr * PITCH + 16u * place<T>(xr, xcol / 8);
  }
  __device__ __forceinline__ void flip() {  // to the other buffer
    dput ^= 2 * HALF;
    xput ^= 2 * HALF;
  }
  __device__ __forceinline__ uint32_t dput_of(int i) const {
    return (DR == 8 && (i & 1) ? dput ^ 32u : dput) + (uint32_t)(i * DR * PITCH);
  }
};

// One stage of the workgroup's work (the same in all its lanes).
struct Stage {
  int32_t row;      // its first row
  int32_t rem;      // rows of the group from there on, at least 1
  uint32_t n0, k0;  // the tile
  int32_t e;        // the group; -1 past the last tile
};

// Rows past the group repeat its last one; drop_rows() clears them in LDS.
template <int FMT, int WT, bool GATHER>
__device__ __forceinline__ void load_src(const WgradParams& p, const Stage& s, uint32_t tid, int i,
                                         Copy<FMT, WT, GATHER>& c) {
  typedef Copy<FMT, WT, GATHER> C;
  const int32_t r = min((int32_t)(tid / (C::T / 16)) + i * C::XR, s.rem - 1);
  if constexpr (GATHER)
    c.src[i] = *reinterpret_cast<const int32_t*>(reinterpret_cast<const char*>(p.row_index + s.row) + 4u * (uint32_t)r);
  else c.src[i] = s.row + r;
}

// What a thread's loads of a stage have in common.
struct Aim {
  const char* base;     // dY at the stage's first row and the tile's first column (uniform)
  uint32_t doff, dlim;  // byte offset of chunk 0, and of the last row of the group
  int32_t row0, rem;    // the thread's first row, rows of the group
  uint32_t cols;        // columns of the thread's dY chunk that exist
  const uint8_t* codes;  // X: row 0 at the thread's columns
  const uint8_t* scales;
};
template <int FMT, int WT, bool GATHER>
__device__ __forceinline__ Aim aim(const WgradParams& p, const Stage& s, uint32_t tid,
                                   const Copy<FMT, WT, GATHER>& c) {
  typedef Copy<FMT, WT, GATHER> C;
  // 64 rows of a pitch below 2^24 elements: 32-bit offsets
  const uint32_t pitch = 2u * (uint32_t)p.ld_dy;
  // columns past N and K are computed from others and not stored
  const uint32_t cc = s.n0 + c.dcol < (uint32_t)p.N ? 2u * c.dcol : 0u;
  const uint32_t kk = s.k0 + c.xcol < (uint32_t)p.K ? c.xcol : 0u;
  Aim a;
  a.base = reinterpret_cast<const char*>(p.dy + (int64_t)s.row * p.ld_dy + s.n0);
  a.doff = tid / (C::T / 8) * pitch + cc;
  a.dlim = (uint32_t)min(s.rem - 1, kStep) * pitch + cc;
  a.row0 = (int32_t)(tid / (C::T / 8));
  a.rem = s.rem;
  a.cols = (uint32_t)p.N - s.n0 - c.dcol;
  a.codes = p.codes + s.k0 + kk;
  a.scales = p.scales + s.k0 / 32 + (C::WORDS ? kk / 128 * 4 : kk / 32);
  return a;
}

template <bool ODD, int FMT, int WT, bool GATHER>
__device__ __forceinline__ void load_d(const WgradParams& p, const Aim& a, int i, Copy<FMT, WT, GATHER>& c) {
  typedef Copy<FMT, WT, GATHER> C;
  const uint32_t off = min(a.doff + (uint32_t)(i * C::DR) * (2u * (uint32_t)p.ld_dy), a.dlim);
  if constexpr (ODD) {  // rows may end inside a chunk, or have a large pitch
    const int64_t row = min((int64_t)a.row0 + i * C::DR, (int64_t)a.rem - 1);
    const uint16_t* at = reinterpret_cast<const uint16_t*>(a.base) + row * p.ld_dy + c.dcol;
    uint32_t w[4] = {};
#pragma unroll
    for (uint32_t e = 0; e < 8; ++e)
      if ((int32_t)a.cols > (int32_t)e) w[e >> 1] |= (uint32_t)at[e] << (16 * (e & 1));
    c.d[i] = u4{w[0], w[1], w[2], w[3]};
  } else {
    c.d[i] = *reinterpret_cast<const u4*>(a.base + off);
  }
}

template <int FMT, int WT, bool GATHER>
__device__ __forceinline__ void load_x(const WgradParams& p, const Aim& a, int i, Copy<FMT, WT, GATHER>& c) {
  const uint32_t src = (uint32_t)min(max(c.src[i], 0), (int32_t)p.x_rows - 1);
  c.x[i] = *reinterpret_cast<const u4*>(a.codes + (uint64_t)src * (uint32_t)p.K);
  const uint8_t* sc = a.scales + (uint64_t)src * (uint32_t)(p.K / 32);
  if constexpr (Copy<FMT, WT, GATHER>::WORDS) c.sc[i] = *reinterpret_cast<const uint32_t*>(sc);
  else c.sc[i] = *sc;
}

// the thread's dY chunk i into LDS
template <int FMT, int WT, bool GATHER>
__device__ __forceinline__ void put_d(int i, const Copy<FMT, WT, GATHER>& c) {
  *(lds_u4)c.dput_of(i) = c.d[i];
}

// The thread's code chunk i on its way: scale, then pair by pair, then into
// LDS by halves.
template <int FMT>
struct Decoded {
  Scale8 s;
  uint32_t o[8];
};
template <int FMT, int WT, bool GATHER>
__device__ __forceinline__ void decode_scale(int i, const Copy<FMT, WT, GATHER>& c, Decoded<FMT>& d) {
  typedef Copy<FMT, WT, GATHER> C;
  d.s = scale8<FMT>(C::WORDS ? (c.sc[i] >> c.sc_shift) & 0xFFu : c.sc[i]);
}
template <int P, int FMT, int WT, bool GATHER>
__device__ __forceinline__ void decode_pair(int i, const Copy<FMT, WT, GATHER>& c, Decoded<FMT>& d) {
  d.o[P] = decode2_bf16<FMT, P & 1>(c.x[i][P / 2], d.s);
}
template <int H, int FMT, int WT, bool GATHER>
__device__ __forceinline__ void put_x(int i, const Copy<FMT, WT, GATHER>& c, const Decoded<FMT>& d) {
  typedef Copy<FMT, WT, GATHER> C;
  *(lds_u4)((c.xput ^ (16u * H)) + i * C::XR * C::PITCH) = u4{d.o[4 * H], d.o[4 * H + 1], d.o[4 * H + 2], d.o[4 * H + 3]};
}
template <int FMT, int WT, bool GATHER>
__device__ __forceinline__ void put_x(int i, const Copy<FMT, WT, GATHER>& c) {
  Decoded<FMT> d;
  decode_scale(i, c, d);
  decode_pair<0>(i, c, d);
  decode_pair<1>(i, c, d);
  decode_pair<2>(i, c, d);
  decode_pair<3>(i, c, d);
  decode_pair<4>(i, c, d);
  decode_pair<5>(i, c, d);
  decode_pair<6>(i, c, d);
  decode_pair<7>(i, c, d);
  put_x<0>(i, c, d);
  put_x<1>(i, c, d);
}

// Clears the rows from `rem` on of the stage that was just written, in both
// operands (a row that is not of the group may hold NaN).  Each thread clears
// what it wrote itself, and a wave's LDS accesses keep their order, so no
// barrier is needed between.
template <int FMT, int WT, bool GATHER>
__device__ __forceinline__ void drop_rows(int32_t rem, uint32_t tid, const Copy<FMT, WT, GATHER>& c) {
  typedef Copy<FMT, WT, GATHER> C;
  const u4 z = u4{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < C::DC; ++i)
    if ((int32_t)(tid / (C::T / 8)) + i * C::DR >= rem) *(lds_u4)c.dput_of(i) = z;
#pragma unroll
  for (int i = 0; i < C::XC; ++i)
    if ((int32_t)(tid / (C::T / 16)) + i * C::XR >= rem) {
      const uint32_t at = i * C::XR * C::PITCH;
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
// the same share of the stage after it, and of the row numbers of the one
// after that.
template <int W, bool ODD, int FMT, int WT, bool GATHER>
__device__ __forceinline__ void copy_share(const WgradParams& p, const Aim& load, const Stage& src, uint32_t tid,
                                           Copy<FMT, WT, GATHER>& c) {
  typedef Copy<FMT, WT, GATHER> C;
#pragma unroll
  for (int i = W * C::DC / 4; i < (W + 1) * C::DC / 4; ++i) {
    put_d(i, c);
    load_d<ODD>(p, load, i, c);
  }
#pragma unroll
  for (int i = W * C::XC / 4; i < (W + 1) * C::XC / 4; ++i) {
    put_x(i, c);
    load_x(p, load, i, c);
    load_src(p, src, tid, i, c);
  }
}

// One window of 16 rows: the products of `f`, and between them the reads of
// the next window's fragments (rows 16 q of the buffer at noff / koff) and the
// share W of the copies.  With one wave on a SIMD the order is the schedule:
// each product (32 cycles of the matrix unit) is followed by what fits beside
// it, and nothing moves over it.
template <int W, bool ODD, int FMT, int WT, bool GATHER, int M = 0>
__device__ __forceinline__ void window(const WgradParams& p, const Aim& load, const Stage& src, uint32_t tid,
                                       Copy<FMT, WT, GATHER>& c, int q, const uint32_t (&noff)[WT / 32],
                                       const uint32_t (&koff)[WT / 32], const Frags<WT / 32>& f, Frags<WT / 32>& next,
                                       v16f (&acc)[WT / 32][WT / 32], Decoded<FMT>& d) {
  typedef Copy<FMT, WT, GATHER> C;
  constexpr int F = WT / 32;
  if constexpr (F == 2) {  // two waves on a SIMD: they fill each other's gaps
    read_frags<WT>(q, noff, koff, next);
    copy_share<W, ODD>(p, load, src, tid, c);
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < F; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.k[i], f.n[j], acc[i][j], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  } else if constexpr (M < F * F) {
    static_assert(C::DC == 8 && C::XC == 4, "shares of two dY chunks and one code chunk");
    acc[M / F][M % F] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.k[M / F], f.n[M % F], acc[M / F][M % F], 0, 0, 0);
    read_nth<M, WT>(q, noff, koff, next);
    if constexpr (M == 0) decode_scale(W, c, d);
    if constexpr (M >= 1 && M <= 8) decode_pair<(M - 1) & 7>(W, c, d);
    if constexpr (M == 5) put_x<0>(W, c, d);
    if constexpr (M == 9) put_x<1>(W, c, d);
    if constexpr (M == 10) put_d(2 * W, c);
    if constexpr (M == 11) put_d(2 * W + 1, c);
    if constexpr (M == 12) load_x(p, load, W, c);
    if constexpr (M == 13) load_d<ODD>(p, load, 2 * W, c);
    if constexpr (M == 14) load_d<ODD>(p, load, 2 * W + 1, c);
    if constexpr (M == 15) load_src(p, src, tid, W, c);
    __builtin_amdgcn_sched_barrier(0);
    window<W, ODD, FMT, WT, GATHER, M + 1>(p, load, src, tid, c, q, noff, koff, f, next, acc, d);
  }
}

// 8 columns of a row of dW
template <int WDT>
__device__ __forceinline__ void put_row(const WgradParams& p, int64_t off, float (&o)[8]) {
  if (p.accumulate) {
    float old[8];
    load_n<WDT>(p.dw, off, 8, p.vec, old);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] += old[e];
  }
  store_n<WDT>(p.dw, off, 8, p.vec, o);
}

// A wave's tile of products, 32 columns of N at a time and PC of K, through
// 4 x 32 x PC bytes of LDS of its own into rows of dW (or, past an edge or
// unaligned, element by element).  Chunk c of 4 columns of row r lies at chunk
// c ^ (r mod chunks): writes of 16 rows and reads of one row are free of
// conflicts.
template <int WT>
__device__ __forceinline__ void store_tile_rows(const WgradParams& p, const Stage& s, uint32_t wn, uint32_t wk, uint32_t lane,
                                       const v16f (&acc)[WT / 32][WT / 32], uint8_t* scratch) {
  constexpr int PC = WT / 2;       // columns of a pass
  constexpr int CH = PC / 4;       // 16-byte chunks of a scratch row
  constexpr int RPI = 64 / (CH / 2);  // rows read at once, 8 columns a lane
  // (opaque, so that the addresses below are not kept over the main loop)
  asm volatile("" : "+v"(lane));
  const uint32_t lr = lane & 31u, lg = lane >> 5;
  const uint32_t rr = lane / (CH / 2), cc = lane % (CH / 2) * 2;
#pragma unroll
  for (int j = 0; j < WT / 32; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i2 = 0; i2 < PC / 32; ++i2)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const v16f& a = acc[h * (PC / 32) + i2][j];
          const uint32_t ch = 8 * i2 + 2 * v + lg;
          *reinterpret_cast<f4*>(scratch + lr * (PC * 4) + 16u * (ch ^ (lr & (CH - 1)))) =
              f4{a[4 * v], a[4 * v + 1], a[4 * v + 2], a[4 * v + 3]};
        }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int t = 0; t < 32 / RPI; ++t) {
        const uint32_t r = t * RPI + rr;
        const f4 lo = *reinterpret_cast<const f4*>(scratch + r * (PC * 4) + 16u * (cc ^ (r & (CH - 1))));
        const f4 hi = *reinterpret_cast<const f4*>(scratch + r * (PC * 4) + 16u * ((cc + 1) ^ (r & (CH - 1))));
        const int64_t n = (int64_t)s.n0 + wn + 32 * j + r, k = (int64_t)s.k0 + wk + PC * h + 4 * cc;
        if (n < p.N && k < p.K) {  // (K is a multiple of 32: a chunk is inside or outside)
          const int64_t off = ((int64_t)s.e * p.N + n) * p.ld_dw + k;
          float o[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
          if (p.f32) put_row<DT_F32>(p, off, o);
          else put_row<DT_BF16>(p, off, o);
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
}

// The workgroup's tiles, as a sequence of stages.  Units id, id + gridDim.x,
// ...: the tiles of a group are dealt to the 8 XCDs (workgroup id mod 8) in
// runs, n fastest, so that the workgroups of an XCD share rows of dY and X in
// its L2.  A group without rows is passed over; its tiles of dW are cleared on
// the way.
template <int T>
__device__ __forceinline__ void clear_tile(const WgradParams& p, uint32_t e, uint32_t n0, uint32_t k0) {
  for (uint32_t q = threadIdx.x; q < T * T; q += 256) {
    const int64_t n = (int64_t)n0 + q / T, k = (int64_t)k0 + q % T;
    if (n < p.N && k < p.K) {
      const int64_t off = (e * p.N + n) * p.ld_dw + k;
      if (p.f32) static_cast<float*>(p.dw)[off] = 0.0f;
      else static_cast<uint16_t*>(p.dw)[off] = 0;
    }
  }
}
// the first stage of unit `id` or of the next one that has rows; if there is
// none, s stays (what is still copied of it is never used) with e = -1
template <int T>
__device__ __forceinline__ void seek(const WgradParams& p, uint32_t& id, Stage& s) {
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
    const uint32_t tk = in / p.tn, n0 = (in - tk * p.tn) * T, k0 = tk * T;
    if (hi > lo) {
      s = {(int32_t)lo, (int32_t)(hi - lo), n0, k0, (int32_t)e};
      return;
    }
    if (!p.accumulate) clear_tile<T>(p, e, n0, k0);
  }
  s.e = -1;
}
template <int T>
__device__ __forceinline__ void advance(const WgradParams& p, uint32_t& id, Stage& s) {
  if (s.rem > kStep) {
    s.row += kStep;
    s.rem -= kStep;
  } else if (s.e >= 0) {
    id += gridDim.x;
    seek<T>(p, id, s);
  }
}

// Stages flow through the pipeline without a break between tiles: while a
// tile's last products run, the next tile's first stages are being copied.
template <int FMT, int WT, bool ODD, bool GATHER>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(WT == 128 ? 1 : 2, WT == 128 ? 1 : 2))) void
k_wgrad(WgradParams p) {
  typedef Copy<FMT, WT, GATHER> C;
  constexpr int F = WT / 32, T = C::T;
  // The workgroup's LDS is addressed by plain offsets from its start (there is
  // no static allocation), so that changing buffers is one exclusive or.
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t wn = (wid >> 1) * WT, wk = (wid & 1u) * WT;
  uint8_t* scratch = smem + 4 * C::HALF + wid * (64 * WT);

  // fragment addresses: 16 lanes read 4 rows x 16 columns
  uint32_t noff[F], koff[F];
  {
    const uint32_t s = lane & 15u, gr = lane >> 4;
    const uint32_t row = 8 * (gr >> 1) + (s >> 2);
#pragma unroll
    for (int i = 0; i < F; ++i) {
      const uint32_t col = 32 * i + 16 * (gr & 1) + 4 * (s & 3);
      noff[i] = row * C::PITCH + 16u * place<T>(row, (wn + col) / 8) + 8 * (s & 1);
      koff[i] = C::HALF + row * C::PITCH + 16u * place<T>(row, (wk + col) / 8) + 8 * (s & 1);
    }
  }

  uint32_t id = blockIdx.x;
  Stage s0 = {0, 0, 0, 0, 0};  // the stage being multiplied; s1 .. s4 follow it
  seek<T>(p, id, s0);
  if (s0.e < 0) return;
  Stage s1 = s0;
  advance<T>(p, id, s1);
  Stage s2 = s1;
  advance<T>(p, id, s2);
  Stage s3 = s2;
  advance<T>(p, id, s3);
  Stage s4 = s3;
  advance<T>(p, id, s4);

  C c;
  c.init(tid);
#pragma unroll
  for (int i = 0; i < C::XC; ++i) load_src(p, s0, tid, i, c);
  {
    const Aim a0 = aim(p, s0, tid, c), a1 = aim(p, s1, tid, c);
#pragma unroll
    for (int i = 0; i < C::DC; ++i) load_d<ODD>(p, a0, i, c);
#pragma unroll
    for (int i = 0; i < C::XC; ++i) load_x(p, a0, i, c);
#pragma unroll
    for (int i = 0; i < C::XC; ++i) load_src(p, s1, tid, i, c);
    copy_share<0, ODD>(p, a1, s2, tid, c);
    copy_share<1, ODD>(p, a1, s2, tid, c);
    copy_share<2, ODD>(p, a1, s2, tid, c);
    copy_share<3, ODD>(p, a1, s2, tid, c);
  }
  if (s0.rem < kStep) drop_rows(s0.rem, tid, c);
  stage_barrier();
  Frags<F> f[2];
  read_frags<WT>(0, noff, koff, f[0]);
  c.flip();
  Aim a = aim(p, s2, tid, c);  // of the stage after the one that is written
  copy_share<3, ODD>(p, a, s3, tid, c);

  for (;;) {  // tiles
    v16f acc[F][F];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < F; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
    const Stage tile = s0;
    bool last, end;
    // Windows of 16 rows.  While a window's products run, the next window's
    // fragments are read and a quarter of a later stage is written.  The barrier
    // comes before the last window, when its fragments are in registers: behind
    // it the stage is free to be overwritten and the next one is complete.
    Decoded<FMT> d;
    do {
      window<0, ODD>(p, a, s3, tid, c, 1, noff, koff, f[0], f[1], acc, d);
      window<1, ODD>(p, a, s3, tid, c, 2, noff, koff, f[1], f[0], acc, d);
      window<2, ODD>(p, a, s3, tid, c, 3, noff, koff, f[0], f[1], acc, d);
      if (s1.rem < kStep) drop_rows(s1.rem, tid, c);
      // the other buffer is read from here on, and this one written
      a = aim(p, s3, tid, c);
      c.flip();
#pragma unroll
      for (int i = 0; i < F; ++i) {
        noff[i] ^= 2 * C::HALF;
        koff[i] ^= 2 * C::HALF;
      }
      stage_barrier();
      window<3, ODD>(p, a, s4, tid, c, 0, noff, koff, f[1], f[0], acc, d);
      last = s0.rem <= kStep;
      end = s1.e < 0;
      s0 = s1;
      s1 = s2;
      s2 = s3;
      s3 = s4;
      advance<T>(p, id, s4);
    } while (!last);
    store_tile_rows<WT>(p, tile, wn, wk, lane, acc, scratch);
    if (end) break;
  }
}

template <int FMT, int WT, bool ODD, bool GATHER>
hipError_t launch_t(const WgradArgs& a, hipStream_t s) {
  typedef Copy<FMT, WT, GATHER> C;
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
  p.tn = (uint32_t)((a.N + C::T - 1) / C::T);
  p.tk = (uint32_t)((a.K + C::T - 1) / C::T);
  p.f32 = a.dwdt == DT_F32;
  p.accumulate = a.accumulate;
  p.vec = (reinterpret_cast<uintptr_t>(a.dw) & 15u) == 0 && (a.ld_dw * (p.f32 ? 4 : 2)) % 16 == 0;
  const int64_t units = ((int64_t)p.tn * p.tk + 7) / 8 * 8 * a.groups;
  if (units > UINT32_MAX / 2) return hipErrorInvalidValue;
  p.units = (uint32_t)units;
  constexpr int smem = 4 * C::HALF + 4 * 64 * WT;  // two stages, and 64 WT bytes of scratch a wave
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
  // as many workgroups as the 256 CUs hold at once
  const uint32_t most = WT == 128 ? 256 : 512;
  hipLaunchKernelGGL(kern, dim3(p.units < most ? p.units : most), dim3(256), smem, s, p);
  return hipGetLastError();
}

template <int FMT, bool GATHER>
hipError_t launch_g(const WgradArgs& a, hipStream_t s) {
  // dY rows that end inside a 16-byte chunk (or of a pitch past 32-bit
  // offsets) are loaded element by element
  if (a.N % 8 || a.ld_dy >= (1 << 24)) return launch_t<FMT, 64, true, GATHER>(a, s);
  // 256 x 256 tiles when they fill the CUs, else 128 x 128
  const int64_t big = ((a.N + 255) / 256) * ((a.K + 255) / 256) * a.groups;
  return big >= 256 && a.K % 128 == 0 ? launch_t<FMT, 128, false, GATHER>(a, s) : launch_t<FMT, 64, false, GATHER>(a, s);
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
