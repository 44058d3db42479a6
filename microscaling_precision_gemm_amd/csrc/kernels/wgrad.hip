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
//
// Bounds.  The matrix unit, where groups are long: 256 x 256 tiles, a wave of
// 128 x 128 to each SIMD with all of its products in accumulators, every other
// instruction placed behind a product, run at the power-limited rate of the
// BF16 instruction on random data (each further 65536 rows x 2048 x 7168 in 32
// even groups: 1585 us, 1214 TFLOP/s).  What a tile costs besides is its store: with one wave a
// SIMD nothing runs beside it, and 256 tiles of 256 KB leave at the rate of
// HBM.  32768 rows in 32 uneven groups x 2048 x 7168 E4M3, gathered: 1075 us
// (895 TFLOP/s; 1.88 GB of FP32 output, 3.4 GB past the L2s in).  Spreading the
// workgroups' phases by waits of 2 .. 36 us did not pay (1200 .. 1230 us
// against 1217 with even groups).  Short groups are bound by latency: a tile's
// first loads, three stages and its store are 8 us.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "../device/decode8.h"
#include "../device/gemm_common.h"
#include "../launch_moe.h"

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
  uint32_t last_word;  // offset of the last 4 scale codes
  const int32_t* row_index;
  const int64_t* offsets;  // nullptr: one group of all rows
  int32_t groups;
  void* dw;
  int64_t ld_dw;
  uint32_t tn, tk;  // tiles along N and K
  uint32_t units;   // tiles of all groups, rounded up for the deal to the XCDs
  // rows of a part of a group, a multiple of kStep; 0: groups are not split.
  // Products of parts go to `parts`, a tile after the other, unless a group is
  // one part; there is place for `slots` tiles.
  int32_t len;
  uint32_t slots;
  float* parts;
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

enum Kind { ANY_SHAPE, PLAIN_SHAPE, WHOLE_WORDS };

// The variants.  WT: columns of a wave's tile (a workgroup's is T = 2 WT
// square).  ANY_SHAPE: any N, K, pitch and size of X, otherwise dY in whole 16-byte
// chunks, at least 4 scale codes and offsets within 32 bits; WHOLE_WORDS: and
// K a multiple of 128, so that the scale codes of a row of X are aligned words.  GATHER: X's rows by the row index.
template <int FMT_, int WT_, int KIND, bool GATHER_>
struct Variant {
  static constexpr int FMT = FMT_, WT = WT_;
  static constexpr bool ANY = KIND == ANY_SHAPE, WORDS = KIND == WHOLE_WORDS, GATHER = GATHER_;
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

// a / b rounded up, for 0 <= a and 0 < b (their sum may pass 31 bits)
__device__ __forceinline__ int32_t parts_of(int32_t a, int32_t b) {
  return (int32_t)(((uint32_t)a + (uint32_t)b - 1u) / (uint32_t)b);
}

// One tile and its rows (the same in all lanes).
struct Unit {
  uint32_t n0, k0;
  int32_t e;         // group; -1: there is none
  int32_t row, cnt;  // its rows, at least one
  int32_t slot;      // where its products go in p.parts; -1: to dW
  // Stages: at least 3, so that the copies, which run ahead of the products,
  // never reach past the tile after this one.
  __device__ __forceinline__ int32_t stages() const { return max(parts_of(cnt, kStep), 3); }
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

// The rows of group e, clamped into [0, R].
__device__ __forceinline__ void group_rows(const WgradParams& p, uint32_t e, int32_t& row, int32_t& cnt) {
  int64_t lo = 0, hi = p.R;
  if (p.offsets) {
    lo = p.offsets[e];
    hi = p.offsets[e + 1];
    lo = lo < 0 ? 0 : (lo > p.R ? p.R : lo);
    hi = hi < lo ? lo : (hi > p.R ? p.R : hi);
  }
  row = (int32_t)lo;
  cnt = (int32_t)(hi - lo);
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
    int32_t row, cnt;
    group_rows(p, e, row, cnt);
    const uint32_t tk = in / p.tn, n0 = (in - tk * p.tn) * V::T, k0 = tk * V::T;
    if (cnt > 0) return {n0, k0, (int32_t)e, row, cnt, -1};
    if (!p.accumulate) clear_tile<V>(p, e, n0, k0);
  }
  return {0, 0, -1, 0, 1, -1};
}

// Parts of the groups g0 .. g0 + 63, a lane each, summed over the lanes up to
// this one.
__device__ __forceinline__ int32_t parts_scan(const WgradParams& p, int32_t g0, uint32_t lane, int32_t& n) {
  int32_t row, cnt = 0;
  if (g0 + (int32_t)lane < p.groups) group_rows(p, g0 + lane, row, cnt);
  n = parts_of(cnt, p.len);
  int32_t sum = n;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int32_t o = __shfl_up(sum, d);
    if ((int)lane >= d) sum += o;
  }
  return sum;
}

// Parts of all groups; 0 when they are not split.  (Offsets that break their
// contract may give groups that share rows, and more parts than there is place
// for: then no group is split.)
__device__ __forceinline__ int32_t parts_of_all(const WgradParams& p, uint32_t lane) {
  int32_t total = 0, n;
  for (int32_t g0 = 0; g0 < p.groups; g0 += 64) total += __builtin_amdgcn_readlane(parts_scan(p, g0, lane, n), 63);
  return (uint32_t)total * p.tn * p.tk <= p.slots ? total : 0;
}

// Group of part `part`, and that part's number within the group, of `of`.
__device__ __forceinline__ int32_t group_of(const WgradParams& p, uint32_t lane, int32_t& part, int32_t& of) {
  for (int32_t g0 = 0;; g0 += 64) {
    int32_t n;
    const int32_t sum = parts_scan(p, g0, lane, n);
    const uint64_t past = __ballot(sum > part);
    if (past) {
      const int l = __builtin_ctzll(past);
      of = __builtin_amdgcn_readlane(n, l);
      part -= __builtin_amdgcn_readlane(sum, l) - of;
      return g0 + l;
    }
    part -= __builtin_amdgcn_readlane(sum, 63);
  }
}

// The only unit of workgroup `id` when groups are split into `total` parts:
// part by part, each part's tiles next to one another and on one XCD as above.
template <class V>
__device__ __forceinline__ Unit seek_part(const WgradParams& p, uint32_t id, uint32_t lane, int32_t total) {
  const uint32_t tiles = p.tn * p.tk, units = (uint32_t)total * tiles, per = (units + 7) / 8;
  const uint32_t slot = (id & 7u) * per + (id >> 3);
  if ((id >> 3) >= per || slot >= units) return {0, 0, -1, 0, 1, -1};
  int32_t part = (int32_t)(slot / tiles), of, row, cnt;
  const uint32_t in = slot - (uint32_t)part * tiles, tk = in / p.tn;
  const int32_t e = group_of(p, lane, part, of);
  group_rows(p, e, row, cnt);
  return {(in - tk * p.tn) * V::T, tk * V::T, e, row + part * p.len, min(cnt - part * p.len, p.len),
          of > 1 ? (int32_t)slot : -1};
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
  uint32_t sc[V::XC], sh[V::XC];
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
    sc_shift = xcol / 32 % 4 * 8;
    xput = V::HALF + xrow * V::PITCH + 16u * place<V::T>(xrow, xcol / 16 * 2);
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

// Aims the loads at the stage at `at` of a tile at columns n0, k0.  `fresh`: the tile, or the
// number of rows, is another than before; the lane offsets of full stages of
// one tile are the same.
template <class V>
__device__ __forceinline__ void aim(const WgradParams& p, uint32_t n0, uint32_t k0, const Cursor& at, bool fresh,
                                    Copy<V>& c) {
  c.dbase = reinterpret_cast<const char*>(p.dy + (int64_t)at.row * p.ld_dy + n0);
  if (fresh || at.rem < kStep) {
    // columns past N and K are computed from others and not stored
    const uint32_t cc = n0 + c.dcol < (uint32_t)p.N ? 2u * c.dcol : 0u;
    c.kk = k0 + c.xcol < (uint32_t)p.K ? c.xcol : 0u;
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
    c.xbase = p.codes + k0;
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
    c.xbase = p.codes + (int64_t)at.row * p.K + k0;
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
// Scale codes: one for 32 codes, so at 1/32 of the code offset from the start.
// The word from there on is loaded (as bytes the compiler would wait for them
// at once), or the last word of the scales and the code is shifted down.
template <class V>
__device__ __forceinline__ void load_sc(const WgradParams& p, int i, Copy<V>& c) {
  if constexpr (V::ANY) c.sc[i] = p.scales[((uint64_t)(c.xbase - p.codes) + c.xoff[i]) / 32];
  else if constexpr (V::WORDS) {
    c.sc[i] = *reinterpret_cast<const uint32_t*>(p.scales + (((uint32_t)(c.xbase - p.codes) + c.xoff[i]) / 32 & ~3u));
  } else {
    typedef uint32_t __attribute__((aligned(1))) word;
    const uint32_t o = (uint32_t)(c.xbase - p.codes) / 32 + c.xoff[i] / 32, in = min(o, p.last_word);
    c.sc[i] = *reinterpret_cast<const word*>(p.scales + in);
    c.sh[i] = (o - in) * 8;
  }
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
  else d.x = scale8_word<V::FMT>(c.sc[i], V::WORDS ? c.sc_shift : c.sh[i]);
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
// 128 PC bytes of LDS of its own into rows at dst.  Chunk c of 4 columns of row
// r lies at chunk c ^ (r mod chunks): writes of 16 rows and reads of one row
// are free of conflicts.  PLAIN: all of the tile is stored, its rows are
// 16-byte aligned, and it is not added to; otherwise chunk by chunk with checks.
template <int WDT, bool PLAIN, class V>
__device__ __forceinline__ void store_tile(const WgradParams& p, const Unit& u, void* dst, int64_t ld, uint32_t wn,
                                           uint32_t wk, uint32_t lane, const v16f (&acc)[V::F][V::F],
                                           uint32_t scratch) {
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
  uint8_t* base = static_cast<uint8_t*>(dst) + ((int64_t)wn * ld + wk) * EB;  // uniform
  const int64_t loff = ((int64_t)rr * ld + 4 * cc) * EB;
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
        uint8_t* at = base + ((int64_t)(32 * j + t * RPI) * ld + PC * h) * EB + loff;
        if constexpr (PLAIN) {
          // streaming stores: the rows of dY and X stay in the L2
          if constexpr (WDT == DT_F32) __builtin_nontemporal_store(f4{o[0], o[1], o[2], o[3]}, reinterpret_cast<f4*>(at));
          else __builtin_nontemporal_store(u4{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]),
                                              pack_bf16(o[6], o[7])}, reinterpret_cast<u4*>(at));
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
  Unit tile;  // whose products run
  const int32_t parts = p.len ? parts_of_all(p, lane) : 0;
  if (parts) {
    tile = seek_part<V>(p, id, lane, parts);
    id = p.units;  // there is no other
  } else {
    tile = seek<V>(p, id);
  }
  if (tile.e < 0) return;
  Unit next = {0, 0, -1, 0, 1, -1};  // the one after it, once the row cursor has come to it
  Cursor rows, load, put;        // the stages whose row numbers are loaded, that are loaded, that are written
  rows.start(tile);
  load.start(tile);
  put.start(tile);
  int32_t left = put.left;
  uint32_t n0 = tile.n0, k0 = tile.k0;  // of the tile that is loaded

  Copy<V> c;
  c.init(tid);
  load_rows(p, rows, lane, c);
  aim(p, n0, k0, load, true, c);
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
  aim(p, n0, k0, load, false, c);
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
  aim(p, n0, k0, load, false, c);
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
      if (fresh) {
        n0 = next.n0;
        k0 = next.k0;
      }
      aim(p, n0, k0, load, fresh, c);
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
    int64_t ld = p.ld_dw;
    void* dst = static_cast<uint8_t*>(p.dw) + (((int64_t)tile.e * p.N + tile.n0) * ld + tile.k0) * (p.f32 ? 4 : 2);
    if (tile.slot >= 0) {
      ld = T;
      dst = p.parts + (int64_t)tile.slot * (T * T);
    }
    if (p.f32 || tile.slot >= 0) {
      if (inside || tile.slot >= 0) store_tile<DT_F32, true, V>(p, tile, dst, ld, wn, wk, lane, acc, scratch);
      else store_tile<DT_F32, false, V>(p, tile, dst, ld, wn, wk, lane, acc, scratch);
    } else {
      if (inside) store_tile<DT_BF16, true, V>(p, tile, dst, ld, wn, wk, lane, acc, scratch);
      else store_tile<DT_BF16, false, V>(p, tile, dst, ld, wn, wk, lane, acc, scratch);
    }
    if (next.e < 0) break;
    tile = next;
    left = tile.stages();
  }
}

// dW of the groups that were split, and of those without rows: the products of
// a group's parts are added in their order.  A workgroup does 1024 elements of
// a tile of T x T, a thread 4 of a row.
__global__ __launch_bounds__(256) void k_wgrad_join(WgradParams p, uint32_t T) {
  const uint32_t lane = threadIdx.x & 63u, pieces = T * T / 1024, tiles = p.tn * p.tk;
  const uint32_t at = blockIdx.x / pieces, e = at / tiles, in = at - e * tiles;
  if (!parts_of_all(p, lane)) return;
  int32_t first = 0, n = 0;
  for (int32_t g0 = 0;; g0 += 64) {
    const int32_t sum = parts_scan(p, g0, lane, n);
    const int l = (int)min(e - g0, 63u);
    first += __builtin_amdgcn_readlane(sum, l);
    if (e < g0 + 64u) {
      n = __builtin_amdgcn_readlane(n, l);
      first -= n;
      break;
    }
  }
  if (n == 1 || (n == 0 && p.accumulate)) return;
  const uint32_t q = ((blockIdx.x - at * pieces) * 256 + threadIdx.x) * 4;  // in the tile
  const int64_t row = (int64_t)(in % p.tn) * T + q / T, col = (int64_t)(in / p.tn) * T + q % T;
  if (row >= p.N || col >= p.K) return;
  const float* src = p.parts + ((int64_t)first * tiles + in) * T * T + q;
  const int64_t pitch = (int64_t)tiles * T * T;
  f4 o = {0, 0, 0, 0};
  int i = 0;
  for (; i + 4 <= n; i += 4) {
    f4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const f4*>(src + (i + j) * pitch);
#pragma unroll
    for (int j = 0; j < 4; ++j) o += v[j];
  }
  for (; i < n; ++i) o += *reinterpret_cast<const f4*>(src + i * pitch);
  const int64_t off = ((int64_t)e * p.N + row) * p.ld_dw + col;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (p.f32) {
      float* d = static_cast<float*>(p.dw) + off + k;
      *d = p.accumulate ? o[k] + *d : o[k];
    } else {
      uint8_t* d = static_cast<uint8_t*>(p.dw);
      store1<DT_BF16>(d, off + k, p.accumulate ? o[k] + load1<DT_BF16>(d, off + k) : o[k]);
    }
  }
}

// The tile of a call and whether the rows of its groups are split: len rows a
// part (0: no), at most `units` parts of tiles in all (R rows in parts of len
// make at most (R + groups (len - 1)) / len parts).  Measured, E4M3 to FP32:
//   rows x N x K, groups     128, whole  128, parts  256, whole  256, parts
//   32768 x 64 x 1024, 1         351          34         667          43 us
//   32768 x 2048 x 2048, 1       421         382          -          283
//   32768 x 1024 x 1024, 4       151          -           -           96
//   8192 x 256 x 512, 16         15.7         28          -           32
//   2000 x 1024 x 1024, 20       24           -           32          -
//   16384 x 512 x 1024, 32       37           -           33          -
//   32768 x 2048 x 2048, 4       316          -          287          -
// (the chosen ones with a workspace at hand and 30 calls in a row: 28, 290, 104 to
// 111, 11 to 14, 24, 32 to 33 and 290 us, by how even the groups are)
struct Plan {
  int64_t T, len, units;
  float us;
};
int64_t most_of(int64_t T) { return T == 256 ? 256 : 512; }  // workgroups that the 256 CUs hold at once

// Estimated time of a plan.  A round of tiles at once takes as long as its
// longest group, so with one round that is taken to be a quarter longer than
// the mean; more rounds even that out.
float time_of(int64_t R, int64_t groups, int64_t tiles, int64_t T, int64_t len) {
  const int64_t most = most_of(T), units = len ? (R + groups * (len - 1) / 2) / len * tiles : groups * tiles;
  const float stages = std::max((float)(len ? len : (R + groups - 1) / groups) / kStep, 3.0f) + 2;
  const float full = (float)(units / most), rest = (float)(units % most);
  const float last = rest == 0 ? 0.0f : T == 256 ? 2.1f : rest > 256 ? 1.25f : 0.85f;
  const float round = T == 256 ? 2.1f : 1.25f;
  const float uneven = len || groups == 1 ? 1.0f : 1.0f + 0.25f / (full + (rest > 0));
  const float join = len ? 5.0f + units * (T * T * 8) / 5e6f : 0.0f;
  return (full * round + last) * stages * uneven + join;
}

// The plan with the least time among 128 x 128 tiles, 256 x 256 tiles (if they
// may be taken) and parts of R / 2, R / 3, R / 4, R / 6, R / 8 ... rows.
Plan plan_of(int64_t R, int64_t N, int64_t K, int64_t groups, bool large) {
  Plan best = {};
  for (int64_t T = 128; T <= (large ? 256 : 128); T *= 2) {
    const int64_t tiles = ((N + T - 1) / T) * ((K + T - 1) / T);
    const float us = time_of(R, groups, tiles, T, 0);
    if (T == 128 || us < best.us) best = {T, 0, 0, us};
    if (groups > 512) continue;
    for (int64_t i = 0; i < 18; ++i) {
      const int64_t n = (i & 1 ? 3 : 2) << (i / 2);
      const int64_t len = ((R + n - 1) / n + kStep - 1) / kStep * kStep;
      const int64_t units = (R + groups * (len - 1)) / std::max<int64_t>(len, 1) * tiles;
      if (len < 3 * kStep || len > INT32_MAX || units > 2 * most_of(T)) break;
      const float us = time_of(R, groups, tiles, T, len);
      if (us < best.us) best = {T, len, units, us};
    }
  }
  return best;
}

template <class V>
hipError_t launch_v(const WgradArgs& a, const Plan& plan, hipStream_t s) {
  WgradParams p = {};
  p.dy = a.dy;
  p.ld_dy = a.ld_dy;
  p.R = a.R;
  p.N = a.N;
  p.codes = a.codes;
  p.scales = a.scales;
  p.x_rows = a.x_rows;
  p.K = a.K;
  p.last_word = (uint32_t)(a.x_rows * a.K / 32 - 4);
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
  const uint32_t most = (uint32_t)most_of(V::T);
  uint32_t grid = p.units < most ? p.units : most;
  if (plan.len) {
    p.len = (int32_t)plan.len;
    p.parts = a.parts;
    p.slots = (uint32_t)plan.units;
    grid = (p.slots + 7) / 8 * 8;
  }
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
  hipLaunchKernelGGL(kern, dim3(grid), dim3(256), V::LDS, s, p);
  if (plan.len)
    hipLaunchKernelGGL(k_wgrad_join, dim3(p.tn * p.tk * (uint32_t)p.groups * (V::T * V::T / 1024)), dim3(256), 0, s, p,
                       (uint32_t)V::T);
  return hipGetLastError();
}

template <int FMT, bool GATHER>
hipError_t launch_g(const WgradArgs& a, hipStream_t s) {
  if (a.N % 8 || a.ld_dy >= (1 << 24) || a.x_rows * a.K < 128 || a.x_rows * a.K >= (int64_t)UINT32_MAX)
    return launch_v<Variant<FMT, 64, ANY_SHAPE, GATHER>>(a, plan_of(a.R, a.N, a.K, a.groups, false), s);
  const Plan plan = plan_of(a.R, a.N, a.K, a.groups, true);
  if (plan.T == 128) return launch_v<Variant<FMT, 64, PLAIN_SHAPE, GATHER>>(a, plan, s);
  return a.K % 128 ? launch_v<Variant<FMT, 128, PLAIN_SHAPE, GATHER>>(a, plan, s)
                   : launch_v<Variant<FMT, 128, WHOLE_WORDS, GATHER>>(a, plan, s);
}

template <int FMT>
hipError_t launch_f(const WgradArgs& a, hipStream_t s) {
  return a.row_index ? launch_g<FMT, true>(a, s) : launch_g<FMT, false>(a, s);
}

}  // namespace

size_t wgrad_workspace_bytes(int64_t R, int64_t N, int64_t K, int64_t groups) {
  const auto bytes = [&](bool large) {
    const Plan plan = plan_of(R, N, K, groups, large);
    return (size_t)(plan.units * plan.T * plan.T) * sizeof(float);
  };
  return std::max(bytes(false), bytes(true));
}

hipError_t launch_wgrad_grouped(const WgradArgs& a, hipStream_t s) {
  if (a.fmt == FMT_MXFP8) return launch_f<FMT_MXFP8>(a, s);
  if (a.fmt == FMT_MXFP8_E5M2) return launch_f<FMT_MXFP8_E5M2>(a, s);
  return launch_f<FMT_MXINT8>(a, s);
}

}  // namespace mxk
