// route.hip -- the router of a mixture-of-experts layer: softmax over the
// experts' scores, the k largest of them, the order in which the grouped
// product takes the routed rows, the per-expert counts and the balance loss,
// and the gradient of the scores.
//
// Forward, for scores x [T, E], V = tokens that are not padding:
//   p = softmax(x) per token; the k largest x, equal ones by lower index;
//   w = p of the chosen (or divided by their sum);
//   c_e = tokens that chose e; S_e = sum_t p[t, e];
//   loss = E / (k V^2) * sum_e c_e S_e;
//   routed rows: by expert, within one by token (a counting sort).
// Backward, with b_e = d_loss * E c_e / (k V^2) and q = the chosen p (divided
// by their sum if the weights are):
//   d_x = p * (b - <p, b>) + q * (d_w - <q, d_w>)            (normalized)
//   d_x = p * (b - <p, b> - <q, d_w>) + q * d_w              (otherwise)
// A score of -inf is never chosen and has p = 0; a padding token chooses
// nothing, adds nothing to S and gets a zero gradient.
//
// A group of G lanes holds one token's scores, VPL consecutive ones a lane.
// Selection works on integer keys of 31 bits or fewer, the score's bits in
// increasing order above the complement of the expert's number, so keys are
// distinct and equal scores come out by lower index: the next key is the
// largest of key - last as an unsigned number (keys not below `last` give less
// than 2^31, the others more), one subtraction and half a max3 a score.  A BF16
// score fits whole.  Of an FP32 score the upper 21 bits do; where two of the
// topk + 1 largest agree in those, the wave selects by comparing scores.
// The sort needs no atomics whose order matters: within 64 tokens an expert's
// tokens are the bits of one 64-bit word, so a token's rank is a population
// count, and the blocks of tokens are put in order by their counts.  S is
// summed per block in a fixed order, then over the blocks.
//
// The bytes (16384 x 256 BF16: 9 MB, 2 us of HBM) are not what bounds it.  Of
// two launches each has a start and an end (an empty kernel takes 1.5 to 2 us).
// Choosing: 900 vector instructions a wave, 4 waves a SIMD, at 16384 x 256 about
// 6 of its 11.7 us; the rest is one chain of load, selection steps and LDS that
// nothing runs beside, since a wave has one pass of tokens.  Placing: every
// workgroup reads the counts of all blocks (33 MB out of the L2s at 256
// experts) and adds them in LDS, where 84% of its accesses conflict.  At 4096 x
// 32 both are chains of dependent loads and LDS steps on 64 of the CUs.
// Measured on the device, top 8: 16384 x 256 BF16 20.5 us (choosing 11.7, placing
// 9.5), 4096 x 32 FP32 13.4 us (6.5 and 6.9), one token of 32 5.5 us, one launch.
// Backward, 16384 x 256: FP32 10.4 us (33 MB: 3.2 TB/s), BF16 10.0.  There a
// group of lanes has one token, and its loads depend on one another: the mask,
// the chosen experts, their scores; 1024 tokens take 6.7 us.
#include "../device/exp.h"
#include "../device/rows.h"
#include "../device/wave.h"
#include "../launch_moe.h"

namespace mxk {

namespace {

// threads of a workgroup, for EP experts (padded): one pass over 64 tokens
// while the sums of its waves fit in LDS
constexpr int threads_for(int EP) { return EP <= 256 ? 1024 : 512; }
constexpr int kSub = 64;     // tokens of one bit word
constexpr int kMaxK = 16;    // slots of a token
constexpr int64_t kMaxBlocks = 256;

struct RouteParams {
  const void* logits;
  int64_t ld;
  const uint8_t* mask;  // nullptr: no padding
  int32_t tokens, experts, topk;
  int32_t normalize;
  int32_t vec;      // rows allow vector loads
  int32_t per;      // tokens of one block (a multiple of kSub)
  int32_t blocks;
  int32_t pitch;    // experts, rounded up to 8: of the workspace's rows
  int32_t* experts_out;
  float* weights;
  int32_t* slot_row;
  int32_t* row_index;
  int64_t* offsets;
  int64_t* counts;
  int64_t* valid;
  float* prob_sum;
  float* loss;
  // workspace (blocks > 1): counts [blocks][pitch], sums of p [blocks][pitch], valid tokens [blocks]
  uint16_t* part_counts;
  float* part_sums;
  int32_t* part_valid;
};

template <int CTRL>
__device__ inline float dpp_f32(float v) {
  return u2f((uint32_t)__builtin_amdgcn_update_dpp(0, (int)f2u(v), CTRL, 0xF, 0xF, false));
}

// all-reduce over the G (16 or 64) lanes of a group
template <int G, class Op>
__device__ inline float group_reduce(float v, Op op) {
  v = op(v, dpp_f32<0xB1>(v));   // lane ^ 1
  v = op(v, dpp_f32<0x4E>(v));   // lane ^ 2
  v = op(v, dpp_f32<0x141>(v));  // the other quad of 8
  v = op(v, dpp_f32<0x140>(v));  // the other 8 of 16
  if constexpr (G == 64) {
    v = op(v, __shfl_xor(v, 16));
    v = op(v, __shfl_xor(v, 32));
  }
  return v;
}
struct OpMax {
  __device__ float operator()(float a, float b) const { return __builtin_fmaxf(a, b); }
};
struct OpAdd {
  __device__ float operator()(float a, float b) const { return a + b; }
};

// Score v of lane gl of a group: chunks of VQ (up to 16 bytes) consecutive
// scores, the chunks of the group's lanes side by side, so that a load of the
// group is one run of memory.
template <int DT, int VPL>
constexpr int chunk_of() {
  return VPL < (DT == DT_BF16 ? 8 : 4) ? VPL : (DT == DT_BF16 ? 8 : 4);
}
template <int DT, int G, int VPL>
__device__ inline int expert_of(int gl, int v) {
  constexpr int VQ = chunk_of<DT, VPL>();
  return (v / VQ) * (VQ * G) + gl * VQ + v % VQ;
}

// the lane's VPL scores of row t; entries past E are -inf
template <int DT, int G, int VPL>
__device__ inline void load_scores(const RouteParams& p, int64_t t, int gl, float (&x)[VPL]) {
  constexpr int VQ = chunk_of<DT, VPL>();
#pragma unroll
  for (int v = 0; v < VPL; v += VQ) {
    const int e = expert_of<DT, G, VPL>(gl, v);
    const int64_t off = t * p.ld + e;
    if (VQ >= 4 && p.vec && e + VQ <= p.experts) {
      if constexpr (DT == DT_BF16 && VQ == 8) {
        float y[8];
        load8<DT_BF16>(p.logits, off, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[v + i] = y[i];
      } else if constexpr (DT == DT_BF16 && VQ == 4) {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.logits) + off);
        x[v] = u2f(w.x << 16);
        x[v + 1] = u2f(w.x & 0xFFFF0000u);
        x[v + 2] = u2f(w.y << 16);
        x[v + 3] = u2f(w.y & 0xFFFF0000u);
      } else if constexpr (DT == DT_F32 && VQ == 4) {
        const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(p.logits) + off);
        x[v] = w.x;
        x[v + 1] = w.y;
        x[v + 2] = w.z;
        x[v + 3] = w.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VQ; ++i) x[v + i] = e + i < p.experts ? load1<DT>(p.logits, off + i) : -__builtin_inff();
    }
  }
}

template <int EP>
struct RouteShared {
  static constexpr int kThreads = threads_for(EP), kWaves = kThreads / 64;
  uint64_t mask[EP];          // tokens of the current 64 that chose the expert
  int32_t run[EP];            // tokens before them in the block that did; then the sort's bases
  int32_t total[EP];
  float sums[kWaves][EP];
  int32_t idx[kSub][kMaxK];   // chosen experts, -1 for none
  int32_t valid;
};

__device__ inline uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
template <int G>
__device__ inline uint32_t group_umax(uint32_t v) {
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));
  if constexpr (G == 64) {
    v = umax(v, lane_read(v, lane_id() ^ 16u));
    v = umax(v, lane_read(v, lane_id() ^ 32u));
  }
  return v;
}

// key of score x of expert e; 0: never chosen (-inf, NaN)
template <int DT>
__device__ inline uint32_t key_of(float x, int e) {
  const uint32_t b = f2u(x + 0.0f);  // (-0 and 0 are equal)
  const uint32_t ord = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  const uint32_t k = (DT == DT_BF16 ? (ord >> 16) << 10 : (ord >> 11) << 10) | (uint32_t)(1023 - e);
  return x > -__builtin_inff() ? k : 0u;
}

// The topk largest scores of each group's token: lane j of the group gets the
// expert of slot j (-1 where there is none) and its score.
template <int DT, int G, int VPL>
__device__ inline int select(const RouteParams& p, int64_t t, const float (&x)[VPL], int gl, float* score) {
  const int topk = p.topk;
  uint32_t key[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) key[v] = key_of<DT>(x[v], expert_of<DT, G, VPL>(gl, v));
  uint32_t last = 0x80000000u, mine = 0;
  bool unsure = false;
  const int n = DT == DT_BF16 ? topk : topk + 1;
  for (int j = 0; j < n; ++j) {
    uint32_t m = key[0] - last;
#pragma unroll
    for (int v = 1; v < VPL; ++v) m = umax(m, key[v] - last);
    m = group_umax<G>(m);
    // none left: the keys below `last` are 0 (or `last` is 0 itself)
    const uint32_t nx = last == 0 ? 0u : last + m;
    if constexpr (DT == DT_F32) unsure = unsure || (nx != 0 && (nx ^ last) < 1024u);
    mine = gl == j ? nx : mine;
    last = nx;
  }
  int at = mine && gl < topk ? 1023 - (int)(mine & 1023u) : -1;
  if constexpr (DT == DT_F32) {
    if (__ballot(unsure)) {
      float y[VPL];
#pragma unroll
      for (int v = 0; v < VPL; ++v) y[v] = x[v] > -__builtin_inff() ? x[v] : -__builtin_inff();
      at = -1;
      for (int j = 0; j < topk; ++j) {
        float m = y[0];
#pragma unroll
        for (int v = 1; v < VPL; ++v) m = __builtin_fmaxf(m, y[v]);
        m = group_reduce<G>(m, OpMax());
        int w = 1 << 20;  // the first of this lane's that has it
#pragma unroll
        for (int v = VPL - 1; v >= 0; --v) w = y[v] == m ? expert_of<DT, G, VPL>(gl, v) : w;
        if (!(m > -__builtin_inff())) w = 1 << 20;
        w = (1 << 20) - (int)group_umax<G>((uint32_t)((1 << 20) - w));  // the lowest of the group's
#pragma unroll
        for (int v = 0; v < VPL; ++v) y[v] = w == expert_of<DT, G, VPL>(gl, v) ? -__builtin_inff() : y[v];
        at = gl == j ? (w < (1 << 20) ? w : -1) : at;
      }
    }
    *score = at >= 0 ? load1<DT>(p.logits, t * p.ld + at) : 0.0f;
  } else {
    const uint32_t ord = mine >> 10;  // the whole score
    *score = at >= 0 ? u2f((ord ^ (ord & 0x8000u ? 0x8000u : 0xFFFFu)) << 16) : 0.0f;
  }
  return at;
}

// 64 tokens from s0 on (those below t1): experts and weights, each expert's
// bit word, the lanes' sums of p.
template <int DT, int G, int VPL>
__device__ inline void choose_64(const RouteParams& p, int s0, int t1, RouteShared<G * VPL>& sh, float (&sum_p)[VPL]) {
  constexpr int kWaves = threads_for(G * VPL) / 64;
  constexpr int TPI = 64 / G;  // tokens a wave handles at once
  constexpr int ITS = kSub / kWaves / TPI;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, gl = lane & (G - 1), grp = lane / G;
  int n_valid = 0;
  float x[2][VPL];
  bool ok[2];
  const auto load = [&](int it, float (&y)[VPL], bool& in) {
    const int t = s0 + wave * (kSub / kWaves) + it * TPI + grp;
    in = t < t1 && (!p.mask || p.mask[t] != 0);
    if (in) {
      load_scores<DT, G, VPL>(p, t, gl, y);
    } else {
#pragma unroll
      for (int v = 0; v < VPL; ++v) y[v] = -__builtin_inff();
    }
  };
  load(0, x[0], ok[0]);
#pragma unroll 2
  for (int it = 0; it < ITS; ++it) {
    if (it + 1 < ITS) load(it + 1, x[(it + 1) & 1], ok[(it + 1) & 1]);
    float(&y)[VPL] = x[it & 1];
    const int lt = wave * (kSub / kWaves) + it * TPI + grp, t = s0 + lt;
    float m = y[0];
#pragma unroll
    for (int v = 1; v < VPL; ++v) m = __builtin_fmaxf(m, y[v]);
    m = group_reduce<G>(__builtin_fmaxf(m, -__builtin_inff()), OpMax());
    const float base = m == -__builtin_inff() ? 0.0f : m;
    float xe;
    const int e = select<DT, G, VPL>(p, t, y, gl, &xe);
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      y[v] = exp_nonpos(y[v] - base);
      s += y[v];
    }
    s = group_reduce<G>(s, OpAdd());
    const float inv = s == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
    for (int v = 0; v < VPL; ++v) sum_p[v] += y[v] * inv;
    float w = e >= 0 ? exp_nonpos(xe - base) : 0.0f;
    if (p.normalize) {
      const float sw = group_reduce<G>(w, OpAdd());
      w = e < 0 ? 0.0f : inv == inv ? w / sw : inv;  // a NaN anywhere in the row shows in its weights
    } else {
      w = e < 0 ? 0.0f : w * inv;
    }
    if (gl == 0) n_valid += ok[it & 1] ? 1 : 0;
    if (gl < p.topk && t < t1) {
      sh.idx[lt][gl] = e;
      p.experts_out[(int64_t)t * p.topk + gl] = e;
      p.weights[(int64_t)t * p.topk + gl] = w;
      if (e >= 0) atomicOr(reinterpret_cast<unsigned long long*>(&sh.mask[e]), 1ull << lt);
    }
  }
  if (n_valid) atomicAdd(&sh.valid, n_valid);
}

// The block's sums of p into sh.sums[0]: over the groups of a wave, then over
// the waves.
template <int DT, int G, int VPL>
__device__ inline void reduce_sums(RouteShared<G * VPL>& sh, float (&sum_p)[VPL]) {
  constexpr int kThreads = threads_for(G * VPL), kWaves = kThreads / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, gl = lane & (G - 1), grp = lane / G;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    float s = sum_p[v];
    if constexpr (G == 16) {
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
    }
    if (grp == 0) sh.sums[wave][expert_of<DT, G, VPL>(gl, v)] = s;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < G * VPL; e += kThreads) {
    float s = sh.sums[0][e];
    for (int w = 1; w < kWaves; ++w) s += sh.sums[w][e];
    sh.sums[0][e] = s;
  }
  __syncthreads();
}

template <int EP>
__device__ inline void clear(RouteShared<EP>& sh) {
  constexpr int kThreads = threads_for(EP);
  for (int e = threadIdx.x; e < EP; e += kThreads) {
    sh.mask[e] = 0;
    sh.run[e] = 0;
    sh.total[e] = 0;
  }
  if (threadIdx.x == 0) sh.valid = 0;
  __syncthreads();
}

// sh.total[e] (counts of all tokens) -> exclusive prefix over the experts,
// in place; returns the number of routed rows.
template <int EP>
__device__ inline int prefix_experts(RouteShared<EP>& sh) {
  constexpr int PER = (EP + 63) / 64;
  __shared__ int rows;
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int c[PER], s = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane * PER + i;
      c[i] = e < EP ? sh.total[e] : 0;
      s += c[i];
    }
    // inclusive scan over the wave: rows of 16 lanes, then the rows' last lanes
    int at = s;
    at += __builtin_amdgcn_update_dpp(0, at, 0x111, 0xF, 0xF, false);
    at += __builtin_amdgcn_update_dpp(0, at, 0x112, 0xF, 0xF, false);
    at += __builtin_amdgcn_update_dpp(0, at, 0x114, 0xF, 0xF, false);
    at += __builtin_amdgcn_update_dpp(0, at, 0x118, 0xF, 0xF, false);
    at += __builtin_amdgcn_update_dpp(0, at, 0x142, 0xA, 0xF, false);
    at += __builtin_amdgcn_update_dpp(0, at, 0x143, 0xC, 0xF, false);
    if (lane == 63) rows = at;
    at -= s;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane * PER + i;
      if (e < EP) sh.total[e] = at;
      at += c[i];
    }
  }
  __syncthreads();
  return rows;
}

// counts, offsets, sums and the loss, from the counts in `count` (LDS) and
// the sums in sh.sums[0]; sh.total holds the exclusive prefix
template <int EP>
__device__ inline void publish(const RouteParams& p, RouteShared<EP>& sh, const int32_t* count, int rows, int valid) {
  constexpr int kThreads = threads_for(EP), kWaves = kThreads / 64;
  __shared__ float red[kWaves];
  float s = 0.0f;
  for (int e = threadIdx.x; e < p.experts; e += kThreads) {
    p.counts[e] = count[e];
    p.offsets[e] = sh.total[e];
    p.prob_sum[e] = sh.sums[0][e];
    s += (float)count[e] * sh.sums[0][e];
  }
  s = group_reduce<64>(s, OpAdd());
  if ((threadIdx.x & 63u) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kWaves; ++w) s += red[w];
    p.offsets[p.experts] = rows;
    *p.valid = valid;
    const float v = (float)valid;
    *p.loss = valid ? s * ((float)p.experts / ((float)p.topk * v)) / v : 0.0f;
  }
}

// At most 64 tokens: everything in one workgroup and one launch.
template <int DT, int G, int VPL>
__global__ __launch_bounds__(threads_for(G * VPL)) void k_route_one(RouteParams p) {
  constexpr int EP = G * VPL;
  constexpr int kThreads = threads_for(EP);
  __shared__ RouteShared<EP> sh;
  clear(sh);
  float sum_p[VPL] = {};
  choose_64<DT, G, VPL>(p, 0, p.tokens, sh, sum_p);
  reduce_sums<DT, G, VPL>(sh, sum_p);
  for (int e = threadIdx.x; e < EP; e += kThreads) sh.run[e] = sh.total[e] = __popcll(sh.mask[e]);
  __syncthreads();
  const int rows = prefix_experts(sh);
  const int n = p.tokens * p.topk;
  for (int o = threadIdx.x; o < n; o += kThreads) {
    const int t = o / p.topk, e = sh.idx[t][o - t * p.topk];
    const int row = e >= 0 ? sh.total[e] + __popcll(sh.mask[e] & ((1ull << t) - 1)) : -1;
    p.slot_row[o] = row;
    if (row >= 0) p.row_index[row] = t;
    if (o >= rows) p.row_index[o] = -1;
  }
  publish(p, sh, sh.run, rows, sh.valid);
}

// One block of tokens: experts, weights, in slot_row the rank of each slot
// among the block's tokens of its expert, and the block's counts and sums.
template <int DT, int G, int VPL>
__global__ __launch_bounds__(threads_for(G * VPL)) void k_route_choose(RouteParams p) {
  constexpr int EP = G * VPL;
  constexpr int kThreads = threads_for(EP);
  __shared__ RouteShared<EP> sh;
  const int b = blockIdx.x;
  const int t0 = b * p.per, t1 = t0 + p.per < p.tokens ? t0 + p.per : p.tokens;
  clear(sh);
  float sum_p[VPL] = {};
  for (int s0 = t0; s0 < t1; s0 += kSub) {
    choose_64<DT, G, VPL>(p, s0, t1, sh, sum_p);
    __syncthreads();
    const int n = (t1 - s0 < kSub ? t1 - s0 : kSub) * p.topk;
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const int lt = i / p.topk, e = sh.idx[lt][i - lt * p.topk];
      p.slot_row[(int64_t)s0 * p.topk + i] = e >= 0 ? sh.run[e] + __popcll(sh.mask[e] & ((1ull << lt) - 1)) : -1;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < EP; e += kThreads) {
      sh.run[e] += __popcll(sh.mask[e]);
      sh.mask[e] = 0;
    }
    __syncthreads();
  }
  reduce_sums<DT, G, VPL>(sh, sum_p);
  for (int e = threadIdx.x; e < p.pitch; e += kThreads) {
    p.part_counts[(int64_t)b * p.pitch + e] = (uint16_t)(e < EP ? sh.run[e] : 0);
    p.part_sums[(int64_t)b * p.pitch + e] = e < EP ? sh.sums[0][e] : 0.0f;
  }
  if (threadIdx.x == 0) p.part_valid[b] = sh.valid;
}

// Blocks 0 .. blocks-1 place their tokens' rows; block `blocks` reduces the
// sums and publishes.  Each adds up the counts of all blocks for itself, 8
// experts a lane and load: 64 K counts of 16 bits at 256 experts, which come
// out of L2.
template <int EP>
__global__ __launch_bounds__(threads_for(EP)) void k_route_place(RouteParams p) {
  constexpr int kThreads = threads_for(EP), kWaves = kThreads / 64;
  __shared__ RouteShared<EP> sh;
  const int b = blockIdx.x, tid = threadIdx.x;
  // this thread's first slot, on its way meanwhile
  const int t0 = b * p.per, t1 = t0 + p.per < p.tokens ? t0 + p.per : p.tokens;
  const int64_t o0 = (int64_t)t0 * p.topk + tid, o1 = (int64_t)t1 * p.topk;
  int e_first = -1, rank_first = 0;
  if (o0 < o1) {
    e_first = p.experts_out[o0];
    rank_first = p.slot_row[o0];
  }
  clear(sh);
  {
    constexpr int LANES = EP / 8;              // lanes along the experts
    constexpr int ROWS = kThreads / LANES;     // blocks read at once
    const int e0 = tid % LANES * 8;
    int all[8] = {}, before[8] = {};
    if (e0 < p.pitch) {
#pragma unroll 4
      for (int i = tid / LANES; i < p.blocks; i += ROWS) {
        const uint4 w = *reinterpret_cast<const uint4*>(p.part_counts + (int64_t)i * p.pitch + e0);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int lo = ww[k] & 0xFFFFu, hi = ww[k] >> 16;
          all[2 * k] += lo;
          all[2 * k + 1] += hi;
          before[2 * k] += i < b ? lo : 0;
          before[2 * k + 1] += i < b ? hi : 0;
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (all[k]) atomicAdd(&sh.total[e0 + k], all[k]);
        if (before[k]) atomicAdd(&sh.run[e0 + k], before[k]);
      }
    }
  }
  if (b == p.blocks) {
    // (before == all here: sh.run holds the counts)  The sums: kWaves runs of
    // blocks, each in order, then the runs in order.
    const int run = (p.blocks + kWaves - 1) / kWaves;
    const int i0 = (tid >> 6) * run, i1 = i0 + run < p.blocks ? i0 + run : p.blocks;
    for (int e = (tid & 63) * 4; e < EP; e += 256) {  // (EP is a multiple of 4)
      float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (e < p.pitch) {
#pragma unroll 8
        for (int i = i0; i < i1; ++i) {
          const float4 v = *reinterpret_cast<const float4*>(p.part_sums + (int64_t)i * p.pitch + e);
          s.x += v.x;
          s.y += v.y;
          s.z += v.z;
          s.w += v.w;
        }
      }
      *reinterpret_cast<float4*>(&sh.sums[tid >> 6][e]) = s;
    }
    for (int i = tid; i < p.blocks; i += kThreads) atomicAdd(&sh.valid, p.part_valid[i]);
  }
  __syncthreads();
  const int rows = prefix_experts(sh);
  if (b == p.blocks) {
    for (int e = tid; e < EP; e += kThreads) {
      float s = sh.sums[0][e];
      for (int w = 1; w < kWaves; ++w) s += sh.sums[w][e];
      sh.sums[0][e] = s;
    }
    __syncthreads();
    publish(p, sh, sh.run, rows, sh.valid);
    return;
  }
  // rank of a slot -> its routed row, and the row's token
  for (int64_t o = o0; o < o1; o += kThreads) {
    const int e = o == o0 ? e_first : p.experts_out[o];
    if (e < 0) continue;
    const int row = sh.total[e] + sh.run[e] + (o == o0 ? rank_first : p.slot_row[o]);
    p.slot_row[o] = row;
    p.row_index[row] = (int32_t)(o / p.topk);
  }
  const int64_t n = (int64_t)p.tokens * p.topk;
  for (int64_t r = rows + (int64_t)b * kThreads + tid; r < n; r += (int64_t)p.blocks * kThreads) p.row_index[r] = -1;
}

// ---- backward ---------------------------------------------------------------
struct RouteBwdParams {
  RouteParams f;  // logits, mask, sizes, experts_out, counts, valid
  const float* d_weights;
  const float* d_loss;
  void* d_logits;
  int64_t ld_d;
  int32_t vec_d;
};

constexpr int kBwdThreads = 256;

// One token of a group on its way in.
template <int VPL>
struct RouteIn {
  float x[VPL];
  int e;         // lane j: the expert of slot j
  float dw, xe;  // the gradient of its weight, its score
  bool ok;
};

// The terms of the chosen experts go to the lanes that hold those experts'
// scores through LDS, one word an expert, zero but for the token's topk words:
// each lane clears again what it wrote.  A group is part of one wave, whose LDS
// accesses keep their order, so no barrier is needed.
template <int DT, int G, int VPL>
__global__ __launch_bounds__(kBwdThreads) void k_route_bwd(RouteBwdParams b) {
  constexpr int GROUPS = kBwdThreads / G;
  constexpr int VQ = chunk_of<DT, VPL>();
  __shared__ __attribute__((aligned(16))) float extra[GROUPS][G * VPL];
  const RouteParams& p = b.f;
  const int gl = threadIdx.x & (G - 1), grp = threadIdx.x / G;
  const int k = p.topk;
  float* mine = extra[grp];
  const auto load = [&](int64_t t, RouteIn<VPL>& in) {
    in.ok = t < p.tokens && (!p.mask || p.mask[t] != 0);
    in.e = -1;
    in.dw = in.xe = 0.0f;
    if (in.ok) {
      if (gl < k) {
        in.e = p.experts_out[t * k + gl];
        in.dw = b.d_weights ? b.d_weights[t * k + gl] : 0.0f;
      }
      load_scores<DT, G, VPL>(p, t, gl, in.x);
      in.e = in.e < p.experts ? in.e : -1;
      if (in.e >= 0) in.xe = load1<DT>(p.logits, t * p.ld + in.e);
      else in.dw = 0.0f;  // (a slot without an expert: its gradient may hold anything)
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) in.x[i] = -__builtin_inff();
    }
  };
  const int64_t step = (int64_t)gridDim.x * GROUPS;
  int64_t t = (int64_t)blockIdx.x * GROUPS + grp;
  RouteIn<VPL> in;
  load(t, in);
  const float v = (float)*p.valid;
  const float scale = b.d_loss && v > 0.0f ? *b.d_loss * ((float)p.experts / ((float)k * v)) / v : 0.0f;
  // some scale * count may not be finite (counts are below 2^63), and 0 times it
  // is no zero for a padding token
  const bool wild = __ballot(!(__builtin_fabsf(scale) <= 1e18f)) != 0;
  float bal[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = expert_of<DT, G, VPL>(gl, i);
    bal[i] = e < p.experts ? scale * (float)p.counts[e] : 0.0f;
    mine[e] = 0.0f;
  }
  // (the groups of a wave leave the loop together: their lanes are shuffled as one)
  for (; __ballot(t < p.tokens) != 0; t += step) {
    float(&x)[VPL] = in.x;
    float m = x[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = __builtin_fmaxf(m, x[i]);
    m = group_reduce<G>(__builtin_fmaxf(m, -__builtin_inff()), OpMax());
    m = m == -__builtin_inff() ? 0.0f : m;
    float s = 0.0f, pb = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      x[i] = exp_nonpos(x[i] - m);
      s += x[i];
      pb = fmaf(x[i], bal[i], pb);
    }
    s = group_reduce<G>(s, OpAdd());
    const float inv = s == 0.0f ? 0.0f : 1.0f / s;
    pb = group_reduce<G>(pb, OpAdd()) * inv;
    const int e = in.e;
    const bool ok = in.ok;
    float q = e >= 0 ? exp_nonpos(in.xe - m) : 0.0f;
    if (p.normalize) {
      const float sq = group_reduce<G>(q, OpAdd());
      q = e >= 0 ? q / sq : 0.0f;
    } else {
      q *= inv;
    }
    const float qd = group_reduce<G>(q * in.dw, OpAdd());
    if (!p.normalize) pb += qd;
    if (e >= 0) mine[e] = p.normalize ? q * (in.dw - qd) : q * in.dw;
    __builtin_amdgcn_wave_barrier();
    float o[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) o[i] = mine[expert_of<DT, G, VPL>(gl, i)];
    __builtin_amdgcn_wave_barrier();
    if (e >= 0) mine[e] = 0.0f;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < VPL; ++i) o[i] = fmaf(x[i] * inv, bal[i] - pb, o[i]);
    if (wild) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) o[i] = ok ? o[i] : 0.0f;
    }
    load(t + step, in);
    if (t < p.tokens) {
#pragma unroll
      for (int i = 0; i < VPL; i += VQ) {
        const int e2 = expert_of<DT, G, VPL>(gl, i);
        const int64_t off = t * b.ld_d + e2;
        if (VQ * (DT == DT_BF16 ? 2 : 4) == 16 && b.vec_d && e2 + VQ <= p.experts) {
          if constexpr (DT == DT_BF16 && VQ == 8)
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(b.d_logits) + off) =
                make_uint4(pack_bf16(o[i], o[i + 1]), pack_bf16(o[i + 2], o[i + 3]), pack_bf16(o[i + 4], o[i + 5]),
                           pack_bf16(o[i + 6], o[i + 7]));
          if constexpr (DT == DT_F32 && VQ == 4)
            *reinterpret_cast<float4*>(static_cast<float*>(b.d_logits) + off) =
                make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        } else {
#pragma unroll
          for (int h = 0; h < VQ; ++h)
            if (e2 + h < p.experts) store1<DT>(b.d_logits, off + h, o[i + h]);
        }
      }
    }
  }
}

RouteParams params_of(const RouteArgs& a) {
  RouteParams p = {};
  p.logits = a.logits;
  p.ld = a.ld;
  p.mask = a.mask;
  p.tokens = (int32_t)a.tokens;
  p.experts = a.experts;
  p.topk = a.topk;
  p.normalize = a.normalize;
  p.vec = (reinterpret_cast<uintptr_t>(a.logits) & 15u) == 0 && (a.ld * (a.dt == DT_F32 ? 4 : 2)) % 16 == 0;
  p.experts_out = a.experts_out;
  p.weights = a.weights;
  p.slot_row = a.slot_row;
  p.row_index = a.row_index;
  p.offsets = a.offsets;
  p.counts = a.counts;
  p.valid = a.valid;
  p.prob_sum = a.prob_sum;
  p.loss = a.loss;
  return p;
}

// tokens of one block and the number of blocks
void split(int64_t tokens, int64_t* per, int64_t* blocks) {
  *per = (tokens + kSub * kMaxBlocks - 1) / (kSub * kMaxBlocks) * kSub;
  *per = *per < kSub ? kSub : *per;
  *blocks = (tokens + *per - 1) / *per;
}

template <int DT, int G, int VPL>
hipError_t route_v(const RouteParams& p, hipStream_t s) {
  if (p.blocks <= 1) {
    hipLaunchKernelGGL((k_route_one<DT, G, VPL>), dim3(1), dim3(threads_for(G * VPL)), 0, s, p);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((k_route_choose<DT, G, VPL>), dim3(p.blocks), dim3(threads_for(G * VPL)), 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_route_place<G * VPL>), dim3(p.blocks + 1), dim3(threads_for(G * VPL)), 0, s, p);
  return hipGetLastError();
}

template <int DT, int G, int VPL>
hipError_t route_bwd_v(const RouteBwdParams& p, hipStream_t s) {
  constexpr int GROUPS = kBwdThreads / G;
  const int64_t need = ((int64_t)p.f.tokens + GROUPS - 1) / GROUPS;
  hipLaunchKernelGGL((k_route_bwd<DT, G, VPL>), dim3((uint32_t)(need < 1024 ? need : 1024)), dim3(kBwdThreads), 0, s,
                     p);
  return hipGetLastError();
}

// A group of 16 lanes while a lane's share is at most 16 scores, else the
// whole wave.
#define MXK_ROUTE(FN, P)                                                \
  const int E = a.experts;                                              \
  if (E <= 16) return FN<DT, 16, 1>(P, s);                              \
  if (E <= 32) return FN<DT, 16, 2>(P, s);                              \
  if (E <= 64) return FN<DT, 16, 4>(P, s);                              \
  if (E <= 128) return FN<DT, 16, 8>(P, s);                             \
  if (E <= 256) return FN<DT, 16, 16>(P, s);                            \
  if (E <= 512) return FN<DT, 64, 8>(P, s);                             \
  return FN<DT, 64, 16>(P, s);

template <int DT>
hipError_t route_d(const RouteArgs& a, const RouteParams& p, hipStream_t s) {
  MXK_ROUTE(route_v, p)
}
template <int DT>
hipError_t route_bwd_d(const RouteArgs& a, const RouteBwdParams& p, hipStream_t s) {
  MXK_ROUTE(route_bwd_v, p)
}
#undef MXK_ROUTE

}  // namespace

size_t route_workspace(int64_t tokens, int32_t experts) {
  int64_t per, blocks;
  split(tokens, &per, &blocks);
  if (blocks <= 1) return 0;
  const size_t cells = (size_t)blocks * (size_t)((experts + 7) / 8 * 8);
  return cells * sizeof(float) + cells * sizeof(uint16_t) + ((size_t)blocks * sizeof(int32_t) + 15) / 16 * 16;
}

hipError_t launch_route(const RouteArgs& a, void* workspace, hipStream_t s) {
  RouteParams p = params_of(a);
  int64_t per, blocks;
  split(a.tokens, &per, &blocks);
  p.per = (int32_t)per;
  p.blocks = (int32_t)blocks;
  if (blocks > 1) {
    p.pitch = (a.experts + 7) / 8 * 8;
    const size_t cells = (size_t)blocks * (size_t)p.pitch;
    p.part_sums = static_cast<float*>(workspace);
    p.part_counts = reinterpret_cast<uint16_t*>(p.part_sums + cells);  // (cells is a multiple of 8)
    p.part_valid = reinterpret_cast<int32_t*>(p.part_counts + cells);
  }
  return a.dt == DT_BF16 ? route_d<DT_BF16>(a, p, s) : route_d<DT_F32>(a, p, s);
}

hipError_t launch_route_bwd(const RouteArgs& a, const float* d_weights, const float* d_loss, void* d_logits,
                            int64_t ld_d, hipStream_t s) {
  RouteBwdParams b = {};
  b.f = params_of(a);
  b.d_weights = d_weights;
  b.d_loss = d_loss;
  b.d_logits = d_logits;
  b.ld_d = ld_d;
  b.vec_d = (reinterpret_cast<uintptr_t>(d_logits) & 15u) == 0 && (ld_d * (a.dt == DT_F32 ? 4 : 2)) % 16 == 0;
  return a.dt == DT_BF16 ? route_bwd_d<DT_BF16>(a, b, s) : route_bwd_d<DT_F32>(a, b, s);
}

}  // namespace mxk
