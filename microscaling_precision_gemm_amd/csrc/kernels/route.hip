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
// The sort needs no atomics whose order matters: within 64 tokens an expert's
// tokens are the bits of one 64-bit word, so a token's rank is a population
// count, and the blocks of tokens are put in order by their counts.  S is
// summed per block in a fixed order, then over the blocks.
#include "../device/rows.h"
#include "../device/wave.h"
#include "../launch.h"

namespace mxk {

namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kSub = 64;     // tokens of one bit word
constexpr int kMaxK = 16;    // slots of a token
constexpr int64_t kMaxBlocks = 256;
constexpr float kLog2e = 1.44269504088896340736f;

struct RouteParams {
  const void* logits;
  int64_t ld;
  const uint8_t* mask;  // nullptr: no padding
  int32_t tokens, experts, topk;
  int32_t normalize;
  int32_t vec;      // rows allow vector loads
  int32_t per;      // tokens of one block (a multiple of kSub)
  int32_t blocks;
  int32_t* experts_out;
  float* weights;
  int32_t* slot_row;
  int32_t* row_index;
  int64_t* offsets;
  int64_t* counts;
  int64_t* valid;
  float* prob_sum;
  float* loss;
  // workspace (blocks > 1): counts [blocks][E], sums of p [blocks][E], valid tokens [blocks]
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

// the lane's VPL scores of row t; entries past E are -inf
template <int DT, int VPL>
__device__ inline void load_scores(const RouteParams& p, int64_t t, int e0, float (&x)[VPL]) {
  const int64_t off = t * p.ld + e0;
  if (VPL >= 4 && p.vec && e0 + VPL <= p.experts) {
    if constexpr (DT == DT_BF16 && VPL >= 8) {
#pragma unroll
      for (int v = 0; v < VPL; v += 8) {
        float y[8];
        load8<DT_BF16>(p.logits, off + v, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[v + i] = y[i];
      }
    } else if constexpr (DT == DT_BF16 && VPL == 4) {
      const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.logits) + off);
      x[0] = u2f(w.x << 16);
      x[1] = u2f(w.x & 0xFFFF0000u);
      x[2] = u2f(w.y << 16);
      x[3] = u2f(w.y & 0xFFFF0000u);
    } else if constexpr (DT == DT_F32 && VPL >= 4) {
#pragma unroll
      for (int v = 0; v < VPL; v += 4) {
        const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(p.logits) + off + v);
        x[v] = w.x;
        x[v + 1] = w.y;
        x[v + 2] = w.z;
        x[v + 3] = w.w;
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < VPL; ++v) x[v] = e0 + v < p.experts ? load1<DT>(p.logits, off + v) : -__builtin_inff();
  }
}

template <int EP>
struct RouteShared {
  uint64_t mask[EP];          // tokens of the current 64 that chose the expert
  int32_t run[EP];            // tokens before them in the block that did; then the sort's bases
  int32_t total[EP];
  float sums[kWaves][EP];
  int32_t idx[kSub][kMaxK];   // chosen experts, -1 for none
  float val[kSub][kMaxK];     // their scores
  float top[kSub], inv[kSub]; // row maximum, 1 / sum of exp
  int32_t valid;
};

// Tokens [t0, t1) of one block: experts, weights, and in slot_row the rank of
// each slot among the block's tokens of its expert.  Leaves the block's
// counts in sh.run, its sums of p in sh.sums[0] and its valid tokens in
// sh.valid.
template <int DT, int G, int VPL>
__device__ inline void choose(const RouteParams& p, int t0, int t1, RouteShared<G * VPL>& sh) {
  constexpr int EP = G * VPL;
  constexpr int TPI = 64 / G;  // tokens a wave handles at once
  const int tid = threadIdx.x;
  const int lane = tid & 63, wave = tid >> 6, gl = lane & (G - 1), grp = lane / G;
  const int e0 = gl * VPL;
  for (int e = tid; e < EP; e += kThreads) {
    sh.mask[e] = 0;
    sh.run[e] = 0;
  }
  if (tid == 0) sh.valid = 0;
  float sum_p[VPL] = {};
  __syncthreads();
  for (int s0 = t0; s0 < t1; s0 += kSub) {
    int n_valid = 0;
#pragma unroll 1
    for (int it = 0; it < kSub / kWaves; it += TPI) {
      const int lt = wave * (kSub / kWaves) + it + grp;  // token within the 64
      const int t = s0 + lt;
      const bool ok = t < t1 && (!p.mask || p.mask[t] != 0);
      float x[VPL];
      if (ok) {
        load_scores<DT, VPL>(p, t, e0, x);
      } else {
#pragma unroll
        for (int v = 0; v < VPL; ++v) x[v] = -__builtin_inff();
      }
      float m = x[0];
#pragma unroll
      for (int v = 1; v < VPL; ++v) m = __builtin_fmaxf(m, x[v]);
      m = group_reduce<G>(__builtin_fmaxf(m, -__builtin_inff()), OpMax());
      const float base = m == -__builtin_inff() ? 0.0f : m;
      float ex[VPL], s = 0.0f;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        ex[v] = __builtin_amdgcn_exp2f((x[v] - base) * kLog2e);
        s += ex[v];
      }
      s = group_reduce<G>(s, OpAdd());
      const float inv = s == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
      for (int v = 0; v < VPL; ++v) sum_p[v] += ex[v] * inv;
      if (gl == 0) {
        sh.top[lt] = base;
        sh.inv[lt] = inv;
        n_valid += ok ? 1 : 0;
      }
      // k times the largest that is left
      for (int j = 0; j < p.topk; ++j) {
        float lm = x[0];
#pragma unroll
        for (int v = 1; v < VPL; ++v) lm = __builtin_fmaxf(lm, x[v]);
        lm = __builtin_fmaxf(lm, -__builtin_inff());  // a lane of NaNs has nothing to offer
        const float gm = j == 0 ? m : group_reduce<G>(lm, OpMax());
        const uint64_t have = __ballot(lm == gm && gm > -__builtin_inff());
        const uint64_t mine = G == 64 ? have : (have >> (grp * G)) & ((1ull << (G & 63)) - 1);
        const int owner = mine ? __builtin_ctzll(mine) : 0;
        if (gl == owner) {
          int at = -1;
          if (mine) {
            bool open = true;
#pragma unroll
            for (int v = 0; v < VPL; ++v) {
              const bool hit = open && x[v] == gm;
              at = hit ? e0 + v : at;
              x[v] = hit ? -__builtin_inff() : x[v];
              open = open && !hit;
            }
            atomicOr(reinterpret_cast<unsigned long long*>(&sh.mask[at]), 1ull << lt);
          }
          sh.idx[lt][j] = at;
          sh.val[lt][j] = gm;
        }
      }
    }
    if (n_valid) atomicAdd(&sh.valid, n_valid);
    __syncthreads();
    for (int i = tid; i < kSub * p.topk; i += kThreads) {
      const int lt = i / p.topk, j = i - lt * p.topk, t = s0 + lt;
      if (t >= t1) break;
      const int e = sh.idx[lt][j];
      float w = 0.0f;
      int rank = -1;
      if (e >= 0) {
        const float base = sh.top[lt], inv = sh.inv[lt];
        w = __builtin_amdgcn_exp2f((sh.val[lt][j] - base) * kLog2e);
        if (p.normalize) {
          float s = 0.0f;
          for (int i2 = 0; i2 < p.topk; ++i2)
            if (sh.idx[lt][i2] >= 0) s += __builtin_amdgcn_exp2f((sh.val[lt][i2] - base) * kLog2e);
          w = inv == inv ? w / s : inv;  // a NaN anywhere in the row shows in its weights
        } else {
          w *= inv;
        }
        rank = sh.run[e] + __popcll(sh.mask[e] & ((1ull << lt) - 1));
      }
      const int64_t o = (int64_t)t * p.topk + j;
      p.experts_out[o] = e;
      p.weights[o] = w;
      p.slot_row[o] = rank;
    }
    __syncthreads();
    for (int e = tid; e < EP; e += kThreads) {
      sh.run[e] += __popcll(sh.mask[e]);
      sh.mask[e] = 0;
    }
    __syncthreads();
  }
  // sums of p: over the groups of a wave, then over the waves
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    float s = sum_p[v];
    if constexpr (G == 16) {
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
    }
    if (grp == 0) sh.sums[wave][e0 + v] = s;
  }
  __syncthreads();
  for (int e = tid; e < EP; e += kThreads) {
    float s = sh.sums[0][e];
    for (int w = 1; w < kWaves; ++w) s += sh.sums[w][e];
    sh.sums[0][e] = s;
  }
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
    int at = s;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(at, off);
      at += lane >= off ? o : 0;
    }
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

// rank of a slot -> its routed row, and the row's token; base[e]: the first
// row of the block's tokens of expert e
__device__ inline void place(const RouteParams& p, int t0, int t1, const int32_t* base) {
  const int64_t o1 = (int64_t)t1 * p.topk;
  for (int64_t o = (int64_t)t0 * p.topk + threadIdx.x; o < o1; o += kThreads) {
    const int e = p.experts_out[o];
    if (e < 0) continue;
    const int row = base[e] + p.slot_row[o];
    p.slot_row[o] = row;
    p.row_index[row] = (int32_t)(o / p.topk);
  }
}

// Few tokens: everything in one workgroup.
template <int DT, int G, int VPL>
__global__ __launch_bounds__(kThreads) void k_route_one(RouteParams p) {
  constexpr int EP = G * VPL;
  __shared__ RouteShared<EP> sh;
  choose<DT, G, VPL>(p, 0, p.tokens, sh);
  for (int e = threadIdx.x; e < EP; e += kThreads) sh.total[e] = sh.run[e];
  __threadfence_block();
  __syncthreads();
  const int rows = prefix_experts(sh);
  place(p, 0, p.tokens, sh.total);
  for (int r = rows + threadIdx.x; r < p.tokens * p.topk; r += kThreads) p.row_index[r] = -1;
  publish(p, sh, sh.run, rows, sh.valid);
}

template <int DT, int G, int VPL>
__global__ __launch_bounds__(kThreads) void k_route_choose(RouteParams p) {
  constexpr int EP = G * VPL;
  __shared__ RouteShared<EP> sh;
  const int b = blockIdx.x;
  const int t0 = b * p.per, t1 = t0 + p.per < p.tokens ? t0 + p.per : p.tokens;
  choose<DT, G, VPL>(p, t0, t1, sh);
  for (int e = threadIdx.x; e < p.experts; e += kThreads) {
    p.part_counts[(int64_t)b * p.experts + e] = (uint16_t)sh.run[e];
    p.part_sums[(int64_t)b * p.experts + e] = sh.sums[0][e];
  }
  if (threadIdx.x == 0) p.part_valid[b] = sh.valid;
}

// Blocks 0 .. blocks-1 place their tokens' rows; block `blocks` reduces the
// sums and publishes.  Each adds up the counts of all blocks for itself: 64 K
// counts at most, which come out of L2.
template <int EP>
__global__ __launch_bounds__(kThreads) void k_route_place(RouteParams p) {
  __shared__ RouteShared<EP> sh;
  const int b = blockIdx.x, E = p.experts;
  for (int e = threadIdx.x; e < EP; e += kThreads) {
    sh.total[e] = 0;
    sh.run[e] = 0;
  }
  if (threadIdx.x == 0) sh.valid = 0;
  __syncthreads();
  constexpr int LANES = EP < kThreads ? EP : kThreads;  // threads along the experts
  constexpr int STEP = kThreads / LANES;                // blocks read at once
  for (int e = threadIdx.x % LANES; e < E; e += LANES) {
    int all = 0, before = 0;
    for (int i = threadIdx.x / LANES; i < p.blocks; i += STEP) {
      const int c = p.part_counts[(int64_t)i * E + e];
      all += c;
      before += i < b ? c : 0;
    }
    atomicAdd(&sh.total[e], all);
    atomicAdd(&sh.run[e], before);
  }
  __syncthreads();
  if (b == p.blocks) {
    // (before == all here: sh.run holds the counts)
    for (int e = threadIdx.x; e < E; e += kThreads) {
      float s = 0.0f;
      for (int i = 0; i < p.blocks; ++i) s += p.part_sums[(int64_t)i * E + e];
      sh.sums[0][e] = s;
    }
    for (int i = threadIdx.x; i < p.blocks; i += kThreads) atomicAdd(&sh.valid, p.part_valid[i]);
  }
  const int rows = prefix_experts(sh);
  if (b == p.blocks) {
    publish(p, sh, sh.run, rows, sh.valid);
    return;
  }
  for (int e = threadIdx.x; e < E; e += kThreads) sh.run[e] += sh.total[e];
  __syncthreads();
  const int t0 = b * p.per, t1 = t0 + p.per < p.tokens ? t0 + p.per : p.tokens;
  place(p, t0, t1, sh.run);
  const int64_t n = (int64_t)p.tokens * p.topk;
  for (int64_t r = rows + (int64_t)b * kThreads + threadIdx.x; r < n; r += (int64_t)p.blocks * kThreads)
    p.row_index[r] = -1;
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

template <int DT, int G, int VPL>
__global__ __launch_bounds__(kBwdThreads) void k_route_bwd(RouteBwdParams b) {
  constexpr int EP = G * VPL;
  constexpr int GROUPS = kBwdThreads / G;
  __shared__ __attribute__((aligned(16))) float extra[GROUPS][EP];
  const RouteParams& p = b.f;
  const int gl = threadIdx.x & (G - 1), grp = threadIdx.x / G;
  const int e0 = gl * VPL, k = p.topk;
  const float v = (float)*p.valid;
  const float scale = b.d_loss && v > 0.0f ? *b.d_loss * ((float)p.experts / ((float)k * v)) / v : 0.0f;
  float bal[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) bal[i] = e0 + i < p.experts ? scale * (float)p.counts[e0 + i] : 0.0f;
  for (int64_t t0 = (int64_t)blockIdx.x * GROUPS; t0 < p.tokens; t0 += (int64_t)gridDim.x * GROUPS) {
    const int64_t t = t0 + grp;
    const bool ok = t < p.tokens && (!p.mask || p.mask[t] != 0);
    float x[VPL];
    if (ok) {
      load_scores<DT, VPL>(p, t, e0, x);
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) x[i] = -__builtin_inff();
    }
    // this lane's slot
    int e = -1;
    float dw = 0.0f, xe = 0.0f;
    if (ok && gl < k) {
      e = p.experts_out[t * k + gl];
      e = e < p.experts ? e : -1;
      if (e >= 0) {
        dw = b.d_weights ? b.d_weights[t * k + gl] : 0.0f;
        xe = load1<DT>(p.logits, t * p.ld + e);
      }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) extra[grp][e0 + i] = 0.0f;
    float m = x[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = __builtin_fmaxf(m, x[i]);
    m = group_reduce<G>(__builtin_fmaxf(m, -__builtin_inff()), OpMax());
    m = m == -__builtin_inff() ? 0.0f : m;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      x[i] = __builtin_amdgcn_exp2f((x[i] - m) * kLog2e);
      s += x[i];
    }
    s = group_reduce<G>(s, OpAdd());
    const float inv = s == 0.0f ? 0.0f : 1.0f / s;
    float pb = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      x[i] *= inv;
      pb = fmaf(x[i], bal[i], pb);
    }
    pb = group_reduce<G>(pb, OpAdd());
    float q = e >= 0 ? __builtin_amdgcn_exp2f((xe - m) * kLog2e) : 0.0f;
    if (p.normalize) {
      const float sq = group_reduce<G>(q, OpAdd());
      q = e >= 0 ? q / sq : 0.0f;
    } else {
      q *= inv;
    }
    const float qd = group_reduce<G>(q * dw, OpAdd());
    if (!p.normalize) pb += qd;
    if (e >= 0) extra[grp][e] = p.normalize ? q * (dw - qd) : q * dw;
    __syncthreads();
    if (t < p.tokens) {
      float o[VPL];
#pragma unroll
      for (int i = 0; i < VPL; ++i) o[i] = fmaf(x[i], bal[i] - pb, extra[grp][e0 + i]);
      const int64_t off = t * b.ld_d + e0;
      if (VPL >= 8 && b.vec_d && e0 + VPL <= p.experts) {
        if constexpr (VPL >= 8) {
#pragma unroll
          for (int i = 0; i < VPL; i += 8) {
            float y[8];
#pragma unroll
            for (int h = 0; h < 8; ++h) y[h] = o[i + h];
            store8<DT>(b.d_logits, off + i, y);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (e0 + i < p.experts) store1<DT>(b.d_logits, off + i, o[i]);
      }
    }
    __syncthreads();
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
    hipLaunchKernelGGL((k_route_one<DT, G, VPL>), dim3(1), dim3(kThreads), 0, s, p);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((k_route_choose<DT, G, VPL>), dim3(p.blocks), dim3(kThreads), 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_route_place<G * VPL>), dim3(p.blocks + 1), dim3(kThreads), 0, s, p);
  return hipGetLastError();
}

template <int DT, int G, int VPL>
hipError_t route_bwd_v(const RouteBwdParams& p, hipStream_t s) {
  constexpr int GROUPS = kBwdThreads / G;
  const int64_t need = ((int64_t)p.f.tokens + GROUPS - 1) / GROUPS;
  hipLaunchKernelGGL((k_route_bwd<DT, G, VPL>), dim3((uint32_t)(need < 2048 ? need : 2048)), dim3(kBwdThreads), 0, s,
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
  const size_t cells = (size_t)blocks * (size_t)experts;
  return (cells * sizeof(float) + (size_t)blocks * sizeof(int32_t) + cells * sizeof(uint16_t) + 15) / 16 * 16;
}

hipError_t launch_route(const RouteArgs& a, void* workspace, hipStream_t s) {
  RouteParams p = params_of(a);
  int64_t per, blocks;
  split(a.tokens, &per, &blocks);
  p.per = (int32_t)per;
  p.blocks = (int32_t)blocks;
  if (blocks > 1) {
    const size_t cells = (size_t)blocks * (size_t)a.experts;
    p.part_sums = static_cast<float*>(workspace);
    p.part_valid = reinterpret_cast<int32_t*>(p.part_sums + cells);
    p.part_counts = reinterpret_cast<uint16_t*>(p.part_valid + blocks);
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
