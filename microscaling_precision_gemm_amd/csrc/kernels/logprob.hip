// logprob.hip -- log probabilities of given tokens, with the entropy of each row
// and its largest entries, and their gradient.  For a row x, s the scale, m its
// largest entry, d_v = s (x_v - m) and S = sum_v e^d_v:
//   log p_v = d_v - log S,   H = log S - (sum_v e^d_v d_v) / S
//   d_x_v   = s (d_logp (delta_v,target - p_v) - d_entropy p_v (log p_v + H))
// One pass over the row: a lane keeps the largest entry it has seen and both sums
// relative to it, and rescales them when it changes.  d is held at -150 and above:
// e^d is 0 there, and 0 times it too, so entries of minus infinity add nothing.
//
// The k largest entries cost that pass nothing.  It leaves the lanes' maxima
// behind; the k-th largest of 64 groups of them is no larger than the k-th largest
// entry, and only lanes whose maximum reaches it hold entries that do: k lanes or a
// few more, whose entries are read once more (1 / 20 of a row for k = 20).  Those
// that reach the bound are collected in LDS and ranked by their keys: an entry's
// value in an order of integers above its index's complement, so equal entries go
// by lower index.  Where ties make more of them than LDS holds, each wave keeps a
// sorted list instead, one key a lane, and the lists are ranked.  (Lists kept during
// the pass: 436 us for 4096 x 128000 BF16 and k = 5, now 190; 27.5 for one token's
// 50257 and k = 20, now 9.9.)
//
// HBM bounds a batch (4096 x 128000 BF16 190 us, 5.5 TB/s; 2048 x 128000 FP32 175 us,
// 6.0 TB/s) with the vector unit right behind it (11 instructions a BF16 entry, and an
// exponential counts four times), one CU's vector unit and the steps after the pass a
// single row: of the 9.3 us for 50257 entries with 20 alternatives, 2.7 find these.
// Sixteen waves for a row instead of eight take longer (11.5 us).
#include "../device/chunk8.h"
#include "../device/exp.h"
#include "../device/wave.h"

namespace mxk {

namespace {

constexpr float kLn2 = 0.693147180559945309417f;
constexpr float kLowest = -3.402823466e38f;  // where a running maximum starts

// An integer order of FP32 values (-0 as 0); -inf, NaN: 0.
__device__ inline uint32_t order_of(float x) {
  const uint32_t u = f2u(x + 0.0f);
  const uint32_t o = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  return x > -__builtin_inff() ? o : 0u;
}
__device__ inline float value_of(uint32_t o) { return u2f(o & 0x80000000u ? o ^ 0x80000000u : ~o); }

__device__ inline uint64_t lane_read64(uint64_t v, uint32_t src) {
  return (uint64_t)lane_read((uint32_t)(v >> 32), src) << 32 | lane_read((uint32_t)v, src);
}
__device__ inline uint64_t uniform64(uint64_t v, int lane) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 |
         (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}

// The k largest keys seen by a wave, one a lane in falling order (0: none).
struct TopList {
  uint64_t key = 0;
  uint64_t kth = 0;  // the k-th (uniform)
  __device__ void insert(uint64_t c, uint32_t lane, int k) {
    if (c <= kth) return;
    const uint32_t at = (uint32_t)__popcll(__builtin_amdgcn_ballot_w64(key > c));
    const uint64_t above = lane_read64(key, lane - 1u);
    key = lane < at ? key : lane == at ? c : above;
    kth = uniform64(key, k - 1);
  }
};

// The largest 16-bit prefix T (as the top half of a word, the rest 0) such that at
// least k lanes have v >= T; 0 if fewer lanes have any.
__device__ inline uint32_t kth_prefix(uint32_t v, int k) {
  uint32_t t = 0;
#pragma unroll
  for (int b = 31; b >= 16; --b) {
    const uint32_t c = t | (1u << b);
    if (__popcll(__builtin_amdgcn_ballot_w64(v >= c)) >= k) t = c;
  }
  return t;
}

// Takes a strip of 512 entries, 8 consecutive ones a lane, the lane's first at
// index `base`; those below `bound` (as order_of) cannot be among the k largest.
// Strips come in the order of their indexes, so that of equal entries the first
// stay.
__device__ inline void take_strip(TopList& list, const float (&v)[8], float largest, int64_t base, uint32_t bound,
                                  uint32_t lane, int k) {
  const uint32_t kth = (uint32_t)(list.kth >> 32) + (list.kth != 0);  // (an equal one loses to the list's)
  bound = kth > bound ? kth : bound;
  const uint32_t mine = order_of(largest);
  bound = bound > 0 ? bound : 1u;
  const uint64_t some = __builtin_amdgcn_ballot_w64(mine >= bound);
  if (some == 0) return;
  if (__popcll(some) > k) {  // many: only what the k-th largest of the lanes' maxima allows can stay
    const uint32_t t = kth_prefix(mine, k);
    bound = t > bound ? t : bound;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t o = order_of(v[i]);
    uint64_t rest = __builtin_amdgcn_ballot_w64(o >= bound);
    while (rest) {
      const int src = __builtin_ctzll(rest);
      rest &= rest - 1;
      const uint32_t value = (uint32_t)__builtin_amdgcn_readlane((int)o, src);
      const uint32_t index = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)base, src) + i;
      list.insert((uint64_t)value << 32 | ~index, lane, k);
    }
  }
}

// Running statistics: the largest entry, the sum of e^d and of e^d d / ln 2.  e^d is the
// hardware's exponential of (x - m) c as rounded, which is off by 2 units of 2^-24, |d|
// for the product and 1.2 |d| for c: of log S that leaves 2 units on average, as much
// as exponentials of d itself do, since most roundings cancel in the sum.  The
// exponential of exp.h, which the backward pass can afford, is 3 to 4 instructions
// more an entry: 4096 x 128000 BF16 232 us instead of 185, for a mean error of log S of
// 1.5e-7 instead of 1.9e-7; so the two passes' p differ by these units.
struct Stats {
  float m = kLowest, s = 0.0f, w = 0.0f;
  // the same relative to a maximum `to` >= m; c = scale / ln 2
  __device__ void move(float to, float c) {
    const float d = __builtin_elementwise_maximum((m - to) * c, -216.0f);
    const float f = __builtin_amdgcn_exp2f(d);
    w = f * fmaf(d, s, w);
    s *= f;
    m = to;
  }
  // 16 more entries, summed among themselves first
  __device__ void add(const float (&v)[16], float largest, float c) {
    move(fmaxf(m, largest), c);
    float s1, w1;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float d = __builtin_elementwise_maximum((v[i] - m) * c, -216.0f);
      const float e = __builtin_amdgcn_exp2f(d);
      s1 = i == 0 ? e : s1 + e;
      w1 = i == 0 ? e * d : fmaf(e, d, w1);
    }
    s += s1;
    w += w1;
  }
  // what was summed behind this; its maximum is no smaller
  __device__ void append(const Stats& run, float c) {
    move(run.m, c);
    s += run.s;
    w += run.w;
  }
  __device__ void join(float m2, float s2, float w2, float c) {
    const float to = fmaxf(m, m2);
    move(to, c);
    Stats o;
    o.m = m2;
    o.s = s2;
    o.w = w2;
    o.move(to, c);
    s += o.s;
    w += o.w;
  }
};

// Entries first .. first + 7 of a row as they lie in memory, those outside it as
// -inf; a chunk inside it is 16-byte aligned if `vec`.
template <int DT>
__device__ inline RawChunk load_part(const void* row, int64_t first, int64_t vocab, bool vec = true) {
  if (first >= 0 && first + 8 <= vocab) return load_raw8<DT>(row, first, 8, vec);
  constexpr uint32_t kNone = DT == DT_BF16 ? 0xFF80FF80u : 0xFF800000u;
  RawChunk r = {{kNone, kNone, kNone, kNone}, {kNone, kNone, kNone, kNone}};
  if (first >= vocab) return r;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (first + i >= 0 && first + i < vocab) {
      if constexpr (DT == DT_BF16) {
        const uint32_t u = static_cast<const uint16_t*>(row)[first + i];
        r.a[i / 2] = i & 1 ? (r.a[i / 2] & 0xFFFFu) | u << 16 : (r.a[i / 2] & 0xFFFF0000u) | u;
      } else (i < 4 ? r.a : r.b)[i & 3] = static_cast<const uint32_t*>(row)[first + i];
    }
  return r;
}
// entries by which a row starts past a 16-byte boundary
template <int DT>
__device__ inline int shift_of(const void* row) {
  return (int)((reinterpret_cast<uintptr_t>(row) & 15u) / (DT == DT_BF16 ? 2 : 4));
}
__device__ inline float max8(const float (&v)[8]) {
  return fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), fmaxf(fmaxf(v[4], v[5]), fmaxf(v[6], v[7])));
}

// What padding gets.
__device__ inline bool skip_padding(const LogprobArgs& a, int64_t t, int64_t target) {
  if (target >= 0 && target < a.vocab) return false;
  if (threadIdx.x == 0) {
    if (a.logp) a.logp[t] = 0.0f;
    a.entropy[t] = 0.0f;
    a.row_max[t] = 0.0f;
    a.log_sum[t] = 0.0f;
  }
  if ((int)threadIdx.x < a.topk) {
    a.top_id[t * a.topk + threadIdx.x] = -1;
    a.top_logp[t * a.topk + threadIdx.x] = -__builtin_inff();
  }
  return true;
}

// A row's results but the alternatives, from its sums; m and log S.
struct RowSums {
  float m, log_sum;
};
__device__ inline RowSums finish_row(const LogprobArgs& a, int64_t t, const Stats& all, float given) {
  // s is 0 only where no entry is above -inf (the largest one adds 1)
  const bool none = all.s == 0.0f;
  const float m = none ? -__builtin_inff() : all.m, log_sum = none ? 0.0f : logf(all.s);
  if (threadIdx.x == 0) {
    a.row_max[t] = m;
    a.log_sum[t] = log_sum;
    a.entropy[t] = none ? 0.0f : log_sum - kLn2 * (all.w / all.s);
    if (a.logp) a.logp[t] = none ? -__builtin_inff() : a.scale * (given - m) - log_sum;
  }
  return {m, log_sum};
}
__device__ inline void write_alternative(const LogprobArgs& a, int64_t t, uint32_t place, uint64_t key, RowSums r) {
  a.top_id[t * a.topk + place] = (int32_t)~(uint32_t)key;
  a.top_logp[t * a.topk + place] = a.scale * (value_of((uint32_t)(key >> 32)) - r.m) - r.log_sum;
}
// the places from n on
__device__ inline void no_alternatives(const LogprobArgs& a, int64_t t, uint32_t n) {
  if ((int)threadIdx.x < a.topk && threadIdx.x >= n) {
    a.top_id[t * a.topk + threadIdx.x] = -1;
    a.top_logp[t * a.topk + threadIdx.x] = -__builtin_inff();
  }
}

// What a workgroup leaves of its part of a row: the sums, then topk keys in falling
// order (0: none).
__device__ inline char* part_of(void* workspace, int64_t part, int topk) {
  return static_cast<char*>(workspace) + part * (16 + 8 * topk);
}

// A lane's sums have three levels: 16 entries, kRunSteps times 16, and the runs: 15 +
// 256 + 1024 roundings for the longest row and 15 + 7 for 50257 entries.  One level
// alone rounds once an entry: a lane that holds 1 and then 2^17 terms of e^-17.5 loses
// them all (2^26 entries: log S off by 1.2e-3), and the mean error of log S over 128000
// BF16 entries is 4.1e-7 instead of 1.9e-7.  The time is the same (4096 x 128000 BF16
// 185 us without alternatives both ways).
constexpr uint32_t kRunSteps = 256;

// One workgroup a row, or one of `parts` for a part of it each (SPLIT: few rows,
// which k_logprob_join puts together).  Lane t of its NW * 64 takes chunks t, t +
// NW * 64, ...
template <int DT, int NW, bool SPLIT>
__global__ __launch_bounds__(NW * 64) void k_logprob(LogprobArgs a, uint32_t parts, void* workspace) {
  constexpr int kLanes = NW * 64, kKeys = 512;
  static_assert(NW * kMaxAlternatives <= kKeys, "the waves' lists");
  __shared__ float part[3][NW];
  __shared__ uint32_t lane_max[kLanes];  // order_of the lanes' maxima; then lanes that reach the bound
  __shared__ uint32_t bound_of, reach[NW], found;
  __shared__ uint64_t keys[kKeys];
  const int64_t t = SPLIT ? blockIdx.x / parts : blockIdx.x;
  const uint32_t lane = threadIdx.x & 63u, wid = threadIdx.x >> 6;
  const int k = a.topk;
  const int64_t target = a.target ? a.target[t] : 0;
  if constexpr (SPLIT) {
    if (target < 0 || target >= a.vocab) return;
  } else {
    if (skip_padding(a, t, target)) return;
  }
  const char* row = static_cast<const char*>(a.logits) + t * a.ld * (DT == DT_BF16 ? 2 : 4);
  const int shift = shift_of<DT>(row);
  const uint32_t all_chunks = (uint32_t)((a.vocab + shift + 7) / 8), number = SPLIT ? blockIdx.x % parts : 0;
  const uint32_t chunk0 = SPLIT ? (uint32_t)((uint64_t)all_chunks * number / parts) : 0;
  const uint32_t chunk1 = SPLIT ? (uint32_t)((uint64_t)all_chunks * (number + 1) / parts) : all_chunks;
  const uint32_t chunks = chunk1 - chunk0;
  const int64_t start = (int64_t)chunk0 * 8 - shift, stop = (int64_t)chunk1 * 8 - shift;
  const int64_t end = stop < a.vocab ? stop : a.vocab;
  const float c = a.scale * kLog2e;
  const float given = !SPLIT && threadIdx.x == 0 && a.logp ? load1<DT>(row, target) : 0.0f;
  Stats st;
  // two chunks at a time, the next two on their way
  auto chunk_at = [&](int64_t q) { return load_part<DT>(row, start + q * 8, end); };
  RawChunk n0 = chunk_at(threadIdx.x), n1 = chunk_at(threadIdx.x + kLanes);
  const uint32_t steps = (chunks + 2 * kLanes - 1) / (2 * kLanes);
  int64_t q = threadIdx.x;
  for (uint32_t i = 0; i < steps;) {
    const uint32_t until = steps - i < kRunSteps ? steps : i + kRunSteps;
    Stats run;
    run.m = st.m;
    for (; i < until; ++i, q += 2 * kLanes) {
      const RawChunk c0 = n0, c1 = n1;
      n0 = chunk_at(q + 2 * kLanes);
      n1 = chunk_at(q + 3 * kLanes);
      float v[16];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = raw_value<DT>(c0, j);
        v[8 + j] = raw_value<DT>(c1, j);
      }
      float largest = v[0];
#pragma unroll
      for (int j = 1; j < 16; ++j) largest = fmaxf(largest, v[j]);
      run.add(v, largest, c);
    }
    st.append(run, c);
  }
  const uint32_t mine = order_of(st.m);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const float m2 = u2f(lane_read(f2u(st.m), lane ^ off)), s2 = u2f(lane_read(f2u(st.s), lane ^ off)),
                w2 = u2f(lane_read(f2u(st.w), lane ^ off));
    // (the lower lane's first in both, so that both get the same bits)
    Stats o;
    const bool low = (lane & off) == 0;
    o.m = low ? st.m : m2;
    o.s = low ? st.s : s2;
    o.w = low ? st.w : w2;
    o.join(low ? m2 : st.m, low ? s2 : st.s, low ? w2 : st.w, c);
    st = o;
  }
  if (lane == 0) {
    part[0][wid] = st.m;
    part[1][wid] = st.s;
    part[2][wid] = st.w;
  }
  if (k > 0) lane_max[threadIdx.x] = mine;
  __syncthreads();
  Stats all;
  all.m = part[0][0];
  all.s = part[1][0];
  all.w = part[2][0];
#pragma unroll
  for (int i = 1; i < NW; ++i) all.join(part[0][i], part[1][i], part[2][i], c);
  RowSums sums = {};
  float* mine_out = nullptr;
  if constexpr (SPLIT) {
    mine_out = reinterpret_cast<float*>(part_of(workspace, blockIdx.x, k));
    if (threadIdx.x == 0) {
      mine_out[0] = all.m;
      mine_out[1] = all.s;
      mine_out[2] = all.w;
    }
  } else {
    sums = finish_row(a, t, all, given);
  }
  if (k == 0) return;

  // the bound: the upper 16 bits of the k-th largest of 64 maxima
  if (wid == 0) {
    uint32_t v = lane_max[lane];
#pragma unroll
    for (int i = 1; i < NW; ++i) {
      const uint32_t o = lane_max[i * 64 + lane];
      v = o > v ? o : v;
    }
    const uint32_t b = kth_prefix(v, k);
    if (lane == 0) {
      bound_of = b > 0 ? b : 1u;
      found = 0;
    }
  }
  __syncthreads();
  // the lanes that reach it, in order
  const uint32_t bound = bound_of;
  const uint64_t here = __builtin_amdgcn_ballot_w64(mine >= bound), below = (1ull << lane) - 1;
  if (lane == 0) reach[wid] = (uint32_t)__popcll(here);
  __syncthreads();
  uint32_t before = 0, lanes = 0;
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    if (i < (int)wid) before += reach[i];
    lanes += reach[i];
  }
  if (mine >= bound) lane_max[before + (uint32_t)__popcll(here & below)] = threadIdx.x;
  __syncthreads();
  // their chunks by index, 64 a strip and wave
  const uint32_t each = (chunks + kLanes - 1) / kLanes, total = each * lanes;
  auto strip = [&](uint32_t e0, float (&v)[8]) {
    const uint32_t e = e0 + lane, i = e / lanes;
    const int64_t first = e < total ? start + ((int64_t)lane_max[e - i * lanes] + (int64_t)i * kLanes) * 8 : end;
    const RawChunk r = load_part<DT>(row, first, end);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = raw_value<DT>(r, j);
    return first;
  };
  for (uint32_t e0 = wid * 64; e0 < total; e0 += kLanes) {
    float v[8];
    const int64_t first = strip(e0, v);
    if (__builtin_amdgcn_ballot_w64(order_of(max8(v)) >= bound) == 0) continue;
    uint64_t mask[8];
    uint32_t n = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      mask[j] = __builtin_amdgcn_ballot_w64(order_of(v[j]) >= bound);
      n += (uint32_t)__popcll(mask[j]);
    }
    uint32_t at = 0;
    if (lane == 0) at = atomicAdd(&found, n);
    at = (uint32_t)__builtin_amdgcn_readfirstlane(at);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t to = at + (uint32_t)__popcll(mask[j] & below);
      if ((mask[j] >> lane & 1) && to < kKeys) keys[to] = (uint64_t)order_of(v[j]) << 32 | ~(uint32_t)(first + j);
      at += (uint32_t)__popcll(mask[j]);
    }
  }
  __syncthreads();
  uint32_t n = found;
  if (n > kKeys) {  // (the same for all)
    TopList list;
    for (uint32_t e0 = wid * 64; e0 < total; e0 += kLanes) {
      float v[8];
      const int64_t first = strip(e0, v);
      take_strip(list, v, max8(v), first, bound, lane, k);
    }
    __syncthreads();
    if ((int)lane < k) keys[wid * k + lane] = list.key;
    n = NW * k;
    __syncthreads();
  }
  // a key's place is the number of larger ones (the lists hold k keys: more than
  // that many were found)
  uint64_t* keys_out = SPLIT ? reinterpret_cast<uint64_t*>(mine_out + 4) : nullptr;
  for (uint32_t i = threadIdx.x; i < n; i += kLanes) {
    const uint64_t key = keys[i];
    uint32_t place = 0;
#pragma unroll 4
    for (uint32_t j = 0; j < n; ++j) place += keys[j] > key;
    if (key && place < (uint32_t)k) {
      if constexpr (SPLIT) keys_out[place] = key;
      else write_alternative(a, t, place, key, sums);
    }
  }
  if constexpr (SPLIT) {
    if ((int)threadIdx.x < k && threadIdx.x >= n) keys_out[threadIdx.x] = 0;
  } else {
    no_alternatives(a, t, n);
  }
}

// The parts of a row put together, their sums in order; of their keys those that
// reach the upper 16 bits of the k-th largest are ranked.
constexpr int kMaxParts = 32;  // (8 threads each)
template <int DT>
__global__ __launch_bounds__(256) void k_logprob_join(LogprobArgs a, uint32_t parts, void* workspace) {
  __shared__ uint64_t every[kMaxParts * kMaxAlternatives], keys[kMaxParts * kMaxAlternatives], bound_of;
  __shared__ float part[kMaxParts][3];
  __shared__ uint32_t found;
  const int64_t t = blockIdx.x;
  const int k = a.topk;
  const int64_t target = a.target ? a.target[t] : 0;
  if (skip_padding(a, t, target)) return;
  const float c = a.scale * kLog2e;
  const char* row = static_cast<const char*>(a.logits) + t * a.ld * (DT == DT_BF16 ? 2 : 4);
  const float given = threadIdx.x == 0 && a.logp ? load1<DT>(row, target) : 0.0f;
  // 8 threads a part fetch what it left
  const uint32_t p0 = threadIdx.x / 8, l0 = threadIdx.x % 8;
  if (p0 < parts) {
    const char* from = part_of(workspace, t * parts + p0, k);
    if (l0 < 3) part[p0][l0] = reinterpret_cast<const float*>(from)[l0];
    for (int i = l0; i < k; i += 8) every[p0 * k + i] = reinterpret_cast<const uint64_t*>(from + 16)[i];
  }
  if (threadIdx.x == 0) found = 0;
  __syncthreads();
  Stats all;
  for (uint32_t p = 0; p < parts; ++p) all.join(part[p][0], part[p][1], part[p][2], c);
  const RowSums sums = finish_row(a, t, all, given);
  if (k == 0) return;
  if (threadIdx.x < 64) {  // (one wave)
    constexpr int kEach = kMaxParts * kMaxAlternatives / 64;
    uint32_t v[kEach], bound = 0;
    const int rows = (int)(parts * k + 63) / 64;
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      v[i] = i * 64 + threadIdx.x < parts * k ? (uint32_t)(every[i * 64 + threadIdx.x] >> 32) : 0;
#pragma unroll 1
    for (int b = 31; b >= 16; --b) {
      const uint32_t next = bound | (1u << b);
      int n = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (i < rows) n += __popcll(__builtin_amdgcn_ballot_w64(v[i] >= next));
      if (n >= k) bound = next;
    }
    if (threadIdx.x == 0) bound_of = bound > 0 ? (uint64_t)bound << 32 : 1;
  }
  __syncthreads();
  const uint64_t bound = bound_of;
  for (uint32_t i = threadIdx.x; i < parts * k; i += 256)
    if (every[i] >= bound) keys[atomicAdd(&found, 1u)] = every[i];
  __syncthreads();
  const uint32_t n = found;
  for (uint32_t i = threadIdx.x; i < n; i += 256) {
    const uint64_t key = keys[i];
    uint32_t place = 0;
#pragma unroll 4
    for (uint32_t j = 0; j < n; ++j) place += keys[j] > key;
    if (place < (uint32_t)k) write_alternative(a, t, place, key, sums);
  }
  no_alternatives(a, t, n);
}

// The gradient: what a thread takes follows from the saved sums and nothing is
// exchanged, so HBM bounds it (4096 x 128000 BF16 372 us, 5.6 TB/s; 2048 x 128000
// FP32 343, 6.1; 509 x 50257 FP32 40, 5.1).  Lanes take 16 bytes next to each other
// in both types: FP32 in pieces of 32 bytes, as two accesses that leave every other
// one out, took 414 and 50 us.  Streaming stores are worth 4% (BF16 386 us without);
// half the units a thread cost as much (383 us; FP32 354 with twice as many).
template <int DT>
constexpr int kBwdUnits = DT == DT_BF16 ? 4 : 2;  // units of a thread
template <int DT>
constexpr int kBwdPart = 256 * kBwdUnits<DT>;     // of a workgroup

template <int DT>
__global__ __launch_bounds__(256) void k_logprob_bwd(LogprobArgs a, const float* __restrict__ d_logp,
                                                     const float* __restrict__ d_entropy, void* d_logits, int64_t ld_d,
                                                     uint32_t parts) {
  constexpr int EB = DT == DT_BF16 ? 2 : 4, U = kUnit<DT>;  // bytes of an entry, entries of a unit
  const int64_t total = a.tokens * parts;
  for (int64_t id = blockIdx.x; id < total; id += gridDim.x) {
    const int64_t t = id / parts, q0 = (id - t * parts) * kBwdPart<DT> + threadIdx.x;
    const char* row = static_cast<const char*>(a.logits) + t * a.ld * EB;
    char* out = static_cast<char*>(d_logits) + t * ld_d * EB;
    const int shift = shift_of<DT>(out);
    const bool vec_in = shift_of<DT>(row) == shift;
    const int64_t target = a.target ? a.target[t] : -1;
    const float m = a.row_max[t], log_sum = a.log_sum[t], H = a.entropy[t];
    const bool nothing = (a.target && (target < 0 || target >= a.vocab)) || m == -__builtin_inff();
    const float dl = a.target && d_logp ? a.scale * d_logp[t] : 0.0f;
    const float dh = d_entropy ? a.scale * d_entropy[t] : 0.0f;
#pragma unroll
    for (int u = 0; u < kBwdUnits<DT>; ++u) {
      const int64_t first = (q0 + u * 256) * U - shift;
      if (first >= a.vocab) break;
      float v[U];
      const bool whole = first >= 0 && first + U <= a.vocab;
      if (nothing) {
#pragma unroll
        for (int i = 0; i < U; ++i) v[i] = 0.0f;
      } else {
        if (whole && vec_in) {
          const raw16 r = load_unit<DT>(row, first, U, true);
#pragma unroll
          for (int i = 0; i < U; ++i) v[i] = unit_value<DT>(r, i);
        } else {
#pragma unroll
          for (int i = 0; i < U; ++i)
            v[i] = first + i >= 0 && first + i < a.vocab ? load1<DT>(row, first + i) : -__builtin_inff();
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const float lp = __builtin_elementwise_maximum(fmaf(a.scale, v[i] - m, -log_sum), -150.0f);
          const float p = exp_nonpos(lp);
          const float d = -p * fmaf(dh, lp + H, dl);
          v[i] = first + i == target ? d + dl : d;
        }
      }
      if (whole) store_unit<DT>(out, first, U, true, v);
      else
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (first + i >= 0 && first + i < a.vocab) store1<DT>(out, first + i, v[i]);
    }
  }
}

}  // namespace

namespace {
// Parts that a row is scored in.  Few rows leave most of the device idle, and
// long ones keep it so: 1 x 262144 BF16 takes 23.4 us in one part and 7.6 in 16
// (27.9 and 14.8 with 20 alternatives), 128 x 128000 14.6 and 11.9.  A second
// kernel is what it costs, the more with alternatives to rank: 1 x 65536 takes 7.9
// us in one part and 7.5 in four, with 20 alternatives 10.4 and 12.8; 1 x 100000
// 14.2 and 13.8 with them, 64 x 128000 17.6 and 15.6, 128 x 100000 16.0 and 18.6.
// Parts of 16384 entries for few tokens (1 x 128000 with 20: 14.2 us, of 8192
// 14.7, of 4096 16.2), of 8192 from 16 tokens on.
uint32_t parts_of(int64_t tokens, int64_t vocab, int32_t topk) {
  if (topk > 0 ? tokens > 64 || vocab < 98304 : tokens > 128 || vocab < 65536) return 1;
  const int64_t fill = (512 + tokens - 1) / tokens, most = vocab / (tokens < 16 ? 16384 : 8192);
  const int64_t p = fill < most ? fill : most;
  return (uint32_t)(p < kMaxParts ? p : kMaxParts);
}
}  // namespace

size_t logprob_workspace(int64_t tokens, int64_t vocab, int32_t topk) {
  const uint32_t parts = parts_of(tokens, vocab, topk);
  return parts > 1 ? (size_t)tokens * parts * (16 + 8 * (size_t)topk) : 0;
}

hipError_t launch_logprob(const LogprobArgs& a, void* workspace, hipStream_t s) {
  const uint32_t parts = parts_of(a.tokens, a.vocab, a.topk);
  const dim3 grid((uint32_t)a.tokens * parts);
#define MXK_LP(NW, SPLIT)                                                                                \
  do {                                                                                                   \
    if (a.dt == DT_BF16)                                                                                 \
      hipLaunchKernelGGL((k_logprob<DT_BF16, NW, SPLIT>), grid, dim3(NW * 64), 0, s, a, parts, workspace); \
    else                                                                                                 \
      hipLaunchKernelGGL((k_logprob<DT_F32, NW, SPLIT>), grid, dim3(NW * 64), 0, s, a, parts, workspace);  \
  } while (0)
  if (parts == 1) {
    if (a.vocab <= 4096) MXK_LP(1, false);
    else if (a.vocab <= 32768) MXK_LP(4, false);
    else MXK_LP(8, false);
    return hipGetLastError();
  }
  MXK_LP(4, true);
#undef MXK_LP
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.dt == DT_BF16)
    hipLaunchKernelGGL((k_logprob_join<DT_BF16>), dim3((uint32_t)a.tokens), dim3(256), 0, s, a, parts, workspace);
  else
    hipLaunchKernelGGL((k_logprob_join<DT_F32>), dim3((uint32_t)a.tokens), dim3(256), 0, s, a, parts, workspace);
  return hipGetLastError();
}

hipError_t launch_logprob_bwd(const LogprobArgs& a, const float* d_logp, const float* d_entropy, void* d_logits,
                              int64_t ld_d, hipStream_t s) {
  const int64_t unit = a.dt == DT_BF16 ? 8 : 4, part = a.dt == DT_BF16 ? kBwdPart<DT_BF16> : kBwdPart<DT_F32>;
  const int64_t parts = ((a.vocab + 2 * unit - 2) / unit + part - 1) / part;  // (a row may start inside a chunk)
  const int64_t total = a.tokens * parts;
  const dim3 grid((uint32_t)(total < (1 << 22) ? total : (1 << 22)));
  if (a.dt == DT_BF16)
    hipLaunchKernelGGL((k_logprob_bwd<DT_BF16>), grid, dim3(256), 0, s, a, d_logp, d_entropy, d_logits, ld_d,
                       (uint32_t)parts);
  else
    hipLaunchKernelGGL((k_logprob_bwd<DT_F32>), grid, dim3(256), 0, s, a, d_logp, d_entropy, d_logits, ld_d,
                       (uint32_t)parts);
  return hipGetLastError();
}

}  // namespace mxk
