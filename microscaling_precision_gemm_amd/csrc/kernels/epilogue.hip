// epilogue.hip -- dropout, and the backward pass of a product's epilogue
//   out = residual + drop(act(z)):   d_z = drop'(d_out) act'(z),  d_bias = sum_r d_z[r, :]
// The mask is drawn again from its counters and never stored.
#include <type_traits>

#include "../device/act.h"
#include "../device/chunk8.h"

namespace mxk {

namespace {

constexpr int kThreads = 256;

// 8 columns a thread, whose draws are one Philox block.  HBM bounds it (16384 x 7168
// BF16 with residual 119 us, 5.9 TB/s; FP32 8192 x 7168 without 77 us, 6.1; some 170
// vector instructions a thread run beside that), a small call its launch (8 x 4096:
// 2.3 us).  Streaming stores: 1% of the first, 5% of the second.
template <int DT>
__global__ __launch_bounds__(kThreads) void k_dropout(DropoutArgs a, uint32_t per_row, bool vec_x, bool vec_r,
                                                      bool vec_o) {
  constexpr int U = kUnit<DT>, R = 8 / U;  // a thread's units: threadIdx.x and kThreads behind it
  const int64_t total = a.M * per_row;
  for (int64_t base = (int64_t)blockIdx.x * kThreads; base < total; base += (int64_t)gridDim.x * kThreads) {
    int64_t q[R], r[R], c[R];
    int n[R];
    raw16 x[R], res[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const uint32_t unit = threadIdx.x + k * kThreads;
      q[k] = base + unit / R;
      r[k] = q[k] / per_row;
      c[k] = (q[k] - r[k] * per_row) * 8 + unit % R * U;
      n[k] = q[k] < total ? (int)(a.N - c[k] < U ? a.N - c[k] : U) : 0;
      x[k] = load_unit<DT>(a.x, r[k] * a.ld_x + c[k], n[k], vec_x);
      if (a.residual) res[k] = load_unit<DT>(a.residual, r[k] * a.ld_r + c[k], n[k], vec_r);
    }
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = unit_value<DT>(x[i / U], i % U);
    if (a.drop.threshold) {
      if constexpr (R == 1) drop_chunk(a.drop, (uint64_t)q[0], v);
      else drop_halves(a.drop, (uint64_t)q[0], (uint64_t)q[1], v);
    }
    if (a.residual) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = unit_value<DT>(res[i / U], i % U) + v[i];
    }
#pragma unroll
    for (int k = 0; k < R; ++k) store_unit<DT>(a.out, r[k] * a.ld_o + c[k], n[k], vec_o, v + k * U);
  }
}

// A workgroup takes `tx` chunks of 8 columns and kThreads / tx rows at a time, in
// turn with the other workgroups of those columns, so that all of them together
// sweep the matrices (16384 x 14336 BF16 silu 277 us, 5.1 TB/s; runs of rows of
// their own 286; 1792 workgroups 2048 columns wide 311).  Each thread sums its
// columns, then the threads of one chunk are added in order through LDS.  HBM bounds
// it, with the slopes' arithmetic close behind (gelu takes 32 vector instructions an
// element, silu with dropout 31).  FP32 goes by units of 16 bytes too, two rows a
// thread: in pieces of 32 bytes, whose two accesses each leave out every other
// unit, 4099 x 2047 with dropout took 29.9 us from HBM, now 24.4, of it 3.8 for the
// joining kernel; 8192 x 14336 took 314, now 295 (4.8 TB/s).
struct BwdPlan {
  uint32_t tx;       // chunks side by side, a power of two
  uint32_t stripes;  // workgroups along the columns
  uint32_t parts;    // workgroups that share a stripe's rows
};

inline BwdPlan plan_bwd(int64_t M, int64_t N) {
  const int64_t chunks = (N + 7) / 8;
  BwdPlan p;
  // Up to 128 rows: narrow workgroups that take all of them, since the second launch
  // costs more (64 x 4096 BF16 10.1 us with it, 7.4; 128 x 14336 10.3 and 7.6; at 256
  // rows 10.3 and 10.8).  Beyond 64 * 1024 chunks the wide ones are one part anyway.
  const bool few = M <= 128 && chunks <= 64 * 1024;
  const uint32_t widest = few ? 8 : 64;
  p.tx = 1;
  while (p.tx < widest && p.tx < chunks) p.tx *= 2;
  p.stripes = (uint32_t)((chunks + p.tx - 1) / p.tx);
  const int64_t ty = kThreads / p.tx;
  const int64_t parts = (1024 + p.stripes - 1) / p.stripes;  // workgroups that fill the card
  const int64_t most = (M + 4 * ty - 1) / (4 * ty);          // at least 4 rows a thread
  p.parts = few || most == 0 ? 1 : (uint32_t)(parts < most ? parts : most);
  return p;
}

template <int DT>
__global__ __launch_bounds__(kThreads) void k_epilogue_bwd(EpilogueBwdArgs a, BwdPlan p, float* sums, bool vec_do,
                                                           bool vec_z, bool vec_dz) {
  constexpr int U = kUnit<DT>, R = 8 / U;  // columns and rows of a thread at a time
  __shared__ float part[kThreads][U + 1];
  const uint32_t wide = p.tx * R, tx = threadIdx.x & (wide - 1), ty = threadIdx.x / wide, ny = kThreads / wide;
  const int64_t chunk = (int64_t)blockIdx.x * p.tx + tx / R, c = chunk * 8 + tx % R * U;
  const int64_t per_row = (a.N + 7) / 8;
  const int n = (int)(a.N - c < U ? a.N - c : U);  // (a chunk's second half may not be there)
  const int64_t step = (int64_t)ny * R * p.parts;
  float sum[U] = {};
  if (chunk < per_row)
    with_act(a.act, [&](auto kind) {
      constexpr int ACT = decltype(kind)::value;
      // (the next rows' operands are loaded before these are used)
      raw16 d_next[R] = {}, z_next[R] = {};
      auto load = [&](int64_t first) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
          const int64_t r = first + k * ny;
          if (r >= a.M) return;
          d_next[k] = load_unit<DT>(a.d_out, r * a.ld_do + c, n, vec_do);
          if constexpr (ACT != ACT_NONE) z_next[k] = load_unit<DT>(a.z, r * a.ld_z + c, n, vec_z);
        }
      };
      const int64_t r0 = (int64_t)blockIdx.y * ny * R + ty;
      load(r0);
      for (int64_t r = r0; r < a.M; r += step) {
        raw16 dr[R], zr[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
          dr[k] = d_next[k];
          zr[k] = z_next[k];
        }
        load(r + step);
        float d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          d[i] = unit_value<DT>(dr[i / U], i % U);
          if constexpr (ACT != ACT_NONE) d[i] *= act_slope<ACT>(unit_value<DT>(zr[i / U], i % U));
        }
        if (a.drop.threshold) {
          const uint64_t q = (uint64_t)(r * per_row + chunk);
          if constexpr (R == 1) drop_chunk(a.drop, q, d);
          else drop_halves(a.drop, q, q + (uint64_t)(ny * per_row), d);
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
          if (r + k * ny >= a.M) break;
#pragma unroll
          for (int i = 0; i < U; ++i) sum[i] += d[k * U + i];
          if (a.d_z) store_unit<DT>(a.d_z, (r + k * ny) * a.ld_dz + c, n, vec_dz, d + k * U);
        }
      }
    });
  if (!sums) return;
#pragma unroll
  for (int i = 0; i < U; ++i) part[threadIdx.x][i] = sum[i];
  __syncthreads();
  if (ty == 0) {
    for (uint32_t y = 1; y < ny; ++y)
#pragma unroll
      for (int i = 0; i < U; ++i) sum[i] += part[y * wide + tx][i];
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (i < n) sums[(int64_t)blockIdx.y * a.N + c + i] = sum[i];
  }
}

// d_bias[c] = the sum over the parts: 16 threads a column take every 16th,
// whose sums are added in order.  (One thread a column waits for each of them in
// turn: 110 of 156 us for 4099 x 2047 FP32.)
__global__ __launch_bounds__(kThreads) void k_join_sums(const float* __restrict__ parts, uint32_t n, int64_t N,
                                                        float* __restrict__ out) {
  __shared__ float part[16][17];
  const uint32_t x = threadIdx.x & 15u, y = threadIdx.x >> 4;
  const int64_t c = (int64_t)blockIdx.x * 16 + x;
  float s = 0.0f;
  if (c < N)
#pragma unroll 8
    for (uint32_t i = y; i < n; i += 16) s += parts[i * N + c];
  part[y][x] = s;
  __syncthreads();
  if (y != 0 || c >= N) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) s += part[i][x];
  out[c] = s;
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs& a, hipStream_t s) {
  const int64_t per_row = (a.N + 7) / 8;
  const int64_t blocks = (a.M * per_row + kThreads - 1) / kThreads;
  const dim3 grid((uint32_t)(blocks < 65536 ? blocks : 65536));
  const bool vx = rows_aligned16(a.x, a.ld_x, a.dt), vr = rows_aligned16(a.residual, a.ld_r, a.dt),
             vo = rows_aligned16(a.out, a.ld_o, a.dt);
  if (a.dt == DT_BF16)
    hipLaunchKernelGGL((k_dropout<DT_BF16>), grid, dim3(kThreads), 0, s, a, (uint32_t)per_row, vx, vr, vo);
  else
    hipLaunchKernelGGL((k_dropout<DT_F32>), grid, dim3(kThreads), 0, s, a, (uint32_t)per_row, vx, vr, vo);
  return hipGetLastError();
}

size_t epilogue_workspace(int64_t M, int64_t N) {
  if (M == 0 || N == 0) return 0;
  const BwdPlan p = plan_bwd(M, N);
  return p.parts > 1 ? (size_t)p.parts * (size_t)N * sizeof(float) : 0;
}

hipError_t launch_epilogue_bwd(const EpilogueBwdArgs& a, hipStream_t s) {
  const BwdPlan p = plan_bwd(a.M, a.N);
  float* sums = !a.d_bias ? nullptr : p.parts > 1 ? a.parts : a.d_bias;
  const dim3 grid(p.stripes, p.parts);
  const bool vd = rows_aligned16(a.d_out, a.ld_do, a.dt), vz = rows_aligned16(a.z, a.ld_z, a.dt),
             vo = rows_aligned16(a.d_z, a.ld_dz, a.dt);
  if (a.dt == DT_BF16)
    hipLaunchKernelGGL((k_epilogue_bwd<DT_BF16>), grid, dim3(kThreads), 0, s, a, p, sums, vd, vz, vo);
  else
    hipLaunchKernelGGL((k_epilogue_bwd<DT_F32>), grid, dim3(kThreads), 0, s, a, p, sums, vd, vz, vo);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && a.d_bias && p.parts > 1) {
    hipLaunchKernelGGL(k_join_sums, dim3((uint32_t)((a.N + 15) / 16)), dim3(kThreads), 0, s, a.parts, p.parts, a.N,
                       a.d_bias);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace mxk
