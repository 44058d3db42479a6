// launch_moe.h -- internal launchers of the operators around the expert
// products of a mixture-of-experts layer, as in launch.h (and apart from it:
// measurements of the GEMMs are kept by the state of the headers they include).
#pragma once
#include "launch.h"

namespace mxk {

// Router (route.hip).  Sizes: 1 <= experts <= 1024, 1 <= topk <= 16, topk <=
// experts, tokens <= 2^23.  The backward pass reads logits, mask, experts_out,
// counts and valid.
struct RouteArgs {
  const void* logits;
  int dt;
  int64_t ld, tokens;
  int32_t experts, topk;
  const uint8_t* mask;  // nullptr: every token counts
  bool normalize;
  int32_t* experts_out;
  float* weights;
  int32_t* slot_row;
  int32_t* row_index;
  int64_t* offsets;
  int64_t* counts;
  int64_t* valid;
  float* prob_sum;
  float* loss;
};
size_t route_workspace(int64_t tokens, int32_t experts);
hipError_t launch_route(const RouteArgs& a, void* workspace, hipStream_t s);
hipError_t launch_route_bwd(const RouteArgs& a, const float* d_weights, const float* d_loss, void* d_logits,
                            int64_t ld_d, hipStream_t s);
// Weighted combination of routed rows (combine.hip) and its gradients.
hipError_t launch_combine(const void* y, int ydt, int64_t ld_y, int64_t rows, const int32_t* slot_row,
                          const float* weights, int64_t tokens, int topk, int64_t cols, void* out, int odt,
                          int64_t ld_out, hipStream_t s);
hipError_t launch_combine_bwd(const void* d_out, int dt, int64_t ld_do, const void* y, int64_t ld_y, int64_t rows,
                              const int32_t* slot_row, const float* weights, int64_t tokens, int topk,
                              int64_t cols, void* dy, int64_t ld_dy, float* d_weights, hipStream_t s);
// Gated activation with an 8-bit checkpoint (swiglu.hip).  fmt 0: nothing is
// saved; otherwise codes / scales of the [rows, 2 cols] tensor.
struct SwigluArgs {
  const void* h;
  int dt;
  int64_t rows, cols, ld_h;
  void* y;
  int64_t ld_y;
  int fmt;
  uint8_t* codes;
  uint8_t* scales;
  bool sr;
  uint64_t seed, counter;
  float* amax;  // or nullptr
};
hipError_t launch_swiglu(const SwigluArgs& a, hipStream_t s);
struct SwigluBwdArgs {
  int fmt;
  const uint8_t* codes;
  const uint8_t* scales;
  const void* dy;
  int dt;
  int64_t rows, cols, ld_dy;
  void* dh;
  int64_t ld_dh;
  int y_fmt;  // 0: y is not written
  uint8_t* y_codes;
  uint8_t* y_scales;
};
hipError_t launch_swiglu_bwd(const SwigluBwdArgs& a, hipStream_t s);
// Grouped weight gradient from an 8-bit checkpoint (wgrad.hip).
struct WgradArgs {
  const uint16_t* dy;
  int64_t ld_dy, R, N;
  int fmt;
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t x_rows, K;
  const int32_t* row_index;
  const int64_t* offsets;
  int32_t groups;
  void* dw;
  int dwdt;
  int64_t ld_dw;
  bool accumulate;
  float* parts;  // wgrad_workspace_bytes(R, N, K, groups) bytes
};
size_t wgrad_workspace_bytes(int64_t R, int64_t N, int64_t K, int64_t groups);
hipError_t launch_wgrad_grouped(const WgradArgs& a, hipStream_t s);

}  // namespace mxk
