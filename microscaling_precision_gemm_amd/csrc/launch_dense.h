// launch_dense.h -- internal launchers of the operators of a dense layer and of
// a head that scores tokens, as in launch.h (and apart from it: measurements of
// the GEMMs are kept by the state of the headers they include).
#pragma once
#include "launch.h"

namespace mxk {

enum Act { ACT_NONE = 0, ACT_RELU = 1, ACT_SILU = 2, ACT_GELU = 3, ACT_GELU_TANH = 4 };

// Dropout: an element whose 16 random bits are below `threshold` is dropped,
// the others are multiplied by `factor` = 65536 / (65536 - threshold).
// threshold 0: no dropout.
struct Drop {
  uint32_t threshold;
  float factor;
  uint64_t seed, counter;
};

// What follows the sum of a product: out = residual + drop(act(z)), z = sum +
// bias, all [M, N] of dtype dt.
struct Epilogue {
  const void* bias;  // [N] of bias_dt, or nullptr
  int bias_dt;
  int act;
  void* z;  // or nullptr
  int64_t ld_z;
  const void* residual;  // or nullptr; may be out
  int64_t ld_r;
  void* out;
  int64_t ld_o;
  int dt;
  Drop drop;
};

// X [M, K] (BF16, 16-byte aligned rows) times the transpose of block-scaled
// weights [N, K] in the row layout (linear.hip): fmt E4M3, E5M2, INT8, E2M1 or
// NVFP4; K % 32 == 0.
struct LinearArgs {
  const uint16_t* x;
  int64_t ld_x, M, N, K;
  int fmt;
  const uint8_t* codes;
  const uint8_t* scales;
  const float* tensor_scale;  // NVFP4
  Epilogue ep;
};
hipError_t launch_linear(const LinearArgs& a, hipStream_t s);

// Backward pass of the epilogue (epilogue.hip): d_z = d_out * drop' * act'(z),
// d_bias = sum of its rows.  z may be nullptr for ACT_NONE, d_z or d_bias when
// not wanted.  parts: epilogue_workspace(M, N) bytes where d_bias is wanted.
struct EpilogueBwdArgs {
  const void* d_out;
  int dt;
  int64_t ld_do, M, N;
  const void* z;
  int64_t ld_z;
  int act;
  Drop drop;
  void* d_z;
  int64_t ld_dz;
  float* d_bias;
  float* parts;
};
size_t epilogue_workspace(int64_t M, int64_t N);
hipError_t launch_epilogue_bwd(const EpilogueBwdArgs& a, hipStream_t s);

// out = residual + drop(x), [M, N] of dtype dt (epilogue.hip)
struct DropoutArgs {
  const void* x;
  int64_t ld_x, M, N;
  const void* residual;  // or nullptr
  int64_t ld_r;
  void* out;
  int64_t ld_o;
  int dt;
  Drop drop;
};
hipError_t launch_dropout(const DropoutArgs& a, hipStream_t s);

// Log probabilities of given tokens (logprob.hip).
struct LogprobArgs {
  const void* logits;
  int dt;
  int64_t ld, tokens, vocab;
  const int64_t* target;  // or nullptr
  float scale;
  int32_t topk;
  float* logp;  // or nullptr (target nullptr)
  float* entropy;
  float* row_max;
  float* log_sum;
  int32_t* top_id;
  float* top_logp;
};
constexpr int kMaxAlternatives = 32;
// workspace: logprob_workspace(tokens, vocab, topk) bytes
size_t logprob_workspace(int64_t tokens, int64_t vocab, int32_t topk);
hipError_t launch_logprob(const LogprobArgs& a, void* workspace, hipStream_t s);
// d_logp, d_entropy: [tokens] or nullptr
hipError_t launch_logprob_bwd(const LogprobArgs& a, const float* d_logp, const float* d_entropy, void* d_logits,
                              int64_t ld_d, hipStream_t s);

}  // namespace mxk
