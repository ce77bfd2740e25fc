// Internal launch interface of the feed-forward half of a decode step and of
// the model's answer: the residual's addition and norm, the gated projections,
// log probabilities.  Not part of the public ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace tq2 {

// ---- the residual's addition and RMS norm ----

struct NormArgs {
  const void* x;
  const void* residual;  // null: none
  void* h_out;           // null: not wanted
  const float* weight;   // null: ones
  void* out;             // of the output type, or int8
  float* scales;         // int8: a scale a token, written here (null: s)
  int64_t x_stride, r_stride;
  int64_t T;
  int32_t D;
  float eps, s;
};
// out_dtype: a tq2_dtype, or kOutI8
constexpr int kOutI8 = 3;
hipError_t launch_add_rms_norm(const NormArgs& a, int x_dtype, int r_dtype, int out_dtype, hipStream_t st);

// ---- the gated projections ----

struct GatedArgs {
  const uint8_t* codes[2];    // gate, up
  const uint16_t* scales[2];
  const void* x;              // fp16 or int8 [M][K]
  const float* x_scales;      // int8: a scale a token (null: s)
  float s;
  void* h;                    // [M][N]
  int64_t N, K, M;
  void* pieces;               // workspace
};
// Most bytes that a call keeps of its activations at a time (it takes its
// tokens in parts), enough for more than a GPU full of workgroups.
constexpr int64_t kGatedWorkspace = (int64_t)48 << 20;
size_t gated_workspace_bytes(int64_t K, int64_t M, bool int8);
hipError_t launch_gated(const GatedArgs& a, bool int8, int out_dtype, hipStream_t st);

// The form for one token: eight waves a workgroup, half of them on gate rows,
// each on four rows, which one, two or four waves share along K.  Its grid has
// up to N * 128 threads; a grid holds less than 2^32.  More rows than that go
// through the form for few tokens, whose workgroups take 32.
constexpr int kGatedOneRows = 4, kGatedOneThreads = 512;
constexpr int64_t kGridThreads = (int64_t)1 << 32;
inline int gated_one_waves(int64_t K) { return K <= 4096 ? 1 : K <= 8192 ? 2 : 4; }
inline int64_t gated_one_groups(int64_t N, int64_t K) {
  const int64_t rows = kGatedOneRows * 4 / gated_one_waves(K);
  return (N + rows - 1) / rows;
}
inline bool gated_one_fits(int64_t N, int64_t K) { return gated_one_groups(N, K) * kGatedOneThreads < kGridThreads; }

// ---- log probabilities ----

struct LogprobArgs {
  const void* logits;
  int64_t stride, T, V;
  float scale;
  float rate;              // scale * log2 e, set by the launch
  const int64_t* tokens;   // null: none
  float* logprobs;
  float* entropy;          // null: not wanted
  int64_t* top_tokens;     // null: top is 0
  float* top_logprobs;
  int32_t top;
  uint8_t* ws;
};
constexpr int kMaxTop = 64;  // a lane each
// Workgroups that share a row, and the bytes in which they leave their parts (0 for one).
int logprob_splits(int64_t T, int64_t V);
size_t logprob_workspace_bytes(int64_t T, int64_t V, int32_t top);
hipError_t launch_token_logprobs(const LogprobArgs& a, int dtype, hipStream_t st);

}  // namespace tq2
