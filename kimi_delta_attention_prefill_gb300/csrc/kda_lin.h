// kda_lin.h -- linear attention with a decay a head (include/kda.h): arguments as the kernels see
// them, and the launches.
#pragma once

#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "kda_internal.h"

namespace kda {

struct LinArgs {
  const void* q = nullptr;
  const void* k = nullptr;
  const void* v = nullptr;
  const float* g = nullptr;
  const void* gate = nullptr;  // bf16 gate logits: with the output stage
  // element strides: sequence (decode only), token, head
  int64_t q_stride[3] = {0, 0, 0};
  int64_t k_stride[3] = {0, 0, 0};
  int64_t v_stride[3] = {0, 0, 0};
  int64_t g_stride[3] = {0, 0, 0};
  int64_t gate_stride[3] = {0, 0, 0};
  float scale = 1.f;
  const float* norm_weight = nullptr;
  float eps = 0.f;
  const float* S_in = nullptr;
  float* S_out = nullptr;  // decode: the states, read and written
  const int32_t* cu = nullptr;        // prefill
  const int32_t* n_commit = nullptr;  // decode
  void* o = nullptr;  // prefill: bf16, decode: fp32
  int n_seq = 0;
  int n_tok = 0;  // decode
  int64_t tokens = 0;
  int H = 0;
  int group = 1;  // heads that share a q/k head
  int n_segments = 0;
  int stall = -1;  // test hook: the copy that each block leaves out
  void* workspace = nullptr;
  int* status = nullptr;
  cudaStream_t stream = nullptr;
};

size_t lin_prefill_workspace(int n_seq, int64_t tokens, int H, int n_segments, int num_sms);
cudaError_t launch_lin_prefill(const LinArgs& a, int num_sms);
cudaError_t launch_lin_decode(const LinArgs& a);

// The step between two blocks (kda_norm.cu).
struct NormArgs {
  const void* x = nullptr;  // residual rows, bf16 or fp32
  const void* y = nullptr;  // the block's output, bf16, or nullptr
  const void* gate = nullptr;
  const float* weight = nullptr;
  const float* post_weight = nullptr;
  void* h = nullptr;
  void* x_out = nullptr;
  int64_t x_stride = 0, y_stride = 0, gate_stride = 0;  // elements a row
  int64_t rows = 0;
  int width = 0;
  bool x_f32 = false;
  bool post_norm = false;
  float scale = 1.f;
  float eps = 0.f;
  cudaStream_t stream = nullptr;
};
constexpr int kMaxNormWidth = 32768;
cudaError_t launch_block_norm(const NormArgs& a, int num_sms);

}  // namespace kda
