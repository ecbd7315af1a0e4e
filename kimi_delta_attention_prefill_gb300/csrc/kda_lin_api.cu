// kda_lin_api.cu -- C entry points of linear attention with a decay a head and of the step between
// blocks (include/kda.h): host-side validation and launch.  Nothing here allocates or keeps anything
// between calls.
#include <cuda_runtime.h>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "kda.h"
#include "kda_lin.h"

namespace {

std::atomic<int> g_stall_copy{-1};  // kda_debug_stall_next_linear: consumed by the next kda_lin_prefill

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Strides of rows that are read 16 bytes at a time (and by tensor maps): positive, whole 16-byte
// units, below 2^40 bytes.
bool row_strides(const int64_t* s, int n, int64_t bytes, int64_t* out) {
  for (int i = 0; i < n; ++i) {
    if (s[i] <= 0 || s[i] >= (int64_t{1} << 40) / bytes || (s[i] * bytes) % 16 != 0) return false;
    out[3 - n + i] = s[i];
  }
  return true;
}

// What the two calls share.  n: the number of leading strides (2 prefill, 3 decode).
kda_status check_lin(const void* q, const int64_t* qs, const void* k, const int64_t* ks, const void* v, const int64_t* vs,
                     const float* g, const int64_t* gs, int n, float scale, const void* gate, const int64_t* gates,
                     const float* norm_weight, float eps, int n_seq, int64_t tokens, const void* o, int qk_heads, int H,
                     int d, const int* status, kda::LinArgs* a) {
  if (d != KDA_HEAD_DIM) return KDA_ERR_UNSUPPORTED;
  if (n_seq < 0 || tokens < 0 || tokens > 0x7fffffffLL || H < 1 || qk_heads < 1 || H % qk_heads != 0) return KDA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(n_seq) * H > 0x7fffffffLL || (n_seq == 0 && tokens > 0)) return KDA_ERR_INVALID_ARG;
  if (H > 65535) return KDA_ERR_UNSUPPORTED;
  if (!std::isfinite(scale)) return KDA_ERR_INVALID_ARG;
  if (gate && (!std::isfinite(eps) || eps < 0.f)) return KDA_ERR_INVALID_ARG;
  if (tokens > 0) {
    if (!q || !k || !v || !g || !o || !qs || !ks || !vs || !gs || (gate && !gates)) return KDA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(g, 4) || !aligned(o, 16) || !aligned(gate, 16) ||
        !aligned(norm_weight, 16) || !aligned(status, 4) || !row_strides(qs, n, 2, a->q_stride) ||
        !row_strides(ks, n, 2, a->k_stride) || !row_strides(vs, n, 2, a->v_stride) ||
        (gate && !row_strides(gates, n, 2, a->gate_stride)))
      return KDA_ERR_ALIGNMENT;
    for (int i = 0; i < n; ++i) {
      if (gs[i] < 0 || gs[i] >= (int64_t{1} << 38)) return KDA_ERR_INVALID_ARG;
      a->g_stride[3 - n + i] = gs[i];
    }
  }
  a->q = q; a->k = k; a->v = v; a->g = g; a->gate = gate; a->scale = scale; a->norm_weight = norm_weight; a->eps = eps;
  a->n_seq = n_seq; a->tokens = tokens; a->H = H; a->group = H / qk_heads; a->o = const_cast<void*>(o);
  return KDA_OK;
}

}  // namespace

extern "C" {

size_t kda_lin_prefill_workspace_size(int n_seq, int H, int d, int64_t total_tokens, int n_segments) {
  if (d != KDA_HEAD_DIM || n_seq < 0 || H < 1 || total_tokens < 0 || n_segments < 0) return 0;
  int sms = 0;
  if (kda::current_device_status(&sms) != KDA_OK) sms = 152;
  return kda::lin_prefill_workspace(n_seq, total_tokens, H, n_segments, sms);
}

kda_status kda_lin_prefill(const kda_bf16* q, const int64_t* q_stride, const kda_bf16* k, const int64_t* k_stride,
                           const kda_bf16* v, const int64_t* v_stride, const float* g, const int64_t* g_stride, float scale,
                           const kda_bf16* gate, const int64_t* gate_stride, const float* norm_weight, float eps,
                           const float* S_in, const int32_t* cu_seqlens, int n_seq, int64_t total_tokens, kda_bf16* o,
                           float* S_out, int qk_heads, int H, int d, int n_segments, void* workspace,
                           size_t workspace_bytes, int* dev_status, cudaStream_t stream) {
  kda::LinArgs a;
  const kda_status st = check_lin(q, q_stride, k, k_stride, v, v_stride, g, g_stride, 2, scale, gate, gate_stride,
                                  norm_weight, eps, n_seq, total_tokens, o, qk_heads, H, d, dev_status, &a);
  if (st != KDA_OK) return st;
  if (n_segments < 0) return KDA_ERR_INVALID_ARG;
  if (n_seq == 0) return KDA_OK;
  if (!cu_seqlens) return KDA_ERR_INVALID_ARG;
  if (!aligned(cu_seqlens, 4) || !aligned(S_in, 16) || !aligned(S_out, 16) || !aligned(workspace, 256)) return KDA_ERR_ALIGNMENT;
  int sms = 152;
  const kda_status dev = static_cast<kda_status>(kda::current_device_status(&sms));
  if (dev != KDA_OK) sms = 152;
  const size_t need = kda::lin_prefill_workspace(n_seq, total_tokens, H, n_segments, sms);
  if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
  if (dev != KDA_OK) return dev;
  a.S_in = S_in; a.S_out = S_out; a.cu = cu_seqlens; a.n_segments = n_segments; a.workspace = workspace;
  a.status = dev_status; a.stream = stream;
  if (g_stall_copy.load(std::memory_order_relaxed) >= 0) a.stall = g_stall_copy.exchange(-1);
  return kda::launch_lin_prefill(a, sms) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_lin_decode(const kda_bf16* q, const int64_t* q_stride, const kda_bf16* k, const int64_t* k_stride,
                          const kda_bf16* v, const int64_t* v_stride, const float* g, const int64_t* g_stride, float scale,
                          const kda_bf16* gate, const int64_t* gate_stride, const float* norm_weight, float eps,
                          float* S_state, const int32_t* n_commit, float* o, int B, int n_tok, int qk_heads, int H, int d,
                          int* dev_status, cudaStream_t stream) {
  if (n_tok < 1 || n_tok > KDA_MAX_DECODE_TOKENS) return KDA_ERR_UNSUPPORTED;
  kda::LinArgs a;
  const kda_status st = check_lin(q, q_stride, k, k_stride, v, v_stride, g, g_stride, 3, scale, gate, gate_stride,
                                  norm_weight, eps, B, static_cast<int64_t>(B) * n_tok, o, qk_heads, H, d, dev_status, &a);
  if (st != KDA_OK || B == 0) return st;
  if (!S_state) return KDA_ERR_INVALID_ARG;
  if (!aligned(S_state, 16) || !aligned(n_commit, 4)) return KDA_ERR_ALIGNMENT;
  const kda_status dev = static_cast<kda_status>(kda::current_device_status(nullptr));
  if (dev != KDA_OK) return dev;
  a.S_out = S_state; a.n_commit = n_commit; a.n_tok = n_tok; a.status = dev_status; a.stream = stream;
  return kda::launch_lin_decode(a) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_block_norm(const void* x, int x_dtype, int64_t x_stride, const float* weight, const kda_bf16* y,
                          int64_t y_stride, int post_norm, const float* post_weight, const kda_bf16* gate,
                          int64_t gate_stride, float scale, float eps, kda_bf16* h, void* x_out, int64_t rows, int width,
                          cudaStream_t stream) {
  if (x_dtype != KDA_ROWS_BF16 && x_dtype != KDA_ROWS_F32) return KDA_ERR_UNSUPPORTED;
  if (rows < 0 || width < 1 || !std::isfinite(eps) || eps < 0.f || !std::isfinite(scale)) return KDA_ERR_INVALID_ARG;
  if (width % 8 != 0 || width > kda::kMaxNormWidth) return KDA_ERR_UNSUPPORTED;
  if (rows == 0) return KDA_OK;
  if (!y && (post_norm || post_weight || gate)) return KDA_ERR_INVALID_ARG;
  if (!h && !x_out) return KDA_ERR_INVALID_ARG;
  if (!y && x_out) return KDA_ERR_INVALID_ARG;  // a copy is not this call's work
  if (!x) return KDA_ERR_INVALID_ARG;
  if (x_out == x && rows > 1 && x_stride != width) return KDA_ERR_INVALID_ARG;  // it would come upon rows not read yet
  const bool f32 = x_dtype == KDA_ROWS_F32;
  int64_t s[3];
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(gate, 16) || !aligned(weight, 16) || !aligned(post_weight, 16) ||
      !aligned(h, 16) || !aligned(x_out, 16) || !row_strides(&x_stride, 1, f32 ? 4 : 2, s) ||
      (y && !row_strides(&y_stride, 1, 2, s)) || (gate && !row_strides(&gate_stride, 1, 2, s)))
    return KDA_ERR_ALIGNMENT;
  int sms = 0;
  const kda_status dev = static_cast<kda_status>(kda::current_device_status(&sms));
  if (dev != KDA_OK) return dev;
  kda::NormArgs a;
  a.x = x; a.y = y; a.gate = gate; a.weight = weight; a.post_weight = post_weight; a.h = h; a.x_out = x_out;
  a.x_stride = x_stride; a.y_stride = y_stride; a.gate_stride = gate_stride; a.rows = rows; a.width = width;
  a.x_f32 = f32; a.post_norm = post_norm != 0; a.scale = scale; a.eps = eps; a.stream = stream;
  return kda::launch_block_norm(a, sms) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

void kda_debug_stall_next_linear(int copy) { g_stall_copy.store(copy < 0 ? -1 : copy); }

}  // extern "C"
