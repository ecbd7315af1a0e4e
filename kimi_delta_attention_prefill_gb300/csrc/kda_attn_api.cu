// kda_attn_api.cu -- the attention cache's C entry points (include/kda.h): host-side
// validation and launch.  Nothing here allocates or keeps anything between calls.
#include <cuda_runtime.h>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "kda.h"
#include "kda_attn.h"

namespace {

std::atomic<int> g_stall_copy{-1};  // kda_debug_stall_next_attention: consumed by the next attention launch

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Strides the kernels and the tensor maps take: positive, whole 16-byte units, below 2^40 bytes.
bool strides_ok(const int64_t* s, int n, int64_t bytes) {
  for (int i = 0; i < n; ++i)
    if (s[i] <= 0 || s[i] >= (int64_t{1} << 40) / bytes || (s[i] * bytes) % 16 != 0) return false;
  return true;
}

kda_status check_cache(const kda_kv_cache* c, int d, kda::KvCache* out) {
  if (d != KDA_HEAD_DIM) return KDA_ERR_UNSUPPORTED;
  if (!c) return KDA_ERR_INVALID_ARG;
  if (c->dtype != KDA_KV_BF16 && c->dtype != KDA_KV_E4M3) return KDA_ERR_UNSUPPORTED;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) return KDA_ERR_UNSUPPORTED;
  if (c->n_pages < 0 || c->n_pages > 0x7fffffffLL || c->n_kv_heads < 1) return KDA_ERR_INVALID_ARG;
  if (c->n_kv_heads > 65535) return KDA_ERR_UNSUPPORTED;
  const bool e4m3 = c->dtype == KDA_KV_E4M3;
  if (!c->k || !c->v || (e4m3 && (!c->k_scale || !c->v_scale))) return KDA_ERR_INVALID_ARG;
  const int64_t bytes = e4m3 ? 1 : 2;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !strides_ok(c->k_stride, 3, bytes) || !strides_ok(c->v_stride, 3, bytes))
    return KDA_ERR_ALIGNMENT;
  if (e4m3 && (!aligned(c->k_scale, 16) || !aligned(c->v_scale, 16) || !strides_ok(c->k_scale_stride, 2, 1) ||
               !strides_ok(c->v_scale_stride, 2, 1)))
    return KDA_ERR_ALIGNMENT;
  out->k = c->k; out->v = c->v; out->ks = c->k_scale; out->vs = c->v_scale;
  for (int i = 0; i < 3; ++i) { out->k_stride[i] = c->k_stride[i]; out->v_stride[i] = c->v_stride[i]; }
  for (int i = 0; i < 2; ++i) { out->ks_stride[i] = c->k_scale_stride[i]; out->vs_stride[i] = c->v_scale_stride[i]; }
  out->n_pages = c->n_pages; out->heads = c->n_kv_heads; out->page_size = c->page_size; out->e4m3 = e4m3;
  out->page_log2 = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
  return KDA_OK;
}

kda_status check_rows(const kda_kv_cache* cache, const void* k, const int64_t* ks, const void* v, const int64_t* vs,
                      const int32_t* page_table, int n_seq, int max_pages, const int32_t* cu, const int32_t* start,
                      int64_t tokens, int d, const int* status, kda::KvRows* a) {
  kda_status st = check_cache(cache, d, &a->cache);
  if (st != KDA_OK) return st;
  if (n_seq < 0 || max_pages < 0 || tokens < 0 || tokens > 0x7fffffffLL) return KDA_ERR_INVALID_ARG;
  if (n_seq == 0 && tokens > 0) return KDA_ERR_INVALID_ARG;
  if (tokens == 0) return KDA_OK;
  if ((tokens + 31) / 32 * cache->n_kv_heads > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;  // a block a head and 32 tokens
  if (!k || !v || !ks || !vs || !cu || !start || (max_pages > 0 && !page_table)) return KDA_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !strides_ok(ks, 2, 2) || !strides_ok(vs, 2, 2) || !aligned(page_table, 4) ||
      !aligned(cu, 4) || !aligned(start, 4) || !aligned(status, 4))
    return KDA_ERR_ALIGNMENT;
  a->k = const_cast<void*>(k); a->v = const_cast<void*>(v);
  for (int i = 0; i < 2; ++i) { a->k_stride[i] = ks[i]; a->v_stride[i] = vs[i]; }
  a->page_table = page_table; a->cu = cu; a->start = start; a->n_seq = n_seq; a->max_pages = max_pages; a->tokens = tokens;
  return static_cast<kda_status>(kda::current_device_status(nullptr));
}

// What the two attention calls share.
kda_status check_attn(const void* q, const int64_t* qs, int n_strides, const kda_kv_cache* cache, const int32_t* page_table,
                      int n_seq, int max_pages, const int32_t* kv_len, int64_t tokens, int H, int d, float scale,
                      int window, int n_sink, const void* o, const float* lse, const void* workspace, const int* status,
                      kda::AttnArgs* a) {
  kda_status st = check_cache(cache, d, &a->cache);
  if (st != KDA_OK) return st;
  if (n_seq < 0 || max_pages < 0 || tokens < 0 || H < 1 || H % cache->n_kv_heads != 0) return KDA_ERR_INVALID_ARG;
  if (tokens > 0x7fffffffLL || tokens * (H / cache->n_kv_heads) > 0x7fffffffLL - 4096) return KDA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(max_pages) * cache->page_size > 0x7fffffffLL - 4096) return KDA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || window < 0 || n_sink < 0) return KDA_ERR_INVALID_ARG;
  if (n_seq == 0 && tokens > 0) return KDA_ERR_INVALID_ARG;
  if (tokens == 0) return KDA_OK;
  if (!q || !qs || !o || !kv_len || (max_pages > 0 && !page_table)) return KDA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !strides_ok(qs, n_strides, 2) || !aligned(page_table, 4) ||
      !aligned(kv_len, 4) || !aligned(lse, 4) || !aligned(status, 4) || !aligned(workspace, 256))
    return KDA_ERR_ALIGNMENT;
  a->q = q; a->page_table = page_table; a->kv_len = kv_len; a->n_seq = n_seq; a->max_pages = max_pages;
  a->tokens = tokens; a->H = H;
  // ceil(2^(31 + b) / G) with 2^b >= G: exact for 31-bit rows, and the product fits 64 bits
  const uint64_t G = static_cast<uint64_t>(H / cache->n_kv_heads);
  int bits = 0;
  while ((uint64_t{1} << bits) < G) ++bits;
  a->g_shift = 31 + bits;
  a->g_magic = ((uint64_t{1} << a->g_shift) + G - 1) / G;
  a->scale_log2 = scale * 1.4426950408889634f;
  // a window no sequence can outgrow is none, and the kernels' 32-bit positions need no more first tokens than fit
  const int64_t most = static_cast<int64_t>(max_pages) * cache->page_size;
  a->window = window >= most ? 0 : window;
  a->n_sink = static_cast<int>(n_sink < most ? n_sink : most);
  a->o = const_cast<void*>(o); a->lse = const_cast<float*>(lse); a->workspace = const_cast<void*>(workspace);
  if (g_stall_copy.load(std::memory_order_relaxed) >= 0) a->stall = g_stall_copy.exchange(-1);
  return KDA_OK;
}

int sm_count() {
  int sms = 0;
  return kda::current_device_status(&sms) == 0 ? sms : 152;
}

}  // namespace

extern "C" {

kda_status kda_kv_append(const kda_kv_cache* cache, const kda_bf16* k, const int64_t* k_stride, const kda_bf16* v,
                         const int64_t* v_stride, const int32_t* page_table, int n_seq, int max_pages,
                         const int32_t* cu_seqlens, const int32_t* kv_start, int64_t total_tokens, int d,
                         int* dev_status, cudaStream_t stream) {
  kda::KvRows a;
  kda_status st = check_rows(cache, k, k_stride, v, v_stride, page_table, n_seq, max_pages, cu_seqlens, kv_start,
                             total_tokens, d, dev_status, &a);
  if (st != KDA_OK || total_tokens == 0) return st;
  a.status = dev_status; a.stream = stream;
  return kda::launch_kv_append(a) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_kv_read(const kda_kv_cache* cache, kda_bf16* k, kda_bf16* v, const int32_t* page_table, int n_seq,
                       int max_pages, const int32_t* cu_seqlens, const int32_t* kv_start, int64_t total_tokens, int d,
                       int* dev_status, cudaStream_t stream) {
  kda::KvRows a;
  const int64_t packed[2] = {cache ? static_cast<int64_t>(cache->n_kv_heads) * KDA_HEAD_DIM : KDA_HEAD_DIM, KDA_HEAD_DIM};
  kda_status st = check_rows(cache, k, packed, v, packed, page_table, n_seq, max_pages, cu_seqlens, kv_start,
                             total_tokens, d, dev_status, &a);
  if (st != KDA_OK || total_tokens == 0) return st;
  a.status = dev_status; a.stream = stream;
  return kda::launch_kv_read(a) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_attn_prefill_workspace_size(int n_seq, int64_t total_tokens, int H, int n_kv_heads, int d) {
  if (d != KDA_HEAD_DIM || n_seq < 0 || total_tokens < 0 || H < 1 || n_kv_heads < 1 || H % n_kv_heads != 0) return 0;
  return kda::attn_prefill_workspace(n_seq, total_tokens, H, n_kv_heads, sm_count());
}

kda_status kda_attn_prefill_paged(const kda_bf16* q, const int64_t* q_stride, const kda_kv_cache* cache,
                                  const int32_t* page_table, int n_seq, int max_pages, const int32_t* cu_seqlens,
                                  const int32_t* kv_len, int64_t total_tokens, int H, int d, float scale, int window,
                                  int n_sink, kda_bf16* o, float* lse, void* workspace, size_t workspace_bytes,
                                  int* dev_status, cudaStream_t stream) {
  kda::AttnArgs a;
  kda_status st = check_attn(q, q_stride, 2, cache, page_table, n_seq, max_pages, kv_len, total_tokens, H, d, scale,
                             window, n_sink, o, lse, workspace, dev_status, &a);
  if (st != KDA_OK || total_tokens == 0) return st;
  if (!cu_seqlens) return KDA_ERR_INVALID_ARG;
  if (!aligned(cu_seqlens, 4)) return KDA_ERR_ALIGNMENT;
  int sms = 152;
  const kda_status dev = static_cast<kda_status>(kda::current_device_status(&sms));
  if (dev != KDA_OK) sms = 152;
  if (!workspace || workspace_bytes < kda::attn_prefill_workspace(n_seq, total_tokens, H, cache->n_kv_heads, sms))
    return KDA_ERR_WORKSPACE;
  if (dev != KDA_OK) return dev;
  a.cu = cu_seqlens; a.q_stride[1] = q_stride[0]; a.q_stride[2] = q_stride[1];
  a.status = dev_status; a.stream = stream;
  return kda::launch_attn_prefill(a, sms) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_attn_decode_workspace_size(int B, int n_tok, int H, int n_kv_heads, int d) {
  if (d != KDA_HEAD_DIM || B < 0 || n_tok < 1 || n_tok > KDA_MAX_DECODE_TOKENS || H < 1 || n_kv_heads < 1 ||
      H % n_kv_heads != 0)
    return 0;
  return kda::attn_decode_workspace(B, n_tok, H, n_kv_heads, sm_count());
}

kda_status kda_attn_decode_paged(const kda_bf16* q, const int64_t* q_stride, const kda_kv_cache* cache,
                                 const int32_t* page_table, int B, int n_tok, int max_pages, const int32_t* kv_len,
                                 int H, int d, float scale, int window, int n_sink, kda_bf16* o, float* lse,
                                 void* workspace, size_t workspace_bytes, int* dev_status, cudaStream_t stream) {
  if (n_tok < 1 || n_tok > KDA_MAX_DECODE_TOKENS) return KDA_ERR_UNSUPPORTED;
  kda::AttnArgs a;
  kda_status st = check_attn(q, q_stride, 3, cache, page_table, B, max_pages, kv_len, static_cast<int64_t>(B) * n_tok, H,
                             d, scale, window, n_sink, o, lse, workspace, dev_status, &a);
  if (st != KDA_OK || B == 0) return st;
  int sms = 152;
  const kda_status dev = static_cast<kda_status>(kda::current_device_status(&sms));
  if (dev != KDA_OK) sms = 152;
  if (!workspace || workspace_bytes < kda::attn_decode_workspace(B, n_tok, H, cache->n_kv_heads, sms))
    return KDA_ERR_WORKSPACE;
  if (dev != KDA_OK) return dev;
  a.n_tok = n_tok;
  for (int i = 0; i < 3; ++i) a.q_stride[i] = q_stride[i];
  a.status = dev_status; a.stream = stream;
  return kda::launch_attn_decode(a, sms) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

int kda_debug_attention_kernel(int n_seq, int64_t total_tokens, int H, int n_kv_heads, int64_t most_keys) {
  if (n_seq < 0 || total_tokens < 0 || H < 1 || n_kv_heads < 1 || H % n_kv_heads != 0 || most_keys < 0) return -1;
  return kda::attn_short_chunks(n_seq, total_tokens, H, n_kv_heads, most_keys) ? 0 : 1;
}

void kda_debug_stall_next_attention(int copy) { g_stall_copy.store(copy < 0 ? -1 : copy); }

}  // extern "C"
