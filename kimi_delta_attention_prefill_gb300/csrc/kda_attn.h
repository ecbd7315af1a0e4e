// kda_attn.h -- the attention cache's shared pieces: the cache as the kernels see it, the
// tiles of keys that a block of query rows has to visit, and the launches.
#pragma once

#include <cuda_runtime.h>
#include <atomic>
#include <cstddef>
#include <cstdint>

#include "kda_internal.h"

namespace kda {

// One layer's cache (kda_kv_cache, checked on the host).
struct KvCache {
  void* k = nullptr;
  void* v = nullptr;
  uint8_t* ks = nullptr;  // scale bytes (e4m3 only)
  uint8_t* vs = nullptr;
  int64_t k_stride[3] = {0, 0, 0};  // elements: page, head, token
  int64_t v_stride[3] = {0, 0, 0};
  int64_t ks_stride[2] = {0, 0};  // bytes: page, head
  int64_t vs_stride[2] = {0, 0};
  int64_t n_pages = 0;
  int heads = 0;
  int page_size = 0;
  int page_log2 = 0;
  bool e4m3 = false;
};

struct KvRows {  // kda_kv_append / kda_kv_read
  KvCache cache;
  void* k = nullptr;
  void* v = nullptr;
  int64_t k_stride[2] = {0, 0};  // elements: token, head
  int64_t v_stride[2] = {0, 0};
  const int32_t* page_table = nullptr;
  const int32_t* cu = nullptr;
  const int32_t* start = nullptr;
  int n_seq = 0;
  int max_pages = 0;
  int64_t tokens = 0;
  int* status = nullptr;
  cudaStream_t stream = nullptr;
};
cudaError_t launch_kv_append(const KvRows& a);
cudaError_t launch_kv_read(const KvRows& a);

struct AttnArgs {
  const void* q = nullptr;
  int64_t q_stride[3] = {0, 0, 0};  // elements: sequence (decode only), token, head
  KvCache cache;
  const int32_t* page_table = nullptr;
  const int32_t* cu = nullptr;  // prefill; nullptr: decode, n_tok tokens of each sequence
  const int32_t* kv_len = nullptr;
  int n_seq = 0;
  int n_tok = 0;
  int max_pages = 0;
  int64_t tokens = 0;
  int H = 0;
  uint64_t g_magic = 0;    // row / (H / kv heads) = row * g_magic >> g_shift (rows below 2^31)
  int g_shift = 0;
  float scale_log2 = 0.f;  // softmax scale in log2 units
  int window = 0;
  int n_sink = 0;
  void* o = nullptr;
  float* lse = nullptr;
  void* workspace = nullptr;
  int* status = nullptr;
  int stall = -1;  // test hook: the copy that each block leaves out
  cudaStream_t stream = nullptr;
};
size_t attn_prefill_workspace(int n_seq, int64_t tokens, int H, int kv_heads, int num_sms);
size_t attn_decode_workspace(int n_seq, int n_tok, int H, int kv_heads, int num_sms);
cudaError_t launch_attn_prefill(const AttnArgs& a, int num_sms);
cudaError_t launch_attn_decode(const AttnArgs& a, int num_sms);
// Whether a chunk of so many tokens, over tables with room for most_keys, is the short kernel's.
bool attn_short_chunks(int n_seq, int64_t tokens, int H, int kv_heads, int64_t most_keys);

// Many rows a sequence: kda_attn_chunk.cu.
size_t attn_chunk_workspace(int n_seq, int64_t tokens, int group, int num_sms);
cudaError_t launch_attn_chunk(const AttnArgs& a, int num_sms);

// Launches a kernel that may begin before the one ahead of it in the stream has ended
// (programmatic dependent launch); it waits for that one's writes itself.
template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// A kernel's dynamic shared memory limit, raised once per device (the call costs a microsecond).
struct SmemOptIn {
  std::atomic<uint64_t> done{0};
  cudaError_t operator()(const void* kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
  }
};

// The split of the work over blocks, and the workspace that joins it (kda_attn_common.cu).
// The items -- (sequence, row tile) x kv head -- lie one after the other on a line of key
// tiles; block c of the first C takes [c W / C, (c + 1) W / C) of its W tiles.  Parts of items
// that two or more blocks share go to slots of the workspace: block c's first part, of an item
// begun by an earlier block, to slot 2c, its last part, of an item that a later block goes on
// with, to slot 2c + 1, and desc[c] says where the latter's rows belong.
struct PartDesc {
  int64_t base;  // packed row of the sequence's first token
  int head;
  int row0;      // the item's first row
  int rows;      // the sequence's
  int last;      // the block that has the item's last part; -1: there is no such part
};
struct AttnSplit {
  PartDesc* desc = nullptr;    // [grid]
  float2* part_ml = nullptr;   // [2 grid][part_rows] (maximum, sum)
  float* part_o = nullptr;     // [2 grid][part_rows][128] unnormalised
  int64_t* plan_total = nullptr;   // prefill: tiles of all items of one kv head
  int64_t* plan_start = nullptr;   // [items + 1] where each begins on one kv head's line
  int2* plan_item = nullptr;       // [items] {sequence, first row}
  int* plan_items = nullptr;       // number of items
  int64_t max_items = 0;
  int grid = 0;
  int part_rows = 0;
  int min_tiles = 1;  // least share of a block
  int item_cost = 0;  // what an item costs besides its key tiles, in key tiles
};
size_t attn_split_bytes(int grid, int part_rows, int64_t max_items);
void attn_split_layout(AttnSplit* s, void* workspace, int grid, int part_rows, int64_t max_items);
// Most row tiles that `tokens` tokens of n_seq sequences can make.
inline int64_t attn_max_items(int n_seq, int64_t tokens, int group, int rows) { return tokens * group / rows + n_seq; }
// Prefill: lists the items (row tiles of `rows` rows, key tiles of `tile` keys) in the workspace.
cudaError_t launch_attn_plan(const AttnArgs& a, const AttnSplit& s, int rows, int tile);
// Joins the parts of split items in block order.
cudaError_t launch_attn_join(const AttnArgs& a, const AttnSplit& s);
// Tensor maps of the cache, one box per (page, kv head): min(page_size, tile) tokens, bf16 rows
// in `panels` (1 or 2) panels of 64 channels.
bool make_cache_maps(const KvCache& c, int tile, int panels, struct CUtensorMap_st* k, struct CUtensorMap_st* v);
// The same of an e4m3 cache's scale bytes.
bool make_scale_maps(const KvCache& c, int tile, struct CUtensorMap_st* ks, struct CUtensorMap_st* vs);

// The key tiles (of `tile` keys) that rows at positions p_first .. p_last have to visit: the
// tiles [0, sink) of the first tokens, then [lo, hi) up to the last visible key.
struct KeyTiles {
  int sink, lo, hi;
  __host__ __device__ int count() const { return sink + hi - lo; }
  // key tile of the i-th visit
  __host__ __device__ int at(int i) const { return i < sink ? i : lo + (i - sink); }
};
__host__ __device__ inline KeyTiles key_tiles(int p_first, int p_last, int window, int n_sink, int tile) {
  KeyTiles t{0, 0, 0};
  if (p_last < 0) return t;
  t.hi = p_last / tile + 1;
  if (window > 0) {
    const int64_t first = static_cast<int64_t>(p_first < 0 ? 0 : p_first) - window + 1;
    t.lo = first > 0 ? static_cast<int>(first / tile) : 0;
    const int s = n_sink > 0 ? (n_sink - 1) / tile + 1 : 0;
    t.sink = s < t.lo ? s : t.lo;
  }
  return t;
}

// Whether the row at position p sees key j (window = 0: no window).
__device__ __forceinline__ bool sees(int p, int j, int window, int n_sink) {
  return j <= p && (window == 0 || p - j < window || j < n_sink);
}

}  // namespace kda
