// kda_attn_common.cu -- the attention kernels' host side and helpers: tensor maps of the paged
// cache, the list of row tiles (prefill), and the joining of items that blocks share.
#include <cuda_runtime.h>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "kda_attn.h"
#include "kda_attn_device.cuh"

namespace kda {

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// One pool: bf16 rows as two 64-channel panels (5-D), `panels` of them a box, e4m3 rows whole
// (4-D), 128-byte swizzle.
bool rows_map(CUtensorMap* m, const void* base, const int64_t* stride, const KvCache& c, int tile, int panels) {
  const cuuint32_t box_tok = static_cast<cuuint32_t>(c.page_size < tile ? c.page_size : tile);
  const cuuint64_t P = c.page_size, H = c.heads, N = c.n_pages > 0 ? c.n_pages : 1;
  const cuuint32_t es[5] = {1, 1, 1, 1, 1};
  CUresult r;
  if (c.e4m3) {
    const cuuint64_t dims[4] = {128, P, H, N};
    const cuuint64_t st[3] = {static_cast<cuuint64_t>(stride[2]), static_cast<cuuint64_t>(stride[1]), static_cast<cuuint64_t>(stride[0])};
    const cuuint32_t box[4] = {128, box_tok, 1, 1};
    r = encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, st, box, es,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  } else {
    const cuuint64_t dims[5] = {64, P, 2, H, N};
    const cuuint64_t st[4] = {2 * static_cast<cuuint64_t>(stride[2]), 128, 2 * static_cast<cuuint64_t>(stride[1]),
                              2 * static_cast<cuuint64_t>(stride[0])};
    const cuuint32_t box[5] = {64, box_tok, static_cast<cuuint32_t>(panels), 1, 1};
    r = encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, st, box, es,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  }
  return r == CUDA_SUCCESS;
}
bool scale_map(CUtensorMap* m, const void* base, const int64_t* stride, const KvCache& c, int tile) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c.page_size), static_cast<cuuint64_t>(c.heads),
                              static_cast<cuuint64_t>(c.n_pages > 0 ? c.n_pages : 1)};
  const cuuint64_t st[2] = {static_cast<cuuint64_t>(stride[1]), static_cast<cuuint64_t>(stride[0])};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(c.page_size < tile ? c.page_size : tile), 1, 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, st, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Lists the row tiles of all sequences in order.  One block; 1024 sequences, then 1024 items,
// at a time.  Offsets or lengths that cannot be are reported and leave their sequence out.
constexpr int kPlanThreads = 1024;

__device__ int64_t warp_scan(int64_t v, int lane) {  // inclusive
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += up;
  }
  return v;
}
__device__ int64_t block_scan(int64_t v, int64_t* sh, int64_t* total) {  // exclusive
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t incl = warp_scan(v, lane);
  __syncthreads();
  if (lane == 31) sh[warp] = incl;
  __syncthreads();
  const int64_t upto = warp_scan(sh[lane], lane);  // every warp, of the 32 warps' sums
  *total = __shfl_sync(0xffffffffu, upto, 31);
  const int64_t before = __shfl_sync(0xffffffffu, upto, warp > 0 ? warp - 1 : 0);
  return (warp > 0 ? before : 0) + incl - v;
}

__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(const __grid_constant__ AttnArgs a,
                                                                 const __grid_constant__ AttnSplit s, int rows, int tile) {
  __shared__ int64_t sh[kPlanThreads / 32];
  __shared__ int64_t first_item[kPlanThreads];
  __shared__ int sh_len[kPlanThreads], sh_tok[kPlanThreads];
  pdl_launch_dependents();
  const int tid = threadIdx.x;
  int64_t items = 0, line = 0;
  for (int b = 0; b < a.n_seq; b += kPlanThreads) {
    Item w;
    int64_t n = 0;
    if (b + tid < a.n_seq) {
      if (item_sequence(a, b + tid, &w))
        n = (w.rows + rows - 1) / rows;
      else if (seq_bad(a, w.len, w.base, w.base + w.n_tok))
        report_status(a.status, 7 /* KDA_ERR_DEVICE_CHECK */);
    }
    sh_len[tid] = w.len;
    sh_tok[tid] = w.n_tok;
    int64_t all;
    first_item[tid] = block_scan(n, sh, &all);
    __syncthreads();
    // offsets that run backwards may repeat tokens: the table holds what sound offsets can need
    if (items + all > s.max_items) {
      if (tid == 0) report_status(a.status, 7 /* KDA_ERR_DEVICE_CHECK */);
      all = s.max_items - items;
    }
    for (int64_t c = 0; c < all; c += kPlanThreads) {
      const int64_t k = c + tid;
      int64_t count = 0;
      int2 d = make_int2(0, 0);
      if (k < all) {
        int lo = 0, hi = kPlanThreads;  // the last sequence whose first item is at most k (empty ones share theirs)
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (first_item[mid] <= k) lo = mid; else hi = mid;
        }
        d = make_int2(b + lo, static_cast<int>(k - first_item[lo]) * rows);
        w.len = sh_len[lo];
        w.n_tok = sh_tok[lo];
        w.G = a.H / a.cache.heads;
        w.rows = w.n_tok * w.G;
        item_tiles(a, d.y, rows, tile, &w);
        count = w.tiles.count() + s.item_cost;
      }
      int64_t sum;
      const int64_t before = block_scan(count, sh, &sum);
      if (k < all) {
        s.plan_item[items + k] = d;
        s.plan_start[items + k] = line + before;
      }
      line += sum;
    }
    items += all;
    __syncthreads();
  }
  if (tid == 0) {
    s.plan_start[items] = line;
    *s.plan_total = line;
    *s.plan_items = static_cast<int>(items);
  }
}

// A warp a row, four channels a lane: the row's parts, weighted to a common maximum, added in
// block order.  The parts were written by other SMs and a dependent load of them costs most of a
// microsecond, so a row is one chain of three -- desc, all of (up to eight) parts with their
// (m, l) at once, the output -- and rows are spread over as many warps as there are.
constexpr int kJoinThreads = 128, kJoinParts = 8;
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const __grid_constant__ AttnArgs a,
                                                                 const __grid_constant__ AttnSplit s) {
  pdl_wait();
  const int c0 = blockIdx.x, lane = threadIdx.x & 31;
  const PartDesc d = s.desc[c0];
  if (d.last < 0) return;
  const int G = a.H / a.cache.heads, R = s.part_rows, n = d.last - c0 + 1;
  for (int lr = blockIdx.y * (kJoinThreads / 32) + (threadIdx.x >> 5); lr < R; lr += gridDim.y * (kJoinThreads / 32)) {
    const int row = d.row0 + lr;
    if (row >= d.rows) return;
    const int64_t at = (2 * static_cast<int64_t>(c0) + 1) * R + lr;  // part i > 0 lies at block c0 + i's first slot
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < n; i0 += kJoinParts) {
      float2 ml[kJoinParts];
      float4 v[kJoinParts];
#pragma unroll
      for (int i = 0; i < kJoinParts; ++i) {
        const int k = i0 + i;
        const int64_t slot = at + (k == 0 ? 0 : (2 * static_cast<int64_t>(k) - 1) * R);
        ml[i] = k < n ? s.part_ml[slot] : make_float2(-INFINITY, 0.f);
        v[i] = k < n ? reinterpret_cast<const float4*>(s.part_o + slot * 128)[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float top = m;
#pragma unroll
      for (int i = 0; i < kJoinParts; ++i) top = fmaxf(top, ml[i].x);
      const float b = top == -INFINITY ? 0.f : top, f0 = exp2_fast(m - b);
      m = top;
      l *= f0;
      o.x *= f0; o.y *= f0; o.z *= f0; o.w *= f0;
#pragma unroll
      for (int i = 0; i < kJoinParts; ++i) {
        const float f = exp2_fast(ml[i].x - b);
        l += ml[i].y * f;
        o.x += v[i].x * f; o.y += v[i].y * f; o.z += v[i].z * f; o.w += v[i].w * f;
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int t = row / G;
    const int64_t orow = (d.base + t) * a.H + static_cast<int64_t>(d.head) * G + (row - t * G);
    reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + orow * 128)[lane] =
        make_uint2(pack_bf162(o.x * inv, o.y * inv), pack_bf162(o.z * inv, o.w * inv));
    if (a.lse && lane == 0) a.lse[orow] = lse_of(m, l);
  }
}

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace

bool make_cache_maps(const KvCache& c, int tile, int panels, CUtensorMap* k, CUtensorMap* v) {
  return encode_fn() && rows_map(k, c.k, c.k_stride, c, tile, panels) && rows_map(v, c.v, c.v_stride, c, tile, panels);
}

bool make_scale_maps(const KvCache& c, int tile, CUtensorMap* ks, CUtensorMap* vs) {
  return encode_fn() && scale_map(ks, c.ks, c.ks_stride, c, tile) && scale_map(vs, c.vs, c.vs_stride, c, tile);
}

size_t attn_split_bytes(int grid, int part_rows, int64_t max_items) {
  const size_t parts = 2 * static_cast<size_t>(grid) * part_rows;
  return up256(sizeof(PartDesc) * static_cast<size_t>(grid)) + up256(8 * parts) + up256(512 * parts) +
         (max_items > 0 ? 256 + up256(8 * static_cast<size_t>(max_items + 1)) + up256(8 * static_cast<size_t>(max_items)) : 0);
}

void attn_split_layout(AttnSplit* s, void* workspace, int grid, int part_rows, int64_t max_items) {
  const size_t parts = 2 * static_cast<size_t>(grid) * part_rows;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  s->grid = grid; s->part_rows = part_rows; s->max_items = max_items;
  s->desc = reinterpret_cast<PartDesc*>(w); w += up256(sizeof(PartDesc) * static_cast<size_t>(grid));
  s->part_ml = reinterpret_cast<float2*>(w); w += up256(8 * parts);
  s->part_o = reinterpret_cast<float*>(w); w += up256(512 * parts);
  if (max_items <= 0) return;
  s->plan_total = reinterpret_cast<int64_t*>(w);
  s->plan_items = reinterpret_cast<int*>(w + 8); w += 256;
  s->plan_start = reinterpret_cast<int64_t*>(w); w += up256(8 * static_cast<size_t>(max_items + 1));
  s->plan_item = reinterpret_cast<int2*>(w);
}

cudaError_t launch_attn_plan(const AttnArgs& a, const AttnSplit& s, int rows, int tile) {
  attn_plan_kernel<<<1, kPlanThreads, 0, a.stream>>>(a, s, rows, tile);
  return cudaGetLastError();
}

cudaError_t launch_attn_join(const AttnArgs& a, const AttnSplit& s) {
  const int y = s.part_rows <= 64 ? s.part_rows / (kJoinThreads / 32) : 32;  // a row a warp; of 256 rows two
  return launch_after(attn_join_kernel, dim3(static_cast<unsigned>(s.grid), static_cast<unsigned>(y)),
                      dim3(kJoinThreads), 0, a.stream, a, s);
}

}  // namespace kda
