// kda_kv.cu -- rows into the paged attention cache (kda_kv_append) and back (kda_kv_read).
//
// An E4M3 row (128 values of one token and head) is stored as codes c and one byte e + 127:
//     e = min { whole e in [-40, 40] : max|x| <= 448 * 2^e },   c = RN_e4m3(x * 2^-e),
// so scaling is exact in both directions and the only rounding is the code's own (half a
// step: 2^-4 relative).  A power of two costs a floating format nothing but the top binade's
// slack; it makes append, read and attention agree bit for bit on what a code stands for.
//
// Bound by memory: each row is read once and written once.  16 lanes hold a row, 16 bytes
// (8 bf16 values) a lane, so a load instruction of a warp covers two whole rows; the row's
// maximum is four shuffles.  A block takes one head's rows of 32 or 64 consecutive tokens, k and v:
// whole stretches of a page (4 or 8 KB of codes), while the blocks of the other heads, next to it in
// the grid, fill in the packed rows between.  Its source loads are issued before it looks up
// which sequence and page each token belongs to, so the two latencies overlap.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "kda_attn.h"

namespace kda {

namespace {

constexpr int kKvThreads = 256;
constexpr int kLanes = 16;                    // lanes a row
constexpr int kGroups = kKvThreads / kLanes;  // rows at a time
// Rows that a group of lanes has in flight.  208873 tokens of 8 heads read: 2 rows 230 us, 4 rows
// 192 us (6.7 TB/s, the copy rate); 130049 tokens appended, e4m3: 1 row 159 us, 2 rows 148 us
// (5.4 TB/s), 4 rows 189 us, whose registers leave fewer blocks.
template <bool kRead>
constexpr int kInFlightRows = kRead ? 4 : 2;

// Where token t (packed) lives: its page, or -1 when nothing may be touched there.
// `strict`: a table entry -1 is an error (read); otherwise it only means "not here".
struct Slot {
  int64_t page;
  int slot;
};
__device__ Slot find_slot(const KvRows& a, int64_t t, bool strict) {
  // The sequence: first where an even packing would have it, then by bisection of
  // cu[lo] <= t < cu[hi] (offsets that run backwards end in some sequence and are refused below).
  int lo = 0, hi = a.n_seq;
  const int guess = static_cast<int>(t * a.n_seq / a.tokens);
  if (a.cu[guess] <= t && t < a.cu[guess + 1]) {
    lo = guess;
  } else {
    while (hi - lo > 1) {
      const int mid = lo + (hi - lo) / 2;
      if (a.cu[mid] <= t) lo = mid; else hi = mid;
    }
  }
  Slot s{-1, 0};
  const int64_t first = a.cu[lo], end = a.cu[lo + 1];
  const int64_t start = a.start[lo];
  const int64_t pos = start + (t - first);
  const int64_t idx = pos >> a.cache.page_log2;
  if (first < 0 || t < first || t >= end || end > a.tokens || start < 0 || idx >= a.max_pages) {
    report_status(a.status, 7 /* KDA_ERR_DEVICE_CHECK */);
    return s;
  }
  const int32_t page = a.page_table[static_cast<int64_t>(lo) * a.max_pages + idx];
  if (page < (strict ? 0 : -1) || page >= a.cache.n_pages) {
    report_status(a.status, 7 /* KDA_ERR_DEVICE_CHECK */);
    return s;
  }
  s.page = page;
  s.slot = static_cast<int>(pos & (a.cache.page_size - 1));
  return s;
}

__device__ __forceinline__ uint32_t cvt_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;  // the second operand lands in the low byte
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

__device__ __forceinline__ float2 bf2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// A row's 8 values of this lane into `dst` (row base), its scale byte into `sb`.
__device__ __forceinline__ void store_e4m3(uint4 x, uint8_t* dst, uint8_t* sb, int lane, bool live) {
  // bf16 magnitudes order like their bit patterns, infinities and NaN above everything
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
#pragma unroll
  for (int off = kLanes / 2; off; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
  // max|x| = 1.f * 2^(E - 127); 448 = 1.75 * 2^8
  int e = static_cast<int>(top >> 7) - 127 - 8 + ((top & 0x7fu) > 0x60u ? 1 : 0);
  const bool bad = e > 40;
  e = max(e, -40);
  const float inv = bad ? 0.f : __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  uint32_t c[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 p = bf2(w[2 * i]), q = bf2(w[2 * i + 1]);
    c[i] = cvt_e4m3x4(p.x * inv, p.y * inv, q.x * inv, q.y * inv);
  }
  if (!live) return;
  *reinterpret_cast<uint2*>(dst + lane * 8) = bad ? make_uint2(0, 0) : make_uint2(c[0], c[1]);
  if (lane == 0) *sb = bad ? 255 : static_cast<uint8_t>(e + 127);
}

__device__ __forceinline__ uint4 load_e4m3(uint2 c, uint32_t byte) {
  const float s = byte == 255 ? __uint_as_float(0x7fffffffu) : byte == 0 ? __uint_as_float(0x00400000u)
                                                                         : __uint_as_float(byte << 23);
  uint32_t out[4];
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h2;
    const uint16_t pair = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(pair));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);
    out[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

template <bool kE4m3, bool kRead>
__global__ void __launch_bounds__(kKvThreads) kv_rows_kernel(const __grid_constant__ KvRows a) {
  constexpr int kInFlight = kInFlightRows<kRead>, kBlockTokens = kGroups * kInFlight;
  __shared__ Slot slots[kBlockTokens];
  const int tid = threadIdx.x, lane = tid & (kLanes - 1), grp = tid / kLanes;
  const unsigned heads = a.cache.heads, tile = blockIdx.x / heads, head = blockIdx.x - tile * heads;
  const int64_t t0 = static_cast<int64_t>(tile) * kBlockTokens;
  const int n_tok = a.tokens - t0 < kBlockTokens ? static_cast<int>(a.tokens - t0) : kBlockTokens;
  uint16_t* k = static_cast<uint16_t*>(a.k) + head * a.k_stride[1] + 8 * lane;
  uint16_t* v = static_cast<uint16_t*>(a.v) + head * a.v_stride[1] + 8 * lane;
  bool live[kInFlight];
  uint4 x[kInFlight][2];
#pragma unroll
  for (int r = 0; r < kInFlight; ++r) {
    const int t = r * kGroups + grp;
    live[r] = t < n_tok;
    if constexpr (!kRead) {
      x[r][0] = x[r][1] = make_uint4(0, 0, 0, 0);
      if (live[r]) {
        x[r][0] = __ldcs(reinterpret_cast<const uint4*>(k + (t0 + t) * a.k_stride[0]));
        x[r][1] = __ldcs(reinterpret_cast<const uint4*>(v + (t0 + t) * a.v_stride[0]));
      }
    }
  }
  if (tid < n_tok) slots[tid] = find_slot(a, t0 + tid, kRead);
  __syncthreads();
  // the rows' places in the pools, in elements and (scales) bytes
  int64_t ko[kInFlight], vo[kInFlight], kso[kInFlight], vso[kInFlight];
#pragma unroll
  for (int r = 0; r < kInFlight; ++r) {
    const Slot s = slots[live[r] ? r * kGroups + grp : 0];
    live[r] = live[r] && s.page >= 0;
    const int64_t page = live[r] ? s.page : 0;
    ko[r] = page * a.cache.k_stride[0] + head * a.cache.k_stride[1] + s.slot * a.cache.k_stride[2];
    vo[r] = page * a.cache.v_stride[0] + head * a.cache.v_stride[1] + s.slot * a.cache.v_stride[2];
    kso[r] = page * a.cache.ks_stride[0] + head * a.cache.ks_stride[1] + s.slot;
    vso[r] = page * a.cache.vs_stride[0] + head * a.cache.vs_stride[1] + s.slot;
  }
  if constexpr (kRead) {
    uint2 c[kInFlight][2];
    uint32_t sb[kInFlight][2];
#pragma unroll
    for (int r = 0; r < kInFlight; ++r) {
      if (!live[r]) continue;
      if constexpr (kE4m3) {
        c[r][0] = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.cache.k) + ko[r]) + lane);
        c[r][1] = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.cache.v) + vo[r]) + lane);
        sb[r][0] = a.cache.ks[kso[r]];
        sb[r][1] = a.cache.vs[vso[r]];
      } else {
        x[r][0] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.cache.k) + ko[r]) + lane);
        x[r][1] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.cache.v) + vo[r]) + lane);
      }
    }
#pragma unroll
    for (int r = 0; r < kInFlight; ++r) {
      if (!live[r]) continue;
      if constexpr (kE4m3) {
        x[r][0] = load_e4m3(c[r][0], sb[r][0]);
        x[r][1] = load_e4m3(c[r][1], sb[r][1]);
      }
      const int64_t t = t0 + r * kGroups + grp;
      __stcs(reinterpret_cast<uint4*>(k + t * a.k_stride[0]), x[r][0]);
      __stcs(reinterpret_cast<uint4*>(v + t * a.v_stride[0]), x[r][1]);
    }
  } else {
#pragma unroll
    for (int r = 0; r < kInFlight; ++r) {
      if constexpr (kE4m3) {
        store_e4m3(x[r][0], static_cast<uint8_t*>(a.cache.k) + ko[r], a.cache.ks + kso[r], lane, live[r]);
        store_e4m3(x[r][1], static_cast<uint8_t*>(a.cache.v) + vo[r], a.cache.vs + vso[r], lane, live[r]);
      } else if (live[r]) {
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.cache.k) + ko[r])[lane] = x[r][0];
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.cache.v) + vo[r])[lane] = x[r][1];
      }
    }
  }
}

template <bool kRead>
cudaError_t launch_rows(const KvRows& a) {
  constexpr int kBlockTokens = kGroups * kInFlightRows<kRead>;
  const unsigned grid = static_cast<unsigned>((a.tokens + kBlockTokens - 1) / kBlockTokens * a.cache.heads);
  if (a.cache.e4m3)
    kv_rows_kernel<true, kRead><<<grid, kKvThreads, 0, a.stream>>>(a);
  else
    kv_rows_kernel<false, kRead><<<grid, kKvThreads, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const KvRows& a) { return launch_rows<false>(a); }
cudaError_t launch_kv_read(const KvRows& a) { return launch_rows<true>(a); }

}  // namespace kda
