// kda_attn_short.cu -- attention of few query rows a sequence over the paged cache.
//
// The mathematics: one pass over the keys with the running maximum m and sum l of a softmax,
//     x_j = scale log2(e) q . k_j,   m' = max(m, max_j x_j),   l <- l 2^(m-m') + sum_j 2^(x_j-m'),
//     O <- O 2^(m-m') + sum_j 2^(x_j-m') v_j,                  o = O / l,  lse = ln 2 (m + log2 l).
// E4M3 rows stand for code * 2^e.  The key's scale multiplies x_j; the value's joins the
// exponent, y_j = x_j + ev_j with m 14 below the maximum of the y_j, so P_j = 2^(y_j - m) <= 2^14 is
// already the weight of the codes (exact in f16) and l sums P_j 2^-ev_j; nothing is rescaled tile
// by tile.  P_j is rounded to f16: by 2^-11 of itself or, below 2^-14, by 2^-25, which is 2^-39 of the
// largest weight times value scale that the row sees.  (With m the maximum itself that was 2^-25: next
// to a value row 2^20 larger, however little attended, the others' weights had few bits left.)
//
// Bound by the cache's bytes: every key and value row is read once per (sequence, kv head),
// whatever the number of query heads that share it.  The H / kv_heads query heads of a kv
// head and the tokens of the step are the rows of one block (row r = token r / G, head r % G),
// 16 rows to a warp's mma.sync tile; at up to 64 rows the products need a small share of even
// the warp-level tensor rate (16 padded rows: 8 KFLOP per key against 512 bytes), so tcgen05's
// 128-row tiles would add latency and win nothing.
//
// Blocks: 4 warps compute, 1 warp walks the block's share and issues the copies (TMA, one box
// per page and tile of keys, 128-byte swizzle) into a ring of stages.  With up to 16 rows the 4
// warps split the keys of a tile (each with its own m, l, O, joined once at the end), with up to
// 32 rows two and two, with more each warp has 16 rows and all keys.  A tile is 64 keys of a
// bf16 cache, 128 of an E4M3 cache: as many bytes, and twice the independent work for a warp,
// whose conversions and products are then what bounds it.
//
// Work: the (sequence, head, row tile) items lie one after the other on a line of key tiles,
// and every block takes an equal share of that line, whole items or parts of them: ragged
// lengths and few long sequences fill the GPU alike.  A block has at most two partial items
// (its first and its last); their O, m, l go to the workspace and a second kernel, launched
// to overlap this one's tail, joins an item's parts in order.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cstdint>
#include <cstring>

#include "kda_attn.h"
#include "kda_attn_device.cuh"
#include "kda_ptx.cuh"

namespace kda {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kTileRows = 16;
constexpr int kMaxRows = kWarps * kTileRows;

template <bool kE4m3>
struct Stage {
  static constexpr int kTile = kE4m3 ? 128 : 64;  // keys
  // A block's least share, 256 keys: below that the joining costs more than it spreads.  One token
  // over 5000 keys, 96 heads on 8: bf16 2 / 4 / 8 tiles 16.1 / 14.5 / 15.0 us, e4m3 1 / 2 / 4 tiles
  // 16.3 / 14.3 / 16.3 us.
  static constexpr int kMinTiles = kE4m3 ? 2 : 4;
  static constexpr int kBytes = kTile * (kE4m3 ? 128 : 256);  // one of K, V
  static constexpr int kScales = kE4m3 ? 8 * 128 : 0;         // a 128-byte slot per page of the tile
  static constexpr int kTotal = 2 * kBytes + 2 * kScales;
  static constexpr int kCount = 3;
};
// What an item costs besides its keys (queries, joining the warps, output), in tiles.  For 1 / 2 / 4 /
// 6 / 8 / 12: 256 sequences of up to 8191 keys, 96 heads on 8, e4m3 389 / 369 / 343 / 346 / 352 /
// 362 us; 64 sequences of 4 tokens, window 4096, bf16 173 / 165 / 163-165 / 159 / 163 / 163 us;
// 37 sequences of up to 2000 keys, e4m3 - / - / 26.0 / 26.9 / 29.5 / 29.6 us.
constexpr int kItemCost = 4;
constexpr float kAbove = 14.f;  // e4m3: log2 of the largest weight
constexpr int kJoinBytes = 32 * 64 * 4 + 32 * 4 * 4;  // one warp's O and its (m, l) pairs
template <bool kE4m3>
constexpr int smem_bytes() {
  return 1024 + Stage<kE4m3>::kTotal * Stage<kE4m3>::kCount + kJoinBytes;
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <bool kHalf>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kHalf)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Address of the c-th 16-byte piece of a key's value row; whether a word holds a non-finite value.
template <bool kE4m3>
__device__ __forceinline__ uint32_t value_piece(uint32_t vb, uint32_t key, int c, int P, int p_log) {
  if constexpr (kE4m3) return vb + sw128(key, 16 * c);
  return vb + (key >> p_log) * (P * 256) + (c >> 3) * (P * 128) + sw128(key & (P - 1), 16 * (c & 7));
}
template <bool kE4m3>
__device__ __forceinline__ bool nonfinite(uint32_t w) {
  if constexpr (kE4m3) return (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

struct ShortParams {
  CUtensorMap tk, tv, tks, tvs;
  AttnArgs a;
  AttnSplit s;
};

template <bool kE4m3, int kRG>
__global__ void __launch_bounds__(kThreads, 2) attn_short_kernel(const __grid_constant__ ShortParams p) {
  using St = Stage<kE4m3>;
  constexpr int kTile = St::kTile;
  constexpr int kKG = kWarps / kRG;            // warps that split a tile's keys
  constexpr int kKeys = kTile / kKG;           // keys of a warp
  constexpr int kStep = kKeys < 32 ? kKeys : 32;  // of which so many at a time
  constexpr int kNT = kStep / 8;               // 8-key column tiles
  constexpr int kRT = kRG * kTileRows;         // rows of an item
  extern __shared__ uint8_t smem_raw[];
  __shared__ alignas(8) uint64_t full[St::kCount], empty[St::kCount];
  __shared__ JobRing jobs;
  uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < St::kCount; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], kWarps); }
    jobs.init(kWarps);
    fence_mbar_init();
    p.s.desc[blockIdx.x].last = -1;
  }
  pdl_launch_dependents();
  if (tid == kWarps * 32) {
    tma_prefetch_desc(&p.tk);
    tma_prefetch_desc(&p.tv);
  }
  const int P = min(a.cache.page_size, kTile), n_blk = kTile / P;
  __syncthreads();

  if (warp == kWarps) {  // ------------------------------------------------------ copies
    ItemWalk<kRT, kTile> walk(p.a, p.s);
    bool more = walk.start(lane);
    uint32_t it = 0;
    bool ok = true;
    const int blk = lane;
    for (uint32_t k = 0; ok; ++k) {
      if (!jobs.put(k, walk, more, lane)) {
        ok = false;
        break;
      }
      if (!more) break;
      const Item& w = walk.item;
      const KeyTiles kt = w.tiles;
      const int p_first = w.p_first(), p_last = w.p_last();
      const int32_t* table = a.page_table + static_cast<int64_t>(w.seq) * a.max_pages;
      for (int i = walk.begin; i < walk.end; ++i, ++it) {
        const int j0 = kt.at(i) * kTile + blk * P;  // first key of this lane's page block
        int page = -1;
        if (blk < n_blk && j0 <= p_last) {
          page = table[j0 >> a.cache.page_log2];
          if (page < 0 || page >= a.cache.n_pages) {
            const bool needed = a.window == 0 || j0 + P - 1 > p_first - a.window || j0 < a.n_sink;
            if (needed) report_status(a.status, 7 /* KDA_ERR_DEVICE_CHECK */);
            page = -1;  // out of the tensor map's range: the copy fills with zeros
          }
        }
        const uint32_t s = it % St::kCount;
        if (it >= St::kCount && !bar_wait(&empty[s], ((it / St::kCount) - 1) & 1)) {
          ok = false;
          break;
        }
        if (it == static_cast<uint32_t>(a.stall)) continue;
        if (lane == 0) mbar_arrive_expect_tx(&full[s], 2 * St::kBytes + (kE4m3 ? 2 * kTile : 0));
        __syncwarp();
        if (blk < n_blk) {
          uint8_t* st = sm + s * St::kTotal;
          const int slot = j0 & (a.cache.page_size - 1);
          if constexpr (kE4m3) {
            tma_load_4d(st + blk * P * 128, &p.tk, &full[s], 0, slot, w.head, page);
            tma_load_4d(st + St::kBytes + blk * P * 128, &p.tv, &full[s], 0, slot, w.head, page);
            tma_load_3d(st + 2 * St::kBytes + blk * 128, &p.tks, &full[s], slot, w.head, page);
            tma_load_3d(st + 2 * St::kBytes + St::kScales + blk * 128, &p.tvs, &full[s], slot, w.head, page);
          } else {
            tma_load_5d(st + blk * P * 256, &p.tk, &full[s], 0, slot, 0, w.head, page);
            tma_load_5d(st + St::kBytes + blk * P * 256, &p.tv, &full[s], 0, slot, 0, w.head, page);
          }
        }
      }
      more = ok && walk.next();
    }
    if (!ok) report_status(a.status, 6 /* KDA_ERR_TIMEOUT */);
    drain_ring(full, St::kCount, it);
    return;
  }

  // -------------------------------------------------------------------------- products
  const int g = lane >> 2, t = lane & 3;
  const int rg = warp / kKG, kg = warp % kKG;
  float* join = reinterpret_cast<float*>(sm + St::kTotal * St::kCount);
  const int p_log = 31 - __clz(P);
  const int G = a.H / a.cache.heads;
  uint32_t it = 0;
  bool dead = false;
  JobFeed feed{jobs, dead};
  for (;;) {
    const Job* jp = feed.next();
    // The four warps leave together: one alone would be missing at the barriers among them.
    dead = named_bar_any(1, kWarps * 32, dead);
    if (dead || !jp) break;
    const Job& w = *jp;
    // this thread's rows g and g + 8 of the warp's 16: position, query fragments
    int pos[2];
    float cs[2];  // scale in log2 units (times the query row's own power of two)
    uint32_t qf[8][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = w.row0 + rg * kTileRows + g + 8 * r;
      const bool live = row < w.rows;
      const int tok = live ? row / G : 0, gh = live ? row - tok * G : 0;
      pos[r] = live ? w.len - w.n_tok + tok : -1;
      const uint16_t* q = static_cast<const uint16_t*>(a.q) + w.q_base + tok * a.q_stride[1] +
                          (static_cast<int64_t>(w.head) * G + gh) * a.q_stride[2];
      cs[r] = a.scale_log2;
      if constexpr (kE4m3) {
        // channel order of the codes' 16-byte loads: this thread's chunks t and t + 4, 4 channels a step
        uint32_t x[16];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 u = live ? *reinterpret_cast<const uint4*>(q + (c >> 1) * 64 + 16 * t + (c & 1) * 8) : make_uint4(0, 0, 0, 0);
          x[4 * c] = u.x; x[4 * c + 1] = u.y; x[4 * c + 2] = u.z; x[4 * c + 3] = u.w;
        }
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < 16; ++c) top = max(top, max(x[c] & 0x7fffu, (x[c] >> 16) & 0x7fffu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = query_exponent(top);
        const float inv = pow2i(-e);
        cs[r] *= pow2i(e);
#pragma unroll
        for (int c = 0; c < 16; ++c)
          qf[c >> 1][r + 2 * (c & 1)] = pack_half2(__uint_as_float(x[c] << 16) * inv, __uint_as_float(x[c] & 0xffff0000u) * inv);
      } else {
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          qf[s][r] = live ? *reinterpret_cast<const uint32_t*>(q + 16 * s + 2 * t) : 0;
          qf[s][r + 2] = live ? *reinterpret_cast<const uint32_t*>(q + 16 * s + 8 + 2 * t) : 0;
        }
      }
    }
    float o[16][4];
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    const int begin = w.begin, end = w.end;
    for (int i = begin; i < end; ++i, ++it) {
      const uint32_t s = it % St::kCount;
      // after a wait that ran out the loop goes on without waiting, so that every barrier is still met
      if (!dead && !bar_wait(&full[s], (it / St::kCount) & 1)) dead = true;
      const uint32_t kb = smem_u32(sm + s * St::kTotal), vb = kb + St::kBytes;
      const int t_first = w.tile(i) * kTile, t_last = t_first + kTile - 1;
      const bool edge = t_last > w.p_first || (a.window > 0 && t_first <= w.p_last - a.window && t_last >= a.n_sink);
      if (edge) {
        // 0 * NaN must not reach a row that does not see the key: value rows with a non-finite
        // value are cleared, and the rows that do see one become NaN here.
        uint32_t bad[(kKeys + 31) / 32];
#pragma unroll
        for (int q = 0; q < (kKeys + 31) / 32; ++q) {
          const uint32_t key = kg * kKeys + 32 * q + lane;
          bool has = false;
          if (32 * q + lane < kKeys) {
#pragma unroll 1
            for (int c = 0; c < (kE4m3 ? 8 : 16); ++c) {
              const uint4 v = lds128(value_piece<kE4m3>(vb, key, c, P, p_log));
              has |= nonfinite<kE4m3>(v.x) | nonfinite<kE4m3>(v.y) | nonfinite<kE4m3>(v.z) | nonfinite<kE4m3>(v.w);
            }
          }
          bad[q] = __ballot_sync(0xffffffffu, has);
        }
        if constexpr (kRG > 1) named_bar_sync(2 + kg, 32 * kRG);  // the warps that share these keys have all looked
#pragma unroll
        for (int q = 0; q < (kKeys + 31) / 32; ++q) {
          if (!bad[q]) continue;
          if ((bad[q] >> lane) & 1) {
#pragma unroll 1
            for (int c = 0; c < (kE4m3 ? 8 : 16); ++c)
              sts128(value_piece<kE4m3>(vb, kg * kKeys + 32 * q + lane, c, P, p_log), make_uint4(0, 0, 0, 0));
          }
          for (uint32_t m = bad[q]; m; m &= m - 1) {
            const int key = t_first + kg * kKeys + 32 * q + __ffs(m) - 1;
#pragma unroll
            for (int r = 0; r < 2; ++r)
              if (sees(pos[r], key, a.window, a.n_sink)) l[r] = __uint_as_float(0x7fffffffu);
          }
        }
        fence_proxy_async_smem();
        if constexpr (kRG > 1) named_bar_sync(2 + kg, 32 * kRG);
        else __syncwarp();
      }
#pragma unroll 1
      for (int k0 = kg * kKeys; k0 < (kg + 1) * kKeys; k0 += kStep) {
      const int key0 = t_first + k0;  // first key of this step
      float x[kNT][4];
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[n][e] = 0.f;
      // ---- q . k
      if constexpr (kE4m3) {
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          const uint32_t row = k0 + n * 8 + g;
          const uint4 u0 = lds128(kb + sw128(row, 16 * t)), u1 = lds128(kb + sw128(row, 64 + 16 * t));
          const uint32_t c[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
#pragma unroll
          for (int e = 0; e < 8; ++e)
          {
            uint32_t lo, hi;
            e4m3_half4(c[e], lo, hi);
            mma16816<true>(x[n], qf[e], lo, hi);
          }
        }
      } else {
#pragma unroll
        for (int n = 0; n < kNT; n += 2) {
          const uint32_t row = k0 + n * 8 + (lane & 7) + ((lane >> 4) << 3);
          const uint32_t base = kb + (row >> p_log) * (P * 256), rr = row & (P - 1);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            uint32_t b[4];
            const uint32_t byte = 32 * (e & 3) + 16 * ((lane >> 3) & 1);
            ldsm4(base + (e >> 2) * (P * 128) + sw128(rr, byte), b);
            mma16816<false>(x[n], qf[e], b[0], b[1]);
            mma16816<false>(x[n + 1], qf[e], b[2], b[3]);
          }
        }
      }
      // ---- scaled scores; hidden ones to -inf
      float rv[kE4m3 ? kNT : 1][2];  // 2^-ev
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        if constexpr (kE4m3) {
          const uint32_t key = k0 + n * 8 + 2 * t;
          const uint8_t* sc = sm + s * St::kTotal + 2 * St::kBytes + (key >> p_log) * 128 + (key & (P - 1));
          const uint32_t k2 = *reinterpret_cast<const uint16_t*>(sc), v2 = *reinterpret_cast<const uint16_t*>(sc + St::kScales);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float ks = scale_value(k2 >> (8 * h)), ev = scale_exponent(v2 >> (8 * h));
            rv[n][h] = scale_inverse(v2 >> (8 * h));
            x[n][h] = fmaf(x[n][h] * ks, cs[0], ev);
            x[n][h + 2] = fmaf(x[n][h + 2] * ks, cs[1], ev);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[n][e] *= cs[e >> 1];
        }
      }
      if (edge) {
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!sees(pos[e >> 1], key0 + n * 8 + 2 * t + (e & 1), a.window, a.n_sink)) x[n][e] = -INFINITY;
      }
      // ---- running maximum and sum
      float corr[2], base[2];
      bool moved = false;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float mx = x[0][2 * r];
#pragma unroll
        for (int n = 0; n < kNT; ++n) mx = fmaxf(mx, fmaxf(x[n][2 * r], x[n][2 * r + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        if constexpr (kE4m3) mx = __fadd_ru(mx, -kAbove);  // never further below, however large
        const float mn = fmaxf(m[r], mx);
        base[r] = mn == -INFINITY ? 0.f : mn;
        corr[r] = exp2_fast(m[r] - base[r]);
        moved |= mn != m[r];
        m[r] = mn;
        l[r] *= corr[r];
      }
      uint32_t pf[kNT][2];
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float p0 = exp2_fast(x[n][2 * r] - base[r]), p1 = exp2_fast(x[n][2 * r + 1] - base[r]);
          // weights rounded once, to the values' type: f16 2^-11, bf16 2^-8 at most; l keeps 32 bits
          if constexpr (kE4m3) {
            float r0 = rv[n][0], r1 = rv[n][1];
            if (edge) {  // a hidden key's scale may be that of a NaN row; that of a visible one counts, however small its weight
              r0 = x[n][2 * r] == -INFINITY ? 0.f : r0;
              r1 = x[n][2 * r + 1] == -INFINITY ? 0.f : r1;
            }
            l[r] = fmaf(p0, r0, fmaf(p1, r1, l[r]));
            pf[n][r] = pack_half2(p0, p1);
          } else {
            l[r] += p0 + p1;
            pf[n][r] = pack_bf162(p0, p1);
          }
        }
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          o[n][0] *= corr[0]; o[n][1] *= corr[0];
          o[n][2] *= corr[1]; o[n][3] *= corr[1];
        }
      }
      // ---- P V
#pragma unroll
      for (int n = 0; n < kNT; n += 2) {  // 16 keys
        const uint32_t pa[4] = {pf[n][0], pf[n][1], pf[n + 1][0], pf[n + 1][1]};
        if constexpr (kE4m3) {
          const uint32_t row = k0 + n * 8 + 2 * t;
          uint32_t c[4][4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const uint4 u = lds128(vb + sw128(row + (r & 1) + 8 * (r >> 1), 16 * g));
            c[r][0] = u.x; c[r][1] = u.y; c[r][2] = u.z; c[r][3] = u.w;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {  // 4 channels: column tiles 4e .. 4e + 3
            const uint32_t a0 = __byte_perm(c[0][e], c[1][e], 0x5140), a1 = __byte_perm(c[0][e], c[1][e], 0x7362);
            const uint32_t b0 = __byte_perm(c[2][e], c[3][e], 0x5140), b1 = __byte_perm(c[2][e], c[3][e], 0x7362);
            uint32_t ba[4], bb[4];
            e4m3_half4(a0, ba[0], ba[1]);
            e4m3_half4(a1, ba[2], ba[3]);
            e4m3_half4(b0, bb[0], bb[1]);
            e4m3_half4(b1, bb[2], bb[3]);
#pragma unroll
            for (int q = 0; q < 4; ++q) mma16816<true>(o[4 * e + q], pa, ba[q], bb[q]);
          }
        } else {
          const uint32_t row = k0 + n * 8 + (lane & 15);
          const uint32_t base_v = vb + (row >> p_log) * (P * 256), rr = row & (P - 1);
#pragma unroll
          for (int c = 0; c < 16; c += 2) {
            uint32_t b[4];
            ldsm4t(base_v + (c >> 3) * (P * 128) + sw128(rr, 16 * ((c & 7) + (lane >> 4))), b);
            mma16816<false>(o[c], pa, b[0], b[1]);
            mma16816<false>(o[c + 1], pa, b[2], b[3]);
          }
        }
      }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }

    // ---- a NaN value row left -inf (see scale_inverse); one row's sum lies over the 4 lanes that share it
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (kE4m3 && l[r] < 0.f) l[r] = __uint_as_float(0x7fffffffu);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
    // ---- join the warps that split the keys, in order
#pragma unroll
    for (int k = 1; k < kKG; ++k) {
#pragma unroll
      for (int q = 0; q < kRG; ++q) {  // one buffer: the row groups take turns
        if (rg == q && kg == k) {
#pragma unroll
          for (int n = 0; n < 16; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) join[(n * 4 + e) * 32 + lane] = o[n][e];
          reinterpret_cast<float4*>(join + 64 * 32)[lane] = make_float4(m[0], m[1], l[0], l[1]);
        }
        named_bar_sync(1, kWarps * 32);
        if (rg == q && kg == 0) {
          const float4 ml = reinterpret_cast<const float4*>(join + 64 * 32)[lane];
          const float om[2] = {ml.x, ml.y}, ol[2] = {ml.z, ml.w};
          float c0[2], c1[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float mn = fmaxf(m[r], om[r]), b = mn == -INFINITY ? 0.f : mn;
            c0[r] = exp2_fast(m[r] - b); c1[r] = exp2_fast(om[r] - b);
            m[r] = mn;
            l[r] = l[r] * c0[r] + ol[r] * c1[r];
          }
#pragma unroll
          for (int n = 0; n < 16; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = o[n][e] * c0[e >> 1] + join[(n * 4 + e) * 32 + lane] * c1[e >> 1];
        }
        named_bar_sync(1, kWarps * 32);
      }
    }
    if (kg == 0) {
      const int slot = w.slot;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int lr = rg * kTileRows + g + 8 * r, row = w.row0 + lr;
        if (row >= w.rows) continue;
        // channels of o[n][2r], o[n][2r + 1]: bf16 8n + 2t, + 1; e4m3 32t + n, 32t + 16 + n
        if (slot >= 0) {
          float* dst = p.s.part_o + (static_cast<int64_t>(slot) * p.s.part_rows + lr) * 128;
          if constexpr (kE4m3) {
#pragma unroll
            for (int n = 0; n < 16; n += 4) {
              *reinterpret_cast<float4*>(dst + 32 * t + n) = make_float4(o[n][2 * r], o[n + 1][2 * r], o[n + 2][2 * r], o[n + 3][2 * r]);
              *reinterpret_cast<float4*>(dst + 32 * t + 16 + n) =
                  make_float4(o[n][2 * r + 1], o[n + 1][2 * r + 1], o[n + 2][2 * r + 1], o[n + 3][2 * r + 1]);
            }
          } else {
#pragma unroll
            for (int n = 0; n < 16; ++n) *reinterpret_cast<float2*>(dst + 8 * n + 2 * t) = make_float2(o[n][2 * r], o[n][2 * r + 1]);
          }
          if (t == 0) p.s.part_ml[static_cast<int64_t>(slot) * p.s.part_rows + lr] = make_float2(m[r], l[r]);
        } else {
          const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
          const int64_t orow = (w.base + row / G) * a.H + static_cast<int64_t>(w.head) * G + row % G;
          uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + orow * 128);
          if constexpr (kE4m3) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int n = 0; n < 16; n += 8)
                *reinterpret_cast<uint4*>(dst + 16 * t + 8 * h + n / 2) =
                    make_uint4(pack_bf162(o[n][2 * r + h] * inv, o[n + 1][2 * r + h] * inv),
                               pack_bf162(o[n + 2][2 * r + h] * inv, o[n + 3][2 * r + h] * inv),
                               pack_bf162(o[n + 4][2 * r + h] * inv, o[n + 5][2 * r + h] * inv),
                               pack_bf162(o[n + 6][2 * r + h] * inv, o[n + 7][2 * r + h] * inv));
          } else {
#pragma unroll
            for (int n = 0; n < 16; ++n) dst[4 * n + t] = pack_bf162(o[n][2 * r] * inv, o[n][2 * r + 1] * inv);
          }
          if (a.lse && t == 0) a.lse[orow] = lse_of(m[r], l[r]);
        }
      }
    }
    feed.done(lane);
  }
  if (dead && lane == 0) report_status(a.status, 6 /* KDA_ERR_TIMEOUT */);
}

template <bool kE4m3, int kRG>
cudaError_t launch_short(const ShortParams& p, int grid) {
  constexpr int bytes = smem_bytes<kE4m3>();
  auto kern = attn_short_kernel<kE4m3, kRG>;
  static SmemOptIn opt_in;
  const cudaError_t e = opt_in(reinterpret_cast<const void*>(kern), bytes);
  if (e != cudaSuccess) return e;
  if (p.a.cu) return launch_after(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), bytes, p.a.stream, p);
  kern<<<grid, kThreads, bytes, p.a.stream>>>(p);
  return cudaGetLastError();
}

int row_groups(int rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }

bool make_maps(ShortParams& p, int tile) {
  const KvCache& c = p.a.cache;
  return make_cache_maps(c, tile, 2, &p.tk, &p.tv) && (!c.e4m3 || make_scale_maps(c, tile, &p.tks, &p.tvs));
}

}  // namespace

size_t attn_decode_workspace(int n_seq, int n_tok, int H, int kv_heads, int num_sms) {
  return attn_split_bytes(2 * num_sms, kTileRows * row_groups(n_tok * (H / kv_heads)), 0);
}

cudaError_t launch_attn_decode(const AttnArgs& a, int num_sms) {
  const int G = a.H / a.cache.heads, rg = row_groups(a.n_tok * G);
  ShortParams p;
  memset(&p, 0, sizeof(p));
  p.a = a;
  const int grid = 2 * num_sms;
  attn_split_layout(&p.s, a.workspace, grid, kTileRows * rg, 0);
  const int tile = a.cache.e4m3 ? Stage<true>::kTile : Stage<false>::kTile;
  p.s.min_tiles = a.cache.e4m3 ? Stage<true>::kMinTiles : Stage<false>::kMinTiles;
  p.s.item_cost = kItemCost;
  if (!make_maps(p, tile)) return cudaErrorInvalidValue;
  cudaError_t e;
  if (a.cache.e4m3)
    e = rg == 1 ? launch_short<true, 1>(p, grid) : rg == 2 ? launch_short<true, 2>(p, grid) : launch_short<true, 4>(p, grid);
  else
    e = rg == 1 ? launch_short<false, 1>(p, grid) : rg == 2 ? launch_short<false, 2>(p, grid) : launch_short<false, 4>(p, grid);
  if (e != cudaSuccess) return e;
  return launch_attn_join(p.a, p.s);
}

// Which kernel takes a chunk.  This one for up to 64 rows (tokens x shared heads) a sequence on
// average, where it reads the keys once, and for little work altogether, where the other's longer
// way to its first product counts: 77 tokens of 3 sequences over 1500 keys, 16 heads on 2: 25 us
// here, 37 us there; but 128 tokens of 8 sequences over 8000 keys, 96 heads on 8: 96 us here,
// 63 us there.  The work is bounded by the page table's width, the lengths being on the device.
bool attn_short_chunks(int n_seq, int64_t tokens, int H, int kv_heads, int64_t most_keys) {
  if (tokens * (H / kv_heads) <= static_cast<int64_t>(kMaxRows) * n_seq) return true;
  return 512.0 * tokens * H * static_cast<double>(most_keys) <= 2.5e9;
}

size_t attn_prefill_workspace(int n_seq, int64_t tokens, int H, int kv_heads, int num_sms) {
  const size_t here = attn_split_bytes(2 * num_sms, kMaxRows, attn_max_items(n_seq, tokens, H / kv_heads, kMaxRows));
  const size_t there = attn_chunk_workspace(n_seq, tokens, H / kv_heads, num_sms);
  return here > there ? here : there;
}

cudaError_t launch_attn_prefill(const AttnArgs& a, int num_sms) {
  if (!attn_short_chunks(a.n_seq, a.tokens, a.H, a.cache.heads, static_cast<int64_t>(a.max_pages) * a.cache.page_size))
    return launch_attn_chunk(a, num_sms);
  const int G = a.H / a.cache.heads;
  ShortParams p;
  memset(&p, 0, sizeof(p));
  p.a = a;
  const int grid = 2 * num_sms;
  attn_split_layout(&p.s, a.workspace, grid, kMaxRows, attn_max_items(a.n_seq, a.tokens, G, kMaxRows));
  const int tile = a.cache.e4m3 ? Stage<true>::kTile : Stage<false>::kTile;
  p.s.min_tiles = a.cache.e4m3 ? Stage<true>::kMinTiles : Stage<false>::kMinTiles;
  p.s.item_cost = kItemCost;
  if (!make_maps(p, tile)) return cudaErrorInvalidValue;
  cudaError_t e = launch_attn_plan(a, p.s, kMaxRows, tile);
  if (e != cudaSuccess) return e;
  e = a.cache.e4m3 ? launch_short<true, 4>(p, grid) : launch_short<false, 4>(p, grid);
  if (e != cudaSuccess) return e;
  return launch_attn_join(p.a, p.s);
}

}  // namespace kda
