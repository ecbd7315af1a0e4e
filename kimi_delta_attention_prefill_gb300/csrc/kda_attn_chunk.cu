// kda_attn_chunk.cu -- attention of a chunk of new tokens over the paged cache (tcgen05).
//
// The mathematics is that of kda_attn_short.cu (one pass with a running maximum); here the
// rows are many, so the products bound it: 4 * 128 FLOPs per visible (query head, key).
//
// A block (one per SM) holds 256 query rows of one kv head -- row r is token r / G, query head
// r % G of the head's group, so 8 tokens of a group of 12 fill 96 rows and no tile is padded
// by the group -- as two 128-row tiles A and B, and visits key tiles of 128:
//     S = Q K^T    tcgen05, both operands in shared memory, S (fp32) in TMEM
//     P = 2^(S c - m), rounded to the values' type, over S's columns
//     O += P V     tcgen05, P from TMEM, V from shared memory (MN-major)
// TMEM: S_A, S_B, O_A, O_B, 128 columns each: all 512.
//
// Warps: two groups of four for the softmax of A and of B (thread = row = TMEM lane: a row's
// maximum and sum need no exchange), one warp each that issues A's and B's products, one for
// the copies; the others bring the next item's queries and, for an E4M3 cache, turn the codes
// into f16 tiles (exact).  The tensor core runs P V and the next Q K^T of one tile while the
// other tile is in its softmax.
//
// The maximum is lazy: O is rescaled only when a row's maximum has grown by more than 2^8 since
// the last time, which random rows do in their first tiles only.
//
// What f16 weights (E4M3) lose: 2^-11 of themselves or, below 2^-14, 2^-25.  A new maximum of the scores
// times the tile's largest value scale weighs 2^7, that scale being at most 2^8 above the one of
// the row that has the maximum: 2^-25 is at most 2^-24 of the largest weight times value scale that a
// query row sees.
//
// Work is split as in kda_attn_short.cu: equal shares of the line of key tiles, at most two
// partial items a block, joined by attn_join_kernel.
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

constexpr int kThreads = 512;
constexpr int kTile = 128;
constexpr int kRows = 256;
constexpr int kPanel = kTile * 128;     // 64 channels of 128 rows, 16-bit
constexpr int kSlot = 2 * kPanel;       // one tile of K or V (or 128 rows of Q) as 16-bit values
constexpr int kStage = kTile * 128;     // a tile of codes
// A block's least share: 1, 2 and 4 tiles took the same time (400 tokens of a prompt, 32 us).
constexpr int kMinTiles = 2;
// What an item costs besides its keys (queries, the pipeline's filling and draining, output), in
// tiles.  A prompt of 8192, 96 heads on 8: 3 / 4 / 5 / 6 / 12 took 1279 / 1270 / 1285 / 1296 / 1373 us
// (bf16), 4 / 5 1719 / 1594 us (e4m3).
constexpr int kItemCost = 5;

template <bool kE4m3>
struct Cfg {
  // Four slots are as good as five; with three the next keys' slot is free only once the last P V
  // has read it, and both wait (2.0 ms against 2.7 ms over 30 K keys).
  static constexpr int kSlots = kE4m3 ? 4 : 5;
  static constexpr int kStages = kE4m3 ? 2 : 0;
  static constexpr int kSmQ = 0;
  static constexpr int kSmKV = 2 * kSlot;
  static constexpr int kSmStage = kSmKV + kSlots * kSlot;
  static constexpr int kSmScale = kSmStage + kStages * kStage;         // [stages][128] scale bytes
  static constexpr int kSmVec = kSmScale + kStages * kTile;            // [2 tiles][keys, values][128] scale bytes (wide tiles)
  static constexpr int kSmExp = kSmVec + (kE4m3 ? 2 * 2 * kTile : 0);  // [2 items][256] query rows' exponents (int8)
  static constexpr int kSmBytes = kSmExp + (kE4m3 ? 2 * kRows : 0) + 1024;
};

constexpr int kReach = 8;
constexpr uint32_t kLeast = 127 - 40;  // the least scale byte that kda_kv_append writes; rows of zeros have it

// E4M3: what the f16 tiles of a key tile were scaled by (see convert_group).
struct TileScale {
  float k;        // 2^E of the keys
  float v;        // E of the values
  int wide_k, wide_v;  // their scales lie too far apart: tiles of codes, scales key by key
};

struct Bars {
  uint64_t full[5], empty[5];      // slots of K / V tiles
  uint64_t v_ask, v_ok;            // bf16: an edge tile's values are there / have been looked through
  uint64_t st_full[2], st_empty[2];  // stages of codes
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_full[2][2], pv_done[2], o_full[2];
  uint64_t turn[2];                // the product warps' turns
  uint64_t drain[2];
  JobRing jobs;
  alignas(16) uint32_t bad[5][4];  // by slot, of bf16 edge tiles only: keys with a non-finite value row
  TileScale tile[2];               // e4m3, by tile parity
  uint32_t tmem;
};

struct ChunkParams {
  CUtensorMap tk, tv;
  AttnArgs a;
  AttnSplit s;
};

using Walk = ItemWalk<kRows, kTile>;

// Whether some row of the item does not see some key of key tile t.
__device__ __forceinline__ bool edge_tile(const AttnArgs& a, int t, int p_first, int p_last) {
  const int first = t * kTile, last = first + kTile - 1;
  return last > p_first || (a.window > 0 && first <= p_last - a.window && last >= a.n_sink);
}

// ---------------------------------------------------------------------------- copies
// The copy warp is furthest ahead of all: it walks the share and hands out the jobs.
template <bool kE4m3>
__device__ void load_warp(const ChunkParams& p, uint8_t* sm, Bars& b, int lane) {
  using C = Cfg<kE4m3>;
  const AttnArgs& a = p.a;
  const int P = min(a.cache.page_size, kTile), n_blk = kTile / P;
  const int blk = kE4m3 ? lane : lane >> 1, panel = kE4m3 ? 0 : lane & 1;
  constexpr int kRing = kE4m3 ? C::kStages : C::kSlots;
  uint64_t* full = kE4m3 ? b.st_full : b.full;
  uint64_t* empty = kE4m3 ? b.st_empty : b.empty;
  if (lane == 0) {
    tma_prefetch_desc(&p.tk);
    tma_prefetch_desc(&p.tv);
  }
  uint32_t n = 0, k = 0;
  Walk walk(p.a, p.s);
  bool more = walk.start(lane), ok = true;
  for (; ok; ++k) {
    if (!b.jobs.put(k, walk, more, lane)) {
      ok = false;
      break;
    }
    const Item& w = walk.item;
    if (!more) break;
    const int p_first = w.p_first(), p_last = w.p_last(), begin = walk.begin, end = walk.end, head = w.head;
    const int32_t* table = a.page_table + static_cast<int64_t>(w.seq) * a.max_pages;
    const KeyTiles kt = w.tiles;
    for (int i = begin; ok && i < end; ++i) {
      const int j0 = kt.at(i) * kTile + blk * P;
      int page = -1;
      if (blk < n_blk && j0 <= p_last) {
        page = table[j0 >> a.cache.page_log2];
        if (page < 0 || page >= a.cache.n_pages) {
          const bool needed = a.window == 0 || j0 + P - 1 > p_first - a.window || j0 < a.n_sink;
          if (needed) report_status(a.status, 7 /* KDA_ERR_DEVICE_CHECK */);
          page = -1;  // out of the tensor map's range: the copy fills with zeros
        }
      }
      const int slot = j0 & (a.cache.page_size - 1);
      const int pages = __popc(__ballot_sync(0xffffffffu, page >= 0));
#pragma unroll
      for (int kv = 0; kv < 2; ++kv, ++n) {
        const uint32_t s = n % kRing;
        if (n >= kRing && !bar_wait(&empty[s], (n / kRing - 1) & 1)) {
          ok = false;
          break;
        }
        if (n == static_cast<uint32_t>(a.stall)) continue;
        if constexpr (kE4m3) {
          if (blk < n_blk && page < 0) {  // no page: rows of zeros, as they are kept
            uint32_t* sc = reinterpret_cast<uint32_t*>(sm + C::kSmScale + s * kTile + blk * P);
            for (int e = 0; e < P / 4; ++e) sc[e] = kLeast * 0x01010101u;
            fence_proxy_async_smem();
          }
          __syncwarp();
        }
        if (lane == 0) mbar_arrive_expect_tx(&full[s], kE4m3 ? kStage + pages * P : kSlot);
        __syncwarp();
        if (blk < n_blk) {
          if constexpr (kE4m3) {
            tma_load_4d(sm + C::kSmStage + s * kStage + blk * P * 128, kv ? &p.tv : &p.tk, &full[s], 0, slot, head, page);
            const int64_t* st = kv ? a.cache.vs_stride : a.cache.ks_stride;
            if (page >= 0)
              bulk_load(sm + C::kSmScale + s * kTile + blk * P, (kv ? a.cache.vs : a.cache.ks) + page * st[0] + head * st[1] + slot,
                        P, &full[s]);
          } else {
            uint8_t* st = sm + C::kSmKV + s * kSlot;
            tma_load_5d(st + panel * kPanel + blk * P * 128, kv ? &p.tv : &p.tk, &full[s], 0, slot, panel, head, page);
          }
        }
      }
    }
    more = ok && walk.next();
  }
  if (!ok) report_status(a.status, 6 /* KDA_ERR_TIMEOUT */);
  drain_ring(full, kRing, n);
}

// -------------------------------------------------------------------------- products
// One warp issues tile A's products, another tile B's.  The whole warp walks, so that
// addresses and descriptors stay in uniform registers; one lane issues.
template <bool kE4m3>
__device__ void mma_warp(const ChunkParams& p, uint8_t* sm, Bars& b, int t) {
  using C = Cfg<kE4m3>;
  const AttnArgs& a = p.a;
  const uint32_t leader = elect_one_sync();
  constexpr uint32_t id_qk = idesc_f16(128, 128, !kE4m3, false, false), id_pv = idesc_f16(128, 128, !kE4m3, false, true);
  const uint64_t dq = smem_desc(smem_u32(sm + C::kSmQ) + t * kSlot, 16, 1024, kSwizzle128B);
  const uint64_t dk = smem_desc(smem_u32(sm + C::kSmKV), 16, 1024, kSwizzle128B);
  const uint64_t dv = smem_desc(smem_u32(sm + C::kSmKV), kPanel, 1024, kSwizzle128B);
  bool dead = false;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!dead && !bar_wait(bar, parity & 1)) dead = true;
  };
  auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
  uint32_t items = 0, edges = 0, tiles = 0, turns = 0;
  uint32_t sk = 0, pk = 0;  // the ring's slot and phase of the next tile to be used
  auto step = [&] {
    if (++sk == C::kSlots) { sk = 0; pk ^= 1; }
  };
  JobFeed feed{b.jobs, dead};
  while (const Job* jp = feed.next()) {
    const int begin = uniform(jp->begin), end = uniform(jp->end), sink = uniform(jp->sink), lo = uniform(jp->lo);
    const int p_first = uniform(jp->p_first), p_last = uniform(jp->p_last);
    const int last_row = uniform(jp->last_row) - uniform(jp->row0);
    const bool mine = last_row >= 128 * t, both = last_row >= 128;  // the item has rows of this tile, of both
    feed.done(threadIdx.x & 31);
    wait(&b.q_full, items);
    ++items;
    // An edge tile's values are looked through by other warps before they are used.  Edge tiles
    // are asked for one by one here, where every phase of the barrier is seen, so that those
    // warps need not follow the ring.
    bool edge = false;
    auto values = [&](int i, uint32_t slot, uint32_t phase) {
        wait(&b.full[slot], phase);
        edge = !kE4m3 && edge_tile(a, i < sink ? i : lo + (i - sink), p_first, p_last);
        if (edge && leader) mbar_arrive(&b.v_ask);
    };
    if (!mine) {  // only keeps the other warps' counts
        if (leader) mbar_arrive(&b.q_empty);
        for (int i = begin; i < end; ++i) {
          wait(&b.full[sk], pk);
          if (leader) mbar_arrive(&b.empty[sk]);
          step();
          values(i, sk, pk);
          if (edge) wait(&b.v_ok, edges++);
          if (leader) mbar_arrive(&b.empty[sk]);
          step();
        }
        continue;
    }
    // The tensor core has products queued while this warp waits: what can be waited for early is
    // waited for behind a product, so that nothing but the softmax comes before P V.  (One loop
    // with one place for each product: this warp's code is fetched anew every time round.)
    uint32_t sv = 0;
#pragma unroll 1
    for (int i = begin - 1; i < end; ++i) {
        const bool pv = i >= begin, more = i + 1 < end;
        if (more) wait(&b.full[sk], pk);
        if (pv) {
          // A and B take turns of one P V and the next Q K^T each.  Left alone their products mix and
          // end together, and then both tiles are in their softmax while the tensor core has nothing.
          if (both && (t == 1 || turns > 0)) wait(&b.turn[t], t == 1 ? turns : turns - 1);
          turns += both;
#pragma unroll
          for (int h = 1; h >= 0; --h) {  // the weights come in two halves of 64 keys, the later keys first
            wait(&b.p_full[t][h], tiles);
            if (h == 1 && edge) wait(&b.v_ok, edges++);
            __syncwarp();
            tc_fence_after();
            const uint64_t db = dv + sv * (kSlot >> 4) + h * (4 * 2048 >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_f16_ta_if(leader, 256 + 128 * t, 128 * t + 64 * h + 8 * kk, db + kk * (2048 >> 4), id_pv,
                            kk > 0 || h == 0 || i > begin);
          }
          mma_commit_if(leader, &b.pv_done[t]);
          if (!more) mma_commit_if(leader, &b.o_full[t]);
          wait(&b.pv_done[t], tiles++);  // P lies over S: the next scores may be written once it has been read
          // The turn goes on before this tile's Q K^T is issued: the other warp takes as long to its
          // first product as this one to issue its eight.
          if (leader) {
            if (both) mbar_arrive(&b.turn[t ^ 1]);
            mbar_arrive(&b.empty[sv]);
          }
        }
        if (more) {
            __syncwarp();
          tc_fence_after();
          const uint64_t db = dk + sk * (kSlot >> 4);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t off = ((kk >> 2) * kPanel + 32 * (kk & 3)) >> 4;
            mma_f16_if(leader, 128 * t, dq + off, db + off, id_qk, kk > 0);
          }
          mma_commit_if(leader, &b.s_full[t]);
          mma_commit_if(leader, &b.empty[sk]);
          if (i + 2 == end) mma_commit_if(leader, &b.q_empty);
          step();
          sv = sk;
          values(i + 1, sk, pk);
          step();
        }
    }
  }
  // nothing of this block's may be in flight when it ends
  mma_commit_if(leader, &b.drain[t]);
  if (!bar_wait(&b.drain[t], 0)) dead = true;
  if (dead && leader) report_status(a.status, 6 /* KDA_ERR_TIMEOUT */);
}

// --------------------------------------------------------------------------- queries
// Four warps bring an item's 256 query rows, 16 lanes a row, zero past the last.  A negative
// scale is the same as negated queries and a scale of 0 as zero queries with any scale, so the
// softmax's scale is positive.
template <bool kE4m3>
__device__ void load_queries(const AttnArgs& a, const Job& w, uint8_t* sm, Bars& b, int tid, uint32_t items, bool& dead) {
  using C = Cfg<kE4m3>;
  const int lane = tid & 31, sub = tid & 15, grp = tid >> 4;
  constexpr int kGroups = 8, kGroupRows = kRows / kGroups;  // of 16 lanes
  const int G = a.H / a.cache.heads;
  const uint32_t q_at = smem_u32(sm + C::kSmQ) + (sub >> 3) * kPanel;
  auto q_piece = [&](int r) { return q_at + (r >> 7) * kSlot + sw128(r & 127, 16 * (sub & 7)); };  // this lane's 8 channels
  const int n_rows = w.rows - w.row0;
  const uint16_t* q0 = static_cast<const uint16_t*>(a.q) + w.q_base + static_cast<int64_t>(w.head) * G * a.q_stride[2];
  // while the last item still uses the tiles, the rows' lines into L2: a few rows a lane
  for (int r = tid; r < min(kRows, n_rows); r += 16 * kGroups) {
    const int tok = row_token(a, w.row0 + r), g = w.row0 + r - tok * G;
    const uint16_t* src = q0 + tok * a.q_stride[1] + g * a.q_stride[2];
    prefetch_l2(src);
    prefetch_l2(src + 64);
  }
  if (items > 0 && !dead && !bar_wait(&b.q_empty, (items - 1) & 1)) dead = true;
  // every piece is on its way before any is waited for; zeros past the last row
  {
    const int first = grp * kGroupRows, tok = row_token(a, w.row0 + first);
    int g = w.row0 + first - tok * G;
    const uint16_t* src = q0 + tok * a.q_stride[1] + g * a.q_stride[2] + 8 * sub;
    const int64_t wrap = a.q_stride[1] - (G - 1) * a.q_stride[2];
#pragma unroll 4
    for (int r = first; r < first + kGroupRows; ++r) {
        cp_async16(q_piece(r), src, r < n_rows);
        const bool end = ++g == G;
        src += end ? wrap : a.q_stride[2];
        g = end ? 0 : g;
    }
  }
  cp_async_wait_all();
  if (kE4m3 || a.scale_log2 <= 0.f) {  // in place: each thread its own pieces
#pragma unroll 4
    for (int r = grp * kGroupRows; r < (grp + 1) * kGroupRows; ++r) {
        uint4 x = lds128(q_piece(r));
        if (a.scale_log2 == 0.f) x = make_uint4(0, 0, 0, 0);
        if constexpr (kE4m3) {
          uint32_t top = max(max(x.x & 0x7fffu, (x.x >> 16) & 0x7fffu), max(x.y & 0x7fffu, (x.y >> 16) & 0x7fffu));
          top = max(top, max(max(x.z & 0x7fffu, (x.z >> 16) & 0x7fffu), max(x.w & 0x7fffu, (x.w >> 16) & 0x7fffu)));
#pragma unroll
          for (int off = 8; off; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
          const int e = query_exponent(top);
          const float inv = a.scale_log2 < 0.f ? -pow2i(-e) : pow2i(-e);
          if (sub == 0) reinterpret_cast<int8_t*>(sm + C::kSmExp)[(items & 1) * kRows + r] = static_cast<int8_t>(e);
          auto half = [&](uint32_t v) { return pack_half2(__uint_as_float(v << 16) * inv, __uint_as_float(v & 0xffff0000u) * inv); };
          x = make_uint4(half(x.x), half(x.y), half(x.z), half(x.w));
        } else if (a.scale_log2 < 0.f) {
          const uint32_t flip = 0x80008000u;
          x = make_uint4(x.x ^ flip, x.y ^ flip, x.z ^ flip, x.w ^ flip);
        }
        sts128(q_piece(r), x);
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(&b.q_full);
}

// bf16 cache: four warps for the queries, which also look the edge tiles' values through (see the softmax).
__device__ void query_warps(const ChunkParams& p, uint8_t* sm, Bars& b, int tid) {
  using C = Cfg<false>;
  const AttnArgs& a = p.a;
  const int lane = tid & 31;
  uint32_t n = 0, items = 0, edges = 0;
  bool dead = false;
  JobFeed feed{b.jobs, dead};
  while (const Job* jp = feed.next()) {
    const Job& w = *jp;
    load_queries<false>(a, w, sm, b, tid, items, dead);
    ++items;
    {
        const int begin = w.begin, end = w.end;
        for (int i = begin; i < end; ++i, n += 2) {
          if (!edge_tile(a, w.tile(i), w.p_first, w.p_last)) continue;
          const uint32_t s = (n + 1) % C::kSlots;
          if (!dead && !bar_wait(&b.v_ask, edges++ & 1)) dead = true;
          // thread = key: a row of 128 values with a NaN or an infinity is cleared and noted
          uint8_t* v = sm + C::kSmKV + s * kSlot;
          bool bad = false;
#pragma unroll 8
          for (int c = 0; c < 16; ++c) {
            const uint4 x = *reinterpret_cast<const uint4*>(v + (c >> 3) * kPanel + sw128(tid, 16 * (c & 7)));
            auto has = [](uint32_t u) { return (u & 0x7f80u) == 0x7f80u || (u & 0x7f800000u) == 0x7f800000u; };
            bad |= has(x.x) | has(x.y) | has(x.z) | has(x.w);
          }
          if (bad) {
#pragma unroll 1
            for (int c = 0; c < 16; ++c)
              *reinterpret_cast<uint4*>(v + (c >> 3) * kPanel + sw128(tid, 16 * (c & 7))) = make_uint4(0, 0, 0, 0);
          }
          const uint32_t m = __ballot_sync(0xffffffffu, bad);
          if (lane == 0) b.bad[s][tid >> 5] = m;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&b.v_ok);
        }
    }
    feed.done(lane);
  }
  if (dead && lane == 0) report_status(a.status, 6 /* KDA_ERR_TIMEOUT */);
}

// ------------------------------------------------------------------- codes to f16 tiles
// Four warps, which also bring the queries; thread = key.  (Eight, four for the keys and four for
// the values, were slower: 3.0 against 2.7 ms for 2048 tokens over 30 K keys, 96 heads on 8.)  With E
// the largest scale exponent of the tile's keys (values), a row becomes code * 2^(e - E) in f16: exact
// for e >= E - 15 (codes go down to 2^-9, f16 to 2^-24), so that one factor 2^E serves the whole tile
// and the softmax has no per-key work.  Where a row's scale lies below E - kReach (all-zero rows
// aside) the tile is "wide": its rows stay plain codes and the softmax takes every key's scale by
// itself.  kReach is less than 15 for the values' sake: their E stands in the reference of the f16
// weights, whoever sees the row that has it.  (15 for the keys and 8 for the values, a register
// more: 2698 us instead of 2600 for 2048 tokens over 30 K keys.)  Rows past the last position, which
// may hold anything, become zeros; so
// do value rows that hold a NaN, noted in bad[].
__device__ void convert_group(const ChunkParams& p, uint8_t* sm, Bars& b, int tid) {
  using C = Cfg<true>;
  const AttnArgs& a = p.a;
  const int lane = tid & 31, warp = tid >> 5;
  uint32_t n = 0, items = 0;
  bool dead = false;
  JobFeed feed{b.jobs, dead};
  while (const Job* jp = feed.next()) {
    const Job& w = *jp;
    load_queries<true>(a, w, sm, b, tid, items++, dead);
    const int begin = w.begin, end = w.end;
    for (int i = begin; i < end; ++i) {
      const int keys = w.p_last + 1 - w.tile(i) * kTile;  // those of the tile that are not past the last position
      const bool past = tid >= keys, edge = edge_tile(a, w.tile(i), w.p_first, w.p_last);
      float k_scale = 1.f;
      int k_wide = 0, k_byte = 127;
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv, ++n) {
        const uint32_t st = n % C::kStages, s = n % C::kSlots;
        if (!dead && !bar_wait(&b.st_full[st], (n / C::kStages) & 1)) dead = true;
        const uint8_t* src = sm + C::kSmStage + st * kStage;
        uint4 c[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) c[k] = *reinterpret_cast<const uint4*>(src + sw128(tid, 16 * k));
        const uint8_t* scales = sm + C::kSmScale + st * kTile;
        const uint32_t byte = scales[tid];
        // A code of NaN matters here where some row does not see the key; elsewhere it makes its own way.
        uint32_t nan = 0;
        if (edge) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            auto has = [](uint32_t u) { return (u & 0x7f7f7f7fu) + 0x01010101u; };  // bit 7 of a byte: it is 0x7f or 0xff
            nan |= (has(c[k].x) | has(c[k].y) | has(c[k].z) | has(c[k].w)) & 0x80808080u;
          }
        }
        // Every warp finds E and the lowest exponent of all 128 rows by itself, four scale bytes a lane.
        // NaN rows and rows past the last position do not count, nor need rows of zeros, which have the
        // least scale: rows of that scale or below (others than kda_kv_append may have filled the
        // cache) are looked into where they decide whether the tile is wide.
        int top, low;
        {
          const int key = 4 * lane;
          uint32_t four = *reinterpret_cast<const uint32_t*>(scales + key);
          int hi4 = 0, lo4 = 1000, few4 = 1000;
          uint32_t least = 0;
#pragma unroll
          for (int q = 0; q < 4; ++q, four >>= 8) {
            const int v = four & 255u;
            const bool in = v != 255 && key + q < keys, few = v <= static_cast<int>(kLeast);
            hi4 = in ? max(hi4, v) : hi4;
            if (in && !few) lo4 = min(lo4, v);
            if (in && few) few4 = min(few4, v);
            least |= in && few ? 1u << q : 0u;
          }
          top = __reduce_max_sync(0xffffffffu, hi4);
          low = __reduce_min_sync(0xffffffffu, lo4);
          if (top - kReach <= static_cast<int>(kLeast)) {
            low = min(low, __reduce_min_sync(0xffffffffu, few4));
          } else {
            uint32_t lanes = __ballot_sync(0xffffffffu, least != 0);
            while (lanes) {  // a warp's work on four keys at a time
              const int from = __ffs(lanes) - 1;
              lanes &= lanes - 1;
              const uint32_t which = __shfl_sync(0xffffffffu, least, from);
              for (int q = 0; q < 4; ++q) {
                const uint32_t part = *reinterpret_cast<const uint32_t*>(src + (4 * from + q) * 128 + 4 * lane);
                if ((which >> q) & 1 && __any_sync(0xffffffffu, (part & 0x7f7f7f7fu) != 0))
                  low = min(low, static_cast<int>(scales[4 * from + q]));
              }
            }
          }
          top = top == 0 ? 0 : top - 127;  // none counts: any factor, but not 0 (hidden scores are -inf)
          low = min(low - 127, top);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&b.st_empty[st]);
        const bool bad = (nan || byte == 255) && !past;
        const uint32_t bad_keys = __ballot_sync(0xffffffffu, bad);
        if (n >= C::kSlots && !dead && !bar_wait(&b.empty[s], (n / C::kSlots - 1) & 1)) dead = true;
        if (kv && lane == 0) b.bad[s][warp] = bad_keys;
        const bool wide = low < top - kReach;
        const int e = static_cast<int>(byte) - 127;
        const bool counts = !past && byte != 255 && e >= low;
        // What the softmax needs of both is written with the values, for whose slot P V of the
        // tile before last has been waited: until then it may still read the words' last tile.
        // Per-key scales, for a tile that is wide in either way: those of the side that is not are in
        // the tile (127: 1), and a zero row's must not raise m.
        if (kv) {
          if (tid == 0) b.tile[(n >> 1) & 1] = TileScale{k_scale, wide ? 0.f : static_cast<float>(top), k_wide, wide};
          uint8_t* vec = sm + C::kSmVec + ((n >> 1) & 1) * 256;
          vec[tid] = k_byte;
          vec[128 + tid] = wide ? (counts ? byte : low + 127) : 127;
        } else {
          k_scale = wide ? 1.f : pow2i(top);
          k_wide = wide;
          k_byte = wide && counts ? byte : 127;
        }
        // the row's factor as an f16 pair; NaN for a key row that holds one
        const int r = wide || !counts ? 0 : e - top;
        __half2 f = __half2half2(__ushort_as_half(static_cast<unsigned short>(r >= -14 ? (15 + r) << 10 : 1 << (24 + r))));
        if (bad && !kv) f = __half2half2(__ushort_as_half(0x7fff));
        const uint32_t keep = past || (bad && kv) ? 0u : 0xffffffffu;
        auto out = [&](uint32_t codes, uint32_t& lo, uint32_t& hi) {
          uint32_t l, h;
          e4m3_half4(codes & keep, l, h);
          const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&l), f), y = __hmul2(*reinterpret_cast<const __half2*>(&h), f);
          lo = *reinterpret_cast<const uint32_t*>(&x);
          hi = *reinterpret_cast<const uint32_t*>(&y);
        };
        uint8_t* dst = sm + C::kSmKV + s * kSlot;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint8_t* row = dst + (k >> 2) * kPanel;
          uint4 x, y;
          out(c[k].x, x.x, x.y);
          out(c[k].y, x.z, x.w);
          out(c[k].z, y.x, y.y);
          out(c[k].w, y.z, y.w);
          *reinterpret_cast<uint4*>(row + sw128(tid, 32 * (k & 3))) = x;
          *reinterpret_cast<uint4*>(row + sw128(tid, 32 * (k & 3) + 16)) = y;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b.full[s]);
      }
    }
    feed.done(lane);
  }
  if (dead && lane == 0) report_status(a.status, 6 /* KDA_ERR_TIMEOUT */);
}

// ---------------------------------------------------------------------------- softmax
// Scores are taken to log2 units as y = S u + off: u the softmax scale (e4m3: times the query
// row's and the tile's powers of two), off the values' E of an e4m3 tile, by which the weights
// 2^(y - m) are those of the scaled tile; the row's sum takes 2^-off back.
template <bool kE4m3>
__device__ void softmax_group(const ChunkParams& p, uint8_t* sm, Bars& b, int t, int tid) {
  using C = Cfg<kE4m3>;
  const AttnArgs& a = p.a;
  // A row's reference m moves only when a score stands more than kMost (log2) above it, and then so
  // that this score's weight is 2^kFresh.  No bf16 weight is above 1: the sums of values are no larger
  // than with the maximum itself.  f16 weights end at 2^16 and lose bits below 2^-14, so they go up to
  // 2^15: see the kernel's head for what is lost.  The price of moving late is that a dominating key's weight is then
  // rarely a power of two, so it is rounded (2^-8).  bf16, kFresh -2 / -8 / -32: 8192 tokens 1395 /
  // 1264 / 1198 us, under a window of 1024 695 / 690 / 633 us, 2048 tokens over 30 K keys 2218 / 2118 /
  // 2055 us; error of 8192 tokens against 64 bits in the norm 1.80e-3 / 2.07e-3 / 2.29e-3 (with weights
  // of 32 bits 1.66e-3, most of it o's own rounding).
  constexpr float kFresh = kE4m3 ? 7.f : -8.f, kMost = kE4m3 ? 15.f : 0.f;
  const int lane = tid & 31;
  const uint32_t tl = static_cast<uint32_t>(tid & 96) << 16;
  const uint32_t ts = tl + 128 * t, to = tl + 256 + 128 * t;
  uint32_t n = 0, tiles = 0, items = 0, edges = 0, seen = 0;  // seen: items of the block, items: those with rows here
  bool dead = false;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!dead && !bar_wait(bar, parity & 1)) dead = true;
  };
  const float scale = a.scale_log2 == 0.f ? 1.f : fabsf(a.scale_log2);  // the queries have its sign (0: are 0)
  JobFeed feed{b.jobs, dead};
  while (const Job* jp = feed.next()) {
    const Job& w = *jp;
    const int begin = w.begin, end = w.end;
    const int row = w.row0 + 128 * t + tid;
    if (w.row0 + 128 * t > w.last_row) {  // no rows of this tile
      if constexpr (!kE4m3) {
        for (int i = begin; i < end; ++i)
          if (edge_tile(a, w.tile(i), w.p_first, w.p_last)) ++edges;
      }
      n += 2 * (end - begin);
      ++seen;
      feed.done(lane);
      continue;
    }
    const bool live = row < w.rows;
    const int G = a.H / a.cache.heads;
    const int tok = row_token(a, row);
    const int pos = live ? w.len - w.n_tok + tok : -1;
    float crow = scale;
    float m = -INFINITY, l = 0.f;
    for (int i = begin; i < end; ++i, n += 2) {
      const int kt = w.tile(i);
      const bool edge = edge_tile(a, kt, w.p_first, w.p_last);
      const uint32_t sv = (n + 1) % C::kSlots;
      wait(&b.s_full[t], tiles);
      ++tiles;
      tc_fence_after();
      // 0 * NaN must not reach a row that does not see the key: value rows with a non-finite value
      // were cleared, and the rows that do see one become NaN here.
      auto poison = [&] {
        const uint4 any = *reinterpret_cast<const uint4*>(b.bad[sv]);
        if ((any.x | any.y | any.z | any.w) == 0) return;
#pragma unroll 1
        for (int k = 0; k < kTile; ++k)
          if (((b.bad[sv][k >> 5] >> (k & 31)) & 1) && sees(pos, kt * kTile + k, a.window, a.n_sink))
            l = __uint_as_float(0x7fffffffu);
      };
      float u = crow, off = 0.f;
      int wide = 0;
      if constexpr (kE4m3) {
        if (i == begin) crow = scale * pow2i(reinterpret_cast<const int8_t*>(sm + C::kSmExp)[(seen & 1) * kRows + 128 * t + tid]);
        wait(&b.full[sv], (n + 1) / C::kSlots);  // the value scales come with the values
        const TileScale& sc = b.tile[(n >> 1) & 1];
        u = fminf(fmaxf(crow * sc.k, 0x1p-126f), 0x1.fp127f);  // hidden scores are -inf, zero keys' 0: neither may meet the other
        off = sc.v;
        wide = sc.wide_k | sc.wide_v;
        poison();
      }
      // ---- in edge and wide tiles, the scores in place first: y of the codes, key by key, after which
      // u = 1 and off = 0; hidden ones -inf.  Rolled: the code is cold whenever it runs.
      const uint8_t* vec = sm + C::kSmVec + ((n >> 1) & 1) * 256;
      const float v_off = off;
      if (edge || (kE4m3 && wide)) {
#pragma unroll 1
        for (int c = 0; c < kTile; c += 16) {
          float x[16];
          tmem_ld16(ts + c, x);
          if (kE4m3 && wide) {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = fmaf(x[e] * scale_value(vec[c + e]), u, scale_exponent(vec[128 + c + e]) + off);
          }
          if (edge) {
            const int first = kt * kTile + c;
            // columns before `end`, from `from` on or before `sink`
            auto below = [](int k) { return k <= 0 ? 0u : k >= 32 ? ~0u : (1u << k) - 1; };
            const uint32_t end = below(pos + 1 - first), sink = below(a.n_sink - first);
            const uint32_t from = a.window > 0 && pos >= a.window ? ~below(pos - a.window + 1 - first) : ~0u;
            const uint32_t see = end & (from | sink);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (!((see >> e) & 1)) x[e] = -INFINITY;
          }
          tmem_st16(ts + c, x);
        }
        tmem_wait_st();
        if (kE4m3 && wide) { u = 1.f; off = 0.f; }
      }
      // ---- the row's maximum, 64 columns at a time; the last 64 stay in registers
      float x[2][32];
      auto load = [&](int c) {
        tmem_ld32_async(ts + c, x[0]);
        tmem_ld32_async(ts + c + 32, x[1]);
        tmem_wait_ld32(x[0]);
        tmem_wait_ld32(x[1]);
      };
      float mx = -INFINITY;
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        load(64 * h);
        float m0 = fmaxf(x[0][0], x[0][1]), m1 = fmaxf(x[1][0], x[1][1]);
        float m2 = fmaxf(x[0][2], x[0][3]), m3 = fmaxf(x[1][2], x[1][3]);
#pragma unroll
        for (int e = 4; e < 32; e += 4) {
          m0 = fmaxf(m0, fmaxf(x[0][e], x[0][e + 1]));
          m1 = fmaxf(m1, fmaxf(x[1][e], x[1][e + 1]));
          m2 = fmaxf(m2, fmaxf(x[0][e + 2], x[0][e + 3]));
          m3 = fmaxf(m3, fmaxf(x[1][e + 2], x[1][e + 3]));
        }
        mx = fmaxf(mx, fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)));
      }
      const float top = fmaf(mx, u, off);
      // Scores past 2^20: what a fused y - m keeps of the product beyond y's own 24 bits would grow to
      // whole powers of two, beyond the weights' type.  There y is rounded first, in place, as m is.
      // (The vote and its cold code cost 1 to 2 % of a prompt; remembering it from tile to tile instead
      // cost as much.)
      if (__any_sync(0xffffffffu, fabsf(top) > 0x1p20f && fabsf(top) < INFINITY)) {
#pragma unroll 1
        for (int c = 0; c < kTile; c += 16) {
          float y[16];
          tmem_ld16(ts + c, y);
#pragma unroll
          for (int e = 0; e < 16; ++e) y[e] = fmaf(y[e], u, off);
          tmem_st16(ts + c, y);
        }
        tmem_wait_st();
        u = 1.f;
        off = 0.f;
        load(64);
      }
      const bool grow = top - m > kMost;  // also from -inf to anything; never for nothing visible
      if (__any_sync(0xffffffffu, grow)) {
        const float to_m = kE4m3 ? __fadd_ru(top, -kFresh) : top - kFresh;  // never further below, however large
        const float f = grow ? exp2_fast(m - to_m) : 1.f;
        m = grow ? to_m : m;
        l *= f;
        if (i > begin) {
          // The scores' barrier stands for every product issued before them, the last P V among them.
#pragma unroll 1
          for (int g = 0; g < 8; ++g) {
            float o[16];
            tmem_ld16(to + 16 * g, o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] *= f;
            tmem_st16(to + 16 * g, o);
          }
        }
      }
      // ---- weights and their sum: keys 64 .. 127 from the registers, over their own scores' first
      // 32 columns, then keys 0 .. 63
      const float ref = m == -INFINITY ? 0.f : m;
      if (kE4m3 && wide) {  // the sum of 2^((y - m) - ev), key by key: of the weights that P V gets, however large y
#pragma unroll 1
        for (int c = 0; c < kTile; c += 16) {
          float y[16];
          tmem_ld16(ts + c, y);
#pragma unroll
          for (int e = 0; e < 16; ++e) l += exp2_fast((y[e] - ref) - (scale_exponent(vec[128 + c + e]) + v_off));
        }
      }
      const uint64_t u2 = f32x2(u, u), nb2 = f32x2(off - ref, off - ref);
      uint64_t sum = f32x2(0.f, 0.f), sum1 = sum;
#pragma unroll 1
      for (int h = 1; h >= 0; --h) {
        if (h == 0) load(0);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 y = unpack_f32x2(fma_f32x2(f32x2(x[q][e], x[q][e + 1]), u2, nb2));
            const float p0 = exp2_fast(y.x), p1 = exp2_fast(y.y);
            if (e & 2) sum = add_f32x2(sum, f32x2(p0, p1)); else sum1 = add_f32x2(sum1, f32x2(p0, p1));
            // rounded once, to the values' type: f16 2^-11, bf16 2^-8; the sum keeps 32 bits
            pk[e >> 1] = __uint_as_float(kE4m3 ? pack_half2(p0, p1) : pack_bf162(p0, p1));
          }
          tmem_st16(ts + 64 * h + 16 * q, pk);
        }
        tmem_wait_st();
        // The look through an edge tile's values must have been seen, and its words read, before the
        // last weights are handed over: P V waits for them, and what follows it asks for the next edge
        // tile's look, whose end is the next phase of the same barrier.
        if (!kE4m3 && h == 0 && edge) {
          wait(&b.v_ok, edges++);
          poison();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b.p_full[t][h]);
      }
      const float2 sums = unpack_f32x2(add_f32x2(sum, sum1));
      if (!kE4m3) l += sums.x + sums.y;
      else if (!wide) l = fmaf(sums.x + sums.y, exp2_fast(-v_off), l);
    }
    // ---- the item's (or part's) rows
    wait(&b.o_full[t], items);
    ++items;
    ++seen;
    tc_fence_after();
    const bool part = w.slot >= 0;
    const int64_t at = static_cast<int64_t>(w.slot) * p.s.part_rows + 128 * t + tid;
    const int64_t orow = (w.base + tok) * a.H + static_cast<int64_t>(w.head) * G + (row - tok * G);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint8_t* dst = part ? reinterpret_cast<uint8_t*>(p.s.part_o + at * 128) : static_cast<uint8_t*>(a.o) + orow * 256;
#pragma unroll 1
    for (int g = 0; g < 8; ++g) {
      float o[16];
      tmem_ld16(to + 16 * g, o);
      if (!live) continue;
      if (part) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          reinterpret_cast<float4*>(dst)[4 * g + e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          reinterpret_cast<uint4*>(dst)[2 * g + e] =
              make_uint4(pack_bf162(o[8 * e] * inv, o[8 * e + 1] * inv), pack_bf162(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                         pack_bf162(o[8 * e + 4] * inv, o[8 * e + 5] * inv), pack_bf162(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
      }
    }
    if (live && part) p.s.part_ml[at] = make_float2(m, l);
    if (live && !part && a.lse) a.lse[orow] = lse_of(m, l);
    tc_fence_before();
    feed.done(lane);
  }
  if (dead && lane == 0) report_status(a.status, 6 /* KDA_ERR_TIMEOUT */);
}

template <bool kE4m3>
__global__ void __launch_bounds__(kThreads, 1) attn_chunk_kernel(const __grid_constant__ ChunkParams p) {
  using C = Cfg<kE4m3>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars b;
  uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < 5; ++i) {
      mbar_init(&b.full[i], kE4m3 ? 4 : 1);
      mbar_init(&b.empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) { mbar_init(&b.st_full[i], 1); mbar_init(&b.st_empty[i], 4); }
    mbar_init(&b.v_ask, 2);
    mbar_init(&b.v_ok, 4);
    mbar_init(&b.q_full, 4);
    mbar_init(&b.q_empty, 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b.s_full[i], 1);
      mbar_init(&b.p_full[i][0], 4);
      mbar_init(&b.p_full[i][1], 4);
      mbar_init(&b.pv_done[i], 1);
      mbar_init(&b.o_full[i], 1);
      mbar_init(&b.turn[i], 1);
      mbar_init(&b.drain[i], 1);
    }
    // a job is read by the two product warps, the query warps, the eight softmax warps and the converters
    b.jobs.init(10 + 4);
    fence_mbar_init();
    p.s.desc[blockIdx.x].last = -1;
  }
  pdl_launch_dependents();
  if (warp == 8) {
    tmem_alloc(&b.tmem, 512);  // all of it, so its addresses begin at 0
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // registers: 128 a thread at launch, 512 over the four groups
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 176;\n" ::: "memory");
    softmax_group<kE4m3>(p, sm, b, warp >> 2, tid & 127);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;\n" ::: "memory");
    if (warp < 10) mma_warp<kE4m3>(p, sm, b, warp - 8);
    else if (warp == 10) load_warp<kE4m3>(p, sm, b, tid & 31);
    else if (warp >= 12) {
      if constexpr (kE4m3) convert_group(p, sm, b, tid - 384);
      else query_warps(p, sm, b, tid - 384);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(b.tmem, 512);
}

template <bool kE4m3>
cudaError_t launch_chunk(const ChunkParams& p) {
  constexpr int bytes = Cfg<kE4m3>::kSmBytes;
  auto kern = attn_chunk_kernel<kE4m3>;
  static SmemOptIn opt_in;
  const cudaError_t e = opt_in(reinterpret_cast<const void*>(kern), bytes);
  if (e != cudaSuccess) return e;
  return launch_after(kern, dim3(static_cast<unsigned>(p.s.grid)), dim3(kThreads), bytes, p.a.stream, p);
}

}  // namespace

size_t attn_chunk_workspace(int n_seq, int64_t tokens, int group, int num_sms) {
  return attn_split_bytes(num_sms, kRows, attn_max_items(n_seq, tokens, group, kRows));
}

cudaError_t launch_attn_chunk(const AttnArgs& a, int num_sms) {
  const int G = a.H / a.cache.heads;
  ChunkParams p;
  memset(&p, 0, sizeof(p));
  p.a = a;
  attn_split_layout(&p.s, a.workspace, num_sms, kRows, attn_max_items(a.n_seq, a.tokens, G, kRows));
  p.s.min_tiles = kMinTiles;
  p.s.item_cost = kItemCost;
  if (!make_cache_maps(a.cache, kTile, 1, &p.tk, &p.tv)) return cudaErrorInvalidValue;
  cudaError_t e = launch_attn_plan(a, p.s, kRows, kTile);
  if (e != cudaSuccess) return e;
  e = a.cache.e4m3 ? launch_chunk<true>(p) : launch_chunk<false>(p);
  if (e != cudaSuccess) return e;
  return launch_attn_join(p.a, p.s);
}

}  // namespace kda
