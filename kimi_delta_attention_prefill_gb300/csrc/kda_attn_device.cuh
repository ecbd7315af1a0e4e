// kda_attn_device.cuh -- device code shared by the attention kernels: the walk of a block over
// its share of the work, scale bytes, and TMA loads of the cache's maps.
#pragma once

#include <cstdint>

#include "kda_attn.h"
#include "kda_ptx.cuh"

namespace kda {

__device__ __forceinline__ void tma_load_4d(void* dst, const void* tmap, uint64_t* bar, int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];\n" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
__device__ __forceinline__ void tma_load_5d(void* dst, const void* tmap, uint64_t* bar, int c0, int c1, int c2, int c3,
                                            int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];\n" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// 16 bytes to shared memory, without registers; zeros (and no read) unless `live`.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Untiled copy of `bytes` (a multiple of 16, both addresses too) into shared memory.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                   smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Programmatic dependent launch: let the next kernel of the stream start its blocks / wait for
// the previous kernel's end and its writes.
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Wait for a barrier's phase, given up after 2^20 polls (false), each of which the hardware
// holds for microseconds: then the caller reports KDA_ERR_TIMEOUT, stops waiting and leaves in
// order.  Kept small: where it stands in a rarely fetched loop, its code is what it costs.
// By a whole warp, whose lanes decide together: a wait that runs out while the barrier flips must
// not send some lanes on and some away, warp-wide instructions coming after it.  (On one GPU with
// and without the vote: a prompt of 8192 1197 and 1210 us, 2048 tokens over 30 K e4m3 keys 2544 and
// 2499 us.  A vote only where a warp's way is decided: 1226 and 2515 us.)
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
  for (uint32_t i = 0; i < (1u << 20); ++i)
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return false;
}

// The copy warp's end, its waits run out or not: a ring's last `uses` copies have landed before
// the block may give its shared memory back (readers that stopped waiting do not see to it).
__device__ __forceinline__ void drain_ring(uint64_t* full, uint32_t slots, uint32_t uses) {
  for (uint32_t u = uses > slots ? uses - slots : 0; u < uses; ++u) bar_wait(&full[u % slots], (u / slots) & 1);
}

// Four e4m3 codes as two pairs of f16 values, exactly.
__device__ __forceinline__ void e4m3_half4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

// Scale bytes of E4M3 rows, in the low 8 bits of b: 2^(b - 127), 2^(127 - b) and b - 127.  Of a row of
// NaN (255, codes 0) they make infinity, by which a score of 0 becomes NaN, -infinity, which
// makes a sum negative, and 128: no instruction is spent on it.
__device__ __forceinline__ float scale_value(uint32_t b) { return __uint_as_float((b << 23) & 0x7f800000u); }
__device__ __forceinline__ float scale_inverse(uint32_t b) { return __uint_as_float(0x7f000000u - ((b << 23) & 0x7f800000u)); }
__device__ __forceinline__ float scale_exponent(uint32_t b) {
  return __uint_as_float(0x4b000000u | (b & 255u)) - (8388608.f + 127.f);
}

__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// Queries against E4M3 keys are f16, as the codes are: a row times 2^-e with its largest value
// (bf16 magnitude bits `top`) in [2^8, 2^9) is exact down to 2^-22 of that value.
__device__ __forceinline__ int query_exponent(uint32_t top) {
  const int e = static_cast<int>(top >> 7) - 127 - 8;
  return top >= 0x7f80u || top == 0 ? 0 : max(e, -100);
}

__device__ __forceinline__ float lse_of(float m, float l) {  // m in log2 units
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// The token of a row, row / (H / kv heads).
__device__ __forceinline__ int row_token(const AttnArgs& a, int row) {
  return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(row)) * a.g_magic) >> a.g_shift);
}

// One (sequence, kv head, row tile): rows [row0, row0 + tile rows) of the sequence's
// rows = n_tok G rows, row r = token r / G, query head head * G + r % G.
struct Item {
  int seq = 0, head = 0, row0 = 0, rows = 0;
  int G = 1, n_tok = 0, len = 0;
  int64_t base = 0;  // packed row of the sequence's first token
  int last_row = 0;  // last live row of the tile
  KeyTiles tiles{0, 0, 0};
  __device__ int p_of_row(int row) const { return len - n_tok + row / G; }
  __device__ int p_first() const { return p_of_row(row0); }
  __device__ int p_last() const { return p_of_row(last_row); }
};

// A kv_len that the table cannot hold, or offsets that run backwards.
__device__ __forceinline__ bool seq_bad(const AttnArgs& a, int len, int64_t first, int64_t end) {
  return len < 0 || len > static_cast<int64_t>(a.max_pages) * a.cache.page_size || first < 0 || end < first || end > a.tokens;
}

// Fills an item's sequence part; false: the sequence is bad or has no new tokens.
__device__ inline bool item_sequence(const AttnArgs& a, int seq, Item* w) {
  const int64_t first = a.cu ? a.cu[seq] : static_cast<int64_t>(seq) * a.n_tok;
  const int64_t end = a.cu ? a.cu[seq + 1] : first + a.n_tok;
  w->seq = seq;
  w->len = a.kv_len[seq];
  w->base = first;
  w->n_tok = static_cast<int>(end - first);
  w->G = a.H / a.cache.heads;
  w->rows = w->n_tok * w->G;
  return !seq_bad(a, w->len, first, end) && end > first;
}
// The tiles of its row tile [row0, row0 + n); never none: a tile that sees nothing has one
// visit, which writes its rows' zeros.
__device__ inline void item_tiles(const AttnArgs& a, int row0, int n, int tile, Item* w) {
  w->row0 = row0;
  w->last_row = min(row0 + n, w->rows) - 1;
  w->tiles = key_tiles(w->p_first(), w->p_last(), a.window, a.n_sink, tile);
  if (w->tiles.count() == 0) w->tiles.hi = w->tiles.lo + 1;
}

// A block's way along the line (AttnSplit).  An item takes its key tiles' length on it and before
// them item_cost more, for what an item costs whatever its length (queries, output); a border
// that falls into that stretch is a border before the first tile.  In decode every sequence's row tiles
// visit the same key tiles, so the line needs only the sequences' counts, which each block adds
// up by itself; in prefill it comes from the plan.
template <int kRows, int kTileKeys>
struct ItemWalk {
  const AttnArgs& a;
  const AttnSplit& s;
  Item item;
  int begin = 0, end = 0;   // key tile visits of the item that are this block's
  int64_t pos = 0, stop = 0, at = 0;  // on the line: where we are, the share's end, where the item begins
  int blocks = 1;
  int64_t total = 0;
  int idx = 0;      // prefill: the plan's item
  int unit = 0, n_units = 1;  // decode: head and row tile within the sequence

  __device__ ItemWalk(const AttnArgs& a_, const AttnSplit& s_) : a(a_), s(s_) {}

  __device__ int length() const { return item.tiles.count() + s.item_cost; }  // the item's on the line
  __device__ int decode_length(int seq) {  // of a row tile of the sequence; 0: bad
    const int len = a.kv_len[seq];
    if (len < 0 || len > static_cast<int64_t>(a.max_pages) * a.cache.page_size) {
      if (blockIdx.x == 0) report_status(a.status, 7 /* KDA_ERR_DEVICE_CHECK */);
      return 0;
    }
    const int n = key_tiles(len - a.n_tok, len - 1, a.window, a.n_sink, kTileKeys).count();
    return (n > 0 ? n : 1) + s.item_cost;
  }

  // a / b of non-negative numbers, without the long division where 32 bits will do
  __device__ static int64_t div(int64_t a, int64_t b) {
    return (a | b) >> 32 ? a / b : static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
  }
  // Prefill: from the plan.
  __device__ bool start_plan() {
    n_units = a.cache.heads;
    total = *s.plan_total * n_units;
    return total > 0 && take_share() && find_plan();
  }
  __device__ bool take_share() {
    blocks = total < int64_t{s.min_tiles} * gridDim.x ? static_cast<int>(total) / s.min_tiles : gridDim.x;
    if (blocks < 1) blocks = 1;
    if (blockIdx.x >= blocks) return false;
    pos = div(blockIdx.x * total, blocks);
    stop = div((blockIdx.x + 1) * total, blocks);
    return true;
  }
  __device__ bool find_plan() {
    const int64_t target = div(pos, n_units);
    int lo = 0, hi = *s.plan_items;  // plan_start[lo] <= target < plan_start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s.plan_start[mid] <= target) lo = mid; else hi = mid;
    }
    idx = lo;
    load_plan();
    return clip();
  }

  // Takes this block's share; false: there is none.  By a whole warp.
  __device__ bool start(int lane) {
    if (a.cu) {
      pdl_wait();  // for the plan; everything else was there before it began
      return start_plan();
    }
    const int rows = a.n_tok * (a.H / a.cache.heads);
    n_units = a.cache.heads * ((rows + kRows - 1) / kRows);
    int64_t sum = 0;
    for (int i = lane; i < a.n_seq; i += 32) sum += decode_length(i);
#pragma unroll
    for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    total = sum * n_units;
    if (total == 0 || !take_share()) return false;
    const int64_t target = div(pos, n_units);
    int64_t run = 0;  // 32 sequences at a time up to the one that holds the share's begin
    int seq = 0;
    for (int b = 0;; b += 32) {
      const int i = b + lane;
      const int64_t c = i < a.n_seq ? decode_length(i) : 0;
      int64_t incl = c;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += up;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, run + incl > target);
      if (past) {
        const int k = __ffs(past) - 1;
        seq = b + k;
        at = (run + __shfl_sync(0xffffffffu, incl - c, k)) * n_units;
        break;
      }
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    item_sequence(a, seq, &item);
    item_tiles(a, 0, rows, kTileKeys, &item);
    unit = static_cast<int>(div(pos - at, length()));
    at += static_cast<int64_t>(unit) * length();
    set_unit();
    return clip();
  }

  __device__ void set_unit() {  // decode: heads outermost, so that row tiles of a head are neighbours
    const int n_rt = n_units / a.cache.heads;
    item.head = unit / n_rt;
    item.row0 = (unit - item.head * n_rt) * kRows;
    item.last_row = min(item.row0 + kRows, item.rows) - 1;
  }
  __device__ void load_plan() {
    const int2 d = s.plan_item[idx];
    item_sequence(a, d.x, &item);
    item_tiles(a, d.y, kRows, kTileKeys, &item);
    at = s.plan_start[idx] * n_units;
    item.head = pos > at ? static_cast<int>(div(pos - at, length())) : 0;
    at += static_cast<int64_t>(item.head) * length();
  }
  __device__ bool clip() {  // false: nothing of the item's tiles is in the share
    const int n = item.tiles.count();
    const int64_t first = at + s.item_cost;
    begin = pos > first ? static_cast<int>(pos - first) : 0;
    end = stop - first < n ? static_cast<int>(stop - first) : n;
    return end > begin;
  }
  // The next item of the share; false: the share is done.
  __device__ bool next() {
    at += length();
    if (at >= stop) return false;
    if (a.cu) {
      if (++item.head == a.cache.heads) {
        ++idx;
        load_plan();
      }
    } else if (++unit == n_units) {
      unit = 0;
      int seq = item.seq + 1;
      while (decode_length(seq) == 0) ++seq;  // there is one: the share goes on
      item_sequence(a, seq, &item);
      item_tiles(a, 0, item.rows, kTileKeys, &item);
      set_unit();
    } else {
      set_unit();
    }
    return clip();
  }
  // Slot of the part at hand, or -1 when the block has the whole item.  The thread that says
  // `names` also names the parts of an item that begins here and ends in a later block.
  __device__ int part_slot(bool names) const {
    const int n = item.tiles.count();
    if (begin == 0 && end == n) return -1;
    if (begin > 0) return 2 * blockIdx.x;
    if (names) {
      // the block that has the item's last tile: c1 = ceil(E C / W) - 1
      const int64_t e = at + length();
      s.desc[blockIdx.x] = PartDesc{item.base, item.head, item.row0, item.rows, static_cast<int>(div(e * blocks + total - 1, total) - 1)};
    }
    return 2 * blockIdx.x + 1;
  }
};

// One item (or part) of a block's share, as the copy warp, which walks, hands it to the others.
struct Job {
  int head, row0, rows, last_row, len, n_tok;
  int sink, lo;         // its key tiles
  int begin, end;       // the visits that are this block's; none: the share is done
  int p_first, p_last;  // positions of its first and last row
  int slot;             // of the workspace, -1: whole
  int64_t base;         // packed row of the sequence's first token
  int64_t q_base;       // its queries' element offset
  __device__ int tile(int i) const { return i < sink ? i : lo + (i - sink); }
};
constexpr int kJobs = 4;
struct JobRing {
  uint64_t full[kJobs], empty[kJobs];
  Job job[kJobs];
  __device__ void init(int readers) {
    for (int i = 0; i < kJobs; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], readers); }
  }
  // The k-th job from the walk, or (more = false) the end.  By a whole warp; false: a wait ran out.
  template <class Walk>
  __device__ bool put(uint32_t k, const Walk& walk, bool more, int lane) {
    if (k >= kJobs && !bar_wait(&empty[k % kJobs], (k / kJobs - 1) & 1)) return false;
    if (lane == 0) {
      Job& j = job[k % kJobs];
      j.begin = j.end = 0;
      if (more) {
        const Item& w = walk.item;
        j.head = w.head; j.row0 = w.row0; j.rows = w.rows; j.last_row = w.last_row; j.len = w.len; j.n_tok = w.n_tok;
        j.sink = w.tiles.sink; j.lo = w.tiles.lo; j.begin = walk.begin; j.end = walk.end;
        j.p_first = w.p_first(); j.p_last = w.p_last(); j.slot = walk.part_slot(true); j.base = w.base;
        j.q_base = walk.a.cu ? w.base * walk.a.q_stride[1] : static_cast<int64_t>(w.seq) * walk.a.q_stride[0];
      }
      mbar_arrive(&full[k % kJobs]);
    }
    return true;
  }
};
// The jobs in order, for one warp: next() waits for the next.
struct JobFeed {
  JobRing& r;
  bool& dead;
  uint32_t k = 0;
  __device__ const Job* next() {
    if (!dead && !bar_wait(&r.full[k % kJobs], (k / kJobs) & 1)) dead = true;
    const Job* j = &r.job[k % kJobs];
    return dead || j->begin == j->end ? nullptr : j;
  }
  // The warp needs nothing of the job any more.
  __device__ void done(int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&r.empty[k % kJobs]);
    ++k;
  }
};

}  // namespace kda
