// kda_lin_prefill.cu -- linear attention with a decay a head over packed sequences, chunk by chunk.
//
// With G_i the inclusive sum of a chunk's log-decays (128 tokens), S the state in front of it:
//     O  = scale ((Q K^T) o D) V + scale diag(e^G) Q S,      D_ij = e^{G_i - G_j} (j <= i), else 0
//     S' = e^{G_last} S + (diag(e^{G_last - G}) K)^T V
// All exponents are differences of sums of values <= 0, so nothing can grow whatever the decays are.
//
// One block walks the chunks of a (sequence, head) or of a segment of one; its warps:
//     0        copies (TMA; two tiles each of q, k and v) and the line of work items
//     1        products (tcgen05)
//     2        decays: sums in 64-bit fixed point (2^-32 of a factor of 2); the weights get them as a whole number and
//              a fraction of 32 bits each, so that a small difference of large sums keeps its bits
//     3        the output stage's gate, into q's tile when q is used
//     4 - 7    weights P = (Q K^T) o D as two bf16 parts over their scores; Q S times e^G in place, on which P V is then
//              added (thread = token)
//     8 - 15   decayed values, transposed into tensor memory as three bf16 parts (24 bits together)
//     16 - 23  the state, in fp32 registers (thread = half a column); its bf16 copy for Q S in shared memory;
//              outputs (thread = half a token's row), through q's tile
//
// Rounded to bf16: the copy of S, for o only, which is bf16 itself.  P has 16 bits: with 8 a row that few weights
// make is off by as much again as its own rounding (o off by 0.0023 instead of 0.0017 of its norm on short
// sequences, by 0.0026 on a few tokens; the second parts' product costs 3 %).  The state sees 24-bit products:
// S^T gets three products, one for each part of the values, with K as it lies.  The decay is on the values'
// side because they can then be an operand in tensor memory: shared memory, whose 128 bytes a cycle the
// products of operands in it take in full, is the block's bottleneck.  The parts go through a ring of four
// units (a part of 64 tokens), so that they are made while the products of the units before them run.
//
// The products of a chunk: Q K^T | units of tokens 0 - 63 | Q S | units of tokens 64 - 127 | P V.  Weights are made
// during the three in the middle, outputs and the next state during P V and the next Q K^T.
//
// What bounds it: the chain of a chunk and the issue of the warps around it.  8192 tokens x 96 heads, one block each
// on 96 of 152 SMs: 196 us, 3 us a chunk, of which the products take 1.9 (tensor pipe 61 %), each scheduler's arithmetic
// pipes 1.2 each; 8 heads x 262144 tokens on all SMs: 3.5 us a chunk, 128 KB of it at 5.5 TB/s; with the output
// stage 3.9 us (12 ragged prompts x 64 heads: 432 - 441 us).  Tried and slower than 196 (or 190,
// before the weights' second parts): scores a chunk ahead in columns of their own with a ring of half the size (232),
// eight warps for weights and outputs (226 - 249), outputs stored from registers (221), loops not unrolled
// (199 - 587), products issued from rolled loops (212), parts by bf16x2 arithmetic (2 cycles an instruction, like the
// conversions that they replace), eight units of 32 tokens (205), with Q S first or last (207, 241), weights made by
// the state's warps too (211); the output stage's sums of squares made by the weights' warps (432 -> 463), q's rows fetched into L2
// before their place is free (no change);
// each of 96 heads in 2 - 6 segments (235 - 275: the rule cuts only what fits the SMs at once; 64 heads
// into 2: 190 -> 167).  Two parts of the values instead of three leave states off by 2e-6.
//
// A token's NaN or infinity must not reach earlier tokens, but 0 * NaN is NaN in P V: values that are not
// finite are cleared in the tile, and the rows that see one get NaN in its channel when they are written.
//
// Few heads: segments_of's rule cuts a sequence into as many segments as its share of the work is worth
// in SMs.  A first pass (the same kernel without q and o) leaves each segment's state from zeros, the second
// begins with the sum over the segments before it, which it takes one after another: cheap for the 19 segments of
// 8 heads, but one head of 100000 tokens in the rule's 97 takes 207 us (in 64: 165; 32: 171; 16: 251), 262144 tokens 396.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cstdint>
#include <cstring>

#include "kda_attn.h"
#include "kda_attn_device.cuh"
#include "kda_lin.h"
#include "kda_ptx.cuh"

namespace kda {
namespace {

constexpr int kD = kHeadDim;
constexpr int kC = 128;  // tokens a chunk
constexpr int kThreads = 768;
constexpr int kRegs = 80;  // at launch
constexpr uint32_t kTile = 32768, kPanel = 16384;
constexpr uint32_t kSmState = 6 * kTile, kSmSmall = kSmState + kTile;
// tensor memory columns: scores and weights; outputs; K^T V, transposed; four units of the values' parts
constexpr uint32_t kTS = 0, kTO = 128, kTKV = 256, kTV = 384;
// The first pass has neither scores nor outputs: K^T V in two places in turn, and twice as many units.
template <bool kFull>
__device__ __forceinline__ uint32_t kv_column(uint32_t n) { return kFull ? kTKV : 128 * (n & 1); }
template <bool kFull>
__device__ __forceinline__ uint32_t unit_column(uint32_t u) { return kFull ? kTV + 32 * (u & 3) : 256 + 32 * (u & 7); }
constexpr int kMinSegment = 8;  // chunks

// ------------------------------------------------------------------------------------ plan
struct Item {
  int seq, first, len;  // first packed row, tokens of the sequence
  int c0, c1;           // chunks
  int seg, base;        // segment number, the sequence's first slot (-1: not split)
  int last;             // the sequence's last segment
};

struct Plan {
  int* counts = nullptr;  // (null: block i has head i % H of sequence i / H) items of pass 2, of pass 1; next item of pass 2, of pass 1; items without tokens, after pass 2's
  Item* items[2] = {nullptr, nullptr};
  float* decay = nullptr;  // [slots][H] factor of a segment's decay
  float* slots = nullptr;  // [slots][H][128][128]: slot base: the sequence's entry state; base + 1 + j: segment j's exit
  int64_t most[2] = {0, 0}, n_slots = 0;
};

__host__ __device__ inline int segments_of(int64_t len, int64_t tokens, int H, int sms, int forced) {
  const int64_t chunks = (len + kC - 1) / kC;
  int64_t n = forced;
  if (forced == 0) {
    n = len * sms / (tokens > 0 ? tokens * H : 1);
    if (n > chunks / kMinSegment) n = chunks / kMinSegment;
  }
  if (n > chunks) n = chunks;
  return n < 1 ? 1 : static_cast<int>(n);
}

// A block for each (sequence, head) and nothing to split: no plan, no workspace (48 items of 97 tokens: 10 us on the
// device instead of 15, and an allocation less).
bool one_item_a_block(int n_seq, int64_t tokens, int H, int forced, int sms) {
  return static_cast<int64_t>(n_seq) * H <= sms && segments_of(tokens, tokens, H, sms, forced) == 1;
}

size_t plan_layout(Plan* p, void* ws, int n_seq, int64_t tokens, int H, int forced, int sms) {
  if (one_item_a_block(n_seq, tokens, H, forced, sms)) {
    p->most[0] = n_seq;
    return 0;
  }
  // Segments beyond a sequence's first.  The rule's counts add up to no more than sms / H, and to one for
  // each kMinSegment chunks of a sequence that has twice as many (its last chunk may hold one token).
  int64_t extra = sms / H - 1;
  const int64_t pays = tokens / (kC * (kMinSegment - 1)), chunks = tokens / kC + n_seq;
  if (forced == 0) extra = extra < pays ? extra : pays;
  else extra = static_cast<int64_t>(n_seq) * (forced - 1) < chunks ? static_cast<int64_t>(n_seq) * (forced - 1) : chunks;
  if (extra < 0) extra = 0;
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  size_t at = 256;
  uint8_t* b = static_cast<uint8_t*>(ws);
  p->counts = reinterpret_cast<int*>(b);
  p->most[0] = n_seq + extra;
  p->most[1] = extra;
  p->n_slots = 2 * extra < n_seq + extra ? 2 * extra : n_seq + extra;
  for (int i = 0; i < 2; ++i) {
    p->items[i] = reinterpret_cast<Item*>(b + at);
    at = up(at + sizeof(Item) * static_cast<size_t>(p->most[i]));
  }
  p->decay = reinterpret_cast<float*>(b + at);
  at = up(at + sizeof(float) * static_cast<size_t>(p->n_slots) * H);
  p->slots = reinterpret_cast<float*>(b + at);
  return at + static_cast<size_t>(p->n_slots) * H * kStateFloats * sizeof(float);
}

// The work items, longest first (by 256 lengths), so that the blocks end together.
__global__ void __launch_bounds__(1024) lin_plan_kernel(const int32_t* __restrict__ cu, int n_seq, int64_t tokens, int H,
                                                       int sms, int forced, Plan p, int* status) {
  __shared__ int at[256];
  __shared__ int longest, n1, slots;
  const int tid = threadIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  if (tid < 256) at[tid] = 0;
  if (tid == 0) { longest = 1; n1 = 0; slots = 0; }
  bool bad = cu[0] != 0 || cu[n_seq] != tokens;
  for (int s = tid; s < n_seq; s += blockDim.x) bad |= cu[s + 1] < cu[s] || cu[s] < 0 || cu[s + 1] > tokens;
  if (__syncthreads_or(bad)) {
    if (tid == 0) {
      report_status(status, 7 /* KDA_ERR_DEVICE_CHECK */);
      for (int i = 0; i < 5; ++i) p.counts[i] = 0;
    }
    return;
  }
  auto chunks = [&](int s) { return static_cast<int>((static_cast<int64_t>(cu[s + 1]) - cu[s] + kC - 1) / kC); };
  auto segments = [&](int s) { return segments_of(cu[s + 1] - cu[s], tokens, H, sms, forced); };
  auto length = [&](int s) { const int n = segments(s); return (chunks(s) + n - 1) / n; };
  for (int s = tid; s < n_seq; s += blockDim.x) atomicMax(&longest, length(s));
  __syncthreads();
  auto bin = [&](int s) { return cu[s + 1] == cu[s] ? 255 : 254 - static_cast<int>(static_cast<int64_t>(length(s)) * 254 / longest); };
  for (int s = tid; s < n_seq; s += blockDim.x) atomicAdd(&at[bin(s)], segments(s));
  __syncthreads();
  if (tid == 0) {
    int sum = 0;
    for (int i = 0; i < 256; ++i) { const int n = at[i]; at[i] = sum; sum += n; }
    p.counts[0] = at[255];
    p.counts[4] = sum - at[255];
    p.counts[2] = p.counts[3] = 0;
  }
  __syncthreads();
  for (int s = tid; s < n_seq; s += blockDim.x) {
    const int n = segments(s), nch = chunks(s), pos = atomicAdd(&at[bin(s)], n);
    int base = -1, pos1 = 0;
    if (n > 1) { base = atomicAdd(&slots, n); pos1 = atomicAdd(&n1, n - 1); }
    for (int j = 0; j < n; ++j) {
      Item it;
      it.seq = s; it.first = cu[s]; it.len = cu[s + 1] - cu[s];
      it.c0 = static_cast<int>(static_cast<int64_t>(nch) * j / n);
      it.c1 = static_cast<int>(static_cast<int64_t>(nch) * (j + 1) / n);
      it.seg = j; it.base = base; it.last = j == n - 1;
      if (pos + j < p.most[0]) p.items[0][pos + j] = it;
      if (j < n - 1 && pos1 + j < p.most[1]) p.items[1][pos1 + j] = it;
    }
  }
  __syncthreads();
  if (tid == 0) p.counts[1] = n1;
}

// ---------------------------------------------------------------------------------- kernel
struct LinParams {
  CUtensorMap tq, tk, tv, tg, to;
  LinArgs a;
  Plan p;
};

struct Job {
  Item item;
  int head;  // -1: no more
};

// G_i of a chunk, in units of log2, as whole + part with 0 <= part <= 1.  A reset counts 192: one float for the sum would
// have a step of up to 2^-9, and after 90 resets weights off by 2^-10 (o off by 20 times what its own roundings leave where values cancel).
struct Decays {
  float whole[kC], part[kC];
};

enum { kK, kV, kQ };  // tiles
// Instances: outputs, outputs with the output stage, states only (the first pass of a split sequence).  The code
// of a chunk has to stay in the instruction caches: what an instance does not need is not in it.
enum { kPlain, kGated, kStates };
// The full kernel has two buffers of each tile; the first pass, without q, three.
template <bool kFull> constexpr int kKinds = kFull ? 3 : 2;
template <bool kFull> constexpr uint32_t kBufs = kFull ? 2 : 3;

struct Small {
  Decays dec;
  // by the chunk's parity
  float cf[2][kC];           // 2^{G at the end of the token's block of 32 - G_t}
  float end[2][4];           // 2^{G_last - G at the end of a block}
  float a[2];                // 2^{G_last}
  float weight[kD];          // the output stage's
  Job job[2];
  uint64_t full[2][3];  // [k and q; v][buffer]
  uint64_t free[3][3];  // [tile][buffer]; in the full kernel only q's: kv and out tell when k and v are free
  uint64_t job_full[2], job_empty[2], dec_full, dec_empty, w_full[2], w_empty[2];
  uint64_t scores, inter, ready, out[2], out_free, gate_full, half_full[2], half_free[2], kv[2], kv_read[2], state, drain;
  uint32_t bad_chunk[4];  // chunk number + 1 with values that are not finite, by its last two bits
  uint32_t tmem;
};
constexpr int kSmBytes = kSmSmall + sizeof(Small);
static_assert(kSmBytes <= 232448, "shared memory");

template <bool kFull>
struct Tiles {  // of chunk n
  uint32_t buf, phase;
  __device__ explicit Tiles(uint32_t n) : buf(n % kBufs<kFull>), phase(n / kBufs<kFull>) {}
  __device__ uint32_t at(int kind) const { return (kind * kBufs<kFull> + buf) * kTile; }
};

// As bar_wait, with few instructions a poll: most warps wait most of the time, and what their polls issue the
// others cannot.  Given up after 2^19 polls, of 4 us at most.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred P;\n\t.reg .b32 i;\n\t"
      "mov.b32 i, 0;\n"
      "POLL%=:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 P, [%1], %2, 4000;\n\t"
      "vote.sync.all.pred P, P, 0xffffffff;\n\t"
      "@P bra DONE%=;\n\t"
      "add.u32 i, i, 1;\n\t"
      "setp.lt.u32 P, i, 524288;\n\t"
      "@P bra POLL%=;\n\t"
      "setp.ne.u32 P, 0, 0;\n"
      "DONE%=:\n\t"
      "selp.b32 %0, 1, 0, P;\n\t}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
#define LIN_WAIT(bar, parity) do { if (!dead && !wait_for(smem_u32(&(bar)), (parity) & 1)) dead = true; } while (0)

// The jobs that warp 0 hands out, in every other warp.
struct Jobs {
  Small& s;
  uint32_t n = 0;
  bool& dead;
  __device__ Jobs(Small& s_, bool& d) : s(s_), dead(d) {}
  __device__ bool next(Job& j) {
    LIN_WAIT(s.job_full[n & 1], n >> 1);
    if (dead) return false;
    j = s.job[n & 1];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&s.job_empty[n & 1]);
    ++n;
    return j.head >= 0;
  }
};

__device__ __forceinline__ int live_rows(const Item& it, int c) { return min(kC, it.len - c * kC); }

// The offsets of all sequences, looked at by one warp.
__device__ __forceinline__ bool offsets_hold(const LinArgs& a, int lane) {
  bool bad = a.cu[0] != 0 || a.cu[a.n_seq] != a.tokens;
  for (int s = lane; s < a.n_seq; s += 32) bad |= a.cu[s + 1] < a.cu[s] || a.cu[s] < 0 || a.cu[s + 1] > a.tokens;
  if (!__any_sync(0xffffffffu, bad)) return true;
  if (lane == 0) report_status(a.status, 7 /* KDA_ERR_DEVICE_CHECK */);
  return false;
}

__device__ __forceinline__ Item whole_sequence(const int32_t* cu, int s) {
  Item it;
  it.seq = s; it.first = cu[s]; it.len = cu[s + 1] - cu[s];
  it.c0 = 0; it.c1 = static_cast<int>((static_cast<int64_t>(it.len) + kC - 1) / kC);
  it.seg = 0; it.base = -1; it.last = 1;
  return it;
}

template <bool kFull>
__device__ void load_warp(const LinParams& p, uint8_t* sm, Small& s, int lane) {
  bool dead = false;
  uint32_t u = 0, n = 0, jobs = 0;
  const int pass = kFull ? 0 : 1;
  const bool planned = !kFull || p.p.counts != nullptr;
  const int64_t total = planned ? static_cast<int64_t>(p.p.counts[pass]) * p.a.H : offsets_hold(p.a, lane) ? gridDim.x : 0;
  int64_t t = blockIdx.x;
  for (;; ++jobs) {
    LIN_WAIT(s.job_empty[jobs & 1], (jobs >> 1) + 1);
    const bool more = t < total && !dead;
    Item it = {};
    int head = -1;
    if (more) {
      head = static_cast<int>(t % p.a.H);
      if (planned) it = p.p.items[pass][t / p.a.H];
      else it = whole_sequence(p.a.cu, static_cast<int>(t / p.a.H));
    }
    if (lane == 0) {
      s.job[jobs & 1].item = it;
      s.job[jobs & 1].head = head;
      mbar_arrive(&s.job_full[jobs & 1]);
    }
    if (!more) break;
    // the next item's number, known by the time that this one's copies are under way
    int next = 0;
    if (planned && lane == 0) next = atomicAdd(&p.p.counts[2 + pass], 1);
    const int hq = head / p.a.group;
    for (int c = it.c0; c < it.c1; ++c, ++n) {
      const int row = it.first + c * kC;
      const Tiles<kFull> tile(n);
#pragma unroll 1
      for (int w = 0; w < kKinds<kFull>; ++w, ++u) {
        const int kind = w;
        if (!kFull || kind == kQ) LIN_WAIT(s.free[kind][tile.buf], tile.phase + 1);
        else if (n > 1) LIN_WAIT(kind == kK ? s.kv[n & 1] : s.out[n & 1], (n >> 1) - 1);
        if (dead || static_cast<int>(u) == p.a.stall) continue;
        if (lane == 0) {
          const CUtensorMap* m = kind == kK ? &p.tk : kind == kQ ? &p.tq : &p.tv;
          const int h = kind == kV ? head : hq;
          uint8_t* dst = sm + tile.at(kind);
          uint64_t* full = &s.full[kind == kV][tile.buf];
          mbar_arrive_expect_tx(full, kTile);
          tma_load_3d(dst, m, full, 0, h, row);
          tma_load_3d(dst + kPanel, m, full, 64, h, row);
        }
        __syncwarp();
      }
    }
    t = gridDim.x + static_cast<int64_t>(__shfl_sync(0xffffffffu, next, 0));
  }
  // the last copies have landed before the block gives its shared memory back; of a barrier without any
  // (a copy left out) both phases are looked at, one of them for nothing
  for (int k = 0; k < 2; ++k)
    for (uint32_t i = 0; i < kBufs<kFull>; ++i) {
      const uint32_t uses = (n + kBufs<kFull> - 1 - i) / kBufs<kFull>;
      if (dead || p.a.stall >= 0) { wait_for(smem_u32(&s.full[k][i]), 0); wait_for(smem_u32(&s.full[k][i]), 1); }
      else if (uses > 0) wait_for(smem_u32(&s.full[k][i]), (uses - 1) & 1);
    }
  if (dead && lane == 0) report_status(p.a.status, 6 /* KDA_ERR_TIMEOUT */);
}

// D = A B^T, both K-major tiles of 128 columns.
__device__ __forceinline__ void product_ss(uint32_t who, uint32_t d, uint64_t a, uint64_t b) {
  constexpr uint32_t id = idesc_f16(128, 128, true, false, false);
#pragma unroll
  for (uint32_t kk = 0; kk < 8; ++kk) {
    const uint64_t off = ((kk & 4) << 8) | ((kk & 3) << 1);  // 16-byte units: panels of 64 columns, 16 columns a step
    mma_f16_if(who, d, a + off, b + off, id, kk);
  }
}
// D (+)= A B, A in tensor memory, B rows of an N-major tile.
template <uint32_t kSteps>
__device__ __forceinline__ void product_ts(uint32_t who, uint32_t d, uint32_t a, uint64_t b, uint32_t more) {
  constexpr uint32_t id = idesc_f16(128, 128, true, false, true);
#pragma unroll
  for (uint32_t kk = 0; kk < kSteps; ++kk) mma_f16_ta_if(who, d, a + 8 * kk, b + 128 * kk, id, more | kk);
}

// D += P B: of each 32 tokens' weights 16 columns are the first parts, the next 16 the second.
__device__ __forceinline__ void product_weights(uint32_t who, uint32_t d, uint32_t a, uint64_t b) {
  constexpr uint32_t id = idesc_f16(128, 128, true, false, true);
#pragma unroll
  for (uint32_t kk = 0; kk < 16; ++kk) {
    const uint32_t step = 2 * (kk >> 2) + (kk & 1);  // 16 tokens
    mma_f16_ta_if(who, d, a + 8 * kk, b + 128 * step, id, 1);
  }
}

template <bool kFull>
__device__ void mma_warp(const LinParams& p, uint8_t* sm, Small& s, int lane) {
  bool dead = false;
  Jobs jobs(s, dead);
  Job j;
  uint32_t n = 0, u = 0;
  const uint32_t who = elect_one_sync();
  const uint64_t d_k = smem_desc(smem_u32(sm), 16, 1024, kSwizzle128B);      // K-major tiles
  const uint64_t d_m = smem_desc(smem_u32(sm), kPanel, 1024, kSwizzle128B);  // the same, N-major
  while (jobs.next(j)) {
    for (int c = j.item.c0; c < j.item.c1; ++c, ++n) {
      const Tiles<kFull> tile(n);
      const uint64_t tk = tile.at(kK) >> 4, tq = tile.at(kQ) >> 4, tv = tile.at(kV) >> 4;
      LIN_WAIT(s.full[0][tile.buf], tile.phase);
      if constexpr (kFull) {
        if (n > 0) LIN_WAIT(s.out[(n - 1) & 1], (n - 1) >> 1);  // the last weights, where the scores go, are used
        tc_fence_after();
        if (dead) break;
        product_ss(who, kTS, d_k + tq, d_k + tk);
        mma_commit_if(who, &s.scores);
        LIN_WAIT(s.state, n);  // the state in front of the chunk is in shared memory, the last K^T V is read
      }
      if (!kFull && n > 1) LIN_WAIT(s.kv_read[n & 1], (n >> 1) - 1);  // K^T V of the last chunk but one is read
      // (the values' parts)^T K, 64 tokens at a time
#pragma unroll 1
      for (uint32_t h = 0; h < 2; ++h) {
        if (kFull && h == 1) {
          if (n > 0) LIN_WAIT(s.out_free, n - 1);
          tc_fence_after();
          if (dead) break;
          product_ss(who, kTO, d_k + tq, d_k + (kSmState >> 4));
          mma_commit_if(who, &s.inter);
        }
        if constexpr (kFull) LIN_WAIT(s.half_full[0], 2 * n + h);
        else LIN_WAIT(s.half_full[h], n);
        tc_fence_after();
        if (dead) break;
#pragma unroll
        for (uint32_t part = 0; part < 3; ++part, ++u) {
          product_ts<4>(who, kv_column<kFull>(n), unit_column<kFull>(u), d_m + tk + 512 * h, h | part);
          if (part == 1) mma_commit_if(who, &s.half_free[kFull ? 0 : h]);  // with the one before, room for the next three
        }
      }
      if (dead) break;
      mma_commit_if(who, &s.kv[n & 1]);
      if constexpr (!kFull) mma_commit_if(who, &s.free[kK][tile.buf]);
      if constexpr (kFull) {
        LIN_WAIT(s.ready, n);  // v has landed before its parts were made
        tc_fence_after();
        if (dead) break;
        product_weights(who, kTO, kTS, d_m + tv);
        mma_commit_if(who, &s.out[n & 1]);
      }
    }
    if (dead) break;
  }
  // products in flight end before the tensor memory is given back
  mma_commit_if(who, &s.drain);
  wait_for(smem_u32(&s.drain), 0);
  if (dead && lane == 0) report_status(p.a.status, 6 /* KDA_ERR_TIMEOUT */);
}

// One warp, four tokens a lane.
template <bool kFull>
__device__ void decay_warp(const LinParams& p, Small& s, int lane) {
  constexpr float kUnit = 4294967296.f;     // 2^32
  constexpr float kLeast = -192.f * kUnit;  // 2^-192 is 0 in 32 bits: what is smaller forgets as well
  bool dead = false;
  Jobs jobs(s, dead);
  Job j;
  uint32_t n = 0;
  while (jobs.next(j)) {
    const float* g = p.a.g + j.head * p.a.g_stride[2];
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    auto load = [&](int c) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = c * kC + 4 * lane + i;
        x[i] = row < j.item.len ? g[(static_cast<int64_t>(j.item.first) + row) * p.a.g_stride[1]] : 0.f;
      }
    };
    if (j.item.c0 < j.item.c1) load(j.item.c0);
    for (int c = j.item.c0; c < j.item.c1; ++c, ++n) {
      long long G[4], sum = 0;
      int bad = kC;  // this lane's first token whose decay is NaN
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool nan = x[i] != x[i];
        if (nan) bad = min(bad, 4 * lane + i);
        sum += nan ? 0 : __float2ll_rn(fminf(fmaxf(x[i] * (1.4426950408889634f * kUnit), kLeast), -kLeast));
        G[i] = sum;
      }
      if (c + 1 < j.item.c1) load(c + 1);
      // it, all later tokens of the chunk and the state are NaN
      const int nan_at = __reduce_min_sync(0xffffffffu, bad);
      const long long own = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, sum, off);
        if (lane >= off) sum += y;
      }
      const long long last = __shfl_sync(0xffffffffu, sum, 31);
      const long long end = __shfl_sync(0xffffffffu, sum, lane | 7);  // of the block of 32 tokens
      auto real = [](long long d) { return static_cast<float>(d) * (1.f / kUnit); };
      const float none = __int_as_float(0x7fffffff);
      float f[4], e = exp2f(real(last - end));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        G[i] += sum - own;
        f[i] = exp2f(real(end - G[i]));
      }
      // the weights' warps are done with these places too: the last chunk but one's dec_empty has been waited for
      LIN_WAIT(s.w_empty[n & 1], (n >> 1) + 1);
      *reinterpret_cast<float4*>(&s.cf[n & 1][4 * lane]) = make_float4(f[0], f[1], f[2], f[3]);
      if ((lane & 7) == 0) s.end[n & 1][lane >> 3] = e;
      if (lane == 0) s.a[n & 1] = nan_at < kC ? none : exp2f(real(last));
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.w_full[n & 1]);
      if constexpr (kFull) {
        float whole[4], part[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          whole[i] = 4 * lane + i >= nan_at ? none : static_cast<float>(static_cast<int>(G[i] >> 32));
          part[i] = static_cast<float>(static_cast<uint32_t>(G[i])) * (1.f / kUnit);
        }
        LIN_WAIT(s.dec_empty, n + 1);
        *reinterpret_cast<float4*>(&s.dec.whole[4 * lane]) = make_float4(whole[0], whole[1], whole[2], whole[3]);
        *reinterpret_cast<float4*>(&s.dec.part[4 * lane]) = make_float4(part[0], part[1], part[2], part[3]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.dec_full);
      }
    }
  }
  if (dead && lane == 0) report_status(p.a.status, 6 /* KDA_ERR_TIMEOUT */);
}

// 32 rows x 64 channels from shared memory to o.
__device__ __forceinline__ void tma_store_3d(const void* tmap, const void* src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];\n" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

// The output stage's gate, into q's tile when q is used.
__device__ void gate_warp(const LinParams& p, uint8_t* sm, Small& s, int lane) {
  bool dead = false;
  Jobs jobs(s, dead);
  Job j;
  uint32_t n = 0;
  while (jobs.next(j)) {
    if (lane == 0 && j.item.c0 < j.item.c1) {
      tma_prefetch_3d(&p.tg, 0, j.head, j.item.first + j.item.c0 * kC);
      tma_prefetch_3d(&p.tg, 64, j.head, j.item.first + j.item.c0 * kC);
    }
    for (int c = j.item.c0; c < j.item.c1; ++c, ++n) {
      const Tiles<true> tile(n);
      const int row = j.item.first + c * kC;
      if (lane == 0 && c + 1 < j.item.c1) {  // the next chunk's, so that its copy comes from L2
        tma_prefetch_3d(&p.tg, 0, j.head, row + kC);
        tma_prefetch_3d(&p.tg, 64, j.head, row + kC);
      }
      LIN_WAIT(s.inter, n);
      if (lane == 0 && !dead) {
        mbar_arrive_expect_tx(&s.gate_full, kTile);
        tma_load_3d(sm + tile.at(kQ), &p.tg, &s.gate_full, 0, j.head, row);
        tma_load_3d(sm + tile.at(kQ) + kPanel, &p.tg, &s.gate_full, 64, j.head, row);
      }
      __syncwarp();
      LIN_WAIT(s.gate_full, n);  // one at a time: the last has landed when the warp ends
    }
  }
  if (dead && lane == 0) report_status(p.a.status, 6 /* KDA_ERR_TIMEOUT */);
}

// A pair of bf16 as two floats.
__device__ __forceinline__ uint64_t floats(uint32_t u) {
  return f32x2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// sigmoid of a pair of gates: the approximations are within 2^-21 of it, and 1 / inf is 0.
__device__ __forceinline__ uint64_t open_gates(uint32_t g) {
  const float l = -1.4426950408889634f;
  const float2 y = unpack_f32x2(mul_f32x2(floats(g), f32x2(l, l)));
  const float2 z = unpack_f32x2(add_f32x2(f32x2(exp2_fast(y.x), exp2_fast(y.y)), f32x2(1.f, 1.f)));
  float r0, r1;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(z.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(z.y));
  return f32x2(r0, r1);
}

// A pair of floats as bf16 and what that leaves of them.
__device__ __forceinline__ void two_parts(uint64_t y, uint32_t& hi, uint32_t& low) {
  hi = bf162_of(y);
  low = bf162_of(fma_f32x2(floats(hi), f32x2(-1.f, -1.f), y));
}

// 32 columns of a row times e, in place.
__device__ __forceinline__ void scale_block(uint32_t at, float e) {
  float x[32];
  tmem_ld32(at, x);
  const uint64_t e2 = f32x2(e, e);
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const float2 y = unpack_f32x2(mul_f32x2(f32x2(x[i], x[i + 1]), e2));
    x[i] = y.x;
    x[i + 1] = y.y;
  }
  tmem_st32(at, x);
}

// NaN for the rows that see a value that is not finite, in its channel, of some channels (cold).  The values were
// cleared in the tile: they are looked at where they came from.
__device__ __forceinline__ void poison(uint32_t tl, const LinArgs& a, const Item& it, int head, int c, int i, int first, int channels) {
  const int live = live_rows(it, c), lane = threadIdx.x & 31;
  const auto* v = static_cast<const uint16_t*>(a.v) + (static_cast<int64_t>(it.first) + c * kC) * a.v_stride[1] + head * a.v_stride[2];
#pragma unroll 1
  for (int ch = first; ch < first + channels; ++ch) {
    int seen = kC;  // the first such token
#pragma unroll 1
    for (int t = 96; t >= 0; t -= 32) {
      const uint32_t bits = t + lane < live ? v[(t + lane) * a.v_stride[1] + ch] : 0;
      const uint32_t m = __ballot_sync(0xffffffffu, (bits & 0x7f80) == 0x7f80);
      if (m) seen = t + __ffs(m) - 1;
    }
    if (!__any_sync(0xffffffffu, seen <= i)) continue;
    uint32_t x;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\ntcgen05.wait::ld.sync.aligned;\n" : "=r"(x) : "r"(tl + ch));
    if (seen <= i) x = 0x7fffffffu;
    __syncwarp();
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};\ntcgen05.wait::st.sync.aligned;\n" ::"r"(tl + ch), "r"(x) : "memory");
  }
}

// Half a row of the staged outputs, where not all of a warp's rows are the sequence's (cold).
__device__ __forceinline__ void copy_row(uint32_t stage, uint4* dst, int i) {
#pragma unroll 1
  for (int q = 0; q < 8; ++q) dst[q] = lds128(stage + sw128(i, 16 * q));
}

__device__ void weight_warps(const LinParams& p, Small& s, int w, int lane) {
  const LinArgs& a = p.a;
  bool dead = false;
  Jobs jobs(s, dead);
  Job j;
  uint32_t n = 0;
  const uint32_t ts = (static_cast<uint32_t>(w) << 21) + kTS, tl = (static_cast<uint32_t>(w) << 21) + kTO;
  const int i = 32 * w + lane;
  while (jobs.next(j)) {
    for (int c = j.item.c0; c < j.item.c1; ++c, ++n) {
      // ---- weights, 32 columns at a time, over the scores of columns that are read already
      LIN_WAIT(s.dec_full, n);
      const Decays& d = s.dec;
      const float* cf = s.cf[n & 1];
      const float whole = d.whole[i], part = d.part[i];
      LIN_WAIT(s.scores, n);
      tc_fence_after();
#pragma unroll 1
      for (int b = 0; b < w; ++b) {  // D_ij = 2^{G_i - G at the block's end} 2^{G at the block's end - G_j}
        float x[32];
        tmem_ld32(ts + 32 * b, x);
        const float rf = exp2_fast((whole - d.whole[32 * b + 31]) + (part - d.part[32 * b + 31]));
        const uint64_t r2 = f32x2(rf, rf);
        uint32_t pk[32];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 f = *reinterpret_cast<const float4*>(&cf[32 * b + e]);
          two_parts(mul_f32x2(f32x2(x[e], x[e + 1]), mul_f32x2(r2, f32x2(f.x, f.y))), pk[e / 2], pk[16 + e / 2]);
          two_parts(mul_f32x2(f32x2(x[e + 2], x[e + 3]), mul_f32x2(r2, f32x2(f.z, f.w))), pk[e / 2 + 1], pk[17 + e / 2]);
        }
        tmem_st32(ts + 32 * b, reinterpret_cast<const float(&)[32]>(pk));
      }
      {
        float x[32];
        uint32_t pk[32];
        const uint64_t whole2 = f32x2(whole, whole), part2 = f32x2(part, part), minus = f32x2(-1.f, -1.f);
        tmem_ld32(ts + 32 * w, x);
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 f = *reinterpret_cast<const float4*>(&d.whole[32 * w + e]), h = *reinterpret_cast<const float4*>(&d.part[32 * w + e]);
          const float2 g0 = unpack_f32x2(add_f32x2(fma_f32x2(f32x2(f.x, f.y), minus, whole2), fma_f32x2(f32x2(h.x, h.y), minus, part2)));
          const float2 g1 = unpack_f32x2(add_f32x2(fma_f32x2(f32x2(f.z, f.w), minus, whole2), fma_f32x2(f32x2(h.z, h.w), minus, part2)));
          const float y0 = e <= lane ? x[e] * exp2_fast(g0.x) : 0.f;
          const float y1 = e + 1 <= lane ? x[e + 1] * exp2_fast(g0.y) : 0.f;
          const float y2 = e + 2 <= lane ? x[e + 2] * exp2_fast(g1.x) : 0.f;
          const float y3 = e + 3 <= lane ? x[e + 3] * exp2_fast(g1.y) : 0.f;
          two_parts(f32x2(y0, y1), pk[e / 2], pk[16 + e / 2]);
          two_parts(f32x2(y2, y3), pk[e / 2 + 1], pk[17 + e / 2]);
        }
        tmem_st32(ts + 32 * w, reinterpret_cast<const float(&)[32]>(pk));
#pragma unroll
        for (int e = 0; e < 32; ++e) pk[e] = 0;
#pragma unroll 1
        for (int b = w + 1; b < 4; ++b) tmem_st32(ts + 32 * b, reinterpret_cast<const float(&)[32]>(pk));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.dec_empty);
      // ---- Q S times e^G
      const float eg = exp2f(whole + part);
      LIN_WAIT(s.inter, n);
      tc_fence_after();
#pragma unroll 1
      for (int b = 0; b < 4; ++b) scale_block(tl + 32 * b, eg);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.ready);
    }
  }
  if (dead && lane == 0) report_status(a.status, 6 /* KDA_ERR_TIMEOUT */);
}

// 8 x 8 tiles of 16-bit values, transposed: lanes 8 m .. 8 m + 7 point to the rows of tile m; of each tile a lane gets
// column lane / 4, rows 2 (lane % 4) and the next.
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// 16 lanes x 8 columns of tensor memory: registers 2 k and 2 k + 1 are column 4 k + lane % 4 of lanes lane / 4 and
// lane / 4 + 8.
__device__ __forceinline__ void tmem_st_16x128b_x2(uint32_t taddr, const uint32_t (&u)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(taddr), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3])
               : "memory");
}

// Values of a warp's 32 channels and 16 tokens that are not finite, cleared in the tile (cold).
__device__ __forceinline__ void clear_bad(uint32_t tile, uint32_t* bad_chunk, uint32_t n, int w, int t0, int lane) {
  const int ch = 32 * w + lane;
  const uint32_t base = tile + (ch >> 6) * kPanel;
#pragma unroll 1
  for (int t = t0; t < t0 + 16; ++t) {
    const uint32_t at = base + sw128(t, 2 * (ch & 63));
    uint16_t x;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(at) : "memory");
    if ((x & 0x7f80) == 0x7f80) asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(static_cast<uint16_t>(0)) : "memory");
  }
  __syncwarp();
  if (lane == 0) bad_chunk[n & 3] = n + 1;
}

// Decayed values, transposed: y = 2^{G_last - G_t} v_t as hi + mid + low, each the nearest bf16 of what is left, in tensor
// memory [channel][token].
// Rows past the sequence's end are cleared in the tiles of k and v: what stands there must not meet the
// state, or P V.
template <bool kFull>
__device__ void value_warps(const LinParams& p, uint8_t* sm, Small& s, int w, int lane) {
  bool dead = false;
  Jobs jobs(s, dead);
  Job j;
  uint32_t n = 0, u = 0;
  const uint64_t minus = f32x2(-1.f, -1.f);
  const int q = w & 3, side = w >> 2;  // channels 32 q .. + 31; tokens 32 side .. + 31 of each 64
  while (jobs.next(j)) {
    for (int c = j.item.c0; c < j.item.c1; ++c, ++n) {
      const Tiles<kFull> tile(n);
      const int live = live_rows(j.item, c);
      const uint32_t v = smem_u32(sm) + tile.at(kV);
      LIN_WAIT(s.full[1][tile.buf], tile.phase);
      if (live < kC) {
        LIN_WAIT(s.full[0][tile.buf], tile.phase);
        if constexpr (kFull) LIN_WAIT(s.scores, n);  // Q K^T has read the keys
        const uint32_t k = smem_u32(sm) + tile.at(kK);
        if (!dead)
          for (int e = lane; e < 4 * 64; e += 32) {  // the warp's tokens, 64 bytes of each
            const int row = (e >> 2 & 31) + 32 * side + 64 * (e >> 7);
            if (row < live) continue;
            const uint32_t at = (q >> 1) * kPanel + sw128(row, 64 * (q & 1) + 16 * (e & 3));
            sts128(k + at, make_uint4(0, 0, 0, 0));
            sts128(v + at, make_uint4(0, 0, 0, 0));
          }
        fence_proxy_async_smem();
        __syncwarp();
      }
      LIN_WAIT(s.w_full[n & 1], n >> 1);
      const float* wp = &s.cf[n & 1][2 * (lane & 3)];
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        const float e = s.end[n & 1][2 * h + side];
        const uint64_t e2 = f32x2(e, e);
#pragma unroll 1
        for (int piece = 0; piece < 2; ++piece) {
          const int t0 = 64 * h + 32 * side + 16 * piece;
          uint32_t part[3][2][4];  // [part][16 channels][..]
          uint64_t any = f32x2(0.f, 0.f);  // NaN if a value is not finite: what is left of it is NaN
#pragma unroll
          for (int b = 0; b < 2; ++b) {  // 8 tokens, 32 channels
            uint32_t r[4];
            const int ch = 32 * q + 8 * (lane >> 3);
            ldsm4_trans(v + (ch >> 6) * kPanel + sw128(t0 + 8 * b + (lane & 7), 2 * (ch & 63)), r);
            const uint64_t f = mul_f32x2(*reinterpret_cast<const uint64_t*>(wp + t0 + 8 * b), e2);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              uint64_t y = mul_f32x2(floats(r[m]), f);
              const uint32_t hi = bf162_of(y);
              y = fma_f32x2(floats(hi), minus, y);
              const uint32_t mid = bf162_of(y);
              y = fma_f32x2(floats(mid), minus, y);
              any = add_f32x2(any, y);
              part[0][m >> 1][2 * b + (m & 1)] = hi;
              part[1][m >> 1][2 * b + (m & 1)] = mid;
              part[2][m >> 1][2 * b + (m & 1)] = bf162_of(y);
            }
          }
          const float2 left = unpack_f32x2(any);
          if (kFull && __any_sync(0xffffffffu, left.x + left.y != left.x + left.y)) {
            clear_bad(v, s.bad_chunk, n, q, t0, lane);
            fence_proxy_async_smem();
          }
          if (piece == 0) {
            if constexpr (kFull) { if (u > 0) LIN_WAIT(s.half_free[0], 2 * n + h - 1); }
            else { if (n > 0) LIN_WAIT(s.half_free[h], n - 1); }
            tc_fence_after();
          }
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const uint32_t at = (static_cast<uint32_t>(q) << 21) + unit_column<kFull>(u + k) + 16 * side + 8 * piece;
            tmem_st_16x128b_x2(at, part[k][0]);
            tmem_st_16x128b_x2(at + (16u << 16), part[k][1]);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.half_full[kFull ? 0 : h]);
        u += 3;
      }
      if (lane == 0) {
        mbar_arrive(&s.w_empty[n & 1]);
        if (!kFull) mbar_arrive(&s.free[kV][tile.buf]);
      }
      __syncwarp();
    }
  }
  if (dead && lane == 0) report_status(p.a.status, 6 /* KDA_ERR_TIMEOUT */);
}

// The final state of a sequence without tokens is its entry state (256 threads).
__device__ __forceinline__ void entry_to_exit(const LinArgs& a, int seq, int head, int thread) {
  if (!a.S_out || a.S_in == a.S_out) return;
  const int64_t at = (static_cast<int64_t>(seq) * a.H + head) * (kStateFloats / 4);
  for (int e = thread; e < kStateFloats / 4; e += 256)
    reinterpret_cast<float4*>(a.S_out)[at + e] = a.S_in ? reinterpret_cast<const float4*>(a.S_in)[at + e] : make_float4(0.f, 0.f, 0.f, 0.f);
}

template <int kMode>
__device__ void state_warps(const LinParams& p, uint8_t* sm, Small& s, int w, int lane) {
  constexpr bool kFull = kMode != kStates, kGate = kMode == kGated;
  const LinArgs& a = p.a;
  bool dead = false;
  Jobs jobs(s, dead);
  Job j;
  uint32_t n = 0;
  const int ch = 32 * (w & 3) + lane, half = w >> 2;  // channel of v: a column of the state; rows 64 half ..
  const uint32_t tl = (static_cast<uint32_t>(w & 3) << 21) + 64 * half;
  const uint32_t copy = smem_u32(sm) + kSmState + half * kPanel;
  constexpr int kHalf = kD / 2;
  // ---- outputs of a chunk: 32 tokens, 64 channels
  auto outputs = [&](const Item& it, int head, int c) {
    const Tiles<kFull> tile(n);
    const int i = ch;  // the thread's token in the chunk
    const uint32_t to_q = (static_cast<uint32_t>(w & 3) << 21) + kTO, to = to_q + 64 * half;
    if constexpr (kGate) LIN_WAIT(s.gate_full, n);
    LIN_WAIT(s.out[n & 1], n >> 1);
    tc_fence_after();
    // with the output stage all 128: both warps of a row sum its squares, and neither waits for the other's mark
    if (s.bad_chunk[n & 3] == n + 1)
      poison(to_q, a, it, head, c, i, kGate ? 0 : 64 * half, kGate ? kD : 64);
    float f = a.scale;
    if constexpr (kGate) {  // the row's sum of squares, by both warps that have it
      uint64_t s0 = f32x2(0.f, 0.f), s1 = s0;
#pragma unroll 1
      for (int b = 0; b < 4; ++b) {
        float x[32];
        tmem_ld32(to_q + 32 * b, x);
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const uint64_t x0 = f32x2(x[e], x[e + 1]), x1 = f32x2(x[e + 2], x[e + 3]);
          s0 = fma_f32x2(x0, x0, s0);
          s1 = fma_f32x2(x1, x1, s1);
        }
      }
      const float2 sum = unpack_f32x2(add_f32x2(s0, s1));
      f *= 1.f / sqrtf((sum.x + sum.y) * a.scale * a.scale * (1.f / kD) + a.eps);
    }
    const uint32_t stage = smem_u32(sm) + tile.at(kQ) + half * kPanel;  // q is used: its tile takes the outputs
#pragma unroll 1
    for (int b = 0; b < 4; ++b) {
      float x[16];
      tmem_ld16(to + 16 * b, x);
      if (b == 3) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.out_free);
      }
      const uint32_t at0 = stage + sw128(i, 32 * b), at1 = stage + sw128(i, 32 * b + 16);
      uint32_t pk[8];
      if constexpr (kGate) {
        const uint4 u0 = lds128(at0), u1 = lds128(at1);
        pk[0] = u0.x; pk[1] = u0.y; pk[2] = u0.z; pk[3] = u0.w; pk[4] = u1.x; pk[5] = u1.y; pk[6] = u1.z; pk[7] = u1.w;
      }
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        uint64_t y = mul_f32x2(f32x2(x[e], x[e + 1]), f32x2(f, f));
        if constexpr (kGate)
          y = mul_f32x2(mul_f32x2(y, *reinterpret_cast<const uint64_t*>(&s.weight[64 * half + 16 * b + e])), open_gates(pk[e >> 1]));
        pk[e >> 1] = bf162_of(y);
      }
      sts128(at0, make_uint4(pk[0], pk[1], pk[2], pk[3]));
      sts128(at1, make_uint4(pk[4], pk[5], pk[6], pk[7]));
    }
    fence_proxy_async_smem();
    __syncwarp();
    const int live = live_rows(it, c), row = it.first + c * kC + 32 * (w & 3);
    if (32 * (w & 3) + 32 <= live) {
      if (lane == 0 && !dead) {
        tma_store_3d(&p.to, sm + tile.at(kQ) + half * kPanel + (w & 3) * 4096, 64 * half, head, row);
        asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
      }
    } else if (i < live && !dead) {  // the next sequence's rows are not this one's to write
      copy_row(stage, reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) +
                                               ((static_cast<int64_t>(row) + lane) * a.H + head) * kD + 64 * half), i);
    }
    __syncwarp();
    if (lane == 0) {  // nothing to do until K^T V of the next chunk, and the next but one's q waits for its place
      asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory");
      mbar_arrive(&s.free[kQ][tile.buf]);
    }
    __syncwarp();
  };
  while (jobs.next(j)) {
    const Item& it = j.item;
    const int mine = half * kHalf * kD + ch;
    auto slot = [&](int k) { return p.p.slots + (static_cast<int64_t>(it.base + k) * a.H + j.head) * kStateFloats + mine; };
    const int64_t unit = (static_cast<int64_t>(it.seq) * a.H + j.head) * kStateFloats + mine;
    if (kFull && it.c0 == it.c1) {  // without a plan an item may be a sequence without tokens
      if (!dead) entry_to_exit(a, it.seq, j.head, 32 * w + lane);
      continue;
    }
    float S[kHalf], A = 1.f;
    auto load = [&](const float* src) {
#pragma unroll
      for (int e = 0; e < kHalf; ++e) S[e] = src[e * kD];
    };
    auto store = [&](float* dst) {
#pragma unroll
      for (int e = 0; e < kHalf; ++e) dst[e * kD] = S[e];
    };
    if (it.seg == 0 && a.S_in) {
      // the second pass of a split sequence reads the copy: S_out may be S_in
      load(kFull && it.base >= 0 ? slot(0) : a.S_in + unit);
      if (!kFull) store(slot(0));
    } else if (kFull && it.seg > 0) {
      load(slot(1));
#pragma unroll 1
      for (int k = 1; k < it.seg; ++k) {
        const float f = p.p.decay[static_cast<int64_t>(it.base + 1 + k) * a.H + j.head];
        const float* src = slot(1 + k);
#pragma unroll
        for (int e = 0; e < kHalf; ++e) S[e] = fmaf(f, S[e], src[e * kD]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < kHalf; ++e) S[e] = 0.f;
    }
    auto publish = [&] {  // rounded to bf16 for Q S
#pragma unroll
      for (int e = 0; e < 8; ++e)
        sts128(copy + sw128(ch, 16 * e), make_uint4(pack_bf162(S[8 * e], S[8 * e + 1]), pack_bf162(S[8 * e + 2], S[8 * e + 3]),
                                                    pack_bf162(S[8 * e + 4], S[8 * e + 5]), pack_bf162(S[8 * e + 6], S[8 * e + 7])));
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.state);
    };
    if constexpr (kFull) publish();
    for (int c = it.c0; c < it.c1; ++c, ++n) {
      LIN_WAIT(s.w_full[n & 1], n >> 1);
      const float f = s.a[n & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.w_empty[n & 1]);
      A *= f;
      LIN_WAIT(s.kv[n & 1], n >> 1);
      tc_fence_after();
      const uint32_t at = tl + kv_column<kFull>(n);
      constexpr int kStep = kFull ? 32 : 16;  // columns at a time: what the registers of either instance take
#pragma unroll
      for (int q = 0; q < kHalf; q += kStep) {
        float x[kStep];
        if constexpr (kFull) tmem_ld32(at + q, x);
        else tmem_ld16(at + q, x);
        if (!kFull && q + kStep == kHalf) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.kv_read[n & 1]);
        }
#pragma unroll
        for (int e = 0; e < kStep; e += 2) {
          const float2 y = unpack_f32x2(fma_f32x2(f32x2(f, f), f32x2(S[q + e], S[q + e + 1]), f32x2(x[e], x[e + 1])));
          S[q + e] = y.x;
          S[q + e + 1] = y.y;
        }
      }
      if constexpr (kFull) {
        if (c + 1 < it.c1) publish();
        else if (it.last && a.S_out && !dead) store(a.S_out + unit);
        outputs(it, j.head, c);
      }
    }
    if constexpr (!kFull) {
      store(slot(1 + it.seg));
      if (w == 0 && lane == 0) p.p.decay[static_cast<int64_t>(it.base + 1 + it.seg) * a.H + j.head] = A;
    }
  }
  tc_fence_before();
  if constexpr (kFull) {
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
  }
  if constexpr (kFull) {  // sequences without tokens, which the plan puts last
    if (p.p.counts && !dead)
      for (int64_t t = blockIdx.x; t < static_cast<int64_t>(p.p.counts[4]) * a.H; t += gridDim.x)
        entry_to_exit(a, p.p.items[0][p.p.counts[0] + t / a.H].seq, static_cast<int>(t % a.H), 32 * w + lane);
  }
  if (dead && lane == 0) report_status(a.status, 6 /* KDA_ERR_TIMEOUT */);
}

template <int kMode>
__global__ void __launch_bounds__(kThreads, 1) lin_chunk_kernel(const __grid_constant__ LinParams p) {
  constexpr bool kFull = kMode != kStates;
  extern __shared__ __align__(1024) uint8_t sm[];
  Small& s = *reinterpret_cast<Small*>(sm + kSmSmall);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(sm) & 1023) {  // the swizzled tiles need it
    if (tid == 0) report_status(p.a.status, 5 /* KDA_ERR_CUDA */);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < 3; ++i) {
      mbar_init(&s.full[0][i], kFull ? 2 : 1);
      mbar_init(&s.full[1][i], 1);
      mbar_init(&s.free[kK][i], 1);
      mbar_init(&s.free[kV][i], 8);
      mbar_init(&s.free[kQ][i], 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.job_full[i], 1);
      mbar_init(&s.job_empty[i], kMode == kGated ? 23 : kMode == kPlain ? 22 : 18);  // warps that read a job
      mbar_init(&s.w_full[i], 1);
      mbar_init(&s.w_empty[i], 16);
      mbar_init(&s.kv[i], 1);
      mbar_init(&s.out[i], 1);
      mbar_init(&s.kv_read[i], 8);
    }
    for (int i = 0; i < 4; ++i) s.bad_chunk[i] = 0;
    for (int i = 0; i < 2; ++i) { mbar_init(&s.half_full[i], 8); mbar_init(&s.half_free[i], 1); }
    mbar_init(&s.dec_full, 1); mbar_init(&s.dec_empty, 4); mbar_init(&s.scores, 1); mbar_init(&s.inter, 1);
    mbar_init(&s.ready, 4); mbar_init(&s.out_free, 8); mbar_init(&s.state, 8); mbar_init(&s.drain, 1);
    mbar_init(&s.gate_full, 1);
    fence_mbar_init();
  }
  pdl_launch_dependents();
  if (warp == 1) {
    tmem_alloc(&s.tmem, 512);  // all of it, so its addresses begin at 0
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  if (kMode == kGated && tid < kD) s.weight[tid] = p.a.norm_weight ? p.a.norm_weight[tid] : 1.f;
  __syncthreads();
  // registers: kRegs a thread at launch, 480 over the six groups of four warps
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;\n" ::: "memory");
    if (warp == 0) load_warp<kFull>(p, sm, s, lane);
    else if (warp == 1) mma_warp<kFull>(p, sm, s, lane);
    else if (warp == 2) decay_warp<kFull>(p, s, lane);
    else if constexpr (kMode == kGated) gate_warp(p, sm, s, lane);
  } else if (warp < 8) {
    if constexpr (kFull) weight_warps(p, s, warp - 4, lane);
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 24;\n" ::: "memory");
  } else if (warp < 16) {
    if constexpr (kFull) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n" ::: "memory");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 88;\n" ::: "memory");
    value_warps<kFull>(p, sm, s, warp - 8, lane);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 112;\n" ::: "memory");
    state_warps<kMode>(p, sm, s, warp - 16, lane);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(s.tmem, 512);
}

// ------------------------------------------------------------------------------- host side
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

// Rows [tokens][heads][128] of bf16 in boxes of some tokens and 64 channels.
bool rows_map(CUtensorMap* m, const void* base, const int64_t* stride, int heads, int64_t tokens, int rows = kC) {
  const auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {kD, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(stride[2]) * 2, static_cast<cuuint64_t>(stride[1]) * 2};
  const cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(rows)}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kMode>
cudaError_t launch_chunks(const LinParams& p, int64_t items, int num_sms) {
  static SmemOptIn opt_in;
  const auto kernel = lin_chunk_kernel<kMode>;
  cudaError_t e = opt_in(reinterpret_cast<const void*>(kernel), kSmBytes);
  if (e != cudaSuccess) return e;
  // setmaxnreg's shares add up to kRegs a thread: with fewer at launch the groups would wait for them forever
  static const int regs = [] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, lin_chunk_kernel<kMode>) == cudaSuccess ? at.numRegs : 0;
  }();
  if (regs < kRegs) return cudaErrorLaunchOutOfResources;
  const unsigned grid = static_cast<unsigned>(items < num_sms ? items : num_sms);
  return launch_after(kernel, dim3(grid), dim3(kThreads), kSmBytes, p.a.stream, p);
}

}  // namespace

size_t lin_prefill_workspace(int n_seq, int64_t tokens, int H, int n_segments, int num_sms) {
  Plan p;
  return plan_layout(&p, nullptr, n_seq, tokens, H, n_segments, num_sms);
}

cudaError_t launch_lin_prefill(const LinArgs& a, int num_sms) {
  LinParams p;
  memset(&p, 0, sizeof(p));
  p.a = a;
  const size_t need = plan_layout(&p.p, a.workspace, a.n_seq, a.tokens, a.H, a.n_segments, num_sms);
  const int64_t o_stride[3] = {0, static_cast<int64_t>(a.H) * kD, kD};
  if (a.tokens > 0 && (!rows_map(&p.tq, a.q, a.q_stride, a.H / a.group, a.tokens) || !rows_map(&p.tk, a.k, a.k_stride, a.H / a.group, a.tokens) ||
                       !rows_map(&p.tv, a.v, a.v_stride, a.H, a.tokens) ||
                       !rows_map(&p.to, a.o, o_stride, a.H, a.tokens, 32) ||
                       (a.gate && !rows_map(&p.tg, a.gate, a.gate_stride, a.H, a.tokens))))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  if (need > 0) {
    e = launch_after(lin_plan_kernel, dim3(1), dim3(1024), 0, a.stream, a.cu, a.n_seq, a.tokens, a.H, num_sms, a.n_segments,
                     p.p, a.status);
    if (e != cudaSuccess) return e;
  }
  // the first pass only where the rule can split: one sequence of all the tokens is cut most
  if (p.p.most[1] > 0 && segments_of(a.tokens, a.tokens, a.H, num_sms, a.n_segments) > 1) {
    e = launch_chunks<kStates>(p, p.p.most[1] * a.H, num_sms);
    if (e != cudaSuccess) return e;
  }
  return a.gate ? launch_chunks<kGated>(p, p.p.most[0] * a.H, num_sms) : launch_chunks<kPlain>(p, p.p.most[0] * a.H, num_sms);
}

}  // namespace kda
