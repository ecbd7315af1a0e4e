// kda_lin_prefill.cu -- linear attention with a decay a head over packed sequences, chunk by chunk.
//
// With G_i the inclusive sum of a chunk's log-decays (128 tokens), S the state in front of it:
//     O  = scale ((Q K^T) o D) V + scale diag(e^G) Q S,      D_ij = e^{G_i - G_j} (j <= i), else 0
//     S' = e^{G_last} S + (diag(e^{G_last - G}) K)^T V
// All exponents are differences of sums of values <= 0, so nothing can grow whatever the decays are.
//
// One block walks the chunks of a (sequence, head) or of a segment of one; its warps:
//     0       copies (TMA, a ring of five 32 KiB tiles: k, q, v, k, q, ..) and the line of work items
//     1       products (tcgen05): Q K^T, Q S, K^T V, P V; 128 x 128 x 128 each, accumulators in tensor memory
//     2       decays: sums in 64-bit fixed point (2^-32 of a factor of 2), so that no difference loses bits
//     4 - 7   weights P = (Q K^T) o D to bf16 over their scores, then the outputs (thread = token)
//     8 - 11  decayed keys, split into two bf16 parts (16 bits together): hi in place of k, lo beside it
//     12 - 19 the state, in fp32 registers (thread = half a row); its bf16 copy for Q S in shared memory
//
// Rounded to bf16: P and the copy of S, for o only, which is bf16 itself.  The state sees 16-bit keys and
// exact values: K^T V is two products.
//
// A token's NaN or infinity must not reach earlier tokens, but 0 * NaN is NaN in P V: a row whose P V part is
// not finite is computed once more from the weights and values of the tokens that it sees (cold).
//
// Few heads: plan_segments' rule cuts a sequence into as many segments as its share of the work is worth
// in SMs.  A first pass (the same kernel without q and o) leaves each segment's state from zeros, the second
// begins with the sum over the segments before it.
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
constexpr int kThreads = 640;
constexpr int kRegs = 96;  // at launch
constexpr int kSlots = 5;
constexpr uint32_t kTile = 32768, kPanel = 16384;
constexpr uint32_t kSmLo = kSlots * kTile, kSmState = kSmLo + kTile, kSmSmall = kSmState + kTile;
// tensor memory columns
constexpr uint32_t kTS = 0, kTO = 128, kTI = 256, kTKV = 384;  // scores / weights; P V; Q S; K^T V
constexpr int kMinSegment = 8;  // chunks

// ------------------------------------------------------------------------------------ plan
struct Item {
  int seq, first, len;  // first packed row, tokens of the sequence
  int c0, c1;           // chunks
  int seg, base;        // segment number, the sequence's first slot (-1: not split)
  int last;             // the sequence's last segment
};

struct Plan {
  int* counts = nullptr;  // items of pass 2, of pass 1; next item of pass 2, of pass 1
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

size_t plan_layout(Plan* p, void* ws, int n_seq, int64_t tokens, int H, int forced, int sms) {
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
      p.counts[0] = p.counts[1] = p.counts[2] = p.counts[3] = 0;
    }
    return;
  }
  auto chunks = [&](int s) { return static_cast<int>((static_cast<int64_t>(cu[s + 1]) - cu[s] + kC - 1) / kC); };
  auto segments = [&](int s) { return segments_of(cu[s + 1] - cu[s], tokens, H, sms, forced); };
  auto length = [&](int s) { const int n = segments(s); return (chunks(s) + n - 1) / n; };
  for (int s = tid; s < n_seq; s += blockDim.x) atomicMax(&longest, length(s));
  __syncthreads();
  auto bin = [&](int s) { return 255 - static_cast<int>(static_cast<int64_t>(length(s)) * 255 / longest); };
  for (int s = tid; s < n_seq; s += blockDim.x) atomicAdd(&at[bin(s)], segments(s));
  __syncthreads();
  if (tid == 0) {
    int sum = 0;
    for (int i = 0; i < 256; ++i) { const int n = at[i]; at[i] = sum; sum += n; }
    p.counts[0] = sum;
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
  CUtensorMap tq, tk, tv;
  LinArgs a;
  Plan p;
};

struct Job {
  Item item;
  int head;  // -1: no more
};

struct Decays {  // of a chunk, in units of log2
  float G[kC];    // G_i
  float cf[kC];   // 2^{G at the end of the token's block of 32 - G_i}
  float wb[4];    // 2^{G_last - G at the end of block b}
  float a;        // 2^{G_last}
  float pad[3];
};

struct Small {
  Decays dec[2];
  Job job[2];
  uint64_t full[kSlots], empty[kSlots];
  uint64_t job_full[2], job_empty[2], dec_full[2], dec_empty[2];
  uint64_t scores, weights, keys, kv, state, out, out_free, drain;
  uint32_t tmem;
};
constexpr int kSmBytes = kSmSmall + sizeof(Small);
static_assert(kSmBytes <= 232448, "shared memory");

constexpr int kReaders = 18;  // warps that read a job

// The jobs that warp 0 hands out, in every other warp.
struct Jobs {
  Small& s;
  uint32_t n = 0;
  bool& dead;
  __device__ Jobs(Small& s_, bool& d) : s(s_), dead(d) {}
  __device__ bool next(Job& j) {
    if (dead || !bar_wait(&s.job_full[n & 1], (n >> 1) & 1)) { dead = true; return false; }
    j = s.job[n & 1];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&s.job_empty[n & 1]);
    ++n;
    return j.head >= 0;
  }
};

#define LIN_WAIT(bar, parity) do { if (!dead && !bar_wait(&(bar), (parity) & 1)) dead = true; } while (0)

__device__ __forceinline__ int live_rows(const Item& it, int c) { return min(kC, it.len - c * kC); }

template <bool kFull>
__device__ void load_warp(const LinParams& p, uint8_t* sm, Small& s, int lane) {
  constexpr int kEach = kFull ? 3 : 2;  // tiles a chunk
  bool dead = false;
  uint32_t u = 0, n = 0, left = 0;
  const int pass = kFull ? 0 : 1;
  const int64_t total = static_cast<int64_t>(p.p.counts[pass]) * p.a.H;
  int64_t t = blockIdx.x;
  for (;; ++n) {
    LIN_WAIT(s.job_empty[n & 1], (n >> 1) + 1);
    const bool more = t < total && !dead;
    Item it = {};
    int head = -1;
    if (more) {
      it = p.p.items[pass][t / p.a.H];
      head = static_cast<int>(t % p.a.H);
    }
    if (lane == 0) {
      s.job[n & 1].item = it;
      s.job[n & 1].head = head;
      mbar_arrive(&s.job_full[n & 1]);
    }
    if (!more) break;
    // the next item's number, known by the time that this one's copies are under way
    int next = 0;
    if (lane == 0) next = atomicAdd(&p.p.counts[2 + pass], 1);
    for (int c = it.c0; c < it.c1; ++c) {
      const int row = it.first + c * kC, hq = head / p.a.group;
#pragma unroll 1
      for (int w = 0; w < kEach; ++w, ++u) {
        const int which = kFull ? w : 2 * w;  // k, q, v
        const uint32_t slot = u % kSlots;
        LIN_WAIT(s.empty[slot], u / kSlots + 1);
        if (static_cast<int>(u) == p.a.stall) { ++left; continue; }
        if (dead) continue;
        if (lane == 0) {
          const CUtensorMap* m = which == 0 ? &p.tk : which == 1 ? &p.tq : &p.tv;
          const int h = which == 2 ? head : hq;
          uint8_t* dst = sm + slot * kTile;
          mbar_arrive_expect_tx(&s.full[slot], kTile);
          tma_load_3d(dst, m, &s.full[slot], 0, h, row);
          tma_load_3d(dst + kPanel, m, &s.full[slot], 64, h, row);
        }
        __syncwarp();
      }
    }
    t = gridDim.x + static_cast<int64_t>(__shfl_sync(0xffffffffu, next, 0));
  }
  // the ring's last copies have landed before the block gives its shared memory back
  if (dead || left) {
    for (uint32_t i = 0; i < kSlots; ++i) { bar_wait(&s.full[i], 0); bar_wait(&s.full[i], 1); }
  } else {
    drain_ring(s.full, kSlots, u);
  }
  if (dead && lane == 0) report_status(p.a.status, 6 /* KDA_ERR_TIMEOUT */);
}

template <bool kFull>
__device__ void mma_warp(const LinParams& p, uint8_t* sm, Small& s, int lane) {
  constexpr int kEach = kFull ? 3 : 2;
  constexpr uint32_t id_kk = idesc_f16(128, 128, true, false, false), id_km = idesc_f16(128, 128, true, false, true),
                     id_mm = idesc_f16(128, 128, true, true, true);
  bool dead = false;
  Jobs jobs(s, dead);
  Job j;
  uint32_t n = 0;
  const uint32_t who = elect_one_sync();
  const uint64_t d_k = smem_desc(smem_u32(sm), 16, 1024, kSwizzle128B);          // K-major tiles
  const uint64_t d_m = smem_desc(smem_u32(sm), kPanel, 1024, kSwizzle128B);      // the same, M- or N-major
  auto at = [](uint32_t slot) { return static_cast<uint64_t>(slot * kTile >> 4); };
  while (jobs.next(j)) {
    for (int c = j.item.c0; c < j.item.c1; ++c, ++n) {
      const uint32_t uk = kEach * n, uq = uk + 1, uv = uk + kEach - 1;
      const uint32_t sk = uk % kSlots, sq = uq % kSlots, sv = uv % kSlots;
      LIN_WAIT(s.full[sk], uk / kSlots);
      if constexpr (kFull) {
        LIN_WAIT(s.full[sq], uq / kSlots);
        if (n > 0) {  // the last chunk's outputs are read: its scores, weights and values are free
          LIN_WAIT(s.out_free, n - 1);
          if (lane == 0) mbar_arrive(&s.empty[(uv - kEach) % kSlots]);
        }
        tc_fence_after();
        if (!dead) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint64_t off = ((kk >> 2) * kPanel + 32 * (kk & 3)) >> 4;
            mma_f16_if(who, kTS, d_k + at(sq) + off, d_k + at(sk) + off, id_kk, kk > 0);
          }
          mma_commit_if(who, &s.scores);
        }
      }
      LIN_WAIT(s.state, n);  // the state in front of the chunk is in shared memory, the last K^T V is read
      tc_fence_after();
      if constexpr (kFull) {
        if (!dead) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_f16_if(who, kTI, d_k + at(sq) + (((kk >> 2) * kPanel + 32 * (kk & 3)) >> 4),
                       d_m + ((kSmState + kk * 2048) >> 4), id_km, kk > 0);
          mma_commit_if(who, &s.empty[sq]);
        }
      }
      LIN_WAIT(s.full[sv], uv / kSlots);
      LIN_WAIT(s.keys, n);
      tc_fence_after();
      if (!dead) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_f16_if(who, kTKV, d_m + at(sk) + ((kk * 2048) >> 4), d_m + at(sv) + ((kk * 2048) >> 4), id_mm, kk > 0);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_f16_if(who, kTKV, d_m + ((kSmLo + kk * 2048) >> 4), d_m + at(sv) + ((kk * 2048) >> 4), id_mm, 1);
        mma_commit_if(who, &s.kv);
        mma_commit_if(who, &s.empty[sk]);
        if constexpr (!kFull) mma_commit_if(who, &s.empty[sv]);
      }
      if constexpr (kFull) {
        LIN_WAIT(s.weights, n);
        tc_fence_after();
        if (!dead) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_f16_ta_if(who, kTO, kTS + 8 * kk, d_m + at(sv) + ((kk * 2048) >> 4), id_km, kk > 0);
          mma_commit_if(who, &s.out);
        }
      }
    }
  }
  // products in flight end before the tensor memory is given back
  mma_commit_if(who, &s.drain);
  bar_wait(&s.drain, 0);
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
      float v[4], f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        G[i] += sum - own;
        v[i] = 4 * lane + i >= nan_at ? none : real(G[i]);
        f[i] = exp2f(real(end - G[i]));
      }
      LIN_WAIT(s.dec_empty[n & 1], (n >> 1) + 1);
      Decays& d = s.dec[n & 1];
      *reinterpret_cast<float4*>(&d.G[4 * lane]) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(&d.cf[4 * lane]) = make_float4(f[0], f[1], f[2], f[3]);
      if ((lane & 7) == 7) d.wb[lane >> 3] = exp2f(real(last - end));
      if (lane == 0) d.a = nan_at < kC ? none : exp2f(real(last));
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.dec_full[n & 1]);
    }
  }
  if (dead && lane == 0) report_status(p.a.status, 6 /* KDA_ERR_TIMEOUT */);
}

// What is not finite in 32 columns of P V, once more from the weights and values of the tokens that a row
// sees.  In place: the caller's registers stay out of memory.
__device__ __noinline__ void seen_only(uint32_t v, uint32_t tl, int row, int block) {
  float x[32], was[32];
#pragma unroll
  for (int e = 0; e < 32; ++e) x[e] = 0.f;
  const uint32_t base = v + (block >> 1) * kPanel;
#pragma unroll 1
  for (int j = 0; j < kC; ++j) {
    uint32_t pair;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\ntcgen05.wait::ld.sync.aligned;\n" : "=r"(pair) : "r"(tl + kTS + (j >> 1)));
    const float w = __uint_as_float(j & 1 ? pair & 0xffff0000u : pair << 16);
    if (j <= row) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4 u = lds128(base + sw128(j, (block & 1) * 64 + 16 * q));
        const uint32_t b[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[8 * q + 2 * e] = fmaf(w, __uint_as_float(b[e] << 16), x[8 * q + 2 * e]);
          x[8 * q + 2 * e + 1] = fmaf(w, __uint_as_float(b[e] & 0xffff0000u), x[8 * q + 2 * e + 1]);
        }
      }
    }
    __syncwarp();
  }
  tmem_ld32(tl + kTO + 32 * block, was);
#pragma unroll
  for (int e = 0; e < 32; ++e) x[e] = fabsf(was[e]) < INFINITY ? was[e] : x[e];
  tmem_st32(tl + kTO + 32 * block, x);
  tmem_wait_st();
}

__device__ void weight_warps(const LinParams& p, uint8_t* sm, Small& s, int w, int lane) {
  const LinArgs& a = p.a;
  bool dead = false;
  Jobs jobs(s, dead);
  Job j;
  uint32_t n = 0;
  const uint32_t tl = static_cast<uint32_t>(w) << 21;
  const int i = 32 * w + lane;
  while (jobs.next(j)) {
    for (int c = j.item.c0; c < j.item.c1; ++c, ++n) {
      // ---- weights, 32 columns at a time, over the scores of columns that are read already
      LIN_WAIT(s.dec_full[n & 1], n >> 1);
      const Decays& d = s.dec[n & 1];
      const float G = d.G[i];
      LIN_WAIT(s.scores, n);
      tc_fence_after();
#pragma unroll 1
      for (int b = 0; b < 4; ++b) {
        float pk[16];
        if (b > w) {
#pragma unroll
          for (int e = 0; e < 16; ++e) pk[e] = 0.f;
        } else {
          float x[32];
          tmem_ld32(tl + kTS + 32 * b, x);
          if (b < w) {
            const float rf = exp2_fast(G - d.G[32 * b + 31]);
            const uint64_t r2 = f32x2(rf, rf);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 f = *reinterpret_cast<const float4*>(&d.cf[32 * b + e]);
              pk[e / 2] = __uint_as_float(bf162_of(mul_f32x2(f32x2(x[e], x[e + 1]), mul_f32x2(r2, f32x2(f.x, f.y)))));
              pk[e / 2 + 1] = __uint_as_float(bf162_of(mul_f32x2(f32x2(x[e + 2], x[e + 3]), mul_f32x2(r2, f32x2(f.z, f.w)))));
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 f = *reinterpret_cast<const float4*>(&d.G[32 * b + e]);
              const float y0 = e <= lane ? x[e] * exp2_fast(G - f.x) : 0.f;
              const float y1 = e + 1 <= lane ? x[e + 1] * exp2_fast(G - f.y) : 0.f;
              const float y2 = e + 2 <= lane ? x[e + 2] * exp2_fast(G - f.z) : 0.f;
              const float y3 = e + 3 <= lane ? x[e + 3] * exp2_fast(G - f.w) : 0.f;
              pk[e / 2] = __uint_as_float(pack_bf162(y0, y1));
              pk[e / 2 + 1] = __uint_as_float(pack_bf162(y2, y3));
            }
          }
        }
        tmem_st16(tl + kTS + 16 * b, pk);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&s.weights);
        mbar_arrive(&s.dec_empty[n & 1]);
      }
      // ---- outputs
      const uint32_t uv = 3 * n + 2, sv = uv % kSlots;
      const bool live = i < live_rows(j.item, c);
      const int64_t t = static_cast<int64_t>(j.item.first) + c * kC + i;
      const float eg = exp2_fast(G);
      LIN_WAIT(s.full[sv], uv / kSlots);  // for the values, should they be needed
      LIN_WAIT(s.out, n);
      tc_fence_after();
      auto block = [&](int b, float (&x)[32]) {  // 32 columns of the row before scale
        float y[32];
        tmem_ld32_async(tl + kTO + 32 * b, x);
        tmem_ld32_async(tl + kTI + 32 * b, y);
        tmem_wait_ld32(x);
        tmem_wait_ld32(y);
        float z = 0.f;
#pragma unroll
        for (int e = 0; e < 32; ++e) z = fmaf(x[e], 0.f, z);
        if (__any_sync(0xffffffffu, live && z != 0.f)) {
          seen_only(smem_u32(sm) + sv * kTile, tl, i, b);
          tmem_ld32(tl + kTO + 32 * b, x);
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = fmaf(eg, y[e], x[e]);
      };
      float f = a.scale;
      if (a.gate) {
        float ss = 0.f;
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {
          float x[32];
          block(b, x);
#pragma unroll
          for (int e = 0; e < 32; ++e) { x[e] *= a.scale; ss = fmaf(x[e], x[e], ss); }
        }
        f *= 1.f / sqrtf(ss * (1.f / kD) + a.eps);
      }
      uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + (t * a.H + j.head) * kD);
      const uint4* gate = a.gate ? reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.gate) + t * a.gate_stride[1] + j.head * a.gate_stride[2]) : nullptr;
#pragma unroll 1
      for (int b = 0; b < 4; ++b) {
        float x[32];
        block(b, x);
        if (b == 3) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.out_free);
        }
        if (live) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = x[8 * q + e] * f;
          if (a.gate) {
            const uint4 u = gate[4 * b + q];
            const uint32_t bits[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              y[2 * e] = __fdividef(y[2 * e], 1.f + __expf(-__uint_as_float(bits[e] << 16)));
              y[2 * e + 1] = __fdividef(y[2 * e + 1], 1.f + __expf(-__uint_as_float(bits[e] & 0xffff0000u)));
            }
            if (a.norm_weight) {
              const float4 w0 = reinterpret_cast<const float4*>(a.norm_weight)[8 * b + 2 * q];
              const float4 w1 = reinterpret_cast<const float4*>(a.norm_weight)[8 * b + 2 * q + 1];
              y[0] *= w0.x; y[1] *= w0.y; y[2] *= w0.z; y[3] *= w0.w; y[4] *= w1.x; y[5] *= w1.y; y[6] *= w1.z; y[7] *= w1.w;
            }
          }
          dst[4 * b + q] = make_uint4(pack_bf162(y[0], y[1]), pack_bf162(y[2], y[3]), pack_bf162(y[4], y[5]), pack_bf162(y[6], y[7]));
        }
        }
        __syncwarp();
      }
    }
  }
  if (dead && lane == 0) report_status(a.status, 6 /* KDA_ERR_TIMEOUT */);
}

// Decayed keys: hi = bf16(w k) in place, lo = bf16(w k - hi) in its own tile.  Rows past the sequence's end are
// cleared, the values' too: what stands there must not meet the state.
template <bool kFull>
__device__ void key_warps(const LinParams& p, uint8_t* sm, Small& s, int tid) {
  constexpr int kEach = kFull ? 3 : 2;
  bool dead = false;
  Jobs jobs(s, dead);
  Job j;
  uint32_t n = 0;
  const int lane = tid & 31;
  while (jobs.next(j)) {
    for (int c = j.item.c0; c < j.item.c1; ++c, ++n) {
      const uint32_t uk = kEach * n, uv = uk + kEach - 1, sk = uk % kSlots, sv = uv % kSlots;
      const int live = live_rows(j.item, c);
      LIN_WAIT(s.dec_full[n & 1], n >> 1);
      LIN_WAIT(s.full[sk], uk / kSlots);
      if constexpr (kFull) LIN_WAIT(s.scores, n);   // Q K^T has read the keys
      if (n > 0) LIN_WAIT(s.kv, n - 1);             // the last K^T V has read the low parts
      if (live < kC) LIN_WAIT(s.full[sv], uv / kSlots);
      const Decays& d = s.dec[n & 1];
      const uint32_t hi = smem_u32(sm) + sk * kTile, lo = smem_u32(sm) + kSmLo, v = smem_u32(sm) + sv * kTile;
      if (!dead) {
#pragma unroll 4
        for (int it = 0; it < 16; ++it) {
          const int row = 8 * it + (tid >> 4), ch = tid & 15;
          const uint32_t at = (ch >> 3) * kPanel + sw128(row, 16 * (ch & 7));
          if (row >= live) {
            sts128(hi + at, make_uint4(0, 0, 0, 0));
            sts128(lo + at, make_uint4(0, 0, 0, 0));
            sts128(v + at, make_uint4(0, 0, 0, 0));
            continue;
          }
          const float w = d.cf[row] * d.wb[row >> 5];
          const uint4 u = lds128(hi + at);
          const uint32_t x[4] = {u.x, u.y, u.z, u.w};
          uint32_t h[4], l[4];
          const uint64_t w2 = f32x2(w, w);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint64_t k2 = f32x2(__uint_as_float(x[e] << 16), __uint_as_float(x[e] & 0xffff0000u));
            h[e] = bf162_of(mul_f32x2(k2, w2));
            l[e] = bf162_of(fma_f32x2(k2, w2, f32x2(-__uint_as_float(h[e] << 16), -__uint_as_float(h[e] & 0xffff0000u))));
          }
          sts128(hi + at, make_uint4(h[0], h[1], h[2], h[3]));
          sts128(lo + at, make_uint4(l[0], l[1], l[2], l[3]));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&s.keys);
        mbar_arrive(&s.dec_empty[n & 1]);
      }
    }
  }
  if (dead && lane == 0) report_status(p.a.status, 6 /* KDA_ERR_TIMEOUT */);
}

template <bool kFull>
__device__ void state_warps(const LinParams& p, uint8_t* sm, Small& s, int w, int lane) {
  const LinArgs& a = p.a;
  bool dead = false;
  Jobs jobs(s, dead);
  Job j;
  uint32_t n = 0;
  const int row = 32 * (w & 3) + lane, half = w >> 2;
  const uint32_t tl = (static_cast<uint32_t>(w & 3) << 21) + kTKV + 64 * half;
  const uint32_t copy = smem_u32(sm) + kSmState + half * kPanel;
  while (jobs.next(j)) {
    const Item& it = j.item;
    const int64_t mine = row * kD + 64 * half;
    auto slot = [&](int k) { return p.p.slots + (static_cast<int64_t>(it.base + k) * a.H + j.head) * kStateFloats + mine; };
    float S[64], A = 1.f;
#pragma unroll
    for (int e = 0; e < 64; ++e) S[e] = 0.f;
    auto load = [&](const float* src) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float4 x = reinterpret_cast<const float4*>(src)[e];
        S[4 * e] = x.x; S[4 * e + 1] = x.y; S[4 * e + 2] = x.z; S[4 * e + 3] = x.w;
      }
    };
    auto store = [&](float* dst) {
#pragma unroll
      for (int e = 0; e < 16; ++e) reinterpret_cast<float4*>(dst)[e] = make_float4(S[4 * e], S[4 * e + 1], S[4 * e + 2], S[4 * e + 3]);
    };
    if (it.seg == 0) {
      if (a.S_in) {
        // the second pass of a split sequence reads the copy: S_out may be S_in
        load(kFull && it.base >= 0 ? slot(0) : a.S_in + (static_cast<int64_t>(it.seq) * a.H + j.head) * kStateFloats + mine);
        if (!kFull) store(slot(0));
      }
    } else if (kFull) {
      load(slot(1));
#pragma unroll 1
      for (int k = 1; k < it.seg; ++k) {
        const float f = p.p.decay[static_cast<int64_t>(it.base + 1 + k) * a.H + j.head];
        const float4* src = reinterpret_cast<const float4*>(slot(1 + k));
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float4 x = src[e];
          S[4 * e] = fmaf(f, S[4 * e], x.x); S[4 * e + 1] = fmaf(f, S[4 * e + 1], x.y);
          S[4 * e + 2] = fmaf(f, S[4 * e + 2], x.z); S[4 * e + 3] = fmaf(f, S[4 * e + 3], x.w);
        }
      }
    }
    for (int c = it.c0; c < it.c1; ++c, ++n) {
      if constexpr (kFull) {  // rounded to bf16 for Q S
#pragma unroll
        for (int e = 0; e < 8; ++e)
          sts128(copy + sw128(row, 16 * e), make_uint4(pack_bf162(S[8 * e], S[8 * e + 1]), pack_bf162(S[8 * e + 2], S[8 * e + 3]),
                                                       pack_bf162(S[8 * e + 4], S[8 * e + 5]), pack_bf162(S[8 * e + 6], S[8 * e + 7])));
        fence_proxy_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.state);
      LIN_WAIT(s.dec_full[n & 1], n >> 1);
      const float f = s.dec[n & 1].a;
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.dec_empty[n & 1]);
      A *= f;
      LIN_WAIT(s.kv, n);
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float x[16];
        tmem_ld16(tl + 16 * q, x);
#pragma unroll
        for (int e = 0; e < 16; ++e) S[16 * q + e] = fmaf(f, S[16 * q + e], x[e]);
      }
    }
    if constexpr (kFull) {
      if (it.last && a.S_out && !dead) store(a.S_out + (static_cast<int64_t>(it.seq) * a.H + j.head) * kStateFloats + mine);
    } else {
      store(slot(1 + it.seg));
      if (w == 0 && lane == 0) p.p.decay[static_cast<int64_t>(it.base + 1 + it.seg) * a.H + j.head] = A;
    }
  }
  tc_fence_before();
  if (dead && lane == 0) report_status(a.status, 6 /* KDA_ERR_TIMEOUT */);
}

template <bool kFull>
__global__ void __launch_bounds__(kThreads, 1) lin_chunk_kernel(const __grid_constant__ LinParams p) {
  extern __shared__ __align__(1024) uint8_t sm[];
  Small& s = *reinterpret_cast<Small*>(sm + kSmSmall);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(sm) & 1023) {  // the swizzled tiles need it
    if (tid == 0) report_status(p.a.status, 5 /* KDA_ERR_CUDA */);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) { mbar_init(&s.full[i], 1); mbar_init(&s.empty[i], 1); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.job_full[i], 1);
      mbar_init(&s.job_empty[i], kFull ? kReaders : kReaders - 4);
      mbar_init(&s.dec_full[i], 1);
      mbar_init(&s.dec_empty[i], kFull ? 16 : 12);
    }
    mbar_init(&s.scores, 1); mbar_init(&s.weights, 4); mbar_init(&s.keys, 4); mbar_init(&s.kv, 1);
    mbar_init(&s.state, 8); mbar_init(&s.out, 1); mbar_init(&s.out_free, 4); mbar_init(&s.drain, 1);
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
  // registers: 96 a thread at launch, 480 over the five groups
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;\n" ::: "memory");
    if (warp == 0) load_warp<kFull>(p, sm, s, lane);
    else if (warp == 1) mma_warp<kFull>(p, sm, s, lane);
    else if (warp == 2) decay_warp<kFull>(p, s, lane);
  } else if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 112;\n" ::: "memory");
    if constexpr (kFull) weight_warps(p, sm, s, warp - 4, lane);
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;\n" ::: "memory");
    key_warps<kFull>(p, sm, s, tid - 256);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 120;\n" ::: "memory");
    state_warps<kFull>(p, sm, s, warp - 12, lane);
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

// Rows [tokens][heads][128] of bf16 in boxes of 128 tokens and 64 channels.
bool rows_map(CUtensorMap* m, const void* base, const int64_t* stride, int heads, int64_t tokens) {
  const auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {kD, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(stride[2]) * 2, static_cast<cuuint64_t>(stride[1]) * 2};
  const cuuint32_t box[3] = {64, 1, kC}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kFull>
cudaError_t launch_chunks(const LinParams& p, int64_t items, int num_sms) {
  static SmemOptIn opt_in;
  const auto kernel = lin_chunk_kernel<kFull>;
  cudaError_t e = opt_in(reinterpret_cast<const void*>(kernel), kSmBytes);
  if (e != cudaSuccess) return e;
  // setmaxnreg's shares add up to kRegs a thread: with fewer at launch the groups would wait for them forever
  static const int regs = [] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, lin_chunk_kernel<kFull>) == cudaSuccess ? at.numRegs : 0;
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
  plan_layout(&p.p, a.workspace, a.n_seq, a.tokens, a.H, a.n_segments, num_sms);
  if (a.tokens > 0 && (!rows_map(&p.tq, a.q, a.q_stride, a.H / a.group, a.tokens) || !rows_map(&p.tk, a.k, a.k_stride, a.H / a.group, a.tokens) ||
                       !rows_map(&p.tv, a.v, a.v_stride, a.H, a.tokens)))
    return cudaErrorInvalidValue;
  cudaError_t e = launch_after(lin_plan_kernel, dim3(1), dim3(1024), 0, a.stream, a.cu, a.n_seq, a.tokens, a.H, num_sms,
                               a.n_segments, p.p, a.status);
  if (e != cudaSuccess) return e;
  // the first pass only where the rule can split: one sequence of all the tokens is cut most
  if (p.p.most[1] > 0 && segments_of(a.tokens, a.tokens, a.H, num_sms, a.n_segments) > 1) {
    e = launch_chunks<false>(p, p.p.most[1] * a.H, num_sms);
    if (e != cudaSuccess) return e;
  }
  return launch_chunks<true>(p, p.p.most[0] * a.H, num_sms);
}

}  // namespace kda
