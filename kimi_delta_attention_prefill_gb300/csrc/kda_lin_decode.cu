// kda_lin_decode.cu -- a decode or verify step of linear attention with a decay a head.
//
// With G_i the sum of the step's decays g_0 .. g_i, the recurrence over n <= 4 tokens unrolls to
//     o_i = scale (e^{G_i} S^T q_i + sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j)
//     S  <- e^{G_m} S + sum_{j < m} e^{G_m - G_j} k_j v_j^T        (m accepted tokens)
// so every output needs the old state only, and the state is read once and written once: the step is
// bound by those 128 KiB a (sequence, head).  One pass over the state's rows takes S^T q of all tokens from what
// comes in and sends the new rows out at once; the rest of the outputs follows while they are on their way.
//
// Work split: 256 threads a (sequence, head), warp w owns columns [16 w, 16 w + 16), lane 4 r + c the columns
// 16 w + 4 c .. + 3 of rows r, r + 8, ..: eight loads of 16 bytes a thread in flight, three blocks an SM.
// Measured (of copy bandwidth): 256 sequences x 96 heads, one token 459 us (104 %); 61 x 64, four tokens with the output
// stage 79 us (89 %).  With the whole state in registers and two blocks an SM the latter took 94 us, and
// 82 with this pass and two blocks.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "kda_lin.h"
#include "kda_ptx.cuh"

namespace kda {
namespace {

constexpr int kD = kHeadDim;
constexpr int kThreads = 256;
constexpr int kRows = 16;  // of the state, a thread

// row i of the state at (i mod 8) x 16 + i / 8: a thread's 16 rows are 16 consecutive floats
__device__ constexpr int at_row(int i) { return (i & 7) * 16 + (i >> 3); }

template <int kTok>
__global__ void __launch_bounds__(kThreads, 3) lin_decode_kernel(const __grid_constant__ LinArgs a, int lookahead) {
  constexpr int kP = kTok == 3 ? 4 : kTok;  // tokens whose sums are spread over the lanes
  __shared__ __align__(16) float sq[kTok][kD], sk[kTok][kD];  // by at_row
  __shared__ __align__(16) float sv[kTok][kD], so[kTok][kD];
  __shared__ float sE[kP];             // e^{g up to token i}
  __shared__ float sqk[kP][kTok];      // q_i . k_j times the decay between them
  const int unit = blockIdx.x, b = unit / a.H, h = unit - b * a.H, hq = h / a.group;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r0 = lane >> 2, col = warp * 16 + (lane & 3) * 4;
  float4* S = reinterpret_cast<float4*>(a.S_out + unit * kStateFloats) + ((r0 * kD + col) >> 2);
  float4 s[8];  // rows r0 + 8 m on their way, eight at a time
#pragma unroll
  for (int m = 0; m < 8; ++m) s[m] = S[m * 2 * kD];
  // the state and the rows of the unit that starts about a third of the resident blocks later, into L2 (a hint;
  // from a third of a wave to one and a half they measured alike)
  if (warp == 1 && unit + lookahead < static_cast<int>(gridDim.x)) {
    const int next = unit + lookahead, nb = next / a.H, nh = next - nb * a.H, nq = nh / a.group;
    if (lane == 0) bulk_prefetch_l2(a.S_out + next * kStateFloats, kStateFloats * sizeof(float));
    const int i = lane >> 3, which = (lane >> 1) & 3;  // token; q, k, v, gate, two lines each
    if (i < kTok && (which < 3 || a.gate)) {
      const void* base = which == 0 ? a.q : which == 1 ? a.k : which == 2 ? a.v : a.gate;
      const int64_t* st = which == 0 ? a.q_stride : which == 1 ? a.k_stride : which == 2 ? a.v_stride : a.gate_stride;
      prefetch_l2(static_cast<const __nv_bfloat16*>(base) + nb * st[0] + i * st[1] + (which < 2 ? nq : nh) * st[2] + 64 * (lane & 1));
    }
  }
  int nc = a.n_commit ? a.n_commit[b] : kTok;
  if (nc < 0 || nc > kTok) {
    if (tid == 0) report_status(a.status, 7 /* KDA_ERR_DEVICE_CHECK */);
    nc = 0;  // the state stays; outputs are made all the same
  }
  float G[kTok];
#pragma unroll
  for (int i = 0; i < kTok; ++i) G[i] = a.g[b * a.g_stride[0] + i * a.g_stride[1] + h * a.g_stride[2]];
  {
    const int c = tid & (kD - 1);
    const auto* q = static_cast<const __nv_bfloat16*>(a.q) + b * a.q_stride[0] + hq * a.q_stride[2] + c;
    const auto* k = static_cast<const __nv_bfloat16*>(a.k) + b * a.k_stride[0] + hq * a.k_stride[2] + c;
    const auto* v = static_cast<const __nv_bfloat16*>(a.v) + b * a.v_stride[0] + h * a.v_stride[2] + c;
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      if (tid < kD) {
        sq[i][at_row(c)] = __bfloat162float(q[i * a.q_stride[1]]);
        sv[i][c] = __bfloat162float(v[i * a.v_stride[1]]);
      } else {
        sk[i][at_row(c)] = __bfloat162float(k[i * a.k_stride[1]]);
      }
    }
  }
  // e^{g_{j+1} + .. + g_{i}}: a sum from its own first term, so that -inf before it does not touch it
  auto decay = [&](int j, int i) {
    float sum = 0.f;
#pragma unroll
    for (int t = 0; t < kTok; ++t)
      if (t > j && t <= i) sum += G[t];
    return expf(sum);
  };
  if (tid < kTok) sE[tid] = decay(-1, tid);
  __syncthreads();
  for (int p = warp; p < kTok * kTok; p += kThreads / 32) {
    const int i = p / kTok, j = p - i * kTok;
    if (j > i) continue;
    const float4 x = *reinterpret_cast<const float4*>(&sq[i][4 * lane]), y = *reinterpret_cast<const float4*>(&sk[j][4 * lane]);
    float d = x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
#pragma unroll
    for (int off = 16; off; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
    if (lane == 0) sqk[i][j] = d * decay(j, i);
  }
  // the state after nc tokens: e times the one before, and each token's values times f = its decay up to there
  const float e = decay(-1, nc - 1);
  const uint64_t e2 = f32x2(e, e);
  uint64_t x[kTok][2];
#pragma unroll
  for (int j = 0; j < kTok; ++j) {
    const float4 u = *reinterpret_cast<const float4*>(&sv[j][col]);
    const float f = decay(j, nc - 1);
    x[j][0] = f32x2(u.x * f, u.y * f);
    x[j][1] = f32x2(u.z * f, u.w * f);
  }
  // one pass over the state's rows: S^T q of what comes in, the new rows on their way out at once
  uint64_t p2[kTok][2];
#pragma unroll
  for (int i = 0; i < kTok; ++i) p2[i][0] = p2[i][1] = f32x2(0.f, 0.f);
#pragma unroll
  for (int m = 0; m < kRows; m += 4) {
    uint64_t y[4][2];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const float4 u = s[(m & 7) + t];
      y[t][0] = f32x2(u.x, u.y);
      y[t][1] = f32x2(u.z, u.w);
    }
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      const float4 q4 = *reinterpret_cast<const float4*>(&sq[i][r0 * 16 + m]);
      const float qv[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint64_t q2 = f32x2(qv[t], qv[t]);
        p2[i][0] = fma_f32x2(q2, y[t][0], p2[i][0]);
        p2[i][1] = fma_f32x2(q2, y[t][1], p2[i][1]);
      }
    }
    if (nc > 0) {
#pragma unroll
      for (int t = 0; t < 4; ++t) { y[t][0] = mul_f32x2(y[t][0], e2); y[t][1] = mul_f32x2(y[t][1], e2); }
#pragma unroll
      for (int j = 0; j < kTok; ++j) {
        if (j >= nc) break;  // a later token's values, whatever they are, do not meet the state
        const float4 k4 = *reinterpret_cast<const float4*>(&sk[j][r0 * 16 + m]);
        const float kv[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint64_t k2 = f32x2(kv[t], kv[t]);
          y[t][0] = fma_f32x2(k2, x[j][0], y[t][0]);
          y[t][1] = fma_f32x2(k2, x[j][1], y[t][1]);
        }
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float2 lo = unpack_f32x2(y[t][0]), hi = unpack_f32x2(y[t][1]);
        __stcs(&S[(m + t) * 2 * kD], make_float4(lo.x, lo.y, hi.x, hi.y));
      }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
      if (m < kRows - 8) s[(m & 7) + t] = S[(m + 8 + t) * 2 * kD];
  }
  // the output stage's gate of token `warp`
  uint2 gb = make_uint2(0, 0);
  float4 w4 = make_float4(1.f, 1.f, 1.f, 1.f);
  if (a.gate && warp < kTok) {
    gb = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.gate) + b * a.gate_stride[0] + warp * a.gate_stride[1] +
                                         h * a.gate_stride[2] + 4 * lane);
    if (a.norm_weight) w4 = *reinterpret_cast<const float4*>(a.norm_weight + 4 * lane);
  }
  // sums over the eight lanes of a column, halving what a lane keeps: value i * 4 + c is column col + c of token i
  float p[kP * 4];
#pragma unroll
  for (int i = 0; i < kP; ++i) {
    const float2 lo = i < kTok ? unpack_f32x2(p2[i % kTok][0]) : make_float2(0.f, 0.f), hi = i < kTok ? unpack_f32x2(p2[i % kTok][1]) : make_float2(0.f, 0.f);
    p[4 * i] = lo.x; p[4 * i + 1] = lo.y; p[4 * i + 2] = hi.x; p[4 * i + 3] = hi.y;
  }
  int first = 0;
  constexpr int kKept = kP == 4 ? 2 : 1;
#pragma unroll
  for (int off = 16, n = kP * 4; off >= 4; off >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool up = lane & off;
#pragma unroll
      for (int t = 0; t < kP * 2; ++t)
        if (t < n) {
          const float other = __shfl_xor_sync(0xffffffffu, up ? p[t] : p[t + n], off);
          p[t] = (up ? p[t + n] : p[t]) + other;
        }
      if (up) first += n;
    } else {
      p[0] += __shfl_xor_sync(0xffffffffu, p[0], off);
    }
  }
  __syncthreads();  // the products of q and k
  const int tok = first >> 2, c0 = col + (first & 3);
  if (tok < kTok && (kP > 1 || r0 % 2 == 0)) {
    const float E = sE[tok];
    float y[kKept];
#pragma unroll
    for (int t = 0; t < kKept; ++t) y[t] = p[t] * E;
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      if (j > tok) break;
      const float f = sqk[tok][j];
#pragma unroll
      for (int t = 0; t < kKept; ++t) y[t] = fmaf(f, sv[j][c0 + t], y[t]);
    }
    float* dst = a.gate ? &so[tok][c0] : static_cast<float*>(a.o) + ((static_cast<int64_t>(b) * kTok + tok) * a.H + h) * kD + c0;
#pragma unroll
    for (int t = 0; t < kKept; ++t) dst[t] = y[t] * a.scale;
  }
  if (a.gate) {  // output stage: warp i normalises and gates token i's row
    __syncthreads();
    if (warp < kTok) {
      const float4 x = *reinterpret_cast<const float4*>(&so[warp][4 * lane]);
      float ss = x.x * x.x + x.y * x.y + x.z * x.z + x.w * x.w;
#pragma unroll
      for (int off = 16; off; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      const float inv = 1.f / sqrtf(ss * (1.f / kD) + a.eps);
      const float2 g01 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&gb.x));
      const float2 g23 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&gb.y));
      float4 y;
      y.x = x.x * inv * w4.x / (1.f + expf(-g01.x)); y.y = x.y * inv * w4.y / (1.f + expf(-g01.y));
      y.z = x.z * inv * w4.z / (1.f + expf(-g23.x)); y.w = x.w * inv * w4.w / (1.f + expf(-g23.y));
      *reinterpret_cast<float4*>(static_cast<float*>(a.o) + ((static_cast<int64_t>(b) * kTok + warp) * a.H + h) * kD + 4 * lane) = y;
    }
  }
}

}  // namespace

cudaError_t launch_lin_decode(const LinArgs& a) {
  int sms = 0;
  current_device_status(&sms);
  const dim3 grid(static_cast<unsigned>(a.n_seq) * static_cast<unsigned>(a.H));
  switch (a.n_tok) {
    case 1: lin_decode_kernel<1><<<grid, kThreads, 0, a.stream>>>(a, sms); break;
    case 2: lin_decode_kernel<2><<<grid, kThreads, 0, a.stream>>>(a, sms); break;
    case 3: lin_decode_kernel<3><<<grid, kThreads, 0, a.stream>>>(a, sms); break;
    default: lin_decode_kernel<4><<<grid, kThreads, 0, a.stream>>>(a, sms); break;
  }
  return cudaGetLastError();
}

}  // namespace kda
