// kda_lin_decode.cu -- a decode or verify step of linear attention with a decay a head.
//
// With G_i the sum of the step's decays g_0 .. g_i, the recurrence over n <= 4 tokens unrolls to
//     o_i = scale (e^{G_i} S^T q_i + sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j)
//     S  <- e^{G_m} S + sum_{j < m} e^{G_m - G_j} k_j v_j^T        (m accepted tokens)
// so every output needs the old state only, and the state is read once and written once: the
// step is bound by those 128 KiB a (sequence, head).  The dot products of all tokens run
// side by side over the state in registers instead of one token after the other.
//
// Work split as the delta rule's step (kda_decode.cu): 256 threads a (sequence, head), warp w owns
// columns [16 w, 16 w + 16), lane 4 r + c the columns 16 w + 4 c .. + 3 of rows r, r + 8, ..: 16 loads of
// 16 bytes a thread in flight, sums over rows by three shuffles.
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
__global__ void __launch_bounds__(kThreads, 2) lin_decode_kernel(const __grid_constant__ LinArgs a, int lookahead) {
  __shared__ __align__(16) float sq[kTok][kD], sk[kTok][kD];  // by at_row
  __shared__ __align__(16) float sv[kTok][kD], so[kTok][kD];
  __shared__ float sqk[kTok][kTok];  // q_i . k_j
  const int unit = blockIdx.x, b = unit / a.H, h = unit - b * a.H, hq = h / a.group;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r0 = lane >> 2, col = warp * 16 + (lane & 3) * 4;
  float4* S = reinterpret_cast<float4*>(a.S_out + unit * kStateFloats);
  float4 s[kRows];
#pragma unroll
  for (int m = 0; m < kRows; ++m) s[m] = S[((r0 + 8 * m) * kD + col) >> 2];
  // the state and the rows of the unit that starts about half the resident blocks later, into L2 (a hint)
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
  // the output stage's gate of token `warp`, for the end
  uint2 gb = make_uint2(0, 0);
  float4 w4 = make_float4(1.f, 1.f, 1.f, 1.f);
  if (a.gate && warp < kTok) {
    gb = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.gate) + b * a.gate_stride[0] + warp * a.gate_stride[1] +
                                         h * a.gate_stride[2] + 4 * lane);
    if (a.norm_weight) w4 = *reinterpret_cast<const float4*>(a.norm_weight + 4 * lane);
  }
  int nc = a.n_commit ? a.n_commit[b] : kTok;
  if (nc < 0 || nc > kTok) {
    if (tid == 0) report_status(a.status, 7 /* KDA_ERR_DEVICE_CHECK */);
    nc = 0;  // the state stays; outputs are made all the same
  }
  // decays up to each token, in every thread
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
  __syncthreads();
  for (int p = warp; p < kTok * kTok; p += kThreads / 32) {
    const int i = p / kTok, j = p - i * kTok;
    if (j > i) continue;
    const float4 x = *reinterpret_cast<const float4*>(&sq[i][4 * lane]), y = *reinterpret_cast<const float4*>(&sk[j][4 * lane]);
    float d = x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
#pragma unroll
    for (int off = 16; off; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
    if (lane == 0) sqk[i][j] = d;
  }
  // w[j][i] = e^{g_{j+1} + .. + g_i}: a sum from its own first term, so that -inf before it does not touch it
  float w[kTok][kTok], E[kTok];
#pragma unroll
  for (int j = 0; j < kTok; ++j) {
    float sum = 0.f;
    w[j][j] = 1.f;
#pragma unroll
    for (int i = j + 1; i < kTok; ++i) {
      sum += G[i];
      w[j][i] = expf(sum);
    }
  }
  {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      sum += G[i];
      E[i] = expf(sum);
    }
  }

  uint64_t s2[kRows][2];
#pragma unroll
  for (int m = 0; m < kRows; ++m) {
    s2[m][0] = f32x2(s[m].x, s[m].y);
    s2[m][1] = f32x2(s[m].z, s[m].w);
  }
  float p[kTok][4];  // S^T q
#pragma unroll
  for (int i = 0; i < kTok; ++i) {
    uint64_t p01 = f32x2(0.f, 0.f), p23 = p01;
#pragma unroll
    for (int m = 0; m < kRows; m += 4) {
      const float4 q4 = *reinterpret_cast<const float4*>(&sq[i][r0 * 16 + m]);
      const float qv[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint64_t q2 = f32x2(qv[e], qv[e]);
        p01 = fma_f32x2(q2, s2[m + e][0], p01);
        p23 = fma_f32x2(q2, s2[m + e][1], p23);
      }
    }
    const float2 lo = unpack_f32x2(p01), hi = unpack_f32x2(p23);
    p[i][0] = lo.x; p[i][1] = lo.y; p[i][2] = hi.x; p[i][3] = hi.y;
  }
#pragma unroll
  for (int off = 4; off < 32; off <<= 1)
#pragma unroll
    for (int i = 0; i < kTok; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) p[i][e] += __shfl_xor_sync(0xffffffffu, p[i][e], off);
  __syncthreads();  // the products of q and k
  if (r0 == 0) {
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) p[i][e] *= E[i];
#pragma unroll
      for (int j = 0; j <= i; ++j) {
        const float f = w[j][i] * sqk[i][j];
        const float4 x = *reinterpret_cast<const float4*>(&sv[j][col]);
        p[i][0] = fmaf(f, x.x, p[i][0]); p[i][1] = fmaf(f, x.y, p[i][1]); p[i][2] = fmaf(f, x.z, p[i][2]); p[i][3] = fmaf(f, x.w, p[i][3]);
      }
      const float4 o4 = make_float4(p[i][0] * a.scale, p[i][1] * a.scale, p[i][2] * a.scale, p[i][3] * a.scale);
      if (a.gate) *reinterpret_cast<float4*>(&so[i][col]) = o4;
      else *reinterpret_cast<float4*>(static_cast<float*>(a.o) + ((static_cast<int64_t>(b) * kTok + i) * a.H + h) * kD + col) = o4;
    }
  }
  if (nc > 0) {
    float f[kTok], e = 0.f;  // of each token in the state after nc of them
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      f[i] = 0.f;
      if (i == nc - 1) e = E[i];
#pragma unroll
      for (int t = i; t < kTok; ++t)
        if (t == nc - 1) f[i] = w[i][t];
    }
    const uint64_t e2 = f32x2(e, e);
#pragma unroll
    for (int m = 0; m < kRows; ++m) { s2[m][0] = mul_f32x2(s2[m][0], e2); s2[m][1] = mul_f32x2(s2[m][1], e2); }
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      if (j >= nc) break;  // a later token's values, whatever they are, do not meet the state
      const float4 x = *reinterpret_cast<const float4*>(&sv[j][col]);
      const uint64_t x01 = f32x2(x.x * f[j], x.y * f[j]), x23 = f32x2(x.z * f[j], x.w * f[j]);
#pragma unroll
      for (int m = 0; m < kRows; m += 4) {
        const float4 k4 = *reinterpret_cast<const float4*>(&sk[j][r0 * 16 + m]);
        const float kv[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint64_t k2 = f32x2(kv[t], kv[t]);
          s2[m + t][0] = fma_f32x2(k2, x01, s2[m + t][0]);
          s2[m + t][1] = fma_f32x2(k2, x23, s2[m + t][1]);
        }
      }
    }
#pragma unroll
    for (int m = 0; m < kRows; ++m) {
      const float2 lo = unpack_f32x2(s2[m][0]), hi = unpack_f32x2(s2[m][1]);
      __stcs(&S[((r0 + 8 * m) * kD + col) >> 2], make_float4(lo.x, lo.y, hi.x, hi.y));
    }
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
