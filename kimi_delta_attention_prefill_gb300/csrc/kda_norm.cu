// kda_norm.cu -- the step between two blocks: the norm after one, its gate and residual scale, the
// residual sum, and the norm before the next, in one pass over the rows.
//     x' = x + scale sigmoid(gate) w_post N(y),   h = w x' / sqrt(mean(x'^2) + eps)
// Bound by memory: 10 bytes an element with all parts in bf16.  A block keeps a row in registers
// (kVec groups of 8 elements a thread) and the weights of its columns too, over all rows that it takes.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "kda_lin.h"
#include "kda_ptx.cuh"

namespace kda {
namespace {

__device__ __forceinline__ void widen(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 narrow(const float (&f)[8]) {
  return make_uint4(pack_bf162(f[0], f[1]), pack_bf162(f[2], f[3]), pack_bf162(f[4], f[5]), pack_bf162(f[6], f[7]));
}

// The sum over the block's threads, in all of them.  `part`: 32 floats that the last call but one may
// still be reading no more (the callers take two in turn).
__device__ __forceinline__ float block_sum(float x, float* part) {
#pragma unroll
  for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return x;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  x = (threadIdx.x & 31) < warps ? part[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

template <int kVec, bool kF32>
__global__ void __launch_bounds__(1024) norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float part[2][2][32];
  const int tid = threadIdx.x, n = a.width >> 3;
  const float inv_w = 1.f / static_cast<float>(a.width);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    float x[kVec][8];
    uint4 yb[kVec], gb[kVec];
    const char* xr = static_cast<const char*>(a.x) + row * a.x_stride * (kF32 ? 4 : 2);
    const char* yr = static_cast<const char*>(a.y) + row * a.y_stride * 2;
    const char* gr = static_cast<const char*>(a.gate) + row * a.gate_stride * 2;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int c = tid + i * blockDim.x;
      if (c < n) {
        if (a.y) yb[i] = *reinterpret_cast<const uint4*>(yr + 16 * static_cast<int64_t>(c));
        if (a.gate) gb[i] = *reinterpret_cast<const uint4*>(gr + 16 * static_cast<int64_t>(c));
        if constexpr (kF32) {
          const float4 u = reinterpret_cast<const float4*>(xr)[2 * c], v = reinterpret_cast<const float4*>(xr)[2 * c + 1];
          x[i][0] = u.x; x[i][1] = u.y; x[i][2] = u.z; x[i][3] = u.w; x[i][4] = v.x; x[i][5] = v.y; x[i][6] = v.z; x[i][7] = v.w;
        } else {
          widen(*reinterpret_cast<const uint4*>(xr + 16 * static_cast<int64_t>(c)), x[i]);
        }
      }
    }
    if (a.y) {
      float f = a.scale;
      if (a.post_norm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          if (tid + i * blockDim.x < n) {
            float y[8];
            widen(yb[i], y);
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
          }
        }
        f *= 1.f / sqrtf(block_sum(ss, part[turn][0]) * inv_w + a.eps);
      }
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int c = tid + i * blockDim.x;
        if (c >= n) continue;
        float y[8];
        widen(yb[i], y);
        if (a.post_weight) {
          const float4 u = reinterpret_cast<const float4*>(a.post_weight)[2 * c], v = reinterpret_cast<const float4*>(a.post_weight)[2 * c + 1];
          y[0] *= u.x; y[1] *= u.y; y[2] *= u.z; y[3] *= u.w; y[4] *= v.x; y[5] *= v.y; y[6] *= v.z; y[7] *= v.w;
        }
        if (a.gate) {
          float g[8];
          widen(gb[i], g);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = __fdividef(y[e], 1.f + __expf(-g[e]));
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = fmaf(f, y[e], x[i][e]);
        if (a.x_out) {
          char* xo = static_cast<char*>(a.x_out) + row * a.width * (kF32 ? 4 : 2);
          if constexpr (kF32) {
            reinterpret_cast<float4*>(xo)[2 * c] = make_float4(x[i][0], x[i][1], x[i][2], x[i][3]);
            reinterpret_cast<float4*>(xo)[2 * c + 1] = make_float4(x[i][4], x[i][5], x[i][6], x[i][7]);
          } else {
            reinterpret_cast<uint4*>(xo)[c] = narrow(x[i]);
          }
        }
      }
    }
    if (!a.h) continue;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      if (tid + i * blockDim.x < n) {
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[i][e], x[i][e], ss);
      }
    }
    const float f = 1.f / sqrtf(block_sum(ss, part[turn][1]) * inv_w + a.eps);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int c = tid + i * blockDim.x;
      if (c >= n) continue;
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = x[i][e] * f;
      if (a.weight) {
        const float4 u = reinterpret_cast<const float4*>(a.weight)[2 * c], v = reinterpret_cast<const float4*>(a.weight)[2 * c + 1];
        y[0] *= u.x; y[1] *= u.y; y[2] *= u.z; y[3] *= u.w; y[4] *= v.x; y[5] *= v.y; y[6] *= v.z; y[7] *= v.w;
      }
      reinterpret_cast<uint4*>(static_cast<char*>(a.h) + row * a.width * 2)[c] = narrow(y);
    }
  }
}

template <int kVec>
void launch(const NormArgs& a, int num_sms) {
  const int threads = (((a.width >> 3) + kVec - 1) / kVec + 31) & ~31;
  const int64_t most = static_cast<int64_t>(num_sms) * (2048 / threads > 32 ? 32 : 2048 / threads);
  const unsigned grid = static_cast<unsigned>(a.rows < most ? a.rows : most);
  if (a.x_f32) norm_kernel<kVec, true><<<grid, threads, 0, a.stream>>>(a);
  else norm_kernel<kVec, false><<<grid, threads, 0, a.stream>>>(a);
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs& a, int num_sms) {
  const int n = a.width >> 3;
  if (n <= 1024) launch<1>(a, num_sms);
  else if (n <= 2048) launch<2>(a, num_sms);
  else launch<4>(a, num_sms);
  return cudaGetLastError();
}

}  // namespace kda
