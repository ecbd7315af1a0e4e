// kda_norm.cu -- the step between two blocks: the norm after one, its gate and residual scale, the
// residual sum, and the norm before the next, in one pass over the rows.
//     x' = x + scale sigmoid(gate) w_post N(y),   h = w x' / sqrt(mean(x'^2) + eps)
// Bound by memory: 10 bytes an element with all parts in bf16.  Few rows: a row a block, in registers (kVec groups
// of 8 elements a thread).  Many: blocks walk over rows with the next ones' loads under way (norm_rows_kernel).
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "kda_attn.h"
#include "kda_attn_device.cuh"
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

constexpr int kStages = 3;
constexpr int kMaxSmem = 227 * 1024 - 1024;

// Eight floats at once where the address allows it: whole sectors, neighbours in neighbouring lanes.
__device__ __forceinline__ void store_f32x8(float* dst, const float (&x)[8], bool whole) {
  if (whole) {
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]),
                 "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
  } else {
    reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// Many rows: a block walks over rows with the loads of the next two under way.  A warp copies what it
// will read itself to its own places in shared memory (cp.async), so that nothing waits for other
// warps, and a thread keeps the weights of its columns in registers.
template <int kVec, bool kF32>
__global__ void __maxnreg__(kVec == 1 ? 64 : kVec == 2 ? 80 : kVec == 3 ? 112 : 128) norm_rows_kernel(const __grid_constant__ NormArgs a) {
  extern __shared__ __align__(16) uint8_t sm[];
  __shared__ float part[2][2][32];
  const int tid = threadIdx.x, n = a.width >> 3, T = blockDim.x;
  const float inv_w = 1.f / static_cast<float>(a.width);
  constexpr int kX = kF32 ? 2 : 1;
  const int parts = kX + (a.y ? 1 : 0) + (a.gate ? 1 : 0);  // 16 bytes each
  const bool whole = (reinterpret_cast<uintptr_t>(a.x_out) & 31) == 0;
  // x, then y and the gate, each of a stage and group in one piece
  auto place = [&](int stage, int i, int k) { return smem_u32(sm) + 16 * T * ((stage * kVec + i) * parts + k); };
  float w[kVec][8], pw[kVec][8];
#pragma unroll
  for (int i = 0; i < kVec; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = 8 * (tid + i * T) + e;
      w[i][e] = a.weight && c < a.width ? a.weight[c] : 1.f;
      pw[i][e] = a.scale * (a.post_weight && c < a.width ? a.post_weight[c] : 1.f);
    }
  auto load = [&](int64_t row, int stage) {
    if (row < a.rows) {
      const char* xr = static_cast<const char*>(a.x) + row * a.x_stride * (kF32 ? 4 : 2);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int c = tid + i * T;
        if (c >= n) continue;
        if (a.y) cp_async16(place(stage, i, kX) + 16 * tid, static_cast<const char*>(a.y) + row * a.y_stride * 2 + 16 * static_cast<int64_t>(c), true);
        if (a.gate) cp_async16(place(stage, i, kX + 1) + 16 * tid, static_cast<const char*>(a.gate) + row * a.gate_stride * 2 + 16 * static_cast<int64_t>(c), true);
        if constexpr (!kF32) cp_async16(place(stage, i, 0) + 16 * tid, xr + 16 * static_cast<int64_t>(c), true);
      }
    }
    if constexpr (kF32) {  // a warp's 1024 bytes by 512: a lane's own 32 would be half of each sector twice
      if (row < a.rows) {
        const char* xr = static_cast<const char*>(a.x) + row * a.x_stride * 4;
        const int first = 2 * (tid & ~31) + (tid & 31);
#pragma unroll
        for (int i = 0; i < kVec; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int at = first + 32 * k;
            if (2 * i * T + at < 2 * n) cp_async16(place(stage, i, 0) + 16 * at, xr + 16 * (static_cast<int64_t>(2 * i * T) + at), true);
          }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int64_t row = blockIdx.x;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) load(row + static_cast<int64_t>(s) * gridDim.x, s);
  int stage = 0, turn = 0;
#pragma unroll 1
  for (; row < a.rows; row += gridDim.x, turn ^= 1) {
    load(row + static_cast<int64_t>(kStages - 1) * gridDim.x, stage == 0 ? kStages - 1 : stage - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    if constexpr (kF32) __syncwarp();
    float x[kVec][8];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      if (tid + i * T >= n) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = 0.f;
        continue;
      }
      const uint4 u = lds128(place(stage, i, 0) + 16 * kX * tid);
      if constexpr (kF32) {
        const uint4 v = lds128(place(stage, i, 0) + 32 * tid + 16);
        x[i][0] = __uint_as_float(u.x); x[i][1] = __uint_as_float(u.y); x[i][2] = __uint_as_float(u.z); x[i][3] = __uint_as_float(u.w);
        x[i][4] = __uint_as_float(v.x); x[i][5] = __uint_as_float(v.y); x[i][6] = __uint_as_float(v.z); x[i][7] = __uint_as_float(v.w);
      } else {
        widen(u, x[i]);
      }
    }
    if (a.y) {
      float f = 1.f;
      if (a.post_norm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          if (tid + i * T >= n) continue;
          float y[8];
          widen(lds128(place(stage, i, kX) + 16 * tid), y);
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
        }
        f = 1.f / sqrtf(block_sum(ss, part[turn][0]) * inv_w + a.eps);
      }
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int c = tid + i * T;
        if (c >= n) continue;
        float y[8];
        widen(lds128(place(stage, i, kX) + 16 * tid), y);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] *= pw[i][e];
        if (a.gate) {
          float g[8];
          widen(lds128(place(stage, i, kX + 1) + 16 * tid), g);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = __fdividef(y[e], 1.f + __expf(-g[e]));
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = fmaf(f, y[e], x[i][e]);
        if (a.x_out) {
          char* xo = static_cast<char*>(a.x_out) + row * a.width * (kF32 ? 4 : 2);
          if constexpr (kF32) {
            store_f32x8(reinterpret_cast<float*>(xo) + 8 * c, x[i], whole);
          } else {
            reinterpret_cast<uint4*>(xo)[c] = narrow(x[i]);
          }
        }
      }
    }
    if constexpr (kF32) __syncwarp();  // the warp has read the stage
    stage = stage == kStages - 1 ? 0 : stage + 1;
    if (!a.h) continue;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kVec; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[i][e], x[i][e], ss);
    const float f = 1.f / sqrtf(block_sum(ss, part[turn][1]) * inv_w + a.eps);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int c = tid + i * T;
      if (c >= n) continue;
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = x[i][e] * f * w[i][e];
      reinterpret_cast<uint4*>(static_cast<char*>(a.h) + row * a.width * 2)[c] = narrow(y);
    }
  }
  cp_async_wait_all();
}

int threads_for(int groups, int vec) { return ((groups + vec - 1) / vec + 31) & ~31; }

template <int kVec, bool kF32>
int registers() {
  static const int regs = [] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, norm_kernel<kVec, kF32>) == cudaSuccess ? (at.numRegs + 7) & ~7 : 64;
  }();
  return regs;
}

// How often all SMs have to be filled for a row a block.
template <int kVec>
int64_t rounds(const NormArgs& a, int num_sms) {
  const int threads = threads_for(a.width >> 3, kVec);
  if (threads > 1024) return INT64_MAX;
  const int fit = 65536 / ((a.x_f32 ? registers<kVec, true>() : registers<kVec, false>()) * threads);
  const int64_t blocks = static_cast<int64_t>(num_sms) * max(1, min(min(32, 2048 / threads), fit));
  return (a.rows + blocks - 1) / blocks;
}

template <int kVec>
void launch(const NormArgs& a, int num_sms) {
  const int threads = threads_for(a.width >> 3, kVec);
  const int64_t most = static_cast<int64_t>(num_sms) * (2048 / threads > 32 ? 32 : 2048 / threads);
  const unsigned grid = static_cast<unsigned>(a.rows < most ? a.rows : most);
  if (a.x_f32) norm_kernel<kVec, true><<<grid, threads, 0, a.stream>>>(a);
  else norm_kernel<kVec, false><<<grid, threads, 0, a.stream>>>(a);
}

template <int kVec, bool kF32>
cudaError_t launch_rows(const NormArgs& a, int num_sms) {
  static SmemOptIn opt_in;
  const auto kernel = norm_rows_kernel<kVec, kF32>;
  const cudaError_t e = opt_in(reinterpret_cast<const void*>(kernel), kMaxSmem);
  if (e != cudaSuccess) return e;
  static const int regs = [] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, norm_rows_kernel<kVec, kF32>) == cudaSuccess ? (at.numRegs + 7) & ~7 : 128;
  }();
  const int threads = threads_for(a.width >> 3, kVec);
  const int bytes = kStages * 16 * threads * kVec * ((kF32 ? 2 : 1) + (a.y ? 1 : 0) + (a.gate ? 1 : 0));
  // as many blocks as an SM holds at once: their rows are then spread evenly
  int blocks = max(1, min(min(32, 2048 / threads), min(65536 / (regs * threads), (kMaxSmem + 1024) / (bytes + 1536))));
  // A stream of 32 bits that is read and written: about 43 KB of it under way on an SM, two blocks at least.  More
  // slows it (30000 rows; blocks an SM: us.  2048 wide 2: 130, 3: 122, 4: 134; 1792 wide 3: 101, 4: 116; 1280 wide 4: 72, 5: 84;
  // 1024 wide 4: 64, 5: 57, 8: 69; 4096 wide 2: 257, 3: 263), a stream of 16 bits or one that is only read does not mind.
  if (kF32 && a.y) blocks = min(blocks, max(2, (43 * 1024 + 4 * a.width) / (8 * a.width)));
  const int64_t most = static_cast<int64_t>(num_sms) * blocks;
  kernel<<<static_cast<unsigned>(a.rows < most ? a.rows : most), threads, bytes, a.stream>>>(a);
  return cudaGetLastError();
}
template <int kVec>
cudaError_t launch_rows(const NormArgs& a, int num_sms) {
  return a.x_f32 ? launch_rows<kVec, true>(a, num_sms) : launch_rows<kVec, false>(a, num_sms);
}

}  // namespace

// What both ways took, in us (8192 x 12288 with all parts in bf16; 30001 x 1928 with an fp32 residual, no gate;
// 4001 x 5128, the norm alone; 1200, 304 and 152 x 4096 with all parts): a row a block 270 / 137 / 42 / 15.5 / 5.0 /
// 3.4, rows in a line 158 / 109 / 18 / 13 / 5.8 / 4.0.  Where no line fits, many rows go a row a block (all parts; of what their bytes
// take at the copy rate: bf16 8192 x 12296 282 us (148), 8192 x 16384 327 (198); fp32 8192 x 12288 223 (208), x 16384 321 (277)).
cudaError_t launch_block_norm(const NormArgs& a, int num_sms) {
  const int n = a.width >> 3, part_bytes = 16 * ((a.x_f32 ? 2 : 1) + (a.y ? 1 : 0) + (a.gate ? 1 : 0));
  // Blocks of up to 256 threads, several on an SM, whose waits overlap; of up to 512 where only one fits
  // (1024 groups, all parts: 132 us with 512 threads, 156 with 256; 641 groups, the norm alone: 28 and 19).
  const int most = 2 * kStages * n * part_bytes > kMaxSmem ? 512 : 256;
  const int vec = (n + most - 1) / most <= 4 ? (n + most - 1) / most : (n + 511) / 512;
  // a line of rows has to fit, counted with the whole warps it is laid out for
  if (a.rows >= 4 * static_cast<int64_t>(num_sms) && vec <= 4 && kStages * part_bytes * vec * threads_for(n, vec) <= kMaxSmem) {
    if (vec <= 1) return launch_rows<1>(a, num_sms);
    if (vec == 2) return launch_rows<2>(a, num_sms);
    return vec == 3 ? launch_rows<3>(a, num_sms) : launch_rows<4>(a, num_sms);
  }
  // A row a block, with as few groups a thread as fill the SMs the fewest times (all parts; 12288 wide: 152 rows 8.0 us
  // with two groups and 9.9 with three, 256 rows 12.9 and 10.9; 8192 wide: 256 rows 10.1 with one and 7.9 with two).
  const int64_t one = rounds<1>(a, num_sms), two = rounds<2>(a, num_sms), three = rounds<3>(a, num_sms);
  if (n <= 1024 && one <= two && one <= three) launch<1>(a, num_sms);
  else if (n <= 2048 && two <= three) launch<2>(a, num_sms);
  else if (n <= 3 * 1024) launch<3>(a, num_sms);
  else launch<4>(a, num_sms);
  return cudaGetLastError();
}

}  // namespace kda
