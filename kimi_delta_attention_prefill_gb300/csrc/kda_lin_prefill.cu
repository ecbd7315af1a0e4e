// kda_lin_prefill.cu -- linear attention with a decay a head over packed sequences, token by token:
//     S <- e^g S + k v^T,      o = scale S^T q
// One block a (sequence, head); thread c holds column c of the state.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "kda_lin.h"

namespace kda {
namespace {

constexpr int kD = kHeadDim;

__global__ void __launch_bounds__(kD) lin_tokens_kernel(const __grid_constant__ LinArgs a) {
  __shared__ float sq[kD], sk[kD], part[4];
  const int seq = blockIdx.x, h = blockIdx.y, c = threadIdx.x;
  const int64_t first = a.cu[seq], end = a.cu[seq + 1];
  bool bad = a.cu[0] != 0 || a.cu[a.n_seq] != a.tokens;
  for (int i = c; i < a.n_seq; i += kD) bad |= a.cu[i + 1] < a.cu[i];
  if (__syncthreads_or(bad)) {
    if (c == 0) report_status(a.status, 7 /* KDA_ERR_DEVICE_CHECK */);
    return;
  }
  const int64_t unit = (static_cast<int64_t>(seq) * a.H + h) * kStateFloats;
  float S[kD];
#pragma unroll
  for (int i = 0; i < kD; ++i) S[i] = a.S_in ? a.S_in[unit + i * kD + c] : 0.f;
  const int hq = h / a.group;
  const auto* q = static_cast<const __nv_bfloat16*>(a.q) + hq * a.q_stride[2] + c;
  const auto* k = static_cast<const __nv_bfloat16*>(a.k) + hq * a.k_stride[2] + c;
  const auto* v = static_cast<const __nv_bfloat16*>(a.v) + h * a.v_stride[2] + c;
  const auto* gate = static_cast<const __nv_bfloat16*>(a.gate) + h * a.gate_stride[2] + c;
  for (int64_t t = first; t < end; ++t) {
    __syncthreads();
    sq[c] = __bfloat162float(q[t * a.q_stride[1]]);
    sk[c] = __bfloat162float(k[t * a.k_stride[1]]);
    const float e = expf(a.g[t * a.g_stride[1] + h * a.g_stride[2]]), x = __bfloat162float(v[t * a.v_stride[1]]);
    __syncthreads();
    float o = 0.f;
#pragma unroll
    for (int i = 0; i < kD; ++i) {
      S[i] = fmaf(sk[i], x, e * S[i]);
      o = fmaf(sq[i], S[i], o);
    }
    o *= a.scale;
    if (a.gate) {
      float ss = o * o;
#pragma unroll
      for (int off = 16; off; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      if ((c & 31) == 0) part[c >> 5] = ss;
      __syncthreads();
      ss = part[0] + part[1] + part[2] + part[3];
      o *= (a.norm_weight ? a.norm_weight[c] : 1.f) / (sqrtf(ss * (1.f / kD) + a.eps) *
           (1.f + expf(-__bfloat162float(gate[t * a.gate_stride[1]]))));
    }
    static_cast<__nv_bfloat16*>(a.o)[(t * a.H + h) * kD + c] = __float2bfloat16(o);
  }
  if (a.S_out)
#pragma unroll
    for (int i = 0; i < kD; ++i) a.S_out[unit + i * kD + c] = S[i];
}

}  // namespace

size_t lin_prefill_workspace(int, int64_t, int, int, int) { return 256; }

cudaError_t launch_lin_prefill(const LinArgs& a, int) {
  lin_tokens_kernel<<<dim3(a.n_seq, a.H), kD, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace kda
