// The backward pass of sparse MLA attention. With K the listed rows (576 columns), V their first
// 512, and the forward's out and lse, the probabilities are recomputed:
//   S = scale q K^T,  P = exp(S - lse),  delta = sum_c dout out - dlse,
//   dS = P (dout V^T - delta) scale,  dq = dS K,  dK = dS^T q,  dV = P^T dout,
// and a cache row's gradient is the sum of dK (+ dV on the latent columns) over the lists that
// hold it. sum over heads of P is each entry's attention weight.
//
// One CTA per (query, 16 list entries): the rows stay in shared memory as fp32, heads go one
// after another, each thread owns three channels of the 16 rows' gradients.
#include <math_constants.h>

#include <cstdint>

#include "device.cuh"
#include "internal.h"

namespace svt {

namespace {

constexpr int kTile = 16;
constexpr int kThreads = 192;  // 3 channels each
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

__global__ void __launch_bounds__(kThreads) backward_kernel(const BackwardParams p) {
  __shared__ float rows[kTile][kRow];
  __shared__ float qs[kRow], dos[kVdim];
  __shared__ float pr[kTile], ds[kTile];
  __shared__ int slot[kTile];
  __shared__ float delta_s;
  __shared__ float dred[kWarps];
  const int tiles = (p.K + kTile - 1) / kTile;
  const int t = blockIdx.x / tiles, j0 = (blockIdx.x - t * tiles) * kTile;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < kTile) slot[tid] = j0 + tid < p.K ? p.slots[static_cast<long long>(t) * p.K + j0 + tid] : -1;
  __syncthreads();
  for (int i = tid; i < kTile * kRow; i += kThreads) {
    const int e = i / kRow, c = i - e * kRow;
    rows[e][c] = slot[e] >= 0
                     ? bf(reinterpret_cast<const uint16_t*>(p.kv + slot[e] * p.row_stride)[c])
                     : 0.f;
  }
  float acc[kTile][3] = {};
  float wsum = 0.f;  // thread e < 16: entry e's weight
  for (int h = 0; h < p.H; ++h) {
    const long long r = static_cast<long long>(t) * p.H + h;
    __syncthreads();
    float d = 0.f;
    for (int c = tid; c < kRow; c += kThreads) qs[c] = bf(p.q[r * kRow + c]);
    for (int c = tid; c < kVdim; c += kThreads) {
      const float g = bf(p.dout[r * kVdim + c]);
      dos[c] = g;
      d += g * bf(p.out[r * kVdim + c]);
    }
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (lane == 0) dred[warp] = d;
    __syncthreads();
    if (tid == 0) {
      float s = p.dlse ? -p.dlse[r] : 0.f;
      for (int w = 0; w < kWarps; ++w) s += dred[w];
      delta_s = s;
    }
    __syncthreads();
    const float lse = p.lse[r];
    for (int e = warp; e < kTile; e += kWarps) {
      float s = 0.f, dp = 0.f;
      for (int c = lane; c < kRow; c += 32) {
        s += qs[c] * rows[e][c];
        if (c < kVdim) dp += dos[c] * rows[e][c];
      }
      for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        dp += __shfl_xor_sync(0xffffffffu, dp, o);
      }
      if (lane == 0) {
        const float pe = slot[e] >= 0 && lse != -CUDART_INF_F ? expf(s * p.scale - lse) : 0.f;
        pr[e] = pe;
        ds[e] = pe != 0.f ? pe * (dp - delta_s) * p.scale : 0.f;
      }
    }
    __syncthreads();
    if (tid < kTile) wsum += pr[tid];
#pragma unroll
    for (int u = 0; u < 3; ++u) {
      const int c = tid + u * kThreads;
      float dq = 0.f;
      const float qc = qs[c], doc = c < kVdim ? dos[c] : 0.f;
#pragma unroll
      for (int e = 0; e < kTile; ++e) {
        dq += ds[e] * rows[e][c];
        acc[e][u] += ds[e] * qc + pr[e] * doc;
      }
      if (dq != 0.f) atomicAdd(p.dq_acc + r * kRow + c, dq);
    }
  }
#pragma unroll
  for (int e = 0; e < kTile; ++e)
    if (slot[e] >= 0)
#pragma unroll
      for (int u = 0; u < 3; ++u)
        atomicAdd(p.dkv_acc + static_cast<long long>(slot[e]) * kRow + tid + u * kThreads, acc[e][u]);
  if (p.weights != nullptr && tid < kTile && j0 + tid < p.K)
    p.weights[static_cast<long long>(t) * p.K + j0 + tid] = wsum;
}

// fp32 sums -> bf16, eight at a time.
__global__ void __launch_bounds__(256) round_kernel(const float* __restrict__ src, uint16_t* __restrict__ dst,
                                                    long long n8) {
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n8; i += gridDim.x * 256ll) {
    const float4 a = reinterpret_cast<const float4*>(src)[2 * i], b = reinterpret_cast<const float4*>(src)[2 * i + 1];
    reinterpret_cast<uint4*>(dst)[i] = make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y),
                                                  pack_bf16x2(b.z, b.w));
  }
}

}  // namespace

cudaError_t launch_backward(const BackwardParams& p, cudaStream_t stream) {
  const int tiles = (p.K + kTile - 1) / kTile;
  cudaError_t e = cudaSuccess;
  if (p.T > 0 && tiles > 0) {
    backward_kernel<<<static_cast<unsigned>(static_cast<long long>(p.T) * tiles), kThreads, 0, stream>>>(p);
    e = cudaGetLastError();
  }
  const long long nq = static_cast<long long>(p.T) * p.H * (kRow / 8), nk = p.num_slots * (kRow / 8);
  if (e == cudaSuccess && nq > 0) {
    round_kernel<<<static_cast<unsigned>(nq / 256 + 1 < 1216 ? nq / 256 + 1 : 1216), 256, 0, stream>>>(p.dq_acc, p.dq, nq);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) {
    round_kernel<<<static_cast<unsigned>(nk / 256 + 1 < 1216 ? nk / 256 + 1 : 1216), 256, 0, stream>>>(p.dkv_acc, p.dkv, nk);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace svt
