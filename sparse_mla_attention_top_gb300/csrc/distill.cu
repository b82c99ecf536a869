// The loss that trains an indexer on a teacher's top entries, and its gradient. For query t with
// student scores x over positions 0 .. len - 1 and a teacher list (position, value):
//   p = the list's values normalised (weights), or softmax(value / tau) (logits),
//   q = softmax(x / tau) over all candidates, or over the listed ones,
//   loss = sum_j p_j (ln p_j - ln q_j),   d loss / d x_n = (q_n - sum of p at n) / tau.
// With W = sum w, A = sum w ln w, B = sum w x / tau and the student's normaliser lse (natural
// log): loss = A / W - ln W - B / W + lse, so one sweep over the list serves the loss.
//
// Bound: reading the scores once and writing the gradient once. A row is cut between the CTAs
// of a cluster so that each part (up to 64 KB) stays in shared memory: it is read from memory
// once, turned into exp(x - max) in place (one exponential per score for loss and gradient),
// and after the cluster has exchanged (max, sum, B) scaled, corrected at the listed positions
// and written. Three CTAs of 512 threads share an SM, so one's reads overlap another's writes.
// Rows longer than eight parts are swept twice from memory.
#include <cooperative_groups.h>
#include <math_constants.h>

#include <cstdint>

#include "device.cuh"
#include "internal.h"

namespace svt {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPart = 16384;  // scores of one part: 64 KB as fp32
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxSplit = 8;

struct Stats {
  float m, s, b;  // running max (log2 units), sum of 2^(x - m), sum of w x (log2 units)
};

struct DistillShared {
  float red[kWarps];
  Stats stats[kMaxSplit];  // every CTA's, pushed by each
};

__device__ __forceinline__ float block_reduce(float v, bool is_max, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = is_max ? fmaxf(v, w) : v + w;
  }
  __syncthreads();  // red is free
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[threadIdx.x & (kWarps - 1)];
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = is_max ? fmaxf(v, w) : v + w;
  }
  return v;
}

__device__ __forceinline__ float load1(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load1(const uint16_t* p) {
  return __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16);
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) {
  *p = static_cast<uint16_t>(pack_bf16x2(v, 0.f) & 0xFFFFu);
}
// Four consecutive scores (16 or 8 bytes, aligned).
__device__ __forceinline__ float4 load4(const float* p) { return __ldcs(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 load4(const uint16_t* p) {
  const uint2 w = __ldcs(reinterpret_cast<const uint2*>(p));
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xFFFF0000u));
}
__device__ __forceinline__ void store4(float* p, float4 v) { __stcs(reinterpret_cast<float4*>(p), v); }
__device__ __forceinline__ void store4(uint16_t* p, float4 v) {
  __stcs(reinterpret_cast<uint2*>(p), make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)));
}

// Scores [a, a + n) times c into part[]; returns this thread's largest.
template <typename E>
__device__ __forceinline__ float fill_part(const E* row, int a, int n, float c, bool vec, float* part) {
  float mx = -CUDART_INF_F;
  int j0 = 0;
  if (vec) {
    const int n4 = n / 4;
    for (int j = threadIdx.x; j < n4; j += 4 * kThreads) {
      float4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (j + u * kThreads < n4) v[u] = load4(row + a + 4 * (j + u * kThreads));
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (j + u * kThreads < n4) {
          v[u].x *= c;
          v[u].y *= c;
          v[u].z *= c;
          v[u].w *= c;
          mx = fmaxf(fmaxf(mx, fmaxf(v[u].x, v[u].y)), fmaxf(v[u].z, v[u].w));
          reinterpret_cast<float4*>(part)[j + u * kThreads] = v[u];
        }
    }
    j0 = 4 * n4;
  }
#pragma unroll 8
  for (int j = j0 + threadIdx.x; j < n; j += kThreads) {
    const float v = load1(row + a + j) * c;
    mx = fmaxf(mx, v);
    part[j] = v;
  }
  return mx;
}

// kAll: the softmax runs over all candidates, else over the listed ones.
template <typename E, bool kAll>
__global__ void __launch_bounds__(kThreads, 3) distill_kernel(const DistillParams p) {
  extern __shared__ float4 dyn[];
  float* part = reinterpret_cast<float*>(dyn);
  __shared__ DistillShared sh;
  const int tid = threadIdx.x;
  const int t = blockIdx.x / p.split, cr = blockIdx.x - t * p.split;
  const E* row = static_cast<const E*>(p.scores) + static_cast<long long>(t) * p.stride;
  E* drow = p.dscores ? static_cast<E*>(p.dscores) + static_cast<long long>(t) * p.dstride : nullptr;
  const int32_t* idx = p.idx + static_cast<long long>(t) * p.K;
  const float* val = p.teacher + static_cast<long long>(t) * p.K;
  int len = p.lens ? p.lens[t] : p.N;
  len = len < 0 ? 0 : (len > p.N ? p.N : len);
  // this CTA's candidates lo .. chi - 1
  const int share = ((len + p.split - 1) / p.split + 7) & ~7;
  const int lo = min(len, cr * share), chi = min(len, lo + share);
  const bool vec = p.vec != 0;
  const float c = p.inv_tau * kLog2e;

  // the teacher's list: every CTA of the row takes the whole list's sums (it is short), and the
  // entries inside its own columns for B. Logits become weights 2^(c (value - max)).
  float tmax = 0.f;
  if (p.logits) {
    tmax = -CUDART_INF_F;
    for (int j = tid; j < p.K; j += kThreads) {
      const int i = __ldg(idx + j);
      if (i >= 0 && i < len) tmax = fmaxf(tmax, __ldg(val + j));
    }
    tmax = block_reduce(tmax, true, sh.red);
    if (tmax == -CUDART_INF_F) tmax = 0.f;  // nothing listed: every weight below is 0
  }
  auto weight = [&](int j, int i) -> float {
    if (i < 0 || i >= len) return 0.f;
    const float v = __ldg(val + j);
    return p.logits ? exp2f((v - tmax) * c) : v;
  };
  float W = 0.f, A = 0.f;
  Stats st{-CUDART_INF_F, 0.f, 0.f};
  for (int j = tid; j < p.K; j += kThreads) {
    const int i = __ldg(idx + j);
    const float w = weight(j, i);
    W += w;
    if (w != 0.f) {
      A += p.logits ? w * ((__ldg(val + j) - tmax) * c) : w * log2f(w);
      if (i >= lo && i < chi) st.b += w * (load1(row + i) * c);
    }
    if (!kAll && i >= 0 && i < len) st.m = fmaxf(st.m, load1(row + i) * c);
  }
  W = block_reduce(W, false, sh.red);
  A = block_reduce(A, false, sh.red);
  st.b = block_reduce(st.b, false, sh.red);

  const int n = chi - lo;
  const bool resident = kAll && n <= kPart;
  if constexpr (kAll) {
    for (int a = lo; a < chi; a += kPart) {
      const int m = min(kPart, chi - a);
      const float mx = block_reduce(fill_part(row, a, m, c, vec, part), true, sh.red);
      const float nm = fmaxf(st.m, mx);
      const float base = nm == -CUDART_INF_F ? 0.f : nm;
      float s = 0.f;
      const int m4 = m / 4;
      for (int j = tid; j < m4; j += kThreads) {
        float4 v = reinterpret_cast<float4*>(part)[j];
        v.x = ex2_approx(v.x - base);
        v.y = ex2_approx(v.y - base);
        v.z = ex2_approx(v.z - base);
        v.w = ex2_approx(v.w - base);
        s += (v.x + v.y) + (v.z + v.w);
        if (resident) reinterpret_cast<float4*>(part)[j] = v;
      }
      for (int j = 4 * m4 + tid; j < m; j += kThreads) {
        const float v = ex2_approx(part[j] - base);
        s += v;
        if (resident) part[j] = v;
      }
      s = block_reduce(s, false, sh.red);
      st.s = (st.m == -CUDART_INF_F ? 0.f : st.s * exp2f(st.m - base)) + s;
      st.m = nm;
    }
  } else {
    // the listed scores only; every CTA takes the whole list
    st.m = block_reduce(st.m, true, sh.red);
    const float base = st.m == -CUDART_INF_F ? 0.f : st.m;
    for (int j = tid; j < p.K; j += kThreads) {
      const int i = __ldg(idx + j);
      if (i >= 0 && i < len) st.s += exp2f(load1(row + i) * c - base);
    }
    st.s = block_reduce(st.s, false, sh.red);
  }

  float M = st.m, Z = st.s, B = st.b;
  if (p.split > 1) {
    auto cl = cooperative_groups::this_cluster();
    cl.sync();  // every CTA of the cluster has started
    if (tid < p.split) cl.map_shared_rank(&sh, static_cast<unsigned>(tid))->stats[cr] = st;
    cl.sync();  // every CTA's statistics are here
    B = 0.f;
    for (int r = 0; r < p.split; ++r) B += sh.stats[r].b;
    if constexpr (kAll) {
      M = -CUDART_INF_F;
      for (int r = 0; r < p.split; ++r) M = fmaxf(M, sh.stats[r].m);
      Z = 0.f;
      for (int r = 0; r < p.split; ++r)
        if (sh.stats[r].m != -CUDART_INF_F) Z += sh.stats[r].s * exp2f(sh.stats[r].m - M);
        else if (sh.stats[r].s != sh.stats[r].s) Z = sh.stats[r].s;  // a NaN score
    }
  }
  // a row without a target, or whose candidates are all -inf, has loss 0 and gradient 0
  const bool some = !(W == 0.f) && !(M == -CUDART_INF_F && !(Z != Z));
  if (p.loss != nullptr && cr == 0 && tid == 0) {
    // the four terms cancel to a small difference: joined in fp64
    const double d = static_cast<double>(A) / W - static_cast<double>(B) / W + static_cast<double>(M) -
                     log2(static_cast<double>(W)) + log2(static_cast<double>(Z));
    p.loss[t] = some ? static_cast<float>(d * 0.69314718055994530942) : 0.f;
  }
  if (drow == nullptr) return;

  const float g = (p.row_weight ? p.row_weight[t] : 1.f) * p.inv_tau;
const int tail = ((p.N - len + p.split - 1) / p.split + 7) & ~7;  // this CTA's share of the columns behind
  const int tlo = min(p.N, len + cr * tail), hi = min(p.N, tlo + tail);
  const float gw = some ? -g / W : 0.f;
  const float base = M == -CUDART_INF_F ? 0.f : M;
  // resident parts hold 2^(x - the CTA's max); parts swept again hold x
  const float scale = some ? (resident ? g / Z * (st.m == -CUDART_INF_F ? 0.f : exp2f(st.m - base)) : g / Z) : 0.f;
  for (int a = lo; a < chi; a += kPart) {
    const int m = min(kPart, chi - a);
    __syncthreads();  // the part is free
    if (!resident) {
      if constexpr (kAll) {
        fill_part(row, a, m, c, vec, part);
      } else {
        for (int j = tid; j < m; j += kThreads) part[j] = 0.f;
      }
      __syncthreads();
    }
    if constexpr (kAll) {
      for (int j = tid; j < m; j += kThreads) {
        const float e = resident ? part[j] : ex2_approx(part[j] - base);
        part[j] = some ? e * scale : 0.f;
      }
      __syncthreads();
    }
    if (some) {
      for (int j = tid; j < p.K; j += kThreads) {
        const int i = __ldg(idx + j);
        if (i < a || i >= a + m) continue;
        float d = weight(j, i) * gw;
        if constexpr (!kAll) d += exp2f(load1(row + i) * c - base) * scale;
        if (d != 0.f) atomicAdd(part + (i - a), d);
      }
    }
    __syncthreads();
    int j0 = 0;
    if (vec) {
      const int m4 = m / 4;
      for (int j = tid; j < m4; j += kThreads) store4(drow + a + 4 * j, reinterpret_cast<float4*>(part)[j]);
      j0 = 4 * m4;
    }
    for (int j = j0 + tid; j < m; j += kThreads) store1(drow + a + j, part[j]);
  }
  // columns behind the candidates
  int j = tlo;
  if (vec) {
    const int al = min(hi, (tlo + 3) & ~3);
    for (int i = tlo + tid; i < al; i += kThreads) store1(drow + i, 0.f);
    const int n4 = (hi - al) / 4;
    for (int i = tid; i < n4; i += kThreads) store4(drow + al + 4 * i, make_float4(0.f, 0.f, 0.f, 0.f));
    j = al + 4 * n4;
  }
  for (int i = j + tid; i < hi; i += kThreads) store1(drow + i, 0.f);
}

template <typename E, bool kAll>
cudaError_t launch_e(DistillParams p, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // CTAs per row: enough that a part fits, and more while the batch leaves SMs idle and the
  // parts stay over 2048 scores
  int split = 1;
  while (split < kMaxSplit && ((p.N + split - 1) / split > kPart ||
                               (static_cast<long long>(p.T) * split < 2ll * sms && p.N / (2 * split) >= 2048)))
    split *= 2;
  p.split = split;
  const int per = (p.N + split - 1) / split + 8;
  const size_t smem = static_cast<size_t>(per < kPart ? (per + 3) & ~3 : kPart) * sizeof(float);
  e = cudaFuncSetAttribute(distill_kernel<E, kAll>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kPart * sizeof(float)));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(p.T) * split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(split);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, distill_kernel<E, kAll>, p);
}

}  // namespace

cudaError_t launch_distill(const DistillParams& p, bool f32, bool all, cudaStream_t stream) {
  if (p.T == 0) return cudaSuccess;
  if (f32) return all ? launch_e<float, true>(p, stream) : launch_e<float, false>(p, stream);
  return all ? launch_e<uint16_t, true>(p, stream) : launch_e<uint16_t, false>(p, stream);
}

}  // namespace svt
