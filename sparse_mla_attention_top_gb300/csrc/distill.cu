// The loss that trains an indexer on a teacher's top entries, and its gradient. For query t with
// student scores x over positions 0 .. len - 1 and a teacher list (position, value):
//   p = the list's values normalised (weights), or softmax(value / tau) (logits),
//   q = softmax(x / tau) over all candidates, or over the listed ones,
//   loss = sum_j p_j (ln p_j - ln q_j),   d loss / d x_n = (q_n - sum of p at n) / tau.
// Everything runs in log2 units (c = log2(e) / tau) and relative to the largest score m and the largest
// teacher value v_m. With w = 2^(c (v - v_m)) (logits) or v / v_m (weights), W = sum w and
// Z = sum 2^(c (x - m)):
//   loss = sum w e / W - log2 W + log2 Z,
//   e = c ((v - x) - (v_m - m)) (logits) or log2 w - c (x - m) (weights),
// so one sweep over the list serves the loss. An entry's two logarithms are subtracted before they are
// summed, which keeps the digits of a small loss of long logarithms, and a list of one entry has
// exactly no loss and no gradient. Scores may be masks of the type's lowest value: the e's are held times
// 2^-32, so that one of 3.4e38 and their sum stay finite, and where the whole row is such a mask, x - m is
// taken first, so that v is not lost in v - x (neither costs time that shows).
//
// Bound: reading the scores once and writing the gradient once. A row is cut between the CTAs
// of a cluster so that each part (up to 64 KB) stays in shared memory: it is read from memory
// once, turned into exp(x - max) in place (one exponential per score for loss and gradient),
// and after the cluster has exchanged its sums scaled on the way out; the listed columns are
// put right behind it. A list of up to 2048 entries stays in registers, each CTA working on those in its
// own columns. Three CTAs of 512 threads share an SM, so one's reads overlap another's writes.
// Longer lists, and rows of more than eight parts, are read again where they are needed. 1024 rows of
// up to 32768 fp32 scores, 2048 listed: 62 us, 3.5 TB/s; the phases of a row wait for one another.
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
constexpr int kWaitTries = 1 << 18;  // of up to 2 us each, before a wait may give up
constexpr float kDown = 1.f / 4294967296.f;  // the e's are held times this
constexpr float kUp = 4294967296.f;

struct Stats {
  float m, s;  // largest score, sum of 2^(c (x - m)) (this CTA's candidates)
  float w, d;  // sums of w and of w e kDown (this CTA's share of the list), e as below
};

struct DistillShared {
  float4 red[2][kWarps];               // one array per reduction, in turns
  alignas(16) Stats stats[kMaxSplit];  // every CTA's, sent by each
  uint64_t arrived;                    // counts their bytes
};
static_assert(sizeof(Stats) == 16, "one message");

// Three sums over the block (x, y, z), or with kMax two maxima (x, y; NaN ignored). One barrier; `red`
// alternates between calls, so that a slow warp still reads the previous array.
template <bool kMax>
__device__ __forceinline__ float4 block_reduce(float4 v, float4* red) {
  const int lane = threadIdx.x & 31;
  auto over = [&](float4 q) {
    if constexpr (kMax) {
      q.x = warp_max_f32(q.x);
      q.y = warp_max_f32(q.y);
    } else {
      // the halves of the warp take x and y; z goes along
      const bool up = (lane & 16) != 0;
      float a = up ? q.y : q.x;
      a += __shfl_xor_sync(0xffffffffu, up ? q.x : q.y, 16);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) q.z += __shfl_xor_sync(0xffffffffu, q.z, o);
      const float b = __shfl_xor_sync(0xffffffffu, a, 16);
      q.x = up ? b : a;
      q.y = up ? a : b;
    }
    return q;
  };
  v = over(v);
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const float none = kMax ? -CUDART_INF_F : 0.f;
  return over(lane < kWarps ? red[lane] : make_float4(none, none, none, none));
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

// Scores [a, a + n) into part[]; returns this thread's largest.
template <typename E>
__device__ __forceinline__ float fill_part(const E* row, int a, int n, bool vec, float* part) {
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
          mx = fmaxf(fmaxf(mx, fmaxf(v[u].x, v[u].y)), fmaxf(v[u].z, v[u].w));
          reinterpret_cast<float4*>(part)[j + u * kThreads] = v[u];
        }
    }
    j0 = 4 * n4;
  }
#pragma unroll 8
  for (int j = j0 + threadIdx.x; j < n; j += kThreads) {
    const float v = load1(row + a + j);
    mx = fmaxf(mx, v);
    part[j] = v;
  }
  return mx;
}

// This thread's sum of 2^(c (x - ref)) over part[0 .. n), which are left in place of x with kKeep. The
// difference comes first: its rounding is relative to x - ref, small where the terms are large.
template <bool kKeep>
__device__ __forceinline__ float exp_part(float* part, int n, float c, float ref) {
  float s = 0.f;
  const int n4 = n / 4;
#pragma unroll 4
  for (int j = threadIdx.x; j < n4; j += kThreads) {
    float4 v = reinterpret_cast<float4*>(part)[j];
    v.x = ex2_approx((v.x - ref) * c);
    v.y = ex2_approx((v.y - ref) * c);
    v.z = ex2_approx((v.z - ref) * c);
    v.w = ex2_approx((v.w - ref) * c);
    s += (v.x + v.y) + (v.z + v.w);
    if (kKeep) reinterpret_cast<float4*>(part)[j] = v;
  }
  for (int j = 4 * n4 + threadIdx.x; j < n; j += kThreads) {
    const float v = ex2_approx((part[j] - ref) * c);
    s += v;
    if (kKeep) part[j] = v;
  }
  return s;
}

// part[0 .. n) times f to out.
template <typename E>
__device__ __forceinline__ void write_part(const float* part, int n, float f, bool vec, E* out) {
  int j0 = 0;
  if (vec) {
    const int n4 = n / 4;
#pragma unroll 4
    for (int j = threadIdx.x; j < n4; j += kThreads) {
      const float4 v = reinterpret_cast<const float4*>(part)[j];
      store4(out + 4 * j, make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
    }
    j0 = 4 * n4;
  }
  for (int j = j0 + threadIdx.x; j < n; j += kThreads) store1(out + j, part[j] * f);
}

constexpr int kHeld = 4;  // list entries a thread keeps in registers: lists of up to 2048

// kAll: the softmax runs over all candidates, else over the listed ones. kFit: the list is held in
// registers and this CTA's columns in shared memory; otherwise both are read again where needed.
template <typename E, bool kAll, bool kFit>
__global__ void __launch_bounds__(kThreads, 3) distill_kernel(const DistillParams p) {
  extern __shared__ float4 dyn[];
  float* part = reinterpret_cast<float*>(dyn);
  __shared__ DistillShared sh;
  if (p.split > 1) {
    if (threadIdx.x == 0) {
      mbar_init(smem_u32(&sh.arrived), 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      mbar_arrive_expect_tx(smem_u32(&sh.arrived), p.split * static_cast<uint32_t>(sizeof(Stats)));
    }
    // (completed below) every CTA of the cluster has started and can be sent to
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  }
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
  const int n = chi - lo;
  const bool vec = p.vec != 0;
  const float c = p.inv_tau * kLog2e;

  float mx = -CUDART_INF_F, tmax = -CUDART_INF_F;  // largest candidate (or listed score), largest teacher value
  int held_i[kHeld];
  float held_v[kHeld];
  if constexpr (kFit) {
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      const int j = tid + u * kThreads;
      held_i[u] = j < p.K ? __ldg(idx + j) : -1;
      held_v[u] = j < p.K ? __ldg(val + j) : 0.f;
    }
  }
  if constexpr (kAll && kFit) mx = fill_part(row, lo, n, vec, part);
  if constexpr (kFit) {
    // only the entries this CTA works on: those in its own columns, or every live one of a listed softmax
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      const bool live = held_i[u] >= 0 && held_i[u] < len;
      if (live) tmax = fmaxf(tmax, held_v[u]);
      if (!live || (kAll && (held_i[u] < lo || held_i[u] >= chi))) held_i[u] = -1;
    }
  }
  float held_x[kHeld];
  if constexpr (!kAll && kFit) {
#pragma unroll
    for (int u = 0; u < kHeld; ++u) held_x[u] = held_i[u] >= 0 ? load1(row + held_i[u]) : -CUDART_INF_F;
  }
  // f(u, position, value, score) for the entries that this thread works on
  auto entries = [&](auto f) {
    if constexpr (kFit) {
#pragma unroll
      for (int u = 0; u < kHeld; ++u)
        if (held_i[u] >= 0) f(u, held_i[u], held_v[u], held_x[u]);
    } else {
      for (int j = tid; j < p.K; j += kThreads) {
        const int i = __ldg(idx + j);
        if (i >= 0 && i < len) f(j / kThreads, i, __ldg(val + j), load1(row + i));
      }
    }
  };
  if (drow != nullptr) {
    // this CTA's share of the columns behind the candidates
    const int tail = ((p.N - len + p.split - 1) / p.split + 7) & ~7;
    const int tlo = min(p.N, len + cr * tail), hi = min(p.N, tlo + tail);
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

  if constexpr (!kAll && kFit) {
    for (int j = tid; j < n; j += kThreads) part[j] = 0.f;
  }
  Stats st{-CUDART_INF_F, 0.f, 0.f, 0.f};
  if constexpr (kAll && !kFit) {
    for (int a = lo; a < chi; a += kPart) {
      const int m = min(kPart, chi - a);
      const float nm = fmaxf(st.m, block_reduce<true>(make_float4(fill_part(row, a, m, vec, part), 0.f, 0.f, 0.f), sh.red[0]).x);
      const float s = block_reduce<false>(
          make_float4(exp_part<false>(part, m, c, nm == -CUDART_INF_F ? 0.f : nm), 0.f, 0.f, 0.f), sh.red[1]).x;
      // (without a largest score so far the sum is 0, or NaN from NaN scores)
      st.s = (st.m == -CUDART_INF_F ? st.s : st.s * exp2f((st.m - nm) * c)) + s;
      st.m = nm;
    }
    mx = st.m;
  }
  if constexpr (!(kAll && kFit))
    entries([&](int, int, float v, float x) {
      if (!kAll) mx = fmaxf(mx, x);
      tmax = fmaxf(tmax, v);
    });
  {
    const float4 r = block_reduce<true>(make_float4(mx, tmax, 0.f, 0.f), sh.red[0]);
    st.m = r.x;
    tmax = r.y == -CUDART_INF_F ? 0.f : r.y;  // nothing listed: every weight is 0
  }
  auto weight = [&](float v) { return p.logits ? exp2f((v - tmax) * c) : (tmax > 0.f ? v / tmax : v); };
  const float ref = st.m == -CUDART_INF_F ? 0.f : st.m;  // of this CTA's exponents
  if constexpr (kAll && kFit) {
#pragma unroll
    for (int u = 0; u < kHeld; ++u) held_x[u] = held_i[u] >= 0 ? part[held_i[u] - lo] : 0.f;
    __syncthreads();  // every thread has read its listed scores
  }
  float held_w[kHeld];
  {
    const float ce = c * kDown;
    // (v - x) - (tmax - ref); beyond 2^10 the differences lose more of v than x - ref loses of x
    const float base = fabsf(ref) > 1024.f ? ref : 0.f;
    const float top = tmax - (ref - base);
    auto gap = [&](float v, float x) { return (v - (x - base)) - top; };
    float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
    if (kAll && kFit) r.x = exp_part<true>(part, n, c, ref);
    entries([&](int u, int, float v, float x) {
      if (!kAll) r.x += exp2f((x - ref) * c);
      const float w = weight(v);
      if (kFit) held_w[u] = w;
      // where CTAs see the same entries, each takes every split-th for the sums
      if (!(kAll && kFit) && ((tid + u * kThreads) & (p.split - 1)) != cr) return;
      r.y += w;
      if (w != 0.f) r.z += w * (p.logits ? gap(v, x) * ce : fmaf(ref - x, ce, log2f(w) * kDown));
    });
    r = block_reduce<false>(r, sh.red[1]);
    if (!(kAll && !kFit)) st.s = r.x;
    st.w = r.y;
    st.d = r.z;
  }

  float M = st.m, Z = st.s, W = st.w, D = st.d;
  bool lost = false;
  if (p.split > 1) {
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (tid < p.split)
      st_async_v4(mapa_shared(smem_u32(&sh.stats[cr]), tid),
                  make_uint4(__float_as_uint(st.m), __float_as_uint(st.s), __float_as_uint(st.w), __float_as_uint(st.d)),
                  mapa_shared(smem_u32(&sh.arrived), tid));
    // every CTA's sums arrive here (a barrier of the cluster would also wait for the zeroes on their way
    // to memory); should one not, the row's loss and gradient are NaN. The time alone does not say so: it
    // runs on while a whole cluster is switched out, whose CTAs still send to each other afterwards
    const uint64_t t0 = globaltimer();
    for (int tries = 0; !mbar_try_wait_cluster(smem_u32(&sh.arrived), 0); ++tries) {
      if (tries > kWaitTries && globaltimer() - t0 > kWaitLimitNs) {
        lost = true;
        break;
      }
    }
    if constexpr (kAll) {
      M = -CUDART_INF_F;
      for (int r = 0; r < p.split; ++r) M = fmaxf(M, sh.stats[r].m);
      Z = 0.f;
    }
    W = D = 0.f;
    for (int r = 0; r < p.split; ++r) {
      const Stats q = sh.stats[r];
      // its exponents and its e's were relative to its own largest score
      const float up = kAll && M != -CUDART_INF_F ? (q.m == -CUDART_INF_F ? 0.f : q.m) - M : 0.f;
      if (q.w != 0.f) {
        W += q.w;
        D += q.d - q.w * (up * (c * kDown));
      }
      if constexpr (kAll) {
        if (q.m != -CUDART_INF_F) Z += q.s * exp2f(up * c);
        else if (q.s != q.s) Z = q.s;  // NaN scores
      }
    }
  }
  if (lost) Z = W = __uint_as_float(0x7FC00000u);
  const float top = M == -CUDART_INF_F ? 0.f : M;  // Z is relative to it
  // a row without a target, or whose candidates are all -inf, has loss 0 and gradient 0
  const bool some = !(W == 0.f) && !(M == -CUDART_INF_F && !(Z != Z));
  if (p.loss != nullptr && cr == 0 && tid == 0) {
    // The terms may cancel to a small difference: a compensated fp32 sum of D / W, the logarithms of
    // mantissas next to exact exponents, and the division's remainder (in fp64, which runs at two lanes a
    // cycle, this took a microsecond that the whole CTA waited for)
    int ez, ew;
    const float mz = frexpf(Z, &ez), mw = frexpf(W, &ew);
    const float quot = __fdiv_rn(D, W);
    float sum = quot * kUp, low = 0.f;
    auto add = [&](float x) {
      const float u = __fadd_rn(sum, x);
      low += fabsf(sum) >= fabsf(x) ? __fadd_rn(__fsub_rn(sum, u), x) : __fadd_rn(__fsub_rn(x, u), sum);
      sum = u;
    };
    add(static_cast<float>(ez - ew));
    add(log2f(mz));
    add(-log2f(mw));
    const float rest = __fmaf_rn(-quot, W, D) / W * kUp;
    const float d = (sum + (low + rest)) * 0.6931471805599453f;
    // a sum that is infinite in log2 units (a weight on a score of -inf, or on one of the lowest value) leaves
    // the logarithms nothing to add; Z is NaN with NaN scores beside it
    p.loss[t] = some ? (fabsf(quot * kUp) == CUDART_INF_F && Z == Z ? quot * 0.6931471805599453f * kUp : d) : 0.f;
  }
  if (drow == nullptr) return;

  const float g = some ? (p.row_weight ? p.row_weight[t] : 1.f) * p.inv_tau : 0.f;
  const float gq = some ? g / Z : 0.f, gw = some ? -g / W : 0.f;
  if constexpr (kAll && kFit) {
    // part holds 2^(c (x - ref)). A listed column is set to q's share, then p's are added (as
    // often as it is listed); the sweep writes q's share everywhere, and the listed columns again
    const float scale = some ? gq * exp2f((ref - top) * c) : 0.f;
    if (some) {
#pragma unroll
      for (int u = 0; u < kHeld; ++u)
        if (held_i[u] >= 0) part[held_i[u] - lo] = ex2_approx((held_x[u] - ref) * c) * scale;
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kHeld; ++u)
        if (held_i[u] >= 0) atomicAdd(part + (held_i[u] - lo), held_w[u] * gw);
      write_part(part, n, scale, vec, drow + lo);
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kHeld; ++u)
        if (held_i[u] >= 0) store1(drow + held_i[u], part[held_i[u] - lo]);
    } else {
      for (int j = tid; j < n; j += kThreads) store1(drow + lo + j, 0.f);
    }
  } else {
    for (int a = lo; a < chi; a += kPart) {
      const int m = min(kPart, chi - a);
      if constexpr (kAll) {
        __syncthreads();
        fill_part(row, a, m, vec, part);
        __syncthreads();
        for (int j = tid; j < m; j += kThreads) part[j] = some ? ex2_approx((part[j] - top) * c) * gq : 0.f;
        __syncthreads();
      } else if constexpr (!kFit) {
        __syncthreads();
        for (int j = tid; j < m; j += kThreads) part[j] = 0.f;
        __syncthreads();
      }
      if (some) {
        entries([&](int, int i, float v, float x) {
          if (i < a || i >= a + m) return;
          float d = weight(v) * gw;
          if (!kAll) d += exp2f((x - top) * c) * gq;
          if (d != 0.f) atomicAdd(part + (i - a), d);
        });
      }
      __syncthreads();
      write_part(part, m, 1.f, vec, drow + a);
    }
  }
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
  const int per = ((p.N + split - 1) / split + 7) & ~7;  // the largest part (the kernel's share for len = N)
  const size_t smem = static_cast<size_t>(per < kPart ? per : kPart) * sizeof(float);
  const bool fit = p.K <= kHeld * kThreads && per <= kPart;
  const auto kernel = fit ? distill_kernel<E, kAll, true> : distill_kernel<E, kAll, false>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kPart * sizeof(float)));
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
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_distill(const DistillParams& p, bool f32, bool all, cudaStream_t stream) {
  if (p.T == 0) return cudaSuccess;
  if (f32) return all ? launch_e<float, true>(p, stream) : launch_e<float, false>(p, stream);
  return all ? launch_e<uint16_t, true>(p, stream) : launch_e<uint16_t, false>(p, stream);
}

}  // namespace svt
