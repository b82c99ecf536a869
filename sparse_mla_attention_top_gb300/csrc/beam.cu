// Beam search's selection. Of every batch item's W beams over V tokens, the K candidates of largest
//   value(w, v) = scores[w] + logits[w, v] - ln sum_u exp(logits[w, u]),
// equal ones in the order of (w, v); a finished beam has one candidate, its end token at its own score.
//
// The logits are read once. Within a beam the values are in the order of the logits, so the first kernel
// keeps, beside the running maximum and sum of the softmax, the K largest logits of its slice of a beam
// (64-bit keys: the logit's order-preserving bits above the complement of the token, so that no two are equal);
// the second joins the slices' sums and ranks the candidates of an item's beams.
//
// What bounds it: 64 x 8 beams x 131072 bf16 logits (a fifth of the beams finished): 34 us, 3.2 TB/s. A logit costs some ten
// instructions (its read, a share of a maximum, a difference, a factor, an exponential, a sum), half of the issue slots of the
// scan's 28 us; at the rankings a CTA's warps wait for one another; the second kernel's 7 us come behind the last scan. 16 x 8 x
// 50257 fp32: 19 us; 4 beams x 32000: 10 us, a chain of dependent steps in each of the two kernels (the first 4 us, the second 6).
//
// Two beams' values may be close, and the order between them is by the normalisers: sums are held per thread in fp32 (over
// some 500 exponentials of a vocabulary of 131072), joined as integers (exact, in any order), and the values are fp64. The
// normalisers are 3e-8 off on average.
#include <algorithm>
#include <cfloat>

#include <cuda_bf16.h>

#include "device.cuh"
#include "internal.h"

namespace svt {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kWords = 16;                 // 4-byte words of a lane a round
constexpr int kSpan = 32 * kWords * 4;     // bytes of a warp a round
constexpr int kStages = 3;                 // a warp's rounds in shared memory
constexpr int kStageBytes = kSpan + 32;    // and what the first piece of 16 bytes holds before them
constexpr int kRounds = 4;                 // rounds between two rankings
constexpr int kBuf = 1024;                 // keys a CTA can hold between two rankings
constexpr int kStep = 3 * kThreads;        // tokens that always fit beside K keys
constexpr int kMaxSlices = 32;
constexpr int kKeys = 4;                   // of a thread of the second kernel, loaded together
constexpr int kSortFrom = 257;             // keys from which sorting is faster than counting the larger ones of each
constexpr float kLog2e = 1.4426950408889634f;
static_assert(kBeamMaxK + kStep <= kBuf);

// Increases with x over all numbers above -inf (+0 and -0 alike); 0 for -inf and NaN.
__device__ __forceinline__ uint32_t ordered(float x) {
  if (!(x > -__int_as_float(0x7f800000))) return 0u;
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t ordered(double x) {
  if (!(x > -__longlong_as_double(0x7ff0000000000000ll))) return 0ull;
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return (b >> 63) ? ~b : b | (1ull << 63);
}
__device__ __forceinline__ double from_ordered(uint64_t k) {
  return __longlong_as_double(static_cast<long long>((k >> 63) ? k & ~(1ull << 63) : ~k));
}

// A lower bound of the K-th largest of the CTA's values, 0 if there are fewer: the K-th largest of each warp's `kept` largest,
// which is the K-th largest itself unless one warp has more than `kept` of the K. `best` is kThreads values of shared memory,
// `found` one. Every thread gets it.
__device__ __forceinline__ uint32_t lower_bar(uint32_t v, int K, uint32_t* best, uint32_t* found) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kept = K <= 16 ? 4 : K <= 64 ? 16 : 32;
  uint32_t mine = 0;
#pragma unroll 1
  for (int i = 0; i < kept; ++i) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, v);
    const bool first_of_them = __ffs(__ballot_sync(0xffffffffu, v == top)) - 1 == lane;
    mine = lane == i ? top : mine;
    v = first_of_them ? 0 : v;
  }
  if (lane < kept) best[warp * kept + lane] = mine;
  __syncthreads();
  const int n = kWarps * kept;
  if (tid < n) {
    const uint32_t x = best[tid];
    int before = 0;
#pragma unroll 4
    for (int j = 0; j < n; j += 4) {
      const uint4 o = *reinterpret_cast<const uint4*>(best + j);
      before += (o.x > x || (o.x == x && j < tid)) + (o.y > x || (o.y == x && j + 1 < tid)) +
                (o.z > x || (o.z == x && j + 2 < tid)) + (o.w > x || (o.w == x && j + 3 < tid));
    }
    if (before == K - 1) *found = x;
  }
  __syncthreads();
  return *found;
}

// A slice's sum of exponentials, at most V and at least 1, as an integer: V of them stay below 2^62.
__device__ __forceinline__ int beam_unit(int V) { return 30 + __clz(V); }
constexpr uint64_t kNoSum = ~0ull;  // NaN

// A bitonic network over `n` (a power of two) places; exchange(i, j) puts the larger first.
template <typename Exchange>
__device__ __forceinline__ void sort_descending(int n, Exchange exchange) {
  for (int k = 2; k <= n; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int t = threadIdx.x; t < n / 2; t += kThreads) {
        const int lo = 2 * t - (t & (j - 1)), hi = lo + j;
        if ((lo & k) == 0) {
          exchange(lo, hi);
        } else {
          exchange(hi, lo);
        }
      }
      __syncthreads();
    }
  }
}
__device__ __forceinline__ int power_of_two(int n) { return n <= 1 ? 1 : 1 << (32 - __clz(n - 1)); }

struct Shared {
  alignas(16) char stage[kWarps][kStages][kStageBytes];
  uint64_t buf[kBuf];
  uint64_t best[kBeamMaxK];
  alignas(16) uint32_t best32[kThreads];
  uint32_t found;
  float part_m[kWarps];
  uint64_t part_s[kWarps];
  int count;
};

// The K largest of buf[0 .. n) in descending order, back in buf.
__device__ __noinline__ void rank_buffer(Shared& sh, int n, int K) {
  if (n >= kSortFrom) {
    const int P = power_of_two(n);
    for (int i = n + threadIdx.x; i < P; i += kThreads) sh.buf[i] = 0;
    __syncthreads();
    sort_descending(P, [&](int i, int j) {
      const uint64_t a = sh.buf[i], b = sh.buf[j];
      if (b > a) {
        sh.buf[i] = b;
        sh.buf[j] = a;
      }
    });
  } else {
    if (threadIdx.x < n) {
      const uint64_t k = sh.buf[threadIdx.x];
      int r = 0;
#pragma unroll 4
      for (int j = 0; j < n; ++j) r += sh.buf[j] > k;
      if (r < K) sh.best[r] = k;
    }
    __syncthreads();
    if (threadIdx.x < min(n, K)) sh.buf[threadIdx.x] = sh.best[threadIdx.x];
  }
  if (threadIdx.x == 0) sh.count = min(n, K);
  __syncthreads();
}

__device__ __forceinline__ uint64_t pack2(float x, float y) {
  return static_cast<uint64_t>(__float_as_uint(y)) << 32 | __float_as_uint(x);
}
__device__ __forceinline__ float first(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float second(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// A beam's row of logits. Its tokens are dealt to the threads by their numbers, not by where memory's 16-byte pieces fall, so
// that equal rows have equal sums wherever they lie: the pieces come into shared memory as they are, and a lane takes word
// lane + 32 i of its warp's tokens from there, at any alignment.
template <bool kF32>
struct Row {
  static constexpr int kSize = kF32 ? 4 : 2, kVec = 16 / kSize, kPer = 4 / kSize;
  static constexpr int kTokens = kSpan / kSize, kRound = kWarps * kTokens;  // of a warp, of the CTA
  const char* base;
  int off, V;

  __device__ __forceinline__ float at(int t) const {
    if constexpr (kF32) return __ldg(reinterpret_cast<const float*>(base) + t);
    return __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(base) + t)) << 16);
  }
  __device__ __forceinline__ static int token(int c0, int i, int half) {
    return c0 + (static_cast<int>(threadIdx.x & 31) + 32 * i) * kPer + half;
  }
  // Starts the copy of the 16-byte pieces of tokens [c0, c0 + n); a piece at the row's edge by its tokens.
  __device__ __forceinline__ void copy(char* stage, long long c0, int n) const {
    const long long q0 = c0 * kSize - off, end = static_cast<long long>(V) * kSize;
    const int lane = threadIdx.x & 31;
    if (n == kTokens && q0 >= 0 && q0 + kSpan + 16 <= end) {
      const char* from = base + q0 + 16 * lane;
      const uint32_t to = smem_u32(stage) + 16 * lane;
#pragma unroll
      for (int i = 0; i < kSpan / 512; ++i) cp_async16(to + 512 * i, from + 512 * i, 16);
      if (off != 0 && lane == 0) cp_async16(to + kSpan, from + kSpan, 16);
      cp_async_commit();
      return;
    }
    const int pieces = n > 0 ? (off + n * kSize + 15) >> 4 : 0;
#pragma unroll 1
    for (int i = lane; i < pieces; i += 32) {
      const long long q = q0 + 16 * i;
      if (q >= 0 && q + 16 <= end) {
        cp_async16(smem_u32(stage + 16 * i), base + q, 16);
      } else {
#pragma unroll 1
        for (int e = 0; e < 16; e += kSize) {
          if (q + e < 0 || q + e >= end) continue;
          if constexpr (kF32) {
            *reinterpret_cast<float*>(stage + 16 * i + e) = *reinterpret_cast<const float*>(base + q + e);
          } else {
            *reinterpret_cast<uint16_t*>(stage + 16 * i + e) = *reinterpret_cast<const uint16_t*>(base + q + e);
          }
        }
      }
    }
    cp_async_commit();
  }
  __device__ __forceinline__ void read(const char* stage, uint32_t (&w)[kWords]) const {
    const uint32_t* from = reinterpret_cast<const uint32_t*>(stage + (off & ~3)) + (threadIdx.x & 31);
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = from[32 * i];
    if (!kF32 && (off & 2)) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = __funnelshift_r(w[i], from[32 * i + 1], 16);
    }
  }
  // -inf for the tokens behind the warp's first n.
  __device__ __forceinline__ static void cut(uint32_t (&w)[kWords], int n) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int t = token(0, i, 0);
      if (t >= n) w[i] = kF32 ? 0xff800000u : 0xff80ff80u;
      if (!kF32 && t + 1 == n) w[i] = (w[i] & 0xffffu) | 0xff800000u;
    }
  }
  __device__ __forceinline__ float from_stage(const char* stage, int t) const {
    if constexpr (kF32) return *reinterpret_cast<const float*>(stage + off + 4 * t);
    return __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(stage + off + 2 * t)) << 16);
  }
  __device__ __forceinline__ static uint64_t pair(uint32_t a, uint32_t b, int i) {  // two tokens of words a and b
    if constexpr (kF32) return static_cast<uint64_t>(b) << 32 | a;
    const uint32_t w = i ? b : a;
    return static_cast<uint64_t>(w & 0xffff0000u) << 32 | w << 16;
  }
  __device__ __forceinline__ static float value(uint32_t w, int half) {
    if constexpr (kF32) return __uint_as_float(w);
    return __uint_as_float(half ? w & 0xffff0000u : w << 16);
  }
  // of four words; NaN only if there is no number
  __device__ __forceinline__ static float largest(const uint32_t* w) {
    if constexpr (kF32) return fmaxf(fmaxf(value(w[0], 0), value(w[1], 0)), fmaxf(value(w[2], 0), value(w[3], 0)));
    const __nv_bfloat162* v = reinterpret_cast<const __nv_bfloat162*>(w);
    const __nv_bfloat162 m = __hmax2(__hmax2(v[0], v[1]), __hmax2(v[2], v[3]));
    return fmaxf(__bfloat162float(m.x), __bfloat162float(m.y));
  }
};

__device__ __forceinline__ uint64_t key_of(float x, int t) {
  return (static_cast<uint64_t>(ordered(x)) << 32) | ~static_cast<uint32_t>(t);
}

// More candidates than the buffer holds (runs of equal logits such as a mask's, rows in ascending order): tokens [begin, end)
// again, a step's worth at a time, against the `held` first keys of the buffer; every step's bar is its K-th key. Of a run of
// equal logits only the first step's pass it. Returns the keys that are held then, to all threads alike (sh.count may be
// counting the next round's by the time a thread looks).
template <bool kF32>
__device__ __noinline__ int select_again(const Row<kF32>& row, int begin, int end, Shared& sh, int held, int K) {
  if (threadIdx.x == 0) sh.count = held;
  __syncthreads();
  float bar = held == K ? from_ordered(static_cast<uint32_t>(sh.buf[K - 1] >> 32)) : -__int_as_float(0x7f800000);
#pragma unroll 1
  for (int done = 0; done < end - begin; done += kStep) {
#pragma unroll
    for (int i = 0; i < kStep / kThreads; ++i) {
      const int left = end - begin - done - i * kThreads - static_cast<int>(threadIdx.x);
      const int t = end - left;
      const float x = left > 0 ? row.at(t) : -__int_as_float(0x7f800000);
      if (x > bar) sh.buf[atomicAdd(&sh.count, 1)] = key_of(x, t);
    }
    __syncthreads();
    const int n = sh.count;
    __syncthreads();
    if (n > held && n >= K) {
      rank_buffer(sh, n, K);
      bar = from_ordered(static_cast<uint32_t>(sh.buf[K - 1] >> 32));
    }
    held = min(n, K);
  }
  return held;
}

// One CTA for a slice of a beam's tokens; a warp's spans come by themselves, the CTA meets at the rankings only.
template <bool kF32>
__global__ void __launch_bounds__(kThreads, 3) beam_scan_kernel(const __grid_constant__ BeamParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  using R = Row<kF32>;
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row_at = blockIdx.x / p.slices, slice = blockIdx.x - row_at * p.slices;
  const int b = row_at / p.W, w = row_at - b * p.W;
  const bool ended = p.finished != nullptr && p.finished[row_at] != 0;
  const float score = p.scores[row_at];
  if (ended || !(score > -__int_as_float(0x7f800000))) return;  // no candidate (-inf, NaN)
  R row;
  row.base = static_cast<const char*>(p.logits) + (b * p.stride_b + w * p.stride_w) * R::kSize;
  row.off = static_cast<int>(reinterpret_cast<uintptr_t>(row.base) & 15);
  row.V = p.V;
  const long long each = ((static_cast<long long>(p.V) + p.slices - 1) / p.slices + R::kVec - 1) / R::kVec * R::kVec;
  const int t_begin = static_cast<int>(min(slice * each, static_cast<long long>(p.V)));
  const int t_end = static_cast<int>(min(t_begin + each, static_cast<long long>(p.V)));
  const int K = p.K;
  // a round's first tokens are the CTA's first warp's; `left`: the tokens from this warp's of the round to the slice's end
  const int rounds = (t_end - t_begin) / R::kRound + ((t_end - t_begin) % R::kRound != 0);
  int left = t_end - t_begin - warp * R::kTokens;
  auto span = [&](int left) { return max(0, min(left, R::kTokens)); };
  if (tid == 0) sh.count = 0;
#pragma unroll
  for (int r = 0; r < kStages; ++r)
    row.copy(sh.stage[warp][r], static_cast<long long>(t_end) - left + r * R::kRound, span(left - r * R::kRound));
  const float neg_inf = -__int_as_float(0x7f800000);
  float m = neg_inf, sum = 0.f;
  // Logits above the bar may be among the K largest. Later tokens come behind equal earlier ones, so that a bar that
  // was ranked is passed by larger logits only.
  float bar = neg_inf;
  int held = 0, from = t_begin;  // since the last ranking
#pragma unroll 1
  for (int r = 0; r < rounds; ++r, left -= R::kRound) {
    char* stage = sh.stage[warp][r % kStages];
    const int n = span(left), c0 = t_end - left;
    uint32_t v[kWords];
    cp_async_wait<kStages - 1>();
    __syncwarp();
    row.read(stage, v);
    if (n < R::kTokens) R::cut(v, n);
    float top[kWords / 4];
#pragma unroll
    for (int g = 0; g < kWords / 4; ++g) top[g] = R::largest(v + 4 * g);
    const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    if (mx > m) {
      sum = m > neg_inf ? sum * ex2_approx((m - mx) * kLog2e) : sum;  // (a NaN stays)
      m = mx;
    }
    // the difference before its factor: what is close to the maximum, and weighs, is exact
    const float ref = m > neg_inf ? -m : 0.f;
    const uint64_t ref2 = pack2(ref, ref), log2e2 = pack2(kLog2e, kLog2e);
    uint64_t part[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < kWords; i += kF32 ? 2 : 1) {
      const uint64_t d = mul2(add2(kF32 ? R::pair(v[i], v[(i + 1) % kWords], 0) : R::pair(v[i], v[i], 0), ref2), log2e2);
      const int at = (kF32 ? i / 2 : i) & 1;
      part[at] = add2(part[at], pack2(ex2_approx(first(d)), ex2_approx(second(d))));
    }
    part[0] = add2(part[0], part[1]);
    sum += first(part[0]) + second(part[0]);

    if (r == 0) {
      const uint32_t lo = lower_bar(ordered(mx), K, sh.best32, &sh.found);
      // the next lower number (the one below +0 is not -0, its equal)
      bar = lo > 0 ? from_ordered(lo - (lo == 0x80000000u ? 2 : 1)) : neg_inf;
    }
    if (__any_sync(0xffffffffu, mx > bar)) {
      uint32_t hits = 0;
#pragma unroll
      for (int g = 0; g < kWords / 4; ++g) {
        if (!(top[g] > bar)) continue;
#pragma unroll
        for (int e = 4 * g * R::kPer; e < 4 * (g + 1) * R::kPer; ++e)
          hits |= R::value(v[e / R::kPer], e % R::kPer) > bar ? 1u << e : 0u;
      }
      int at = hits != 0 ? atomicAdd(&sh.count, __popc(hits)) : 0;
#pragma unroll 1
      for (; hits != 0; hits &= hits - 1, ++at) {
        const int e = __ffs(hits) - 1, t = R::token(0, e / R::kPer, e % R::kPer);
        if (at < kBuf) sh.buf[at] = key_of(row.from_stage(stage, t), c0 + t);
      }
    }
    __syncwarp();
    row.copy(stage, static_cast<long long>(c0) + kStages * R::kRound, span(left - kStages * R::kRound));

    if ((r + 1) % kRounds != 0 && r + 1 < rounds) continue;
    __syncthreads();
    const int count = sh.count;
    __syncthreads();
    const int to = r + 1 < rounds ? t_begin + (r + 1) * R::kRound : t_end;
    int got = count;
    if (count > kBuf) {
      got = select_again(row, from, to, sh, held, K);
    } else if (count > held && count >= K) {
      rank_buffer(sh, count, K);
    }
    if (got >= K) bar = from_ordered(static_cast<uint32_t>(sh.buf[K - 1] >> 32));
    held = min(got, K);
    from = to;
  }
  __syncthreads();
  // the slice's maximum, sum and keys
  float M = m;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  if (lane == 0) sh.part_m[warp] = M;
  const bool nan = __syncthreads_or(sum != sum);
#pragma unroll
  for (int i = 0; i < kWarps; ++i) M = fmaxf(M, sh.part_m[i]);
  // in units of 2^-unit from here: exact sums, in whatever order
  uint64_t s = m > neg_inf && !nan ? __float2ull_rn(ldexpf(sum * ex2_approx((m - M) * kLog2e), beam_unit(p.V))) : 0;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  if (lane == 0) sh.part_s[warp] = s;
  __syncthreads();
  const long long at = blockIdx.x;
  if (tid == 0) {
#pragma unroll
    for (int i = 1; i < kWarps; ++i) s += sh.part_s[i];
    p.part_sum[at] = nan ? kNoSum : s;
    p.part_max[at] = M;
  }
  const int n = min(sh.count, K);
  for (int i = tid; i < K; i += kThreads) p.part_keys[at * K + i] = i < n ? sh.buf[i] : 0;
}

// One CTA for a batch item. A candidate's value is an fp64 sum, of which an SM makes few: all get bounds in fp32 first, and
// only those that may be among the K have it made. These few are ranked by counting, or sorted if they are many
// (equal values).
__global__ void __launch_bounds__(kThreads) beam_pick_kernel(const __grid_constant__ BeamParams p) {
  extern __shared__ uint64_t dyn[];
  __shared__ alignas(16) uint32_t best[kThreads];
  __shared__ uint32_t found;
  __shared__ double shift[kBeamMaxW];  // score - ln of the sum, NaN: no candidate
  __shared__ float shift32[kBeamMaxW];
  __shared__ float largest[kBeamMaxW];
  __shared__ float end_score[kBeamMaxW];  // of a finished beam, else -inf
  __shared__ int survivors;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x, W = p.W, K = p.K, S = p.slices;
  const int n = W * S * K, P = power_of_two(n);
  uint64_t* const all = dyn;  // the candidates' keys
  uint64_t* const value = dyn + P;  // of those that are left, in order of value and place w * V + token
  uint32_t* const place = reinterpret_cast<uint32_t*>(dyn + 2 * P);
  uint32_t* const upper = place + P;  // the candidates' upper bounds
  const double none = __longlong_as_double(0x7ff8000000000000ll);
  const float neg_inf = -__int_as_float(0x7f800000);
  const int unit = beam_unit(p.V);
  if (tid == 0) survivors = 0;
  const uint64_t* const keys = p.part_keys + static_cast<long long>(b) * n;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  uint64_t key[kKeys];
#pragma unroll
  for (int i = 0; i < kKeys; ++i) key[i] = tid + i * kThreads < n ? keys[tid + i * kThreads] : 0;
  for (int w = warp; w < W; w += kWarps) {
    const int row = b * W + w;
    const float score = p.scores[row];
    const bool ended = p.finished != nullptr && p.finished[row] != 0;
    const float m = lane < S ? p.part_max[row * S + lane] : neg_inf;
    uint64_t s = lane < S ? p.part_sum[row * S + lane] : 0;
    if (!(score > neg_inf) || ended) {  // (its parts were not written)
      if (lane == 0) {
        shift[w] = none;
        shift32[w] = __int_as_float(0x7fc00000);
        end_score[w] = ended ? score : neg_inf;
      }
      continue;
    }
    const bool nan = __any_sync(0xffffffffu, s == kNoSum);
    float M = m;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    if (m < M) s = m > neg_inf ? __float2ull_rn(__ull2float_rn(s) * ex2_approx((m - M) * kLog2e)) : 0;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (lane == 0) {
      // ln s from a mantissa in [1, 2): within 2^-24 for its rounding and as much for logf; fp64 for the exponent's share
      const int e = 63 - __clzll(s);
      const float mantissa = ldexpf(__ull2float_rn(s), -e);
      // a sum of 0 (no number at all) or NaN leaves no candidate
      const double c = s != 0 && !nan ? static_cast<double>(score) - (logf(mantissa) + (e - unit) * 0.6931471805599453) : none;
      shift[w] = c;
      shift32[w] = static_cast<float>(c);
      largest[w] = M;
      end_score[w] = neg_inf;
    }
  }
  __syncthreads();
  const int per = S * K, w_step = kThreads / per, j_step = kThreads - w_step * per;
  int w = tid / per, j = tid - w * per;
  uint32_t top = 0;
  for (int i = tid; i < n;) {
#pragma unroll
    for (int u = 0; u < kKeys; ++u) {
      if (i < n) {
        uint32_t high = 0;
        const float c = shift32[w], end = end_score[w];
        const bool alive = c == c;
        if (alive ? key[u] != 0 : j == 0 && end > neg_inf) {
          // three roundings of at most 2^-24 of |v| + 2 |c| together; what is beyond the type's range is at its end
          const float x = from_ordered(static_cast<uint32_t>(key[u] >> 32));
          const float v = alive ? fminf(fmaxf((x - largest[w]) + c, -FLT_MAX), FLT_MAX) : end;
          const float slack = 0x1p-21f * (fabsf(v) + (alive ? fabsf(c) : 0.f));
          const uint32_t low = ordered(fmaxf(v - slack, -FLT_MAX));
          high = ordered(fminf(v + slack, FLT_MAX));
          top = max(top, low);
        }
        all[i] = key[u];
        upper[i] = high;
        i += kThreads;
        w += w_step;
        j += j_step;
        if (j >= per) {
          j -= per;
          ++w;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kKeys; ++u) key[u] = i + u * kThreads < n ? keys[i + u * kThreads] : 0;
  }
  const uint32_t bar = max(lower_bar(top, K, best, &found), 1u);
  for (int i = tid; i < n; i += kThreads)
    if (upper[i] >= bar) place[atomicAdd(&survivors, 1)] = i;
  __syncthreads();
  const int m = survivors;
  for (int i = tid; i < m; i += kThreads) {
    const int c_at = place[i], row = c_at / per;
    const uint64_t k = all[c_at];
    const double c = shift[row];
    const bool alive = c == c;
    // (the difference of the logits first: masks of the type's lowest value leave no room for the rest)
    const double x = static_cast<double>(from_ordered(static_cast<uint32_t>(k >> 32))) - static_cast<double>(largest[row]);
    const uint32_t token = alive ? ~static_cast<uint32_t>(k) : static_cast<uint32_t>(p.end_token);
    value[i] = ordered(alive ? x + c : static_cast<double>(end_score[row]));
    place[i] = static_cast<uint32_t>(row) * static_cast<uint32_t>(p.V) + token;
  }
  __syncthreads();
  const bool many = m >= kSortFrom;
  if (many) {
    const int padded = power_of_two(m);
    for (int i = m + tid; i < padded; i += kThreads) value[i] = 0;
    __syncthreads();
    sort_descending(padded, [&](int i, int j) {
      const uint64_t x = value[i], y = value[j];
      const uint32_t at = place[i], other = place[j];
      if (y > x || (y == x && other < at)) {
        value[i] = y;
        value[j] = x;
        place[i] = other;
        place[j] = at;
      }
    });
  }
  for (int i = tid; i < (many ? K : m); i += kThreads) {
    const uint64_t v = value[i];
    const uint32_t at = place[i];
    int r = i;
    if (!many) {
      r = 0;
#pragma unroll 4
      for (int j = 0; j < m; ++j) r += (value[j] > v) | ((value[j] == v) & (place[j] < at));
    }
    if (r < K) {
      const long long to = static_cast<long long>(b) * K + r;
      p.out_scores[to] = static_cast<float>(from_ordered(v));
      p.parents[to] = static_cast<int32_t>(at / static_cast<uint32_t>(p.V));
      p.tokens[to] = static_cast<int32_t>(at % static_cast<uint32_t>(p.V));
    }
  }
  for (int i = m + tid; i < K; i += kThreads) {
    const long long to = static_cast<long long>(b) * K + i;
    p.out_scores[to] = neg_inf;
    p.parents[to] = -1;
    p.tokens[to] = -1;
  }
}

}  // namespace

// Slices of a beam: enough CTAs for three on every SM, which is what their registers leave room for, each with at least a
// round of half its threads' loads, and no more candidates for an item's CTA than 2048 (or one slice's). More and smaller
// slices cost more rankings than they even out (64 x 8 x 131072 bf16: 33 us with one slice a beam, 35 with two, 38 with
// four; 16 x 8 x 50257 fp32: 20 us with three, 25 with eight).
void plan_beam(BeamParams& p, int sms) {
  const long long rows = static_cast<long long>(p.B) * p.W;
  long long s = rows > 0 ? (3ll * sms + rows - 1) / rows : 1;
  s = std::min(s, (p.V + static_cast<long long>(kThreads) * 8 - 1) / (kThreads * 8));
  s = std::min(s, 2048ll / (static_cast<long long>(p.W) * p.K));
  s = std::min<long long>(s, kMaxSlices);
  p.slices = static_cast<int>(std::max(1ll, s));
}

cudaError_t launch_beam(const BeamParams& p, bool f32, cudaStream_t stream) {
  const long long ctas = static_cast<long long>(p.B) * p.W * p.slices;
  if (f32)
    beam_scan_kernel<true><<<static_cast<unsigned>(ctas), kThreads, 0, stream>>>(p);
  else
    beam_scan_kernel<false><<<static_cast<unsigned>(ctas), kThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  size_t smem = 24;  // a candidate, twice; as many as the next power of two
  while (smem < 24ull * p.W * p.slices * p.K) smem *= 2;
  if (smem > 40000) {  // (always the largest: a call in another thread may set it at the same time)
    e = cudaFuncSetAttribute(beam_pick_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 24 * kBeamMaxWK);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.B));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, beam_pick_kernel, p);
}

}  // namespace svt
