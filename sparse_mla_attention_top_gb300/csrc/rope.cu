// Rotary positions, and the write of rotated rows into the paged latent cache.
//
// A pair (a, b) of a token's columns is turned by the angle pos * freq of its pair index and
// scaled by `amplitude`:  a' = A (a cos - b sin),  b' = A (a sin + b cos). The pairs are
// columns (2 i, 2 i + 1) ("interleaved") or (i, i + dim / 2) ("half"). The rotation's
// transpose (its gradient, and its inverse up to A^2) is the same with the angle negated.
//
// Angles: a frequency arrives in radians per position as fp64 and becomes a 64-bit fraction of
// a turn, so pos * fraction modulo 2^64 is the angle modulo a turn exactly, for any 32-bit
// position; only the reduced angle is rounded to fp32 (relative 2^-24) for sincospif. An fp32
// product would be off by 0.06 rad at position 10^6. The table of a CTA's tokens is computed
// once in shared memory and used by all of their heads.
//
// Bound: reading and writing the columns, and next to that the instructions that find them: a thread
// takes two units, of one or two 16-byte pieces each, loaded before the angles are known; six CTAs of
// 256 threads share an SM. 8192 tokens x 64 heads x 192 columns (64 rotated): 64.3 us, 6.3 TB/s, against
// 63.4 for a plain copy of them (one piece a unit: 74 us; the quarters of a turn taken off in integers, for
// a smaller angle to round: 65.2). Rows that do not start on 16-byte boundaries (or dims that do not split
// into 16-byte pieces) take the same kernel on single pairs.
#include <cuda_bf16.h>

#include <cstdint>
#include <type_traits>

#include "device.cuh"
#include "internal.h"

namespace svt {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeUnroll = 2;   // units a thread loads at once
constexpr int kRopeCtas = 6;     // resident CTAs per SM (40 registers a thread)
constexpr int kRopeBatches = 1;  // batches of a full CTA

// The angle of position `pos` at `freq` radians per position, in half turns in [-1, 1). The fraction
// of a turn, freq / 2 pi modulo 1 in units of 2^-64, comes from the double's 53-bit mantissa times
// 2^64 / 2 pi in integers (an SM runs two lanes of fp64 a cycle), off by at most (|freq| + 1) 2^-64 turns.
// No frequency (NaN, infinite, or of 2^52 and above, whose fraction of a turn these bits do not hold): NaN.
__device__ __forceinline__ float half_turns(int32_t pos, double freq) {
  const unsigned long long bits = static_cast<unsigned long long>(__double_as_longlong(freq));
  const int e = static_cast<int>((bits >> 52) & 0x7FF);
  const unsigned long long m = (bits & 0xFFFFFFFFFFFFFull) | 0x10000000000000ull;
  const unsigned long long k = 2935890503282001226ull;  // 2^64 / (2 pi)
  const unsigned long long lo = m * k, hi = __umul64hi(m, k);
  const int s = 1075 - e;  // freq = m 2^-s
  if (s <= 0) return __uint_as_float(0x7FC00000u);
  unsigned long long turn = 0;
  if (s > 0 && s < 64) turn = (lo >> s) | (hi << (64 - s));
  else if (s >= 64 && s < 128) turn = hi >> (s - 64);  // (further right there is nothing left)
  if (bits >> 63) turn = 0ull - turn;
  const long long a = static_cast<long long>(static_cast<unsigned long long>(static_cast<long long>(pos)) * turn);
  return __ll2float_rn(a) * 1.0842021724855044e-19f;  // 2^-63
}

// n / d for 0 <= n < 2^16, 1 <= d < 2^16, with m = ceil(2^32 / d) (d = 1: m = 0 marks it).
__device__ __forceinline__ uint32_t fast_div(uint32_t n, uint32_t m) { return m == 0u ? n : __umulhi(n, m); }

template <typename E>
__device__ __forceinline__ float to_f32(E v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ float to_f32<uint16_t>(uint16_t v) {
  return __uint_as_float(static_cast<uint32_t>(v) << 16);
}
template <typename E>
__device__ __forceinline__ E from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ uint16_t from_f32<uint16_t>(float v) {
  return static_cast<uint16_t>(pack_bf16x2(v, 0.f) & 0xFFFFu);
}

__device__ __forceinline__ void unpack(const uint4& v, float (&f)[8], uint16_t*) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[4], float*) {
  f[0] = __uint_as_float(v.x);
  f[1] = __uint_as_float(v.y);
  f[2] = __uint_as_float(v.z);
  f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ uint4 pack(const float (&f)[8], uint16_t*) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ uint4 pack(const float (&f)[4], float*) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

// Rows blk * p.rows_per_cta .. of the [T * H] rows. E: uint16_t (bf16 bits) or float. kVec: 16-byte
// units, else single pairs and single copied columns. kHalf: pairs (i, i + dim / 2).
template <typename E, bool kVec, bool kHalf>
__device__ __forceinline__ void rope_rows(const RopeParams& p, long long blk, float2* table) {
  constexpr int kE = kVec ? 16 / static_cast<int>(sizeof(E)) : 1;  // elements of a unit (of each half)
  const int tid = threadIdx.x;
  const long long row0 = blk * p.rows_per_cta;
  const long long total = static_cast<long long>(p.T) * p.H;
  const int rows = static_cast<int>(total - row0 < p.rows_per_cta ? total - row0 : p.rows_per_cta);
  const long long t0 = row0 / p.H;
  const uint32_t h0 = static_cast<uint32_t>(row0 - t0 * p.H);
  const int tokens = static_cast<int>((h0 + rows - 1) / p.H) + 1;
  const int items = rows * p.units;
  const E* x = static_cast<const E*>(p.x);
  E* out = static_cast<E*>(p.out);
  const int pairs = p.dim / 2;

  using Reg = typename std::conditional<kVec, uint4, E>::type;
  struct Batch {
    Reg a[kRopeUnroll], b[kRopeUnroll];
    int unit[kRopeUnroll], tl[kRopeUnroll];
    long long dst[kRopeUnroll];
  };
  auto load = [&](Batch& q, int base) {
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      const int it = base + u * kRopeThreads + tid;
      q.unit[u] = -1;
      if (it < items) {
        const uint32_t r = fast_div(it, p.magic_units);
        const int un = it - static_cast<int>(r) * p.units;
        const uint32_t hr = h0 + r;
        const uint32_t t = fast_div(hr, p.magic_h);
        const uint32_t h = hr - t * p.H;
        // unit order: the rotated units first, then the copied ones
        int col;
        if (un < p.rot_units) {
          col = p.offset + un * (kVec || kHalf ? kE : 2);
        } else {
          col = (un - p.rot_units) * p.copy_cols;
          if (col >= p.offset) col += p.dim;
        }
        const E* src = x + (t0 + t) * p.x_stride_t + h * p.x_stride_h + col;
        q.dst[u] = (t0 + t) * p.out_stride_t + h * p.out_stride_h + col;
        q.unit[u] = un;
        q.tl[u] = static_cast<int>(t);
        q.a[u] = *reinterpret_cast<const Reg*>(src);
        if (un < p.rot_units) {
          if (kHalf) q.b[u] = *reinterpret_cast<const Reg*>(src + pairs);
          else if (!kVec) q.b[u] = *reinterpret_cast<const Reg*>(src + 1);
        } else if (p.copy_cols > kE) {
          q.b[u] = *reinterpret_cast<const Reg*>(src + kE);
        }
      }
    }
  };
  auto turn = [&](const Batch& q) {
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      if (q.unit[u] < 0) continue;
      E* dst = out + q.dst[u];
      if (q.unit[u] >= p.rot_units) {
        *reinterpret_cast<Reg*>(dst) = q.a[u];
        if (p.copy_cols > kE) *reinterpret_cast<Reg*>(dst + kE) = q.b[u];
        continue;
      }
      const float2* cs = table + q.tl[u] * pairs;
      if constexpr (!kVec) {
        const float2 w = cs[q.unit[u]];
        const float fa = to_f32<E>(q.a[u]), fb = to_f32<E>(q.b[u]);
        dst[0] = from_f32<E>(fa * w.x - fb * w.y);
        dst[kHalf ? pairs : 1] = from_f32<E>(fa * w.y + fb * w.x);
      } else if constexpr (kHalf) {
        float fa[kE], fb[kE], ra[kE], rb[kE];
        unpack(q.a[u], fa, static_cast<E*>(nullptr));
        unpack(q.b[u], fb, static_cast<E*>(nullptr));
#pragma unroll
        for (int i = 0; i < kE; ++i) {
          const float2 w = cs[q.unit[u] * kE + i];
          ra[i] = fa[i] * w.x - fb[i] * w.y;
          rb[i] = fa[i] * w.y + fb[i] * w.x;
        }
        *reinterpret_cast<uint4*>(dst) = pack(ra, static_cast<E*>(nullptr));
        *reinterpret_cast<uint4*>(dst + pairs) = pack(rb, static_cast<E*>(nullptr));
      } else {
        float f[kE], r[kE];
        unpack(q.a[u], f, static_cast<E*>(nullptr));
#pragma unroll
        for (int i = 0; i < kE; i += 2) {
          const float2 w = cs[(q.unit[u] * kE + i) / 2];
          r[i] = f[i] * w.x - f[i + 1] * w.y;
          r[i + 1] = f[i] * w.y + f[i + 1] * w.x;
        }
        *reinterpret_cast<uint4*>(dst) = pack(r, static_cast<E*>(nullptr));
      }
    }
  };
  constexpr int kStep = kRopeThreads * kRopeUnroll;
  Batch q0;
  load(q0, 0);
  for (int i = tid; i < tokens * pairs; i += kRopeThreads) {
    const int t = i / pairs;
    float s, c;
    sincospif(half_turns(p.positions[t0 + t], p.freqs[i - t * pairs]), &s, &c);
    table[i] = make_float2(c * p.amplitude, s * p.amplitude * p.sign);
  }
  __syncthreads();
  for (int base = 0;; load(q0, base)) {
    turn(q0);
    base += kStep;
    if (base >= items) break;
  }
}

template <typename E, bool kVec, bool kHalf>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_kernel(const RopeParams p) {
  extern __shared__ float2 table[];
  rope_rows<E, kVec, kHalf>(p, blockIdx.x, table);
}

// One warp writes one cache row: lane l holds latent channels 16 l .. 16 l + 15 and rotates one
// of the 32 rope pairs. e4m3 rows: the four blocks of 128 channels are eight lanes each; a
// block's scale is its largest magnitude / 448 (1 for a block of zeros) and each code the e4m3
// nearest to value / scale, both in IEEE fp32 division, so that a code is the same wherever it
// is computed.
template <bool kF8, bool kHalf>
__device__ __forceinline__ void append_row(const AppendParams& p, int t) {
  const int lane = threadIdx.x & 31;
  const int slot = p.slots[t];
  if (slot < 0) return;
  if (slot >= p.num_slots) {
    if (lane == 0) atomicOr(p.status, SVT_DEV_ERR_INDEX_RANGE);
    return;
  }
  const uint16_t* lat = p.latent + t * p.latent_stride;
  const uint16_t* kr = p.k_rope + t * p.k_rope_stride;
  uint8_t* row = p.kv + slot * p.row_stride;
  const int ia = kHalf ? lane : 2 * lane, ib = kHalf ? lane + 32 : 2 * lane + 1;
  const uint4 v0 = __ldg(reinterpret_cast<const uint4*>(lat) + 2 * lane);
  const uint4 v1 = __ldg(reinterpret_cast<const uint4*>(lat) + 2 * lane + 1);
  const float fa = to_f32<uint16_t>(__ldg(kr + ia)), fb = to_f32<uint16_t>(__ldg(kr + ib));
  float s, c;
  sincospif(half_turns(p.positions[t], p.freqs[lane]), &s, &c);
  s *= p.amplitude;
  c *= p.amplitude;
  const float ra = fa * c - fb * s, rb = fa * s + fb * c;
  uint16_t* rope_dst;
  bool beyond = false;
  if constexpr (kF8) {
    float f[16];
    {
      float g[8];
      unpack(v0, g, static_cast<uint16_t*>(nullptr));
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = g[i];
      unpack(v1, g, static_cast<uint16_t*>(nullptr));
#pragma unroll
      for (int i = 0; i < 8; ++i) f[8 + i] = g[i];
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      amax = fmaxf(amax, fabsf(f[i]));
      beyond |= !(fabsf(f[i]) <= 65504.f);  // also NaN: not a value the e4m3 cache can hold
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float scale = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
    uint32_t codes[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint16_t lo, hi;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
          : "=h"(lo)
          : "f"(__fdiv_rn(f[4 * i + 1], scale)), "f"(__fdiv_rn(f[4 * i], scale)));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
          : "=h"(hi)
          : "f"(__fdiv_rn(f[4 * i + 3], scale)), "f"(__fdiv_rn(f[4 * i + 2], scale)));
      codes[i] = static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
    }
    reinterpret_cast<uint4*>(row)[lane] = make_uint4(codes[0], codes[1], codes[2], codes[3]);
    if ((lane & 7) == 0) reinterpret_cast<float*>(row + kVdim)[lane >> 3] = scale;
    rope_dst = reinterpret_cast<uint16_t*>(row + kVdim + 16);
  } else {
    reinterpret_cast<uint4*>(row)[2 * lane] = v0;
    reinterpret_cast<uint4*>(row)[2 * lane + 1] = v1;
    rope_dst = reinterpret_cast<uint16_t*>(row) + kVdim;
  }
  const uint32_t packed = pack_bf16x2(ra, rb);
  if constexpr (kF8) beyond |= bf16x2_beyond_f16(packed);
  if constexpr (kHalf) {
    rope_dst[lane] = static_cast<uint16_t>(packed & 0xFFFFu);
    rope_dst[lane + 32] = static_cast<uint16_t>(packed >> 16);
  } else {
    reinterpret_cast<uint32_t*>(rope_dst)[lane] = packed;
  }
  if constexpr (kF8) {
    if (__any_sync(0xffffffffu, beyond) && lane == 0) atomicOr(p.status, SVT_DEV_ERR_FP8_RANGE);
  }
}

// CTAs below row_ctas write cache rows (a warp each); the others rotate q's rope columns, so a
// decode step's two writes are one launch (128 e4m3 rows and 64 heads: 4.2 us, the launch; 8192 bf16
// rows and 16 heads: 12.5 us, of which the bytes are 7.7 and the launch 4.1).
template <bool kF8, bool kHalf, bool kVec>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) append_kernel(const AppendParams p, const RopeParams q) {
  extern __shared__ float2 table[];
  if (static_cast<int>(blockIdx.x) < p.row_ctas) {
    const int t = blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
    if (t < p.T) append_row<kF8, kHalf>(p, t);
    return;
  }
  rope_rows<uint16_t, kVec, kHalf>(q, blockIdx.x - p.row_ctas, table);
}

uint32_t magic_of(int d) { return d <= 1 ? 0u : static_cast<uint32_t>(((1ull << 32) + d - 1) / d); }

// Fills the launch fields (units, rows per CTA) and says whether 16-byte units apply; returns the
// CTAs. rows_per_cta keeps a CTA's items, tokens and table inside the limits of fast_div and of
// 32 KB of table.
long long plan_rope(RopeParams& p, int elem, bool half, int sms, bool* vec) {
  const int e = 16 / elem;
  auto al = [&](long long v) { return v % e == 0; };
  *vec = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && reinterpret_cast<uintptr_t>(p.out) % 16 == 0 &&
         al(p.x_stride_t) && al(p.x_stride_h) && al(p.out_stride_t) && al(p.out_stride_h) && al(p.offset) && al(p.D) &&
         al(half ? p.dim / 2 : p.dim);
  const bool copy = p.x != p.out;
  p.rot_units = *vec ? (half ? p.dim / 2 : p.dim) / e : p.dim / 2;
  // copied columns go two 16-byte pieces a unit where both sides of the rotated ones allow it
  p.copy_cols = *vec ? (p.offset % (2 * e) == 0 && (p.D - p.dim - p.offset) % (2 * e) == 0 ? 2 * e : e) : 1;
  p.units = p.rot_units + (copy ? (p.D - p.dim) / p.copy_cols : 0);
  const long long total = static_cast<long long>(p.T) * p.H;
  // a full CTA takes one batch; when that leaves SMs idle, fewer rows
  long long rows = kRopeThreads * kRopeUnroll * kRopeBatches / p.units;
  const long long fill = (total + 2ll * sms - 1) / (2ll * sms);
  if (rows > fill) rows = fill;
  const long long by_table = (4096 / (p.dim / 2) - 1) * static_cast<long long>(p.H);  // tokens spanned <= rows / H + 2
  if (rows > by_table) rows = by_table;
  if (rows < 1) rows = 1;
  p.rows_per_cta = static_cast<int>(rows);
  p.magic_units = magic_of(p.units);
  p.magic_h = magic_of(p.H);
  return (total + rows - 1) / rows;
}

size_t table_bytes(const RopeParams& p) {
  const long long tokens = (static_cast<long long>(p.rows_per_cta) + p.H - 2) / p.H + 1;
  return static_cast<size_t>(tokens) * (p.dim / 2) * sizeof(float2);
}

cudaError_t current_sms(int* sms) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

template <typename E>
cudaError_t launch_rope_e(RopeParams p, bool half, int sms, cudaStream_t stream) {
  bool vec = false;
  const long long ctas = plan_rope(p, static_cast<int>(sizeof(E)), half, sms, &vec);
  const unsigned grid = static_cast<unsigned>(ctas);
  const size_t smem = table_bytes(p);
  if (vec && half) rope_kernel<E, true, true><<<grid, kRopeThreads, smem, stream>>>(p);
  else if (vec) rope_kernel<E, true, false><<<grid, kRopeThreads, smem, stream>>>(p);
  else if (half) rope_kernel<E, false, true><<<grid, kRopeThreads, smem, stream>>>(p);
  else rope_kernel<E, false, false><<<grid, kRopeThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, bool f32, bool half, cudaStream_t stream) {
  if (p.T == 0 || p.H == 0) return cudaSuccess;
  int sms = 0;
  const cudaError_t e = current_sms(&sms);
  if (e != cudaSuccess) return e;
  return f32 ? launch_rope_e<float>(p, half, sms, stream) : launch_rope_e<uint16_t>(p, half, sms, stream);
}

cudaError_t launch_append(const AppendParams& append, const RopeParams& rope, bool f8, bool half, cudaStream_t stream) {
  if (append.T == 0) return cudaSuccess;
  int sms = 0;
  const cudaError_t e = current_sms(&sms);
  if (e != cudaSuccess) return e;
  AppendParams p = append;
  RopeParams q = rope;
  constexpr int kWarps = kRopeThreads / 32;
  p.row_ctas = (p.T + kWarps - 1) / kWarps;
  long long ctas = p.row_ctas;
  bool vec = true;
  size_t smem = 0;
  if (q.H > 0) {
    ctas += plan_rope(q, 2, half, sms, &vec);
    smem = table_bytes(q);
  }
  const unsigned grid = static_cast<unsigned>(ctas);
  auto go = [&](auto f, auto h, auto v) {
    append_kernel<decltype(f)::value, decltype(h)::value, decltype(v)::value><<<grid, kRopeThreads, smem, stream>>>(p, q);
  };
  using T = std::true_type;
  using F = std::false_type;
  if (f8) {
    if (half) vec ? go(T{}, T{}, T{}) : go(T{}, T{}, F{});
    else vec ? go(T{}, F{}, T{}) : go(T{}, F{}, F{});
  } else {
    if (half) vec ? go(F{}, T{}, T{}) : go(F{}, T{}, F{});
    else vec ? go(F{}, F{}, T{}) : go(F{}, F{}, F{});
  }
  return cudaGetLastError();
}

}  // namespace svt
