// The backward pass of sparse MLA attention. With K the listed rows (576 columns), V their first
// 512, and the forward's out and lse, the probabilities are recomputed:
//   S = scale q K^T,  P = exp(S - lse),  delta = sum_c dout out - dlse,
//   dS = P (dout V^T - delta) scale,  dq = dS K,  dK = dS^T q,  dV = P^T dout,
// and a cache row's gradient is the sum of dK (+ dV on the latent columns) over the lists that
// hold it. sum over heads of P is each entry's attention weight.
//
// Three kernels. prepare resolves the lists, forms delta and zeroes the cache rows' sums. The main
// kernel walks (row-set, 64-entry tile) pairs, a row-set being up to 64 heads of one query, one
// persistent CTA per SM with an equal share of all tiles (stream-K). finish joins the dq of row-sets
// cut between CTAs (fp32, in a fixed order) and rounds the cache rows' sums to bf16.
//
// Main kernel, per tile, on tcgen05 with fp32 accumulators in tensor memory (e = entry, r = head
// row, c = channel; the contractions' operands are the tiles as they lie, read K- or MN-major):
//   1. [S^T | dP^T][e, r]  = K [q | dout]^T     one 64 x 128 product: q and dout lie interleaved
//                                               in 64-channel blocks, so both share the reads of K
//   2. dq^T[c, r]         += K^T dS             stays in tensor memory over the row-set's tiles
//   3. dKV^T[c, e]         = q^T dS + dout^T P  128 channels at a time; each block leaves for
//                                               fp32 atomic additions as it is done
// P and dS are the only values rounded before the end (to bf16, as operands).
//
// Warps: 8 softmax (S^T, dP^T -> P, dS; two of the five dKV^T blocks -> additions; dq out), 8 scatter
// (the other blocks -> additions), 3 gather (cp.async, rows zero-filled where there is none), 1 that
// issues the MMAs. q and dout of 64 heads (136 KB) and one 72 KB tile of rows fill shared memory, so the
// next tile is gathered while step 3 runs. Calls of at most 32 heads keep q and dout in half of that and
// two tiles of rows (Lay<32>).
//
// What bounds it: of 64 heads, a tile takes about 4.9 us (9300 cycles). The chain product 1 (2200 cycles) -> softmax
// (1500) -> product 2 (900) -> product 3 (2300) is 7800 with the additions left out, and the additions
// alone, 147 KB a tile, 7200 at the 6 TB/s that the L2 takes; they meet in the few buffers between.
// 1024 queries x 64 heads x 2048 entries: 1.07 ms (1.02 in this kernel), 690 TFLOP/s, 4.8 GB of additions.
// Of 32 heads or fewer, a tile takes 4.3 us: the additions beside the reads of the rows (4.2 us at the
// measured 5.4 TB/s); 333 x 16 x 2048: 338 us, with the schedule of 64 heads 369.
#include <math_constants.h>

#include <cstdint>
#include <type_traits>

#include "device.cuh"
#include "internal.h"
#include "resolve_entry.cuh"

namespace svt {

namespace {

constexpr int kRows = 64;     // heads of a row-set
constexpr int kEntries = 64;  // list entries of a tile
constexpr float kLog2e = 1.4426950408889634f;

constexpr uint32_t kBlk = 8192;  // 64 x 64 bf16 in the 128-byte swizzle
struct Misc {
  int slot[4][kEntries];  // the tile's cache rows, a ring: scatter may trail the gather by two tiles
  float weight[2][kEntries];
  uint64_t bars[22];
  uint32_t tmem;
  int abort_flag;
};

// barriers
enum { kBarKvFull, kBarKvFree = kBarKvFull + 2, kBarS = kBarKvFree + 2, kBarP, kBarPFree, kBarSeg, kBarDq, kBarDqFree,
       kBarBlock, kBarBlockFree = kBarBlock + 5, kBarDone = kBarBlockFree + 5, kNumBars };
static_assert(kNumBars <= 22, "barriers");

// Shared memory (bytes from a 1024-byte boundary) and tensor memory (columns) for row-sets of R heads,
// R = 64 or 32. Tensor memory: dq^T in five blocks of R (channels 128 mb .. +127, then the 64 rope ones),
// S^T, dP^T, blocks of dKV^T.
template <int R>
struct Lay;

// R = 64: q0 dout0 q1 dout1 .. q7 dout7 q8, one tile of rows. The S^T columns hold blocks 0 and 3 of dKV^T
// and the dP^T columns block 1 once the softmax has read them; the others go to the last 64.
template <>
struct Lay<64> {
  static constexpr uint32_t kQBlocks = 17, kKvBufs = 1;
  static constexpr uint32_t kTmS = 320, kTmDp = kTmS + 64;
  static __device__ constexpr uint32_t block(int cb) { return cb == 1 ? kTmDp : (cb == 2 || cb == 4 ? kTmDp + 64 : kTmS); }
};
// R = 32: a block's rows are 32 heads of q, then the same of dout (the last block: rows 32 .. 63 unused),
// which leaves room for a second tile of rows; and blocks 0 to 3 have columns of their own (block 4: block
// 1's, as the same warps drain both), so that a tile's additions run beside the next tile's products.
template <>
struct Lay<32> {
  static constexpr uint32_t kQBlocks = 9, kKvBufs = 2;
  static constexpr uint32_t kTmS = 160, kTmDp = kTmS + 32;
  static __device__ constexpr uint32_t block(int cb) { return kTmS + 64 + 64 * (cb == 4 ? 1 : cb); }
};
constexpr uint32_t kTmDq = 0, kOffQ = 0;
template <int R>
constexpr uint32_t kOffKv = Lay<R>::kQBlocks* kBlk;  // 9 blocks a tile
template <int R>
constexpr uint32_t kOffP = kOffKv<R> + Lay<R>::kKvBufs * 9 * kBlk;  // 64 entries x R heads
template <int R>
constexpr uint32_t kOffDs = kOffP<R> + 128 * R;
template <int R>
constexpr uint32_t kOffMisc = kOffDs<R> + 128 * R;
template <int R>
constexpr uint32_t kSmem = kOffMisc<R> + sizeof(Misc) + 1024;
static_assert(kSmem<64> <= 232448 && kSmem<32> <= 232448, "backward shared memory");

// The 16-byte chunk of a row of 64 bytes in the 64-byte swizzle.
__device__ __forceinline__ uint32_t sw64_offset(uint32_t row, uint32_t chunk) {
  return row * 64u + ((chunk ^ ((row >> 1) & 3u)) << 4);
}

constexpr int kSoftWarps = 8, kScatWarps = 8, kFillWarps = 3;
constexpr int kScatWarp0 = kSoftWarps, kFillWarp0 = kScatWarp0 + kScatWarps, kMmaWarp = kFillWarp0 + kFillWarps;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr int kFillThreads = 32 * kFillWarps;
constexpr int kFillStep = kFillThreads / 8;                       // rows filled at once, 8 threads each
constexpr int kFillRows = (kEntries + kFillStep - 1) / kFillStep;  // rows per thread

template <int R>
constexpr uint32_t kIdescS = idesc_f32acc(64, 2 * R, 0, 0, kFmtBf16);
template <int R>
constexpr uint32_t kIdescSRope = idesc_f32acc(64, R, 0, 0, kFmtBf16);
template <int R>
constexpr uint32_t kIdescDq = idesc_f32acc(128, R, 1, 1, kFmtBf16);
template <int R>
constexpr uint32_t kIdescDqRope = idesc_f32acc(64, R, 1, 1, kFmtBf16);
constexpr uint32_t kIdescKv = idesc_f32acc(128, 64, 1, 0, kFmtBf16);
constexpr uint32_t kIdescKvRope = idesc_f32acc(64, 64, 1, 0, kFmtBf16);

// Programmatic dependent launch: lets the next kernel of the stream begin; waits until the last one has
// ended and its writes are visible.
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The part of one row-set that this CTA walks: live tiles j0 .. j1 - 1 (none when j0 >= j1). CTAs whose
// lists are in step add to the same rows at a time, which costs nothing that shows (1024 x 64 x 2048, every
// list the same ascending one 1068 us, independent lists 1067; beginning each CTA at another place of its
// list took 2 to 5 us more in both).
struct Seg {
  int rowset, t;
  long long base;  // first of its rows in [T * H, ...]
  int nvalid;
  int j0, j1;
  bool whole;      // this CTA has every tile of the row-set
  int part;        // where its dq goes otherwise
};

// Walks the segments of CTA blockIdx.x; every role runs its own copy.
struct SegIter {
  const BackwardParams& p;
  long long pos, hi;
  __device__ explicit SegIter(const BackwardParams& q) : p(q) {
    pos = streamk_lo(blockIdx.x, p.total_tiles, p.num_ctas);
    hi = streamk_lo(blockIdx.x + 1ll, p.total_tiles, p.num_ctas);
  }
  __device__ bool next(Seg& s) {
    if (pos >= hi) return false;
    const int r = static_cast<int>(pos / p.tiles);
    const long long first = static_cast<long long>(r) * p.tiles;
    const long long end = first + p.tiles < hi ? first + p.tiles : hi;
    s.rowset = r;
    s.t = r / p.hchunks;
    const int chunk = r - s.t * p.hchunks;
    s.base = static_cast<long long>(s.t) * p.H + chunk * kRows;
    s.nvalid = min(kRows, p.H - chunk * kRows);
    int reach = 0;
    for (int i = 0; i < p.chunks; ++i) reach = max(reach, p.live_len[static_cast<long long>(s.t) * p.chunks + i]);
    const int live = (reach + kEntries - 1) / kEntries;
    s.j0 = static_cast<int>(pos - first);
    s.j1 = min(static_cast<int>(end - first), live);
    s.whole = pos == first && end == first + p.tiles;
    s.part = static_cast<int>(streamk_part_slot(blockIdx.x, first, p.total_tiles, p.num_ctas));
    pos = end;
    return true;
  }
};

template <int R>
__device__ __forceinline__ void gather_role(const BackwardParams& p, uint8_t* smem, Misc* misc, uint32_t bars,
                                            const WaitCtl& wc) {
  const int tid = static_cast<int>(threadIdx.x) - 32 * kFillWarp0;
  const uint32_t base = smem_u32(smem);
  const int c = tid & 7, r0 = tid >> 3;  // 16-byte chunk of a block, first row
  auto bar = [&](int i) -> uint32_t { return bars + 8u * static_cast<uint32_t>(i); };
  uint32_t g = 0, segs = 0;
  SegIter it(p);
  Seg s;
  while (it.next(s)) {
    if (s.j0 >= s.j1) continue;
    // the last segment's products are done: q and dout may be replaced
    if (segs > 0 && !mbar_wait(bar(kBarSeg), (segs - 1) & 1, wc)) return;
    for (int r = r0; r < R; r += kFillStep) {
      const uint32_t ok = r < s.nvalid ? 16u : 0u;
      const uint16_t* q = p.q + (s.base + (ok ? r : 0)) * kRow + c * 8;
      const uint16_t* d = p.dout + (s.base + (ok ? r : 0)) * kVdim + c * 8;
      const uint32_t at = base + kOffQ + sw128_offset(r, c);
      constexpr uint32_t kStep = (Lay<R>::kQBlocks - 1) / 8 * kBlk;
      constexpr uint32_t kDout = R == 64 ? kBlk : R * 128;  // from a row of q to dout's
#pragma unroll
      for (int kb = 0; kb < 8; ++kb) {
        cp_async16(at + kb * kStep, q + 64 * kb, ok);
        cp_async16(at + kb * kStep + kDout, d + 64 * kb, ok);
      }
      cp_async16(at + 8 * kStep, q + 512, ok);
    }
    const int32_t* list = p.slots + static_cast<long long>(s.t) * p.K;
    int slot[kFillRows];
    auto load_slots = [&](int j) {
#pragma unroll
      for (int i = 0; i < kFillRows; ++i) {
        const int r = r0 + kFillStep * i, k = j * kEntries + r;
        slot[i] = r < kEntries && k < p.K ? __ldg(list + k) : -1;
      }
    };
    load_slots(s.j0);
    for (int j = s.j0; j < s.j1; ++j, ++g) {
      constexpr uint32_t kBufs = Lay<R>::kKvBufs;
      const uint32_t buf = g % kBufs;
      if (g >= kBufs && !mbar_wait(bar(kBarKvFree + static_cast<int>(buf)), (g / kBufs - 1) & 1, wc)) {
        cp_async_wait_all();  // none in flight when the CTA ends
        return;
      }
#pragma unroll
      for (int i = 0; i < kFillRows; ++i) {
        const int r = r0 + kFillStep * i;
        if (r >= kEntries) break;
        const uint32_t ok = slot[i] >= 0 ? 16u : 0u;
        const uint8_t* row = p.kv + (ok ? slot[i] * p.row_stride : 0) + c * 16;
        const uint32_t at = base + kOffKv<R> + buf * 9 * kBlk + sw128_offset(r, c);
#pragma unroll
        for (int kb = 0; kb < 9; ++kb) cp_async16(at + kb * kBlk, row + 128 * kb, ok);
        if (c == 0) misc->slot[g & 3][r] = slot[i];
      }
      if (j + 1 < s.j1) load_slots(j + 1);
      cp_async_wait_all();
      fence_proxy_async_smem();  // the rows (generic proxy) -> MMA operand reads
      if (!(g == 0 && (p.fault & kFaultWithholdFirstFill))) mbar_arrive(bar(kBarKvFull + static_cast<int>(buf)));
    }
    ++segs;
  }
}

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// Four MMAs of K = 16 each, or the first `steps` of them: a and b are the first one's descriptors,
// which advance by kA and kB bytes.
template <uint32_t kIdesc, uint32_t kA, uint32_t kB>
__device__ __forceinline__ void umma_x4(uint32_t d, uint64_t a, uint64_t b, bool accumulate, int steps = 4) {
#pragma unroll
  for (int ks = 0; ks < 4; ++ks)
    if (ks < steps) umma_f16(d, a + ((ks * kA) >> 4), b + ((ks * kB) >> 4), kIdesc, ks > 0 || accumulate);
}

// The one thread that issues the MMAs. Per tile: dq (which frees the rows' tile), four blocks of dKV
// while the next rows land, the next tile's S^T and dP^T, the last block. The issue has to keep up
// with products of 32 to 64 cycles: one elected lane of a uniform warp (a lane chosen by its number:
// 70 cycles an MMA, elected: 45), descriptors that advance by constants, loops of a few MMAs.
__device__ __forceinline__ void mma_role64(const BackwardParams& p, uint8_t* smem, uint32_t tmem, uint32_t bars,
                                           const WaitCtl& wc) {
  using L = Lay<64>;
  const uint32_t base = smem_u32(smem);
  const uint64_t q_k = smem_desc_sw128(base + kOffQ, 16, 1024), q_mn = smem_desc_sw128(base + kOffQ, 2 * kBlk, 1024);
  const uint64_t kv_k = smem_desc_sw128(base + kOffKv<64>, 16, 1024), kv_mn = smem_desc_sw128(base + kOffKv<64>, kBlk, 1024);
  const uint64_t p_k = smem_desc_sw128(base + kOffP<64>, 16, 1024), ds_k = smem_desc_sw128(base + kOffDs<64>, 16, 1024);
  const uint64_t ds_mn = smem_desc_sw128(base + kOffDs<64>, kBlk, 1024);
  auto bar = [&](int i) -> uint32_t { return bars + 8u * static_cast<uint32_t>(i); };
  uint32_t segs = 0;
  auto scores = [&](uint32_t g) -> bool {
    // the S^T and dP^T columns last held the previous tile's blocks 3 and 1
    if (!mbar_wait(bar(kBarKvFull), g & 1, wc)) return false;
    if (g > 0 && !(mbar_wait(bar(kBarBlockFree + 1), (g - 1) & 1, wc) &&
                   mbar_wait(bar(kBarBlockFree + 3), (g - 1) & 1, wc)))
      return false;
    tc_fence_after();
#pragma unroll 1
    for (uint32_t kb = 0; kb < 8; ++kb)
      umma_x4<kIdescS<64>, 32, 32>(tmem + L::kTmS, kv_k + kb * (kBlk >> 4), q_k + kb * (2 * kBlk >> 4), kb > 0);
    umma_x4<kIdescSRope<64>, 32, 32>(tmem + L::kTmS, kv_k + 8 * (kBlk >> 4), q_k + 16 * (kBlk >> 4), true);
    umma_commit(bar(kBarS));
    return true;
  };
  uint32_t g = 0;
  bool ok = true;
  SegIter it(p);
  Seg s;
  while (ok && it.next(s)) {
    if (s.j0 >= s.j1) continue;
    ok = scores(g);
    const int steps = (s.nvalid + 15) / 16;  // rows past the last head add nothing to dKV
    for (int j = s.j0; ok && j < s.j1; ++j, ++g) {
      ok = mbar_wait(bar(kBarP), g & 1, wc);
      if (ok && j == s.j0 && segs > 0) ok = mbar_wait(bar(kBarDqFree), (segs - 1) & 1, wc);
      if (!ok) break;
      tc_fence_after();
#pragma unroll 1
      for (uint32_t mb = 0; mb < 4; ++mb)
        umma_x4<kIdescDq<64>, 2048, 2048>(tmem + kTmDq + 64 * mb, kv_mn + mb * (2 * kBlk >> 4), ds_mn, j > s.j0);
      umma_x4<kIdescDqRope<64>, 2048, 2048>(tmem + kTmDq + 256, kv_mn + 8 * (kBlk >> 4), ds_mn, j > s.j0);
      umma_commit(bar(kBarKvFree));
#pragma unroll 1
      for (uint32_t cb = 0; cb < 4; ++cb) {
        // what the block's columns held before has been read
        if (cb == 2 && g > 0) ok = mbar_wait(bar(kBarBlockFree + 4), (g - 1) & 1, wc);
        if (cb == 3) ok = mbar_wait(bar(kBarBlockFree), g & 1, wc);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + L::block(static_cast<int>(cb));
        umma_x4<kIdescKv, 2048, 32>(d, q_mn + cb * (4 * kBlk >> 4), ds_k, false, steps);
        umma_x4<kIdescKv, 2048, 32>(d, q_mn + cb * (4 * kBlk >> 4) + (kBlk >> 4), p_k, true, steps);
        umma_commit(bar(kBarBlock + static_cast<int>(cb)));
      }
      if (ok && j + 1 < s.j1) ok = scores(g + 1);
      if (ok) ok = mbar_wait(bar(kBarBlockFree + 2), g & 1, wc);
      if (!ok) break;
      tc_fence_after();
      umma_x4<kIdescKvRope, 2048, 32>(tmem + L::block(4), q_mn + 16 * (kBlk >> 4), ds_k, false, steps);
      umma_commit(bar(kBarBlock + 4));
      umma_commit(bar(kBarPFree));
    }
    umma_commit(bar(kBarSeg));
    umma_commit(bar(kBarDq));
    ++segs;
  }
  umma_commit(bar(kBarDone));
  mbar_wait_ignoring_abort(bar(kBarDone), 0, wc);  // nothing runs when tensor memory is released
}

// The same for row-sets of 32 heads. Per tile: four blocks of dKV, the next tile's S^T and dP^T (its rows have
// a buffer of their own), dq, the last block.
__device__ __forceinline__ void mma_role32(const BackwardParams& p, uint8_t* smem, uint32_t tmem, uint32_t bars,
                                           const WaitCtl& wc) {
  using L = Lay<32>;
  const uint32_t base = smem_u32(smem);
  const uint64_t q_k = smem_desc_sw128(base + kOffQ, 16, 1024), q_mn = smem_desc_sw128(base + kOffQ, kBlk, 1024);
  const uint64_t kv_k0 = smem_desc_sw128(base + kOffKv<32>, 16, 1024);
  const uint64_t kv_mn0 = smem_desc_sw128(base + kOffKv<32>, kBlk, 1024);
  const uint64_t p_k = smem_desc_sw64(base + kOffP<32>, 16, 512), ds_k = smem_desc_sw64(base + kOffDs<32>, 16, 512);
  const uint64_t ds_mn = smem_desc_sw64(base + kOffDs<32>, 4096, 512);
  constexpr uint64_t kDout = 32 * 128 >> 4;  // from q's rows of a block to dout's
  auto bar = [&](int i) -> uint32_t { return bars + 8u * static_cast<uint32_t>(i); };
  auto scores = [&](uint32_t g) -> bool {
    const uint32_t buf = g & 1;
    // (the softmax has read the last S^T and dP^T: it has arrived with their P and dS)
    if (!mbar_wait(bar(kBarKvFull + static_cast<int>(buf)), (g >> 1) & 1, wc)) return false;
    tc_fence_after();
    const uint64_t kv_k = kv_k0 + buf * (9 * kBlk >> 4);
#pragma unroll 1
    for (uint32_t kb = 0; kb < 8; ++kb)
      umma_x4<kIdescS<32>, 32, 32>(tmem + L::kTmS, kv_k + kb * (kBlk >> 4), q_k + kb * (kBlk >> 4), kb > 0);
    umma_x4<kIdescSRope<32>, 32, 32>(tmem + L::kTmS, kv_k + 8 * (kBlk >> 4), q_k + 8 * (kBlk >> 4), true);
    umma_commit(bar(kBarS));
    return true;
  };
  uint32_t g = 0, segs = 0;
  bool ok = true;
  SegIter it(p);
  Seg s;
  while (ok && it.next(s)) {
    if (s.j0 >= s.j1) continue;
    ok = scores(g);
    const int steps = (s.nvalid + 15) / 16;  // rows past the last head add nothing to dKV
    for (int j = s.j0; ok && j < s.j1; ++j, ++g) {
      ok = mbar_wait(bar(kBarP), g & 1, wc);
#pragma unroll 1
      for (uint32_t cb = 0; ok && cb < 4; ++cb) {
        // the last tile's block in these columns has been read
        if (g > 0) ok = mbar_wait(bar(kBarBlockFree + static_cast<int>(cb == 1 ? 4 : cb)), (g - 1) & 1, wc);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + L::block(static_cast<int>(cb));
        umma_x4<kIdescKv, 2048, 32>(d, q_mn + cb * (2 * kBlk >> 4), ds_k, false, steps);
        umma_x4<kIdescKv, 2048, 32>(d, q_mn + cb * (2 * kBlk >> 4) + kDout, p_k, true, steps);
        umma_commit(bar(kBarBlock + static_cast<int>(cb)));
      }
      if (ok && j + 1 < s.j1) ok = scores(g + 1);
      if (ok && j == s.j0 && segs > 0) ok = mbar_wait(bar(kBarDqFree), (segs - 1) & 1, wc);
      if (!ok) break;
      tc_fence_after();
      const uint64_t kv_mn = kv_mn0 + (g & 1) * (9 * kBlk >> 4);
#pragma unroll 1
      for (uint32_t mb = 0; mb < 4; ++mb)
        umma_x4<kIdescDq<32>, 2048, 1024>(tmem + kTmDq + 32 * mb, kv_mn + mb * (2 * kBlk >> 4), ds_mn, j > s.j0);
      umma_x4<kIdescDqRope<32>, 2048, 1024>(tmem + kTmDq + 128, kv_mn + 8 * (kBlk >> 4), ds_mn, j > s.j0);
      umma_commit(bar(kBarKvFree + static_cast<int>(g & 1)));
      ok = mbar_wait(bar(kBarBlockFree + 1), g & 1, wc);
      if (!ok) break;
      tc_fence_after();
      umma_x4<kIdescKvRope, 2048, 32>(tmem + L::block(4), q_mn + 8 * (kBlk >> 4), ds_k, false, steps);
      umma_commit(bar(kBarBlock + 4));
      umma_commit(bar(kBarPFree));
    }
    umma_commit(bar(kBarSeg));
    umma_commit(bar(kBarDq));
    ++segs;
  }
  umma_commit(bar(kBarDone));
  mbar_wait_ignoring_abort(bar(kBarDone), 0, wc);  // nothing runs when tensor memory is released
}

// The cache rows' sums keep their channels in an order that suits add_rows: each 32 latent channels as
// 8 x 4 (channels c, c + 8, c + 16, c + 24 side by side), each 16 rope channels as 4 x 4 (c, c + 4, c + 8,
// c + 12). finish_kernel puts them right.

// Adds v[e] of this lane's channel to cache row slots[e], e < 32; the warp's lanes are 32 consecutive
// latent channels, or with kRope the lower 16 lanes 16 rope channels; dst is the first one in row 0.
// Lanes exchange four entries' values (two butterfly steps), after which a lane holds four channels of
// one entry, 16 consecutive bytes of the sums, and neighbours continue the line: a quarter of the
// instructions that single additions take.
template <bool kRope>
__device__ __forceinline__ void add_rows(float* dst, const int* slots, const uint32_t (&v)[32]) {
  const int lane = threadIdx.x & 31;
  constexpr int kLow = kRope ? 4 : 8;      // lanes that hold one entry afterwards
  constexpr int kStep = kRope ? 8 : 4;     // entries per instruction
  constexpr int kBatch = 16 / kStep;       // instructions prepared together
  const bool up = (lane & kLow) != 0, top = (lane & (2 * kLow)) != 0;
  dst += (lane & (kLow - 1)) * 4;
#pragma unroll
  for (int i0 = 0; i0 < 32; i0 += kBatch * kStep) {
    uint32_t x[kBatch][4];
    int slot[kBatch];
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      const int i = i0 + n * kStep;
      slot[n] = slots[i + (lane / kLow)];
#pragma unroll
      for (int u = 0; u < 4; ++u) x[n][u] = v[i + u];
      if constexpr (kRope) {
        // the upper lanes hold nothing: they take entries i + 4 .. i + 7
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t o = __shfl_sync(0xffffffffu, v[i + 4 + u], lane & 15);
          if (lane >= 16) x[n][u] = o;
        }
      }
    }
#pragma unroll
    for (int n = 0; n < kBatch; ++n)
#pragma unroll
      for (int u = 0; u < 4; u += 2) {
        const uint32_t o = __shfl_xor_sync(0xffffffffu, up ? x[n][u] : x[n][u + 1], kLow);
        if (up) x[n][u] = o;
        else x[n][u + 1] = o;
      }
#pragma unroll
    for (int n = 0; n < kBatch; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t o = __shfl_xor_sync(0xffffffffu, top ? x[n][u] : x[n][u + 2], 2 * kLow);
        if (top) x[n][u] = o;
        else x[n][u + 2] = o;
      }
#pragma unroll
    for (int n = 0; n < kBatch; ++n)
      if (slot[n] >= 0)
        asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(dst + static_cast<long long>(slot[n]) * kRow),
                     "f"(__uint_as_float(x[n][0])), "f"(__uint_as_float(x[n][1])), "f"(__uint_as_float(x[n][2])),
                     "f"(__uint_as_float(x[n][3]))
                     : "memory");
  }
}

// This role and scatter_role end at the first block of dKV^T whose wait gives up: a barrier that stays in its
// phase answers the next tile's parity as if it had completed, for a block that was never written and rows
// that the gather never named. The other waits may give up: what follows them stays in this CTA and the
// call's outputs. (The loops are left by their variables: a return at this place, or one at every wait,
// makes 333 x 16 x 2048 take 345 us instead of 338.)
template <int R>
__device__ __forceinline__ void softmax_role(const BackwardParams& p, uint8_t* smem, Misc* misc, uint32_t tmem,
                                             uint32_t bars, const WaitCtl& wc) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = warp & 3, half = warp >> 2;
  auto bar = [&](int i) -> uint32_t { return bars + 8u * static_cast<uint32_t>(i); };
  // S^T and dP^T (64 entries in lanes 0-15 of each quadrant): this thread's entries e and e + 8, and
  // their heads kHeads half + 8 k + 2 (lane & 3) and the next, k < kOcts
  constexpr int kHeads = R / 2, kOcts = kHeads / 8;
  const int e = 16 * quad + (lane >> 2), pair = lane & 3;
  const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quad) << 16);
  // where this lane's row of the stored 8 x 8 matrices goes: matrix lane >> 3 is chunk 4 half + that, of
  // entries e; with R = 32 chunks 2 half and 2 half + 1 of entries e, then of entries e + 8
  const uint32_t at0 = smem_u32(smem) + (R == 64 ? sw128_offset(16 * quad + (lane & 7), 4 * half + (lane >> 3))
                                                 : sw64_offset(16 * quad + 8 * (lane >> 4) + (lane & 7),
                                                               2 * half + ((lane >> 3) & 1)));
  // an entry's weight: the two warps of a quadrant hold half of the heads each. Lanes 0 and 1 of four
  // keep the sums of e and e + 8
  const int we = e + 8 * (pair & 1);
  uint32_t g = 0, segs = 0;
  SegIter it(p);
  Seg s;
  while (it.next(s)) {
    const bool any = s.j0 < s.j1;
    // the exponent S - lse is one fma and takes its factor log2 e afterwards: lse in log2 units would be
    // off by 2^-24 of itself, here the rounding is relative to the difference
    float lse[2 * kOcts], delta[2 * kOcts];  // delta times the softmax scale
#pragma unroll
    for (int i = 0; i < 2 * kOcts; ++i) {
      const int r = kHeads * half + 8 * (i >> 1) + 2 * pair + (i & 1);
      const float2 v = r < s.nvalid ? p.stats[s.base + r] : make_float2(CUDART_INF_F, 0.f);
      lse[i] = v.x;
      delta[i] = v.y * p.scale;
    }
    // the second half leaves its sums in shared memory; the first adds them once the tile's first block of
    // dKV is there, which the MMAs began when both had arrived
    float held = 0.f;
    bool held_live = false;
    auto put_weight = [&](int j) {
      const int k = j * kEntries + we;
      if (half == 0 && pair < 2 && held_live && k < p.K) {
        float* dst = p.weights + static_cast<long long>(s.t) * p.K + k;
        const float w = held + misc->weight[g & 1][we];
        // two head chunks add to a zero: the same sum in either order
        if (p.hchunks > 1) atomicAdd(dst, w);
        else *dst = w;
      }
    };
    for (int j = s.j0; j < s.j1; ++j, ++g) {
      mbar_wait(bar(kBarS), g & 1, wc);
      tc_fence_after();
      uint32_t sv[4 * kOcts], dv[4 * kOcts];
      tmem_ld_16x256b(lanes + Lay<R>::kTmS + kHeads * half, sv);
      tmem_ld_16x256b(lanes + Lay<R>::kTmDp + kHeads * half, dv);
      const bool live0 = misc->slot[g & 3][e] >= 0, live8 = misc->slot[g & 3][e + 8] >= 0;
      tmem_ld_wait();
      uint32_t pp[2 * kOcts], pd[2 * kOcts];  // [2 k]: entry e, [2 k + 1]: entry e + 8
      float w0 = 0.f, w8 = 0.f;
#pragma unroll
      for (int k = 0; k < kOcts; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float pr[2], d[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int i = 4 * k + 2 * h + u;
            // a dead entry's row is zero: with P = 0, its dS is 0 too
            const float x = ex2_approx(fmaf(__uint_as_float(sv[i]), p.scale, -lse[2 * k + u]) * kLog2e);
            pr[u] = (h ? live8 : live0) ? x : 0.f;
            d[u] = pr[u] * fmaf(__uint_as_float(dv[i]), p.scale, -delta[2 * k + u]);
            if (h) w8 += pr[u];
            else w0 += pr[u];
          }
          pp[2 * k + h] = pack_bf16x2(pr[0], pr[1]);
          pd[2 * k + h] = pack_bf16x2(d[0], d[1]);
        }
      // the last tile's products with P and dS are done
      if (g > 0) mbar_wait(bar(kBarPFree), (g - 1) & 1, wc);
      if constexpr (R == 64) {
        const uint32_t at8 = at0 + 8 * 128;
        stmatrix_x4(at0 + kOffP<R>, pp[0], pp[2], pp[4], pp[6]);
        stmatrix_x4(at8 + kOffP<R>, pp[1], pp[3], pp[5], pp[7]);
        stmatrix_x4(at0 + kOffDs<R>, pd[0], pd[2], pd[4], pd[6]);
        stmatrix_x4(at8 + kOffDs<R>, pd[1], pd[3], pd[5], pd[7]);
      } else {
        stmatrix_x4(at0 + kOffP<R>, pp[0], pp[2], pp[1], pp[3]);
        stmatrix_x4(at0 + kOffDs<R>, pd[0], pd[2], pd[1], pd[3]);
      }
      if (p.weights != nullptr) {
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          w0 += __shfl_xor_sync(0xffffffffu, w0, o);
          w8 += __shfl_xor_sync(0xffffffffu, w8, o);
        }
        held = pair ? w8 : w0;
        held_live = pair ? live8 : live0;
        if (half == 1 && pair < 2) misc->weight[g & 1][we] = held;
      }
      fence_proxy_async_smem();  // P and dS -> MMA operand reads
      tc_fence_before();
      mbar_arrive(bar(kBarP));
      // these warps wait for the next scores now: meanwhile they add blocks 0 and 3 of dKV^T, half of the
      // entries each
#pragma unroll 1
      for (int cb = 0; cb < 4; cb += 3) {
        if (!__all_sync(0xffffffffu, mbar_wait(bar(kBarBlock + cb), g & 1, wc))) {
          j = s.j1;  // no further tile
          it.pos = it.hi;
          break;
        }
        if (cb == 0 && p.weights != nullptr) put_weight(j);
        tc_fence_after();
        uint32_t v[32];
        tmem_ld32(lanes + Lay<R>::block(cb) + 32 * half, v);
        tmem_ld_wait();
        tc_fence_before();
        mbar_arrive(bar(kBarBlockFree + cb));
        add_rows<false>(p.dkv_acc + 128 * cb + 32 * quad, misc->slot[g & 3] + 32 * half, v);
      }
    }
    // dq^T: lane = channel, this warp's heads kHeads half and on
    if (any) {
      mbar_wait(bar(kBarDq), segs & 1, wc);
      tc_fence_after();
    }
#pragma unroll 1
    for (int mb = 0; mb < 5; ++mb) {
      uint32_t v[kHeads];
      if (any) {
        if constexpr (R == 64) tmem_ld32(lanes + kTmDq + R * mb + kHeads * half, v);
        else tmem_ld16(lanes + kTmDq + R * mb + kHeads * half, v);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int i = 0; i < kHeads; ++i) v[i] = 0u;
      }
      if (mb == 4 && lane >= 16) continue;
      const int c = 128 * mb + (mb < 4 ? 32 : 16) * quad + lane;
      if (s.whole) {
        uint16_t* dst = p.dq + (s.base + kHeads * half) * kRow + c;
#pragma unroll
        for (int i = 0; i < kHeads; ++i)
          if (kHeads * half + i < s.nvalid) dst[i * kRow] = static_cast<uint16_t>(pack_bf16x2(__uint_as_float(v[i]), 0.f));
      } else {
        float* dst = p.dq_part + (static_cast<long long>(s.part) * kRows + kHeads * half) * kRow + c;
#pragma unroll
        for (int i = 0; i < kHeads; ++i)
          if (kHeads * half + i < s.nvalid) dst[i * kRow] = __uint_as_float(v[i]);
      }
    }
    if (any) {
      tc_fence_before();
      mbar_arrive(bar(kBarDqFree));
      ++segs;
    }
  }
}

template <int R>
__device__ __forceinline__ void scatter_role(const BackwardParams& p, Misc* misc, uint32_t tmem, uint32_t bars,
                                             const WaitCtl& wc) {
  const int warp = (threadIdx.x >> 5) - kScatWarp0;
  const int quad = warp & 3;
  const int group = warp >> 2;  // takes blocks 1 and 4, or 2
  auto bar = [&](int i) -> uint32_t { return bars + 8u * static_cast<uint32_t>(i); };
  const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quad) << 16);
  uint32_t g = 0;
  SegIter it(p);
  Seg s;
  while (it.next(s)) {
    for (int j = s.j0; j < s.j1; ++j, ++g) {
#pragma unroll 1
      for (int cb = 1 + group; cb < 5; cb += 3) {
        const uint32_t from = Lay<R>::block(cb);
        if (!__all_sync(0xffffffffu, mbar_wait(bar(kBarBlock + cb), g & 1, wc))) return;
        tc_fence_after();
        uint32_t v[2][32];
        tmem_ld32(lanes + from, v[0]);
        tmem_ld32(lanes + from + 32, v[1]);
        tmem_ld_wait();
        tc_fence_before();
        mbar_arrive(bar(kBarBlockFree + cb));
        const int* slots = misc->slot[g & 3];
        if (cb < 4) {
          add_rows<false>(p.dkv_acc + 128 * cb + 32 * quad, slots, v[0]);
          add_rows<false>(p.dkv_acc + 128 * cb + 32 * quad, slots + 32, v[1]);
        } else {
          add_rows<true>(p.dkv_acc + kVdim + 16 * quad, slots, v[0]);
          add_rows<true>(p.dkv_acc + kVdim + 16 * quad, slots + 32, v[1]);
        }
      }
    }
  }
}

template <int R>
__global__ void __launch_bounds__(kThreads, 1) backward_kernel(const BackwardParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Misc* misc = reinterpret_cast<Misc*>(smem + kOffMisc<R>);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // a uniform value
  const uint32_t bars = smem_u32(misc->bars);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      int count = 1;
      if (i < kBarKvFree) count = kFillThreads;
      if (i == kBarP || i == kBarDqFree) count = 32 * kSoftWarps;
      if (i >= kBarBlockFree && i < kBarBlockFree + 5) count = 128;
      if (i == kBarBlockFree || i == kBarBlockFree + 3) count = 32 * kSoftWarps;
      mbar_init(bars + 8 * i, count);
    }
    misc->abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // no row before the gather names one
  if (threadIdx.x < 4 * kEntries) misc->slot[threadIdx.x / kEntries][threadIdx.x % kEntries] = -1;
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&misc->tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc->tmem;
  const WaitCtl wc{p.status, &misc->abort_flag, p.wait_limit_ns ? p.wait_limit_ns : kWaitLimitNs};
  grid_launch_dependents();
  grid_wait();  // for prepare_kernel, beside whose end the above ran
  if (warp < kScatWarp0) {
    softmax_role<R>(p, smem, misc, tmem, bars, wc);
  } else if (warp < kFillWarp0) {
    scatter_role<R>(p, misc, tmem, bars, wc);
  } else if (warp < kMmaWarp) {
    gather_role<R>(p, smem, misc, bars, wc);
  } else if (elect_one()) {
    if constexpr (R == 64) mma_role64(p, smem, tmem, bars, wc);
    else mma_role32(p, smem, tmem, bars, wc);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// The first T * chunks CTAs: 2048 entries of a query's list as cache rows, and how far the live ones
// reach. The next delta_ctas, 32 heads of any queries each: (lse, delta); a head without a live entry
// (lse = -inf) gets +inf, so that P = 0. The others zero the cache rows' sums.
constexpr int kPrepThreads = 256;
constexpr int kPrepHeads = 32;
constexpr int kListChunk = 2048;
__global__ void __launch_bounds__(kPrepThreads) prepare_kernel(const BackwardParams p, const ListParams l,
                                                               int delta_ctas) {
  const int tid = threadIdx.x, lane = tid & 31;
  grid_launch_dependents();
  const int lists = p.T * p.chunks;
  if (static_cast<int>(blockIdx.x) < lists) {
    __shared__ int reach;
    const int t = blockIdx.x / p.chunks, k0 = (blockIdx.x - t * p.chunks) * kListChunk;
    const int k1 = min(p.K, k0 + kListChunk);
    if (tid == 0) reach = 0;
    __syncthreads();
    const ReqContext ctx = request_context(t, l.req_of_token, l.block_table, l.num_reqs, l.max_blocks, l.seq_lens);
    const int len = l.topk_len ? l.topk_len[t] : p.K;
    int err = 0, last = 0;
#pragma unroll 4
    for (int k = k0 + tid; k < k1; k += kPrepThreads) {
      const long long at = static_cast<long long>(t) * p.K + k;
      int slot = -1;
      if (k < len) {
        const int pos = __ldg(l.topk + at);
        slot = slot_of(pos, page_of(pos, ctx, l.max_blocks, l.page_size), ctx, l.block_table != nullptr, l.max_blocks,
                       l.page_size, l.num_pages, &err);
      }
      p.slots[at] = slot;
      if (p.weights != nullptr) p.weights[at] = 0.f;
      if (slot >= 0) last = k + 1;
    }
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 0 && last > 0) atomicMax(&reach, last);
    if (__any_sync(0xffffffffu, err != 0) && lane == 0) atomicOr(p.status, SVT_DEV_ERR_INDEX_RANGE);
    __syncthreads();
    if (tid == 0) p.live_len[blockIdx.x] = reach;
    return;
  }
  const int cta = blockIdx.x - lists;
  if (cta >= delta_ctas) {
    const long long n = p.num_slots * (kRow / 4), step = (gridDim.x - lists - delta_ctas) * static_cast<long long>(kPrepThreads);
    for (long long i = (cta - delta_ctas) * static_cast<long long>(kPrepThreads) + tid; i < n; i += step)
      reinterpret_cast<float4*>(p.dkv_acc)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    return;
  }
  // a warp takes two heads at a time: eight 16-byte loads in flight a lane
  const long long rows = static_cast<long long>(p.T) * p.H;
#pragma unroll 1
  for (int i = 0; i < kPrepHeads; i += 2 * kPrepThreads / 32) {
    const long long r0 = static_cast<long long>(cta) * kPrepHeads + i + 2 * (tid >> 5);
    if (r0 >= rows) break;
    const int count = r0 + 1 < rows ? 2 : 1;
    uint4 a[2][2], b[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (u < count) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          a[u][k] = __ldg(reinterpret_cast<const uint4*>(p.out + (r0 + u) * kVdim) + lane + 32 * k);
          b[u][k] = __ldg(reinterpret_cast<const uint4*>(p.dout + (r0 + u) * kVdim) + lane + 32 * k);
        }
      }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (u >= count) break;
      const long long r = r0 + u;
      float d = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t aw[4] = {a[u][k].x, a[u][k].y, a[u][k].z, a[u][k].w};
        const uint32_t bw[4] = {b[u][k].x, b[u][k].y, b[u][k].z, b[u][k].w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          d = fmaf(__uint_as_float(aw[w] << 16), __uint_as_float(bw[w] << 16), d);
          d = fmaf(__uint_as_float(aw[w] & 0xFFFF0000u), __uint_as_float(bw[w] & 0xFFFF0000u), d);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
      if (lane == 0) {
        const float lse = p.lse[r];
        p.stats[r] = make_float2(lse == -CUDART_INF_F ? CUDART_INF_F : lse, d - (p.dlse ? p.dlse[r] : 0.f));
      }
    }
  }
}

// CTAs below join_ctas join the dq of the row-set that the border before CTA c + 1 of the main
// kernel cuts (the first such border of the row-set does it), four rows each; the others round the
// cache rows' sums to bf16.
constexpr int kJoinRows = 4;
__global__ void __launch_bounds__(256) finish_kernel(const BackwardParams p, int join_ctas) {
  grid_wait();
  if (static_cast<int>(blockIdx.x) < join_ctas) {
    const int c = 1 + blockIdx.x / (kRows / kJoinRows), part0 = (blockIdx.x % (kRows / kJoinRows)) * kJoinRows;
    const long long lo = streamk_lo(c, p.total_tiles, p.num_ctas);
    const int r = static_cast<int>(lo / p.tiles);
    const long long first = static_cast<long long>(r) * p.tiles;
    if (lo == first || streamk_lo(c - 1, p.total_tiles, p.num_ctas) > first) return;
    const int c1 = static_cast<int>(streamk_owner(first + p.tiles - 1, p.total_tiles, p.num_ctas));
    const int t = r / p.hchunks, chunk = r - t * p.hchunks;
    const int nvalid = min(kRows, p.H - chunk * kRows);
    const long long base = static_cast<long long>(t) * p.H + chunk * kRows;
    // CTA c - 1's part may be its second; every later one begins inside the row-set: its first
    const float* a = p.dq_part + streamk_part_slot(c - 1, first, p.total_tiles, p.num_ctas) * (kRows * kRow);
    const float* b = p.dq_part + 2ll * c * (kRows * kRow);
    const int more = c1 - c + 1;
    for (int i = threadIdx.x; i < kJoinRows * (kRow / 4); i += 256) {
      const int row = part0 + i / (kRow / 4), at = row * kRow + 4 * (i % (kRow / 4));
      if (row >= nvalid) break;
      float4 sum = *reinterpret_cast<const float4*>(a + at);
#pragma unroll 4
      for (int k = 0; k < more; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(b + at + 2ll * k * (kRows * kRow));
        sum.x += v.x;
        sum.y += v.y;
        sum.z += v.z;
        sum.w += v.w;
      }
      *reinterpret_cast<uint2*>(p.dq + base * kRow + at) = make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
    }
    return;
  }
  // 16 bytes of the sums hold four channels a stride apart (add_rows): neighbours exchange two each and
  // write pairs
  const long long n = p.num_slots * (kRow / 4), step = (gridDim.x - join_ctas) * 256ll;
  const bool odd = (threadIdx.x & 1) != 0;
  for (long long i = (blockIdx.x - join_ctas) * 256ll + threadIdx.x; i < n; i += 4 * step) {
    float4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + u * step < n) v[u] = reinterpret_cast<const float4*>(p.dkv_acc)[i + u * step];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const long long at = i + u * step;
      // (n and step are even: both lanes of a pair are here)
      const unsigned pair = 3u << (threadIdx.x & 30);
      if (at >= n) break;
      const float a = __shfl_xor_sync(pair, odd ? v[u].x : v[u].z, 1);
      const float b = __shfl_xor_sync(pair, odd ? v[u].y : v[u].w, 1);
      const long long row = at / (kRow / 4);
      const int c4 = static_cast<int>(at - row * (kRow / 4));
      const bool rope = c4 >= kVdim / 4;
      const int stride = rope ? 4 : 8, k = rope ? c4 - kVdim / 4 : c4;
      const int first = (rope ? kVdim + 16 * (k >> 2) + (k & 3) : 32 * (k >> 3) + (k & 7)) - odd;
      uint16_t* dst = p.dkv + row * kRow + first + (odd ? 2 * stride : 0);
      *reinterpret_cast<uint32_t*>(dst) = odd ? pack_bf16x2(a, v[u].z) : pack_bf16x2(v[u].x, a);
      *reinterpret_cast<uint32_t*>(dst + stride) = odd ? pack_bf16x2(b, v[u].w) : pack_bf16x2(v[u].y, b);
    }
  }
}

}  // namespace

void plan_backward(BackwardParams& p, int sms) {
  p.hchunks = (p.H + kRows - 1) / kRows;
  p.tiles = (p.K + kEntries - 1) / kEntries;
  p.chunks = (p.K + kListChunk - 1) / kListChunk;
  p.total_tiles = static_cast<long long>(p.T) * p.hchunks * p.tiles;
  p.num_ctas = static_cast<int>(p.total_tiles < sms ? p.total_tiles : sms);
}

cudaError_t launch_backward(const BackwardParams& p, const ListParams& l, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  const bool any = p.total_tiles > 0;
  if (!any && p.T > 0) {  // empty lists: no gradient
    e = cudaMemsetAsync(p.dq, 0, static_cast<size_t>(p.T) * p.H * kRow * sizeof(uint16_t), stream);
    if (e != cudaSuccess) return e;
  }
  if (!any) return cudaMemsetAsync(p.dkv, 0, static_cast<size_t>(p.num_slots) * kRow * sizeof(uint16_t), stream);
  // the two schedules, us for 32 and for 64 heads a row-set: 333 x 32 x 2048 355 and 381, 1024 x 16 x 2048 934 and
  // 1015, 512 x 8 x 512 147 and 161, 64 x 32 x 200 38 and 41. More heads in sets of 32 would add every row twice
  const bool packed = p.H <= 32;
  const auto kernel = packed ? backward_kernel<32> : backward_kernel<64>;
  const uint32_t smem = packed ? kSmem<32> : kSmem<64>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const long long zero = (p.num_slots * (kRow / 4) + kPrepThreads - 1) / kPrepThreads;
  const int delta_ctas = static_cast<int>((static_cast<long long>(p.T) * p.H + kPrepHeads - 1) / kPrepHeads);
  prepare_kernel<<<static_cast<unsigned>(p.T * p.chunks + delta_ctas + (zero < 1216 ? zero : 1216)), kPrepThreads, 0, stream>>>(
      p, l, delta_ctas);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // each kernel may begin while the last one ends, and waits for its results (programmatic dependent
  // launch: the short calls are mostly the kernels' beginnings and ends)
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(p.num_ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e != cudaSuccess) return e;
  const int join = (p.num_ctas - 1) * (kRows / kJoinRows);
  const long long n = (p.num_slots * (kRow / 4) + 1023) / 1024;
  cfg.gridDim = dim3(static_cast<unsigned>(join + (n < 1216 ? n : 1216)));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, finish_kernel, p, join);
}

}  // namespace svt
