// Decode attention over the paged latent cache for a batch whose queries share long prefixes (dense: a query attends to every
// row of its request up to its length). Per query row r and the rows j it attends to:
//   s_j = scale * q_r . k_j,  out_r = softmax(s) . V,  lse_r = ln sum_j exp(s_j)
// with k_j the whole 576-wide cache row and V its first 512 columns.
//
// The queries of a group share the rows of its prefix: 128 packed rows (query, head) of the group are one row tile, and a prefix row
// that is staged serves all 128. A row tile's list is its prefix followed by the rows that each of its queries has to itself, in
// pieces of 16 positions; a tile of the list is 8 pieces. The rows a query has to itself go through the same accumulators with the
// other queries' rows masked, so that nothing is merged but what the schedule cuts: all tiles of all row tiles, laid end to end, are
// dealt out evenly to the CTA pairs, and a row tile that two pairs share leaves normalised f16 rows and their lse for the merge.
//
// GB300 design. 128 rows x 512 channels of O in fp32 are all 512 TMEM columns, so a cluster of two CTAs holds a row tile, 64 rows
// each, and both work on one tcgen05.mma of cta_group::2 with M = 128: the accumulator's lanes 0-63 hold a CTA's rows in the lower
// half of N, lanes 64-127 the same rows in the upper half, so that O takes 256 columns, S (128 list rows) 64. Such an MMA runs at the full
// rate for N = 128 and 256 (measured: 32 and 64 cycles for K = 16), each CTA staging half of the B operand:
//   S  [128 x 128] = Q . K^T: CTA c stages list rows 64 c .. + 63, all 576 channels (K-major);
//   O  [128 x 512] += P . V, two MMAs of N = 256: CTA c stages channels 256 h + 128 c .. + 127 of all 128 list rows (MN-major).
// A ring of seven 16 KB units feeds them: five for K (128 channels each, the last one the 64 rope channels), four for V (64
// list rows by 128 channels). Units are consumed in the order K(0), K(1), V(0), K(2), V(1), ..: the scores of the next tile run while
// the softmax of this one does.
//
// An e4m3 cache: K is its codes as they are (f16 holds them exactly), V codes times scales in f16, rounded once. A score's four
// blocks of 128 channels have a scale each, so that each K unit's sums go to one of four slots of 64 TMEM columns, from which the
// softmax warps collect them, times their scales, in fp32.
//
// What bounds it: bf16, 128 queries x 64 heads over 32768 rows: 382 to 390 us, 1.55 PFLOP/s (a step of the loop is 2200 to 2450 cycles, the
// MMAs of a tile alone 2180; the rest is power and the last pairs' tails); 64 x 64 x 8192: 67 us, of which the plan and the merge are
// some 12. e4m3, 120 x 16 x 12007: 100 us, 9000 cycles a tile: a warp takes some 6000 to load and convert a unit, and the
// softmax warps as long for five units of scores and their P.
//
// Warps of each CTA: 0 issues the MMAs (in CTA 0 of the pair), 1 and 3 load by TMA, 2 resolves list positions to cache rows, 4-11
// softmax and epilogue, 12-15 (12-18 with an e4m3 cache) fill the units of tiles that TMA cannot (rows that end inside a piece, pages of fewer than 16
// rows, an e4m3 cache). Every wait is bounded.
#include <algorithm>
#include <mutex>

#include <cuda_fp16.h>
#include <math_constants.h>

#include "device.cuh"
#include "internal.h"

namespace svt {

namespace {

// The loading warps are none of the MMA warp's SM sub-partition: there their loads wait behind the MMAs that are being issued
// (1700 cycles late).
constexpr int kMmaWarp = 0, kTmaWarp0 = 1, kResolveWarp = 2, kTmaWarp1 = 3, kSoftWarp0 = 4, kSoftWarps = 8, kFillWarp0 = 12;
// An e4m3 cache has all of its units filled (and converted) by threads: by a warp for each unit of the ring. (Two warps a
// unit took as long, 109 us against 107 then: the softmax warps then have 72 registers and spill.)
__host__ __device__ constexpr int fill_warps(bool f16) { return f16 ? 7 : 4; }
__host__ __device__ constexpr int block_threads(bool f16) { return 32 * (kFillWarp0 + fill_warps(f16)); }

constexpr int kRows = 64;                       // query rows of a CTA
constexpr int kTile = 128;                      // list rows of a tile
constexpr int kPieces = kTile / kListPiece;     // 8
constexpr int kBlk = 64 * 128;                  // 64 rows x 64 channels, 128-byte swizzle
constexpr int kUnit = 2 * kBlk;                 // 16 KB
constexpr int kUnits = 7;
constexpr int kPBytes = 2 * kBlk;               // two blocks of 64 rows x 64 list rows, twice
constexpr int kKUnits = 5, kVUnits = 4;         // units of a tile
constexpr int kInfos = 4;                       // tiles resolved ahead
constexpr int kSlots = 4;                       // of S: bf16 two of a tile each, e4m3 four of a unit of K each
constexpr float kTau = 8.0f;                    // the reference maximum moves when a score passes it by 2^8

// What the resolver says of a tile.
struct alignas(16) TileInfo {
  int slot[kTile];       // cache row, -1: none
  int base[kPieces];     // cache row of the piece's first row (any one for a piece without rows)
  int pos[kPieces];      // position of the piece's first row
  int lo[kPieces], hi[kPieces];  // positions of the piece that its queries attend to
  int owner[kPieces];    // the query they belong to, -1: all of the group
  int mode;              // kFill*
  int whole;             // no entry is masked for any row of the row tile
  int fix;               // loaded by TMA, with rows that are none: zeroes take their place in V
  int pad;
};
// How a tile is loaded: row by row, in pieces of 16 rows, in halves of 64.
enum FillMode : int { kFillThreadwise = 0, kFillPieces = 1, kFillHalves = 2, kFillNone = 3 };

// shared memory map (offsets from a 1024-aligned base)
constexpr int kOffQ = 0;                                  // 9 blocks
constexpr int kOffRing = kOffQ + 9 * kBlk;
constexpr int kOffP = kOffRing + kUnits * kUnit;
constexpr int kOffInfo = kOffP + 2 * kPBytes;
constexpr int kOffRed = kOffInfo + kInfos * static_cast<int>(sizeof(TileInfo));  // float[4][64]
constexpr int kOffSum = kOffRed;  // float[4][64]: the last reader of either passes a barrier before the other is written
constexpr int kOffScales = kOffRed + 4 * kRows * 4;       // e4m3: float[kSoftWarps][4][32]
constexpr int kOffBars = kOffScales + kSoftWarps * 4 * 32 * 4;

// barriers (those marked L are used in CTA 0 of the pair by both)
constexpr int kBarFull = 0;             // L kUnits: both CTAs' parts of the unit have landed
constexpr int kBarEmpty = kBarFull + kUnits;    // kUnits: the MMAs have read the unit
constexpr int kBarQFull = kBarEmpty + kUnits;   // L
constexpr int kBarQLand = kBarQFull + 1;        // e4m3: this CTA's q has landed (and is to become f16)
constexpr int kBarQEmpty = kBarQLand + 1;       // the row tile's scores are done
constexpr int kBarSFull = kBarQEmpty + 1;       // kSlots
constexpr int kBarSFree = kBarSFull + kSlots;   // L kSlots
constexpr int kBarPFull = kBarSFree + kSlots;   // L 2
constexpr int kBarPvDone = kBarPFull + 2;       // 2
constexpr int kBarInfoFull = kBarPvDone + 2;    // kInfos
constexpr int kBarInfoFree = kBarInfoFull + kInfos;  // kInfos
constexpr int kBarGrant = kBarInfoFree + kInfos;     // kUnits: the unit is the fill warps' to fill
constexpr int kBarDrain = kBarGrant + kUnits;
constexpr int kNumBars = kBarDrain + 1;
constexpr int kOffMisc = kOffBars + kNumBars * 8;  // tmem base, abort flag
constexpr int kSmemBytes = kOffMisc + 16 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory map exceeds 227 KB");
static_assert(sizeof(TileInfo) % 16 == 0, "");

constexpr int kNamedAll = 3;    // the eight of them
constexpr int kNamedRows0 = 1;  // the four softmax warps of 32 rows meet on 1 + (rows' half)

constexpr int kTmemCols = 512;
constexpr int kTmemO = 0;    // 256 columns: 128 for each half of the channels
constexpr int kTmemS = 256;  // 64 columns a slot

__device__ __forceinline__ void tmem_alloc2(uint32_t dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}
// One MMA of the pair: the descriptors' addresses hold in both CTAs. Of a descriptor only the lower half (the start address)
// changes from one MMA to the next.
__device__ __forceinline__ void umma2_f16(uint32_t d, uint32_t a, uint32_t a_hi, uint32_t b, uint32_t b_hi, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 a, {%1, %2};\n\t"
      "mov.b64 b, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
      "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on the barrier at this offset in both CTAs when this thread's MMAs so far are done.
__device__ __forceinline__ void umma2_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
// A TMA load into this CTA whose bytes are counted on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma2_load_2d(uint32_t dst, const void* tmap, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// Arrivals on a barrier of CTA 0 of the pair, which its MMA thread waits for at cluster scope. arrive_lead announces what the
// warp's threads have written to their own CTA's shared memory for the MMAs (each thread behind a proxy fence, then all
// behind a __syncwarp); its release is of that memory only. A release of everything at cluster scope waits for all that the
// thread has in flight (128 x 64 x 32768: 459 us against 387). Relaxed arrivals hand back what has been read, or announce loads
// whose bytes the barrier counts.
__device__ __forceinline__ void arrive_lead(uint32_t bar) {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
  mbar_arrive_remote_relaxed(bar);
}
__device__ __forceinline__ void arrive_lead_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void tma2_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// Barriers that the other CTA of the pair, or the MMAs of CTA 0, arrive on are observed at cluster scope.
__device__ __forceinline__ bool mbar_test_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// The bounded wait of a single thread that is waited for: it looks again and again for a while before it sleeps. (A thread that
// sleeps in a wait was seen to wake up to 1200 cycles behind the commit of MMAs that it waited for; more than a few
// threads that look keep the others from their barriers.)
template <bool kCluster>
__device__ __forceinline__ bool mbar_wait_awake(uint32_t bar, uint32_t parity, const WaitCtl& wc) {
#pragma unroll 1
  for (int i = 0; i < 256; ++i)
    if (kCluster ? mbar_test_wait_cluster(bar, parity) : mbar_test_wait(bar, parity)) return true;
  return kCluster ? mbar_wait_cluster(bar, parity, wc) : mbar_wait<true>(bar, parity, wc);
}
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}

// The tiles of pair c: [lo, hi) of all row tiles' tiles laid end to end, walked in segments of one row tile.
struct Segments {
  const SharedPrefixParams& p;
  long long at, hi, start, first, end;  // `first`, `end`: the tiles of row tile rt
  int rt;
  __device__ explicit Segments(const SharedPrefixParams& params) : p(params) {
    const PairStart s = p.pairs[blockIdx.x >> 1];
    at = start = s.lo;
    hi = s.hi;
    first = s.first;
    end = s.end;
    rt = s.row_tile;
  }
  // The next segment: row tile, first tile in it, tiles; whether it is all of the row tile; where it goes if not.
  int row_tile, t0, nt, part;
  bool complete;
  __device__ bool next() {
    if (at >= hi) return false;
    while (at >= end) {  // (row tiles without a tile are passed over)
      ++rt;
      first = end;
      end = p.tile_first[rt + 1];
    }
    row_tile = rt;
    t0 = static_cast<int>(at - first);
    const long long to = end < hi ? end : hi;
    nt = static_cast<int>(to - at);
    complete = at == first && to == end;
    part = static_cast<int>(2 * (blockIdx.x >> 1)) + (at == start ? 0 : 1);
    at = to;
    return true;
  }
};

// ---------------------------------------------------------------------------------- resolver
// One warp: lane l looks up list rows 4 l .. 4 l + 3, all of piece l / 4.
__device__ void resolve_role(const SharedPrefixParams& p, uint8_t* smem, uint32_t bars, uint32_t crank, const WaitCtl& wc) {
  const int lane = threadIdx.x & 31;
  auto bar = [&](int i) -> uint32_t { return bars + 8u * static_cast<uint32_t>(i); };
  TileInfo* infos = reinterpret_cast<TileInfo*>(smem + kOffInfo);
  Segments seg(p);
  uint32_t k = 0;
  bool err = false;
  const int P = p.page_size;
  const int room = static_cast<int>(min(static_cast<long long>(p.max_blocks) * P, 0x7fffffffll));
  while (seg.next()) {
    const RowTile rt = p.row_tiles[seg.row_tile];
    const long long own0 = p.own_before[rt.t_first];
    const int own_all = static_cast<int>(p.own_before[rt.t_last + 1] - own0);
    // query rt.t_first + lane (a row tile of more than 32 queries is looked up in memory)
    const int queries = rt.t_last - rt.t_first + 1, mine = rt.t_first + lane;
    int q_before = 0, q_len = 0, q_req = 0;
    if (lane < queries) {
      q_before = static_cast<int>(p.own_before[mine] - own0);
      q_len = p.token_len[mine];
      q_req = p.req_of_token != nullptr ? p.req_of_token[mine] : mine;
    }
    for (int t = seg.t0; t < seg.t0 + seg.nt; ++t, ++k) {
      const uint32_t r = k % kInfos;
      const int piece = t * kPieces + (lane >> 2);
      int owner = -1, pos = 0, lo = 0, hi = 0, req = 0;
      const int in = piece - rt.shared_pieces;  // among the pieces that the queries have to themselves
      // the last query whose own pieces begin at or before this one
      int a = 0;
      if (queries <= 32) {
#pragma unroll
        for (int step = 16; step > 0; step >>= 1) {
          const int v = __shfl_sync(0xffffffffu, q_before, (a + step) & 31);
          if (a + step < queries && v <= in) a += step;
        }
      } else if (in >= 0) {
        int z = queries - 1;
        while (a < z) {
          const int mid = (a + z + 1) >> 1;
          if (p.own_before[rt.t_first + mid] - own0 <= in)
            a = mid;
          else
            z = mid - 1;
        }
      }
      int before = __shfl_sync(0xffffffffu, q_before, a & 31), len = __shfl_sync(0xffffffffu, q_len, a & 31),
          its = __shfl_sync(0xffffffffu, q_req, a & 31);
      if (in < 0) {
        pos = piece * kListPiece;
        hi = rt.shared_len;
        req = rt.req;
      } else if (in < own_all) {
        owner = rt.t_first + a;
        if (queries > 32) {
          before = static_cast<int>(p.own_before[owner] - own0);
          len = p.token_len[owner];
          its = p.req_of_token != nullptr ? p.req_of_token[owner] : owner;
        }
        pos = (rt.prefix_len / kListPiece + in - before) * kListPiece;
        lo = rt.prefix_len;
        hi = len;
        req = its;
      }
      hi = min(hi, room);
      // the cache rows of positions pos + 4 (lane % 4) .. + 3; with pages of whole pieces, by one look at the table
      const int at0 = pos + 4 * (lane & 3);
      const int32_t* row = p.block_table + static_cast<long long>(req) * p.max_blocks;
      int slot[4], base = 0;
      if (p.pieces) {
        bool live = max(pos, lo) < min(pos + kListPiece, hi);
        if (live) {
          const int in_table = p.page_shift >= 0 ? pos >> p.page_shift : pos / P;
          const int page = __ldg(row + in_table);
          if (page >= 0 && page < p.num_pages)
            base = page * P + (pos - in_table * P);  // (below 2^31)
          else
            err = true, live = false;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) slot[i] = live && at0 + i >= lo && at0 + i < hi ? base + 4 * (lane & 3) + i : -1;
        // a piece without rows is loaded from behind the half's first one, whatever is there
        const int first = __shfl_sync(0xffffffffu, base, lane & 16);
        if (!live) base = first + kListPiece * ((lane >> 2) & 3);
      } else {
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          int at = -1;
          if (at0 + i >= lo && at0 + i < hi) {
            const int in_table = (at0 + i) / P;
            const int page = __ldg(row + in_table);
            if (page >= 0 && page < p.num_pages)
              at = page * P + (at0 + i - in_table * P);
            else
              err = true;
          }
          slot[0] = i == 0 ? at : slot[0];
          slot[1] = i == 1 ? at : slot[1];
          slot[2] = i == 2 ? at : slot[2];
          slot[3] = i == 3 ? at : slot[3];
        }
      }
      const int half0 = __shfl_sync(0xffffffffu, base, lane & 16);
      const bool halves = __all_sync(0xffffffffu, base == half0 + kListPiece * ((lane >> 2) & 3));
      const bool all = __all_sync(0xffffffffu, slot[0] >= 0 && slot[1] >= 0 && slot[2] >= 0 && slot[3] >= 0);
      const bool whole = __all_sync(0xffffffffu, owner < 0 && pos + kListPiece <= min(hi, rt.min_len)) && all;
      const bool owned = __any_sync(0xffffffffu, owner >= 0);
      uint32_t dead = 0;  // rows of the piece inside its range without a cache row
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (at0 + i >= lo && at0 + i < hi && slot[i] < 0) dead = 1;
      dead |= __shfl_xor_sync(0xffffffffu, dead, 1);
      dead |= __shfl_xor_sync(0xffffffffu, dead, 2);
      const bool freed = k < kInfos || mbar_wait<true>(bar(kBarInfoFree + r), ((k / kInfos) - 1) & 1u, wc);
      if (!__all_sync(0xffffffffu, freed)) return;
      TileInfo& info = infos[r];
      reinterpret_cast<int4*>(info.slot)[lane] = make_int4(slot[0], slot[1], slot[2], slot[3]);
      if ((lane & 3) == 0) {
        const int g = lane >> 2;
        info.base[g] = base;
        info.pos[g] = pos;
        info.lo[g] = lo | static_cast<int>(dead) << 31;
        info.hi[g] = hi;
        info.owner[g] = owner;
      }
      if (lane == 0) {
        info.mode = !p.pieces ? kFillThreadwise : halves ? kFillHalves : kFillPieces;
        info.whole = whole;
        info.fix = p.pieces && !all;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarInfoFull + r));
      if (owned) {
        // rows of a query's own come from DRAM: into the L2 ahead of their loads (each CTA half of them)
#pragma unroll 1
        for (int j = 0; j < 2; ++j) {
          const int at = info.slot[64 * crank + 32 * j + lane];
          if (at >= 0) {
            const uint8_t* src = p.kv + at * p.row_stride;
#pragma unroll 1
            for (int c = 0; c < p.row_bytes; c += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + c));
          }
        }
      }
    }
  }
  if (__any_sync(0xffffffffu, err) && lane == 0) atomicOr(p.status, SVT_DEV_ERR_INDEX_RANGE);
}

// ---------------------------------------------------------------------------------- units
// A place in the ring and the parity of its laps.
struct Ring {
  uint32_t at = 0, lap = 0;
  __device__ __forceinline__ void step(uint32_t n = 1) {
    at += n;
    if (at >= kUnits) {
      at -= kUnits;
      lap ^= 1u;
    }
  }
};

// A segment's units are staged and consumed in the order K(0), K(1), V(0), K(2), V(1), .. V(nt - 1). The roles' code for them stands
// in one place each and is kept short: it has to fit the instruction cache. (With the loops unrolled, 100 KB in all, a
// third of the warps' waiting was for instructions.)

// Two threads, each every second unit in the order of their use: a unit costs a thread some 300 cycles (its wait, an arrival and
// one load), the MMAs 256. They load what TMA can and grant the other units to the fill warps, or have them know of loads that are
// to be mended. A wait tells a phase from the next one, not from the one after: when a thread waits for unit u - 7 to be read,
// unit u - 14 must have been; it knows that from its unit before, u - 2. The fill warps, which may be tiles behind or
// ahead, could not know: they wait for grants.
template <bool kF16>
__device__ void tma_role(const SharedPrefixParams& p, uint8_t* smem, uint32_t bars, uint32_t crank, uint32_t me,
                         const WaitCtl& wc) {
  const uint32_t ring0 = smem_u32(smem) + kOffRing;
  auto bar = [&](int i) -> uint32_t { return bars + 8u * static_cast<uint32_t>(i); };
  const uint32_t lead_full = mapa_shared(bars, 0) + 8u * kBarFull;
  const TileInfo* infos = reinterpret_cast<const TileInfo*>(smem + kOffInfo);
  Segments seg(p);
  // this thread's next unit: its place in the ring and the parity of its lap (in the first one the waits pass: they are for
  // the phase before a barrier's first)
  uint32_t at = me, lap = 0;
  int turn = static_cast<int>(me);  // 0: the next unit of all is this thread's
  const uint32_t empty0 = bar(kBarEmpty);
  uint32_t k0 = 0;
  bool withhold = (p.fault & kFaultWithholdFirstFill) != 0;
  uint32_t s = 0;
  for (; seg.next(); ++s) {
    if (me == 0) {
      // this CTA's 64 query rows (past the row tile's end: rows that nobody stores; past q's: zeroes)
      if (s > 0 && !mbar_wait_cluster(bar(kBarQEmpty), (s - 1) & 1u, wc)) return;
      const int row = p.row_tiles[seg.row_tile].row0 + kRows * static_cast<int>(crank);
      const uint32_t on = kF16 ? bar(kBarQLand) : mapa_shared(bar(kBarQFull), 0);
      if (kF16)
        mbar_arrive_expect_tx(on, 9 * kBlk);
      else
        arrive_lead_expect_tx(on, 9 * kBlk);
#pragma unroll 1
      for (int b = 0; b < 9; ++b) tma2_load_2d(smem_u32(smem) + kOffQ + b * kBlk, &p.q_map, 64 * b, row, on);
    }
    const int nt = seg.nt;
    for (int t = 0; t <= nt; ++t) {
      // step t: the units of K(t), then of V(t - 1)
      const uint32_t rk = (k0 + t) % kInfos, rv = (k0 + t - 1) % kInfos;
      if (t < nt && !mbar_wait_awake<false>(bar(kBarInfoFull + rk), ((k0 + t) / kInfos) & 1u, wc)) return;
      const TileInfo &ik = infos[rk], &iv = infos[rv];
      const int mode_k = t < nt ? ik.mode : kFillNone, mode_v = t > 0 ? iv.mode : kFillNone;
      if (mode_k == kFillHalves && mode_v == kFillHalves && iv.fix == 0 && !withhold) {
        // the long run of a prefix: nothing that can be left out of a unit
        const int yk = ik.base[4 * crank], y0 = iv.base[0], y1 = iv.base[4];
        // turn 0: K blocks 0, 4, 8 (behind the rope columns the box's second block is filled with zeroes) and channels 256 .. of V; turn
        // 1: K blocks 2, 6 and channels 0 .. of V
        const int nk = 3 - turn, zv = 2 * static_cast<int>(crank) + 4 * (1 - turn);
#pragma unroll 1
        for (int j = 0; j < nk + 2; ++j) {
          if (!mbar_wait_awake<true>(empty0 + 8u * at, lap ^ 1u, wc)) return;
          const uint32_t full = lead_full + 8u * at;
          arrive_lead_expect_tx(full, kUnit);
          tma2_load_3d(ring0 + at * kUnit, &p.kv_map64, 0, j < nk ? yk : j == nk ? y0 : y1, j < nk ? 2 * turn + 4 * j : zv, full);
          at += 2;
          if (at >= kUnits) {
            at -= kUnits;
            lap ^= 1u;
          }
        }
        turn ^= 1u;
      } else {
        int i = 0;
        const int units = (t < nt ? kKUnits : 0) + (t > 0 ? kVUnits : 0);
#pragma unroll 1
        for (i = turn; i < units; i += 2) {
          const bool v = t == nt || i >= kKUnits;
          const int j = v && t < nt ? i - kKUnits : i;
          const int mode = v ? mode_v : mode_k;
          const TileInfo& info = v ? iv : ik;
          if (!mbar_wait_awake<true>(empty0 + 8u * at, lap ^ 1u, wc)) return;
          const uint32_t dst = ring0 + at * kUnit;
          const int* base = info.base + 4 * (v ? j >> 1 : static_cast<int>(crank));
          const int block = v ? 4 * (j & 1) + 2 * static_cast<int>(crank) : 2 * j;
          const bool fix = v && info.fix != 0;  // by way of a fill warp
          const uint32_t on = fix ? bar(kBarGrant + at) : lead_full + 8u * at;
          const int bytes = mode == kFillPieces && block == 8 ? kBlk : kUnit;
          if (mode == kFillThreadwise) {
            mbar_arrive_relaxed(bar(kBarGrant + at));
          } else if (!withhold) {
            if (fix)
              mbar_arrive_expect_tx(on, bytes);
            else
              arrive_lead_expect_tx(on, bytes);
            if (mode == kFillHalves) {
              tma2_load_3d(dst, &p.kv_map64, 0, base[0], block, on);
            } else {
              const int4 rows = *reinterpret_cast<const int4*>(base);
#pragma unroll 1
              for (int g = 0; g < (block == 8 ? 1 : 2); ++g) {
                const uint32_t to = dst + g * kBlk;
                const int x = 64 * (block + g);
                tma2_load_2d(to, &p.kv_map16, x, rows.x, on);
                tma2_load_2d(to + kListPiece * 128, &p.kv_map16, x, rows.y, on);
                tma2_load_2d(to + 2 * kListPiece * 128, &p.kv_map16, x, rows.z, on);
                tma2_load_2d(to + 3 * kListPiece * 128, &p.kv_map16, x, rows.w, on);
              }
            }
          }
          withhold = false;
          at += 2;
          if (at >= kUnits) {
            at -= kUnits;
            lap ^= 1u;
          }
        }
        turn = (turn + units) & 1;
      }
      if (t > 0) mbar_arrive_relaxed(bar(kBarInfoFree + rv));
    }
    k0 += nt;
  }
  if (me == 0 && s > 0) mbar_wait_cluster(bar(kBarQEmpty), (s - 1) & 1u, wc);  // (the last one lands before the CTA leaves)
}

// The fill warps fill the units that are granted to them: 16-byte pieces of 64 rows, zeroes where there is no row; or put the zeroes
// into a unit of V that TMA has loaded. (What a masked row of K holds is masked in S. In V it would meet a P of zero, and a
// cache row that no token has been written to may hold NaN.) A place of the ring is always the same warp's: so it has waited
// for each of the place's grants, and a wait cannot take one for the next but one.
template <bool kF16>
__device__ void fill_role(const SharedPrefixParams& p, uint8_t* smem, uint32_t bars, uint32_t crank, const WaitCtl& wc) {
  constexpr int kFillWarps = fill_warps(kF16), kFillThreads = 32 * kFillWarps;
  const int lane = threadIdx.x & 31;
  const uint32_t me = (threadIdx.x >> 5) - kFillWarp0;
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return bars + 8u * static_cast<uint32_t>(i); };
  const uint32_t lead_bars = mapa_shared(bars, 0);
  const TileInfo* infos = reinterpret_cast<const TileInfo*>(smem + kOffInfo);
  Segments seg(p);
  Ring ring;
  uint32_t k0 = 0, s = 0;
  uint32_t granted = 0;  // the parity of the next grant of each of the warp's places
  bool range = false, withhold = (p.fault & kFaultWithholdFirstFill) != 0;
  int pending = -1;  // bf16: the unit whose copies are in flight
  auto announce = [&](int unit) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) arrive_lead(lead_bars + 8u * (kBarFull + unit));
  };
  auto flush = [&] {
    if (kF16 || pending < 0) return;
    cp_async_wait<0>();
    announce(pending);
    pending = -1;
  };
  // Until the unit may be filled, what is in flight is waited for and announced.
  auto unit_free = [&](uint32_t st) -> bool {
    const uint32_t parity = (granted >> st) & 1u;
    granted ^= 1u << st;
    if (pending >= 0 && !__all_sync(0xffffffffu, mbar_test_wait(bar(kBarGrant + st), parity))) flush();
    return __all_sync(0xffffffffu, mbar_wait<true>(bar(kBarGrant + st), parity, wc));
  };
  auto mend = [&](const TileInfo& info, int i) -> bool {
    const uint32_t st = ring.at;
    const int* slots = info.slot + 64 * (i >> 1);
    if (!unit_free(st)) return false;
    uint8_t* to = smem + kOffRing + st * kUnit;
#pragma unroll 1
    for (int row = lane; row < 64; row += 32) {
      if (slots[row] < 0) {
#pragma unroll
        for (int c = 0; c < 16; ++c)
          *reinterpret_cast<uint4*>(to + (c >> 3) * kBlk + row * 128 + 16 * (c & 7)) = make_uint4(0, 0, 0, 0);
      }
    }
    announce(st);
    return true;
  };
  auto fill = [&](const TileInfo& info, bool v, int i) -> bool {
    const uint32_t st = ring.at;
    const bool rope = !v && i == kKUnits - 1;
    const int x0 = v ? 256 * (i & 1) + 128 * static_cast<int>(crank) : 128 * i;
    const int* slots = info.slot + 64 * (v ? i >> 1 : static_cast<int>(crank));
    if constexpr (!kF16) {
      if (!unit_free(st)) return false;
      const uint32_t dst = sbase + kOffRing + st * kUnit;
      // 16-byte pieces of the unit's columns: 16 (rope: 8) of a row by neighbouring lanes
      const int log = rope ? 3 : 4, chunk = lane & ((1 << log) - 1), rows = 32 >> log;
      const uint32_t to = dst + (chunk >> 3) * kBlk;
      const long long col = x0 * 2 + chunk * 16;
#pragma unroll 4
      for (int row = lane >> log; row < 64; row += rows) {
        const int slot = slots[row];
        cp_async16(to + sw128_offset(row, chunk & 7), p.kv + (slot >= 0 ? slot * p.row_stride + col : 0), slot >= 0 ? 16u : 0u);
      }
      cp_async_commit();
      if (pending >= 0) {
        cp_async_wait<1>();
        announce(pending);
      }
      pending = withhold ? -1 : static_cast<int>(st);
    } else {
      // 16 bytes: 16 codes, or 8 rope values; a row's 8 pieces by neighbouring lanes, four rows at a time, four times that in
      // registers while four before are converted
      const int chunk = lane & 7, row0 = lane >> 3;
      const long long col = (rope ? kVdim + 16 : x0) + chunk * 16;
      uint8_t* to = smem + kOffRing + st * kUnit + (rope ? 0 : (chunk >> 2) * kBlk);
      uint4 raw[2][4];
      float scale[2][4];
      auto load = [&](int h, uint4 (&w)[4], float (&f)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int slot = slots[16 * h + 4 * j + row0];
          w[j] = make_uint4(0, 0, 0, 0);
          f[j] = 0.f;
          if (slot >= 0) {
            const uint8_t* src = p.kv + slot * p.row_stride;
            w[j] = __ldg(reinterpret_cast<const uint4*>(src + col));
            if (!rope) f[j] = v ? __ldg(reinterpret_cast<const float*>(src + kVdim) + (x0 >> 7)) : 1.f;
          }
        }
      };
      auto convert = [&](int h, const uint4 (&raw4)[4], const float (&f)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = 16 * h + 4 * j + row0;
          const uint32_t w[4] = {raw4[j].x, raw4[j].y, raw4[j].z, raw4[j].w};
          if (rope) {
            uint32_t o[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              range |= bf16x2_beyond_f16(w[q]);
              o[q] = bf16x2_to_f16x2(w[q]);
            }
            *reinterpret_cast<uint4*>(to + sw128_offset(row, chunk)) = make_uint4(o[0], o[1], o[2], o[3]);
          } else {
            uint32_t hi2, lo2, o[8];
            split_scale_f16x2(f[j], hi2, lo2);
            range |= !(448.f * fabsf(f[j]) <= 65504.f);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              o[2 * q] = e4m3x2_times_f16x2(w[q] & 0xffffu, hi2, lo2);
              o[2 * q + 1] = e4m3x2_times_f16x2(w[q] >> 16, hi2, lo2);
            }
            // 16 channels: two pieces of the block that holds them
            *reinterpret_cast<uint4*>(to + sw128_offset(row, 2 * (chunk & 3))) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(to + sw128_offset(row, 2 * (chunk & 3) + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
          }
        }
      };
      load(0, raw[0], scale[0]);
      load(1, raw[1], scale[1]);
      if (!unit_free(st)) return false;
#pragma unroll 1
      for (int h = 0; h < 4; h += 2) {
        convert(h, raw[0], scale[0]);
        if (h == 0) load(2, raw[0], scale[0]);
        convert(h + 1, raw[1], scale[1]);
        if (h == 0) load(3, raw[1], scale[1]);
      }
      if (!withhold) announce(st);
    }
    return true;
  };
  bool ok = true;
  while (ok && seg.next()) {
    if (kF16) {
      // q: bf16 -> f16 in place
      ok = __all_sync(0xffffffffu, mbar_wait<true>(bar(kBarQLand), s & 1u, wc));
      if (!ok) break;
      const int rows = p.row_tiles[seg.row_tile].nrows - kRows * static_cast<int>(crank);
#pragma unroll 2
      for (int i = static_cast<int>(threadIdx.x) - kFillWarp0 * 32; i < 9 * kBlk / 16; i += kFillThreads) {
        uint4* at = reinterpret_cast<uint4*>(smem + kOffQ) + i;
        uint4 w = *at;
        if (((i >> 3) & 63) < rows)  // (rows of other queries, not stored, say nothing about the range)
          range |= bf16x2_beyond_f16(w.x) || bf16x2_beyond_f16(w.y) || bf16x2_beyond_f16(w.z) || bf16x2_beyond_f16(w.w);
        *at = make_uint4(bf16x2_to_f16x2(w.x), bf16x2_to_f16x2(w.y), bf16x2_to_f16x2(w.z), bf16x2_to_f16x2(w.w));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive_lead(lead_bars + 8u * kBarQFull);
      ++s;
    }
    for (int step = 0; ok && step < 2 * seg.nt + 2; ++step) {
      const bool v = (step & 1) != 0;
      const int t = (step >> 1) - (v ? 1 : 0), units = v ? kVUnits : kKUnits;
      if (t < 0 || t >= seg.nt) continue;
      const uint32_t k = k0 + t, r = k % kInfos;
      const TileInfo& info = infos[r];
      if (!v) ok = __all_sync(0xffffffffu, mbar_wait<true>(bar(kBarInfoFull + r), (k / kInfos) & 1u, wc));
      if (!ok) break;
      const bool threadwise = info.mode == kFillThreadwise;
      if (!threadwise && !(v && info.fix != 0)) {
        ring.step(units);
        withhold = false;
      } else {
#pragma unroll 1
        for (int i = 0; i < units; ++i) {
          if (ring.at % kFillWarps == me && !(threadwise ? fill(info, v, i) : mend(info, i))) {
            ok = false;
            break;
          }
          ring.step();
          withhold = false;
        }
        if (!ok) break;
        flush();
      }
      if (v) {
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(bar(kBarInfoFree + r));
      }
    }
    k0 += seg.nt;
  }
  if (!kF16) cp_async_wait_all();
  if (kF16 && __any_sync(0xffffffffu, range) && lane == 0) atomicOr(p.status, SVT_DEV_ERR_FP8_RANGE);
}

// ---------------------------------------------------------------------------------- MMA issuer
// One thread.
template <bool kF16>
__device__ void mma_role(const SharedPrefixParams& p, uint8_t* smem, uint32_t tmem, uint32_t bars, const WaitCtl& wc) {
  constexpr int kFmt = kF16 ? kFmtF16 : kFmtBf16;
  constexpr uint32_t kIdescS = idesc_f32acc(128, 128, 0, 0, kFmt);
  constexpr uint32_t kIdescPv = idesc_f32acc(128, 256, 0, 1, kFmt);
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return bars + 8u * static_cast<uint32_t>(i); };
  auto wait = [&](int i, uint32_t parity) -> bool {
    return mbar_test_wait_cluster(bar(i), parity) || mbar_wait_cluster(bar(i), parity, wc);
  };
  const uint64_t dk = smem_desc_sw128(sbase, 16, 1024), dv = smem_desc_sw128(sbase, kBlk, 1024);
  const uint32_t k_hi = static_cast<uint32_t>(dk >> 32), v_hi = static_cast<uint32_t>(dv >> 32);
  const uint32_t k_lo = static_cast<uint32_t>(dk), v_lo = static_cast<uint32_t>(dv);
  Segments seg(p);
  uint32_t k0 = 0, s = 0;
  Ring ring;
  while (seg.next()) {
    if (!wait(kBarQFull, s & 1u)) return;
    ++s;
    for (int t = 0; t <= seg.nt; ++t) {
      if (t < seg.nt) {
        const uint32_t k = k0 + t, b = k & 1u;
        uint32_t d = tmem + kTmemS + 64 * b;
        if (!kF16 && k >= 2 && !wait(kBarSFree + b, ((k >> 1) - 1) & 1u)) return;
#pragma unroll
        for (int i = 0; i < kKUnits; ++i) {
          const uint32_t st = ring.at, u = kKUnits * k + i, slot = u % kSlots;
          if (kF16) {
            d = tmem + kTmemS + 64 * slot;
            if (u >= kSlots && !wait(kBarSFree + slot, (u / kSlots - 1) & 1u)) return;
          }
          if (!wait(kBarFull + st, ring.lap)) return;
          ring.step();
          tc_fence_after();
          const uint32_t from = k_lo + (kOffRing >> 4) + st * (kUnit >> 4);
#pragma unroll
          for (int ks = 0; ks < (i == kKUnits - 1 ? 4 : 8); ++ks) {
            const uint32_t off = (ks >> 2) * (kBlk >> 4) + (ks & 3) * 2;
            umma2_f16(d, k_lo + ((kOffQ + i * kUnit) >> 4) + off, k_hi, from + off, k_hi, kIdescS, ((kF16 ? 0 : i) | ks) != 0);
          }
          umma2_commit(bar(kBarEmpty + st));
          if (kF16) umma2_commit(bar(kBarSFull + slot));
        }
        if (!kF16) umma2_commit(bar(kBarSFull + b));
        if (t == seg.nt - 1) umma2_commit(bar(kBarQEmpty));
      }
      if (t > 0) {
        const uint32_t k = k0 + t - 1, b = k & 1u;
        if (!wait(kBarPFull + b, (k >> 1) & 1u)) return;
        const uint32_t p_lo = k_lo + (kOffP >> 4) + b * (kPBytes >> 4);
#pragma unroll
        for (int i = 0; i < kVUnits; ++i) {
          const uint32_t st = ring.at;
          if (!wait(kBarFull + st, ring.lap)) return;
          ring.step();
          tc_fence_after();
          const uint32_t from = v_lo + (kOffRing >> 4) + st * (kUnit >> 4);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            umma2_f16(tmem + kTmemO + 128 * (i & 1), p_lo + (i >> 1) * (kBlk >> 4) + ks * 2, k_hi, from + ks * (2048 >> 4), v_hi,
                      kIdescPv, (i >> 1 | ks) != 0 || t > 1);
          umma2_commit(bar(kBarEmpty + st));
        }
        umma2_commit(bar(kBarPvDone + b));
      }
    }
    k0 += seg.nt;
  }
}

// ---------------------------------------------------------------------------------- softmax
// Thread: TMEM lane 32 q + lane, that is row (q & 1) * 32 + lane of the CTA and the list rows 64 (q >> 1) + 32 hs .. + 31 of a
// tile; of O the channels 256 hs + 128 (q >> 1) .. + 127.
template <bool kF16>
__device__ void softmax_role(const SharedPrefixParams& p, uint8_t* smem, uint32_t tmem, uint32_t bars, uint32_t crank,
                             const WaitCtl& wc) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = warp & 3, hs = (warp - kSoftWarp0) >> 2;
  const int row = (q & 1) * 32 + lane, quarter = (q >> 1) * 2 + hs;
  const int col0 = 32 * quarter;
  const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * q) << 16);
  auto bar = [&](int i) -> uint32_t { return bars + 8u * static_cast<uint32_t>(i); };
  auto lead_bar = [&](int i) -> uint32_t { return mapa_shared(bar(i), 0); };
  const TileInfo* infos = reinterpret_cast<const TileInfo*>(smem + kOffInfo);
  float* red = reinterpret_cast<float*>(smem + kOffRed);
  float* sums = reinterpret_cast<float*>(smem + kOffSum);
  const uint32_t named = kNamedRows0 + (q & 1);
  Segments seg(p);
  const int r = kRows * static_cast<int>(crank) + row;
  // what is to be known of a segment, read while the one before is computed
  struct Coming {
    RowTile rt;
    int nt, part, token, len;
    bool complete, valid;
  } coming;
  auto look = [&]() -> bool {
    if (!seg.next()) return false;
    coming.rt = p.row_tiles[seg.row_tile];
    coming.nt = seg.nt;
    coming.part = seg.part;
    coming.complete = seg.complete;
    coming.valid = r < coming.rt.nrows;
    coming.token = coming.valid ? (coming.rt.row0 + r) / p.H : -2;
    coming.len = coming.valid ? p.token_len[coming.token] : 0;
    return true;
  };
  uint32_t k = 0;
  bool more = look();
  while (more) {
    const RowTile rt = coming.rt;
    const int nt = coming.nt, part = coming.part, token = coming.token, len = coming.len;
    const bool complete = coming.complete, valid = coming.valid;
    more = look();
    float m = -CUDART_INF_F, l = 0.f;
    for (int t = 0; t < nt; ++t, ++k) {
      const uint32_t b = k & 1u, ring = k % kInfos;
      const bool told = mbar_wait<true>(bar(kBarInfoFull + ring), (k / kInfos) & 1u, wc);
      const TileInfo& info = infos[ring];
      const bool whole = info.whole != 0;
      uint32_t live = 0xffffffffu;
      if (!whole) {
        live = 0;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int at = 2 * quarter + g;
          const int pos = info.pos[at], owner = info.owner[at], lo = info.lo[at] & 0x7fffffff;
          const int a = max(lo - pos, 0), z = min(min(info.hi[at], len) - pos, kListPiece);
          uint32_t bits = 0;
          if (z > a && (owner < 0 || owner == token)) bits = ((1u << z) - 1u) & ~((1u << a) - 1u);
          if (info.lo[at] < 0) {  // rows whose page is out of range
            for (int i = 0; i < kListPiece; ++i)
              if (info.slot[kListPiece * at + i] < 0) bits &= ~(1u << i);
          }
          live |= bits << (kListPiece * g);
        }
      }
      float scales[4] = {0.f, 0.f, 0.f, 0.f};
      if (kF16) {
        const int slot = info.slot[32 * quarter + lane];
        if (told && slot >= 0) {  // (after a wait that gave up, the slots say nothing)
          const float4 of = __ldg(reinterpret_cast<const float4*>(p.kv + slot * p.row_stride + kVdim));
          scales[0] = of.x, scales[1] = of.y, scales[2] = of.z, scales[3] = of.w;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarInfoFree + ring));
      // e4m3: a unit of K holds its codes as they are (f16 holds them exactly), and the four sums of a score's 128 channels
      // each meet their scales here, in fp32. (Codes times scales in f16 had scores 2^-12 of their terms off: 7e-5 of the lse of ten rows.)
      float acc[32];
      if (kF16) {
        float* const mine = reinterpret_cast<float*>(smem + kOffScales) + (warp - kSoftWarp0) * 128;
#pragma unroll
        for (int i = 0; i < 4; ++i) mine[32 * i + lane] = scales[i];
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 32; ++c) acc[c] = 0.f;
#pragma unroll 1
        for (int i = 0; i < kKUnits; ++i) {
          const uint32_t u = kKUnits * k + i, slot = u % kSlots;
          mbar_wait_cluster(bar(kBarSFull + slot), (u / kSlots) & 1u, wc);
          tc_fence_after();
          uint32_t sv[32];
          tmem_ld32(lanes + kTmemS + 64 * slot + 32 * hs, sv);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote_relaxed(lead_bar(kBarSFree + slot));
          if (i == kKUnits - 1) {
#pragma unroll
            for (int c = 0; c < 32; ++c) acc[c] += __uint_as_float(sv[c]);
          } else {
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              const float4 f = *reinterpret_cast<const float4*>(mine + 32 * i + c);
              acc[c] = fmaf(__uint_as_float(sv[c]), f.x, acc[c]);
              acc[c + 1] = fmaf(__uint_as_float(sv[c + 1]), f.y, acc[c + 1]);
              acc[c + 2] = fmaf(__uint_as_float(sv[c + 2]), f.z, acc[c + 2]);
              acc[c + 3] = fmaf(__uint_as_float(sv[c + 3]), f.w, acc[c + 3]);
            }
          }
        }
      } else {
        mbar_wait_cluster(bar(kBarSFull + b), (k >> 1) & 1u, wc);
        tc_fence_after();
      }
      // the PV before the last has read this buffer of P
      if (t > 1) mbar_wait_cluster(bar(kBarPvDone + b), ((k >> 1) - 1) & 1u, wc);
      const uint32_t from = lanes + kTmemS + 64 * b + 32 * hs;
      uint8_t* pb = smem + kOffP + b * kPBytes + (col0 >> 6) * kBlk;
      // P relative to the reference maximum as it is; only if a score passes it by 2^8 (or is the first) it is moved and P made again
      float sum = 0.f, over = -CUDART_INF_F;
      auto make = [&] {
        const float ref = m == -CUDART_INF_F ? 0.f : m;
        float s0 = 0.f, s1 = 0.f;
#pragma unroll(kF16 ? 2 : 1)
        for (int h = 0; h < 2; ++h) {
          uint32_t sv[16];
          if (kF16) {
#pragma unroll
            for (int c = 0; c < 16; ++c) sv[c] = __float_as_uint(acc[16 * h + c]);
          } else {
            tmem_ld16(from + 16 * h, sv);
            tmem_ld_wait();
          }
          // (the mask behind the scale, which may be 0 or negative)
#pragma unroll
          for (int c = 0; c < 16; ++c) sv[c] = __float_as_uint(fmaf(__uint_as_float(sv[c]), p.scale_log2, -ref));
          if (!whole) {
#pragma unroll
            for (int c = 0; c < 16; ++c) sv[c] = (live >> (16 * h + c)) & 1u ? sv[c] : 0xff800000u;
          }
          uint32_t w[8];
#pragma unroll
          for (int c = 0; c < 16; c += 2) {
            const float x = __uint_as_float(sv[c]), y = __uint_as_float(sv[c + 1]);
            over = fmaxf(over, fmaxf(x, y));
            const float a = ex2_approx(x), z = ex2_approx(y);
            s0 += a;
            s1 += z;
            w[c >> 1] = kF16 ? pack_f16x2(a, z) : pack_bf16x2(a, z);
          }
#pragma unroll
          for (int c = 0; c < 2; ++c)
            *reinterpret_cast<uint4*>(pb + sw128_offset(row, ((col0 & 63) >> 3) + 2 * h + c)) =
                make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        }
        sum = s0 + s1;
      };
      for (int pass = 0;; ++pass) {
        make();
        if (pass == 1) break;
        // (the first score of all moves the reference too: m is -inf, and any score is above it)
        const bool keep = m == -CUDART_INF_F ? over == -CUDART_INF_F : !(over > kTau);
        if (named_bar_red_and(named, 128, keep)) break;
        const float ref = m == -CUDART_INF_F ? 0.f : m;
        red[quarter * kRows + row] = over + ref;
        named_bar_sync(named, 128);
        float mn = m;
#pragma unroll
        for (int i = 0; i < 4; ++i) mn = fmaxf(mn, red[i * kRows + row]);
        named_bar_sync(named, 128);  // (red is written again by a later tile)
        const float alpha = m == -CUDART_INF_F ? 0.f : ex2_approx(m - mn);
        m = mn;
        l *= alpha;
        if (t > 0) {
          // O holds the tiles before this one once their PV is done
          mbar_wait_cluster(bar(kBarPvDone + (b ^ 1u)), ((k - 1) >> 1) & 1u, wc);
          tc_fence_after();
          if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
            for (int c = 0; c < 128; c += 16) {
              uint32_t o[16];
              tmem_ld16(lanes + kTmemO + 128 * hs + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st16(lanes + kTmemO + 128 * hs + c, o);
            }
            tmem_st_wait();
          }
          tc_fence_before();
        }
      }
      l += sum;
      tc_fence_before();
      __syncwarp();
      if (!kF16 && lane == 0) mbar_arrive_remote_relaxed(lead_bar(kBarSFree + b));
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_lead(lead_bar(kBarPFull + b));
    }
    // ------------------------------------------------------------------ epilogue
    sums[quarter * kRows + row] = l;
    named_bar_sync(named, 128);
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) total += sums[i * kRows + row];
    named_bar_sync(named, 128);  // (sums is written again by the next segment)
    mbar_wait_cluster(bar(kBarPvDone + ((k - 1) & 1u)), ((k - 1) >> 1) & 1u, wc);
    tc_fence_after();
    const float inv = total > 0.f ? 1.f / total : (total == total ? 0.f : total);
    const float lse2 = total > 0.f ? m + __log2f(total) : (total == total ? -CUDART_INF_F : total);
    const int ch0 = 256 * hs + 128 * (q >> 1);
    const long long grow = static_cast<long long>(rt.row0) + r;
    if (quarter == 0 && valid) {
      if (complete) {
        if (p.lse != nullptr) p.lse[grow] = lse2 * 0.69314718055994530942f;
      } else {
        p.part_lse[part * kTile + r] = lse2;
      }
    }
    // A partial row goes to the merge in f16, times a power of two for each 128 channels that brings their largest magnitude to
    // 2^14 .. 2^15: half of fp32's bytes (26 MB of them in a burst), with a relative error of 2^-11.
    float scale = inv;
    if (!complete) {
      float big = 0.f;
#pragma unroll 1
      for (int c = 0; c < 128; c += 16) {
        uint32_t o[16];
        tmem_ld16(lanes + kTmemO + 128 * hs + c, o);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) big = fmaxf(big, fabsf(__uint_as_float(o[i])));
      }
      const int e = total > 0.f ? static_cast<int>(__float_as_uint(big * inv) >> 23) : 0;  // biased; 255: inf (or NaN)
      const int shift = e == 255 || e == 0 ? 0 : min(127 + 14 - e, 100);
      scale = inv * __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
      if (valid)
        p.part_scale[(static_cast<long long>(part) * kTile + r) * 4 + (ch0 >> 7)] =
            __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
    }
    // 128 bytes of each of the warp's 32 rows at a time, turned round in P's place (its last reader is done) so that eight lanes
    // store a row's.
    const int row0 = kRows * static_cast<int>(crank) + (q & 1) * 32;
    uint8_t* turn = smem + kOffP + (4 * hs + q) * 4096;
    const long long first = complete ? static_cast<long long>(rt.row0) + row0 : static_cast<long long>(part) * kTile + row0;
    uint8_t* to = reinterpret_cast<uint8_t*>((complete ? p.out : p.part_o) + first * kVdim + ch0);
#pragma unroll 1
    for (int c = 0; c < 128; to += 128) {
#pragma unroll 1
      for (int j = 0; j < 8; j += 2, c += 16) {
        uint32_t o[16], w[8];
        tmem_ld16(lanes + kTmemO + 128 * hs + c, o);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = total > 0.f ? __uint_as_float(o[2 * i]) * scale : inv;
          const float y = total > 0.f ? __uint_as_float(o[2 * i + 1]) * scale : inv;
          w[i] = complete ? pack_bf16x2(x, y) : pack_f16x2(x, y);
        }
        *reinterpret_cast<uint4*>(turn + sw128_offset(lane, j)) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(turn + sw128_offset(lane, j + 1)) = make_uint4(w[4], w[5], w[6], w[7]);
      }
      __syncwarp();
#pragma unroll 4
      for (int it = 0; it < 8; ++it) {
        const int rr = 4 * it + (lane >> 3);
        const uint4 w = *reinterpret_cast<const uint4*>(turn + sw128_offset(rr, lane & 7));
        if (row0 + rr < rt.nrows) *reinterpret_cast<uint4*>(to + static_cast<long long>(rr) * (kVdim * 2) + (lane & 7) * 16) = w;
      }
      __syncwarp();
    }
    named_bar_sync(kNamedAll, kSoftWarps * 32);  // (P may be written again)
    tc_fence_before();
  }
}

// One thread of each CTA, behind the roles' last use of the MMAs: waits until they are done and each of their arrivals on this
// CTA's barriers has landed, the last ones too, which no role needs. (What a parity cannot tell, that the phase before a
// barrier's last is over, is known: the last one's unit or P was made behind a wait for it or for MMAs issued later.)
__device__ void drain(const SharedPrefixParams& p, uint32_t bars, const WaitCtl& wc) {
  auto bar = [&](int i) -> uint32_t { return bars + 8u * static_cast<uint32_t>(i); };
  if (!mbar_wait_ignoring_abort(bar(kBarDrain), 0, wc)) return;
  const PairStart s = p.pairs[blockIdx.x >> 1];
  const long long tiles = s.hi - s.lo;
  auto last = [&](int i, long long phases) {
    if (phases > 0) mbar_wait_cluster(bar(i), static_cast<uint32_t>(phases - 1) & 1u, wc);
  };
#pragma unroll 1
  for (int i = 0; i < kUnits; ++i) last(kBarEmpty + i, ((kKUnits + kVUnits) * tiles - i + kUnits - 1) / kUnits);
  last(kBarPvDone, (tiles + 1) / 2);
  last(kBarPvDone + 1, tiles / 2);
}

template <bool kF16>
__global__ void __launch_bounds__(block_threads(kF16), 1) shared_prefix_kernel(const __grid_constant__ SharedPrefixParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t bars = smem_u32(smem) + kOffBars;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  const int warp = threadIdx.x >> 5;
  const uint32_t crank = cluster_ctarank();
  if (threadIdx.x == 0) {
    auto bar = [&](int i) -> uint32_t { return bars + 8u * static_cast<uint32_t>(i); };
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(bar(kBarFull + i), 2);
      mbar_init(bar(kBarEmpty + i), 1);
      mbar_init(bar(kBarGrant + i), 1);
    }
    mbar_init(bar(kBarQFull), kF16 ? 2 * fill_warps(kF16) : 2);
    mbar_init(bar(kBarQLand), 1);
    mbar_init(bar(kBarQEmpty), 1);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(bar(kBarSFull + i), 1);
      mbar_init(bar(kBarSFree + i), 2 * kSoftWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarPFull + i), 2 * kSoftWarps);
      mbar_init(bar(kBarPvDone + i), 1);
    }
    for (int i = 0; i < kInfos; ++i) {
      mbar_init(bar(kBarInfoFull + i), 1);
      mbar_init(bar(kBarInfoFree + i), 2 + fill_warps(kF16) + kSoftWarps);
    }
    mbar_init(bar(kBarDrain), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) tmem_alloc2(smem_u32(tmem_slot), kTmemCols);
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl wc{p.status, abort_flag, p.wait_limit_ns > 0 ? p.wait_limit_ns : kWaitLimitNs};
  // the merge may come when the plan is done: it reads the plan while this kernel runs
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp >= kFillWarp0) {
    fill_role<kF16>(p, smem, bars, crank, wc);
  } else if (warp >= kSoftWarp0) {
    softmax_role<kF16>(p, smem, tmem, bars, crank, wc);
  } else if (warp == kResolveWarp) {
    resolve_role(p, smem, bars, crank, wc);
  } else if (warp == kMmaWarp) {
    if (crank == 0 && elect_one()) {
      mma_role<kF16>(p, smem, tmem, bars, wc);
      umma2_commit(bars + 8u * kBarDrain);
    }
  } else if (warp == kTmaWarp0 || warp == kTmaWarp1) {
    if (elect_one()) tma_role<kF16>(p, smem, bars, crank, warp == kTmaWarp0 ? 0 : 1, wc);
  }
  __syncwarp();
  // No MMA may still read shared memory or write TMEM when the CTAs let go of them, and nothing may be on its way to a CTA that has
  // left: the MMAs' arrivals are waited for here, loads were by the MMAs, and the threads' own arrivals are behind the cluster's
  // barrier. (A softmax thread waits, whose role ends with the MMAs: the limit of a wait is not one of the kernel's whole time.)
  if (threadIdx.x == 32 * kSoftWarp0) drain(p, bars, wc);
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  if (threadIdx.x == 0 && *abort_flag) {
    // after a wait that gave up, loads and arrivals that nobody waited for land first
    const uint64_t t0 = globaltimer();
    for (int i = 0; i < 4096 && globaltimer() - t0 < 50000u; ++i) __nanosleep(64);
  }
  __syncwarp();
  cluster_sync_all();
  if (warp == 0) tmem_dealloc2(tmem, kTmemCols);
}

// ---------------------------------------------------------------------------------- plan
// One CTA: the queries' lengths and own pieces, the row tiles, and the tiles' places end to end.
constexpr int kPlanThreads = 1024, kPlanNear = 1024;
// What a tile of a prefix costs, and a row tile's end: its epilogue and the pipeline's new start (4 us, three such tiles).
constexpr int kCost = 2, kTurnCost = 6;

__device__ __forceinline__ long long plan_scan(long long v, long long* part, long long* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long s = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += o;
  }
  if (lane == 31) part[warp] = s;
  __syncthreads();
  if (warp == 0) {
    long long t = part[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, t, d);
      if (lane >= d) t += o;
    }
    part[lane] = t;
  }
  __syncthreads();
  const long long before = warp > 0 ? part[warp - 1] : 0;
  *all = part[31];
  __syncthreads();
  return before + s - v;
}

__global__ void __launch_bounds__(kPlanThreads) shared_prefix_plan_kernel(const __grid_constant__ SharedPrefixParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ long long part[32];
  // what this kernel itself reads again (up to these sizes)
  __shared__ long long near_first[kPlanNear + 1], near_cost[kPlanNear + 1];
  __shared__ long long near_lo[kMaxPairs + 1];
  __shared__ int near_len[kPlanNear], near_before[kPlanNear + 1];
  const int tid = threadIdx.x;
  const bool near = p.T <= kPlanNear && p.max_row_tiles <= kPlanNear && static_cast<long long>(p.T) * p.max_blocks * p.page_size < (1ll << 31);
  const long long room = static_cast<long long>(p.max_blocks) * p.page_size;
  bool err = false;
  // queries first .. end of group g (starts that go back, or out of range, leave the group empty)
  auto group_begin = [&](int g) { return min(max(p.group_start[g], 0), p.T); };
  auto group_end = [&](int g) { return max(group_begin(g), min(max(p.group_start[g + 1], 0), p.T)); };
  auto prefix_of = [&](int g) -> int {
    const int n = p.prefix_lens[g];
    return static_cast<int>(min(static_cast<long long>(max(n, 0)), room));
  };
  for (int g = tid; g < p.groups; g += kPlanThreads) {
    const int a = p.group_start[g], z = p.group_start[g + 1];
    if (a < 0 || z < a || z > p.T || p.prefix_lens[g] < 0 || p.prefix_lens[g] > room) err = true;
  }
  long long base = 0;
  for (int t0 = 0; t0 < p.T; t0 += kPlanThreads) {
    const int t = t0 + tid;
    long long own = 0;
    if (t < p.T) {
      int a = 0, z = p.groups - 1;  // the last group that begins at or before t
      while (a < z) {
        const int mid = (a + z + 1) >> 1;
        if (p.group_start[mid] <= t)
          a = mid;
        else
          z = mid - 1;
      }
      int len = 0;
      if (t >= group_begin(a) && t < group_end(a)) {
        len = p.lens[t];
        const int req = p.req_of_token != nullptr ? p.req_of_token[t] : t;
        if (len < 0 || len > room || req < 0 || req >= p.num_reqs) {
          err = true;
          len = req < 0 || req >= p.num_reqs ? 0 : static_cast<int>(min(static_cast<long long>(max(len, 0)), room));
        }
        const int pre = prefix_of(a);
        if (len > pre) own = (len + kListPiece - 1) / kListPiece - pre / kListPiece;
      }
      p.token_len[t] = len;
      if (near) near_len[t] = len;
    }
    long long all;
    const long long s = plan_scan(own, part, &all);
    if (t < p.T) {
      p.own_before[t] = base + s;
      if (near) near_before[t] = static_cast<int>(base + s);
    }
    base += all;
  }
  if (tid == 0) {
    p.own_before[p.T] = base;
    if (near) near_before[p.T] = static_cast<int>(base);
  }
  // row tiles of the groups: group g's are from group_tile[g]
  long long tiles = 0;
  for (int g0 = 0; g0 < p.groups; g0 += kPlanThreads) {
    const int g = g0 + tid;
    long long n = 0;
    if (g < p.groups) n = (static_cast<long long>(group_end(g) - group_begin(g)) * p.H + kTile - 1) / kTile;
    long long all;
    const long long s = plan_scan(n, part, &all);
    if (g < p.groups) p.group_tile[g] = static_cast<int>(tiles + s);
    tiles += all;
  }
  // (groups that overlap, which is refused above, may not run over the arrays)
  const int row_tiles = static_cast<int>(min(tiles, static_cast<long long>(p.max_row_tiles)));
  if (tiles > p.max_row_tiles) err = true;
  __syncthreads();
  long long total = 0, cost_total = 0;
  for (int r0 = 0; r0 < row_tiles; r0 += kPlanThreads) {
    const int r = r0 + tid;
    long long n = 0, cost = 0;
    if (r < row_tiles) {
      int a = 0, z = p.groups - 1;
      while (a < z) {
        const int mid = (a + z + 1) >> 1;
        if (p.group_tile[mid] <= r)
          a = mid;
        else
          z = mid - 1;
      }
      const int begin = group_begin(a), i = r - p.group_tile[a];
      const long long rows = static_cast<long long>(group_end(a) - begin) * p.H, first = static_cast<long long>(i) * kTile;
      RowTile rt;
      rt.row0 = static_cast<int>(static_cast<long long>(begin) * p.H + first);
      rt.nrows = static_cast<int>(min(static_cast<long long>(kTile), rows - first));
      rt.t_first = begin + static_cast<int>(first / p.H);
      rt.t_last = begin + static_cast<int>((first + rt.nrows - 1) / p.H);
      rt.prefix_len = prefix_of(a);
      rt.min_len = 0x7fffffff;
      int most = 0, longest = begin;
      for (int t = rt.t_first; t <= rt.t_last; ++t) {
        const int len = near ? near_len[t] : p.token_len[t];
        rt.min_len = min(rt.min_len, len);
        if (len > most) most = len, longest = t;
      }
      rt.shared_len = min(rt.prefix_len, most);
      rt.shared_pieces = (rt.shared_len + kListPiece - 1) / kListPiece;
      // The prefix is read through the group's first query's table; if that one has no request, through that of the row
      // tile's longest query (which has one, unless all are empty).
      auto request = [&](int t) { return p.req_of_token != nullptr ? p.req_of_token[t] : t; };
      rt.req = request(begin);
      if (rt.req < 0 || rt.req >= p.num_reqs) rt.req = most > 0 ? request(longest) : 0;
      p.row_tiles[r] = rt;
      const long long own = near ? near_before[rt.t_last + 1] - near_before[rt.t_first]
                                 : p.own_before[rt.t_last + 1] - p.own_before[rt.t_first];
      n = (rt.shared_pieces + own + kPieces - 1) / kPieces;
      cost = p.own_cost * n - (p.own_cost - kCost) * (rt.shared_pieces / kPieces) + (n > 0 ? kTurnCost : 0);
    }
    long long all;
    const long long s = plan_scan(n, part, &all);
    if (r < row_tiles) {
      p.tile_first[r] = total + s;
      if (near) near_first[r] = total + s;
    }
    total += all;
    const long long u = plan_scan(cost, part, &all);
    if (r < row_tiles) (near ? near_cost : p.cost_first)[r] = cost_total + u;
    cost_total += all;
  }
  long long pairs = (total + p.min_tiles - 1) / p.min_tiles;
  if (pairs > p.max_pairs) pairs = p.max_pairs;
  if (tid == 0) {
    p.tile_first[row_tiles] = total;
    if (near) near_first[row_tiles] = total;
    p.plan->total = total;
    p.plan->pairs = static_cast<int>(pairs);
    p.plan->row_tiles = row_tiles;
  }
  __syncthreads();
  const long long* tile_first = near ? near_first : p.tile_first;
  const long long* cost_first = near ? near_cost : p.cost_first;
  auto row_tile_at = [&](const long long* firsts, long long at) {  // the last row tile that begins at or before
    int a = 0, z = row_tiles - 1;
    while (a < z) {
      const int mid = (a + z + 1) >> 1;
      if (firsts[mid] <= at)
        a = mid;
      else
        z = mid - 1;
    }
    return a;
  };
  // Pairs of many tiles are dealt even shares of cost, each above any tile's and row tile's end's, so that none is left without.
  const bool weigh = total >= 8 * pairs;
  for (int c = tid; c <= pairs; c += kPlanThreads) {
    long long lo = streamk_lo(c, weigh ? cost_total : total, max(pairs, 1ll));
    if (c == pairs) {
      lo = total;
    } else if (weigh) {
      const int a = row_tile_at(cost_first, lo);
      const long long in = lo - cost_first[a], shared = p.row_tiles[a].shared_pieces / kPieces;
      lo = min(tile_first[a] + (in < kCost * shared ? in / kCost : shared + (in - kCost * shared) / p.own_cost), tile_first[a + 1]);
    }
    near_lo[c] = lo;
  }
  __syncthreads();
  for (int c = tid; c < p.max_pairs; c += kPlanThreads) {
    PairStart s = {};
    s.part0 = -1;
    if (c < pairs) {
      s.lo = near_lo[c];
      s.hi = near_lo[c + 1];
      s.row_tile = row_tile_at(tile_first, s.lo);
      s.first = tile_first[s.row_tile];
      s.end = tile_first[s.row_tile + 1];
      if (s.lo > s.first && near_lo[c - 1] <= s.first) s.part0 = 2 * (c - 1) + (near_lo[c - 1] == s.first ? 0 : 1);
      int a = c, z = static_cast<int>(pairs) - 1;
      while (a < z) {
        const int mid = (a + z + 1) >> 1;
        if (near_lo[mid] < s.end)
          a = mid;
        else
          z = mid - 1;
      }
      s.last = a;
    }
    p.pairs[c] = s;
  }
  if (__syncthreads_or(err) && tid == 0) atomicOr(p.status, SVT_DEV_ERR_INDEX_RANGE);
}

// ---------------------------------------------------------------------------------- merge
// CTA (x, y): rows 4 y .. 4 y + 3, a warp each, of the row tile that the beginning of pair x's range cuts, if pair x is the
// first to begin inside it; then the row tiles without any tile (out = 0, lse = -inf). (CTAs of 128 threads, which fit beside the
// attention's: they look up the plan while it runs.)
constexpr int kMergeRows = 4;
__global__ void __launch_bounds__(32 * kMergeRows, 9) shared_prefix_merge_kernel(const __grid_constant__ SharedPrefixParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row_tiles = __ldcg(&p.plan->row_tiles);
  const int c = blockIdx.x;
  const PairStart* s = p.pairs + c;
  const int part0 = __ldcg(&s->part0), r = __ldcg(&s->row_tile), last = __ldcg(&s->last);
  int row0 = 0, nrows = 0;
  if (part0 >= 0) {
    row0 = __ldcg(&p.row_tiles[r].row0);
    nrows = __ldcg(&p.row_tiles[r].nrows);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  {
    if (part0 >= 0) {
      const int row = kMergeRows * blockIdx.y + warp;
      const int parts = last - (c - 1) + 1;
      if (row < nrows) {
        auto slot = [&](int i) -> long long { return i == 0 ? part0 : 2ll * (c - 1 + i); };
        float m = -CUDART_INF_F;
        bool nan = false;
        for (int i = lane; i < parts; i += 32) {
          const float v = p.part_lse[slot(i) * kTile + row];
          nan |= v != v;
          m = fmaxf(m, v);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        nan = __any_sync(0xffffffffu, nan);
        const float ref = m == -CUDART_INF_F ? 0.f : m;
        float z = 0.f;
        for (int i = lane; i < parts; i += 32) z += ex2_approx(p.part_lse[slot(i) * kTile + row] - ref);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
        const float inv = z > 0.f ? 1.f / z : 0.f;
        float acc[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = 0.f;
#pragma unroll 4
        for (int i = 0; i < parts; ++i) {
          const long long at = slot(i) * kTile + row;
          // (lane: channels 16 lane .. + 15)
          const float w = ex2_approx(p.part_lse[at] - ref) * inv * p.part_scale[at * 4 + (lane >> 3)];
          const uint4* src = reinterpret_cast<const uint4*>(p.part_o + at * kVdim) + 2 * lane;
          const uint4 v[2] = {__ldcg(src), __ldcg(src + 1)};
          if (w != 0.f || nan) {  // (a part without live entries may hold anything)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t e[4] = {v[h].x, v[h].y, v[h].z, v[h].w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&e[j]));
                acc[8 * h + 2 * j] = fmaf(f.x, w, acc[8 * h + 2 * j]);
                acc[8 * h + 2 * j + 1] = fmaf(f.y, w, acc[8 * h + 2 * j + 1]);
              }
            }
          }
        }
        const long long grow = static_cast<long long>(row0) + row;
        uint4* dst = reinterpret_cast<uint4*>(p.out + grow * kVdim) + 2 * lane;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          dst[h] = make_uint4(pack_bf16x2(acc[8 * h], acc[8 * h + 1]), pack_bf16x2(acc[8 * h + 2], acc[8 * h + 3]),
                              pack_bf16x2(acc[8 * h + 4], acc[8 * h + 5]), pack_bf16x2(acc[8 * h + 6], acc[8 * h + 7]));
        if (lane == 0 && p.lse != nullptr)
          p.lse[grow] = nan ? CUDART_NAN_F : z > 0.f ? (m + __log2f(z)) * 0.69314718055994530942f : -CUDART_INF_F;
      }
    }
  }
  const int ctas = gridDim.x * gridDim.y, cta = blockIdx.x * gridDim.y + blockIdx.y;
  for (int r = cta; r < row_tiles; r += ctas) {
    if (p.tile_first[r] != p.tile_first[r + 1]) continue;
    const RowTile rt = p.row_tiles[r];
    for (int i = threadIdx.x; i < rt.nrows * (kVdim / 8); i += blockDim.x)
      reinterpret_cast<uint4*>(p.out + static_cast<long long>(rt.row0) * kVdim)[i] = make_uint4(0, 0, 0, 0);
    if (p.lse != nullptr)
      for (int i = threadIdx.x; i < rt.nrows; i += blockDim.x) p.lse[rt.row0 + i] = -CUDART_INF_F;
  }
}

template <bool kF16>
int max_pairs_of() {
  if (cudaFuncSetAttribute(shared_prefix_kernel<kF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) !=
      cudaSuccess)
    return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(block_threads(kF16));
  cfg.dynamicSmemBytes = kSmemBytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, shared_prefix_kernel<kF16>, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  return n;
}

cudaLaunchAttribute behind() {
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}

}  // namespace

int shared_prefix_pairs() {
  static std::mutex mu;
  static int cache[64] = {};  // per device; 0 = not asked yet, -1 = the query failed
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (cache[dev] == 0) {
    const int a = max_pairs_of<false>(), b = max_pairs_of<true>();
    const int n = a < b ? a : b;
    cache[dev] = n > 0 ? n : -1;
  }
  return cache[dev] > 0 ? cache[dev] : 0;
}

cudaError_t launch_shared_prefix(const SharedPrefixParams& p, bool f16, cudaStream_t stream) {
  shared_prefix_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * static_cast<unsigned>(p.max_pairs));
  cfg.blockDim = dim3(block_threads(f16));
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = behind();
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = f16 ? cudaLaunchKernelEx(&cfg, shared_prefix_kernel<true>, p) : cudaLaunchKernelEx(&cfg, shared_prefix_kernel<false>, p);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t mc = {};
  mc.gridDim = dim3(static_cast<unsigned>(p.max_pairs), kTile / kMergeRows);
  mc.blockDim = dim3(32 * kMergeRows);
  mc.stream = stream;
  cudaLaunchAttribute ma[1] = {behind()};
  mc.attrs = ma;
  mc.numAttrs = 1;
  return cudaLaunchKernelEx(&mc, shared_prefix_merge_kernel, p);
}

}  // namespace svt
