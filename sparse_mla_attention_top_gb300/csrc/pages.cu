// The pages of a cache: rows of a block table that go on as others (a beam search's parents, samples of one prompt),
// grow, or end, with the pages' reference counts; and the live pages moved to the lowest numbers.
//
// A count is the number of table entries that hold the page; a page is free while it is 0. Free pages are found in their
// order without a list: the first kernel makes a bitmap of them with the number before each word and in each chunk, and the
// k-th free page is then two binary searches away, for any thread. The second kernel does all the rest, as what it writes (counts,
// tables, rows of pages) nothing else in it reads. What bounds them: the copies' bytes where pages move, the launches
// and a few dependent reads otherwise.
#include <algorithm>

#include "device.cuh"
#include "internal.h"

namespace svt {

namespace {

constexpr int kThreads = 256;
constexpr int kScanThreads = 1024;

// Exclusive sums over a CTA of kN threads; *all gets the total. `part` is kN / 32 values of shared memory.
template <int kN, typename T>
__device__ __forceinline__ T block_scan(T v, T* part, T* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T s = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T o = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += o;
  }
  if (lane == 31) part[warp] = s;
  __syncthreads();
  if (warp == 0) {
    T t = lane < kN / 32 ? part[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const T o = __shfl_up_sync(0xffffffffu, t, d);
      if (lane >= d) t += o;
    }
    if (lane < kN / 32) part[lane] = t;
  }
  __syncthreads();
  const T before = warp > 0 ? part[warp - 1] : 0;
  *all = part[kN / 32 - 1];
  __syncthreads();
  return before + s - v;
}

// What the first kernel leaves of the pages: per word of 32 pages the free ones and how many are free before it in its
// chunk; per chunk the free ones. kFree: free pages, else live ones.
struct PageMap {
  const uint32_t* bits;
  const int* word_before;
  const int* chunk_before;  // shared memory: exclusive sums of the chunks' counts of free pages, and the total
  int chunk_pages, chunks;
  long long num_pages;

  // Pages of the kind before page p.
  template <bool kFree>
  __device__ long long before(long long p) const {
    const long long word = p >> 5;
    const int free_before = chunk_before[p / chunk_pages] + word_before[word] +
                            __popc(bits[word] & ((1u << (p & 31)) - 1u));
    return kFree ? free_before : p - free_before;
  }
  // The k-th page of the kind (there are more than k).
  template <bool kFree>
  __device__ long long at(long long k) const {
    auto chunk_first = [&](int c) -> long long {
      return kFree ? chunk_before[c] : static_cast<long long>(c) * chunk_pages - chunk_before[c];
    };
    int lo = 0, hi = chunks - 1;  // the last chunk that begins at or before the k-th
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (chunk_first(mid) <= k)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int in = static_cast<int>(k - chunk_first(lo));
    const long long w0 = static_cast<long long>(lo) * chunk_pages / 32;
    const long long words = (num_pages + 31) / 32;
    long long a = w0, z = min(w0 + chunk_pages / 32, words) - 1;
    while (a < z) {
      const long long mid = (a + z + 1) >> 1;
      const int n = kFree ? word_before[mid] : static_cast<int>((mid - w0) * 32) - word_before[mid];
      if (n <= in)
        a = mid;
      else
        z = mid - 1;
    }
    const int n = kFree ? word_before[a] : static_cast<int>((a - w0) * 32) - word_before[a];
    // (past the last page a word's bits are neither)
    uint32_t v = kFree ? bits[a] : ~bits[a];
    for (int i = in - n; i > 0; --i) v &= v - 1;
    return a * 32 + (__ffs(static_cast<int>(v)) - 1);
  }
};

// The counts of the chunks as exclusive sums in `sums` (chunks + 1 of them); every thread of kN calls it.
template <int kN>
__device__ void chunk_sums(const int* counts, int chunks, int* sums, int* part) {
  int base = 0;
  for (int c0 = 0; c0 < chunks; c0 += kN) {
    const int c = c0 + static_cast<int>(threadIdx.x);
    int all;
    const int s = block_scan<kN>(c < chunks ? counts[c] : 0, part, &all);
    if (c < chunks) sums[c] = base + s;
    base += all;
  }
  if (threadIdx.x == 0) sums[chunks] = base;
  __syncthreads();
}

// Bitmap, counts and (where they are to be kept apart) a copy of the reference counts of chunk `c`.
__device__ void scan_chunk(const PoolParams& p, int c, int* part) {
  const long long p0 = static_cast<long long>(c) * p.chunk_pages;
  const long long p1 = min(p0 + p.chunk_pages, p.num_pages);
  const int lane = threadIdx.x & 31;
  int base = 0;
  for (long long q0 = p0; q0 < p1; q0 += kScanThreads) {
    const long long q = q0 + threadIdx.x;
    const int r = q < p1 ? p.refs[q] : 1;
    if (p.copy_refs && q < p1) p.refs_out[q] = r;
    const uint32_t free = __ballot_sync(0xffffffffu, r <= 0);
    int all;
    const int before = block_scan<kScanThreads>(lane == 0 ? __popc(free) : 0, part, &all);
    if (lane == 0 && q < p1) {
      p.bits[q >> 5] = free;
      p.word_before[q >> 5] = base + before;
    }
    base += all;
  }
  if (threadIdx.x == 0) p.counts[c] = base;
}

// Whether the entries in use of the table's rows are pages that are held.
__device__ bool rows_are_bad(const ForkParams& p, int cta, int ctas) {
  bool bad = false;
  for (int r = cta; r < p.R; r += ctas) {
    const int len = p.lens[r];
    if (len < 0 || len > static_cast<long long>(p.M) * p.page_size) {
      bad = true;
      continue;
    }
    const int n = (len + p.page_size - 1) / p.page_size;
    for (int j = threadIdx.x; j < n; j += kScanThreads) {
      const int page = p.table[static_cast<long long>(r) * p.M + j];
      if (page < 0 || page >= p.pool.num_pages || p.pool.refs[page] <= 0) bad = true;
    }
  }
  return bad;
}

// For each row to come: what of its parent it keeps, and the place of its new pages among all. One CTA.
// (Their sum is in 64 bits: a row alone may ask for 2^30 pages, of which the pool need not have any.)
__device__ void plan_rows(const ForkParams& p) {
  extern __shared__ int first[];  // [R] the first row that names a parent
  __shared__ long long part[32];
  __shared__ int void_call;
  const int P = p.page_size;
  const long long room = static_cast<long long>(p.M_out) * P;
  for (int r = threadIdx.x; r < p.R; r += kScanThreads) first[r] = 0x7fffffff;
  if (threadIdx.x == 0) void_call = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < p.N; i += kScanThreads) {
    const int from = p.parents[i];
    if (from >= 0 && from < p.R) atomicMin(&first[from], i);
  }
  __syncthreads();
  long long base = 0;
  bool bad = false;
  for (int i0 = 0; i0 < p.N; i0 += kScanThreads) {
    const int i = i0 + static_cast<int>(threadIdx.x);
    long long need = 0;
    if (i < p.N) {
      const int from = p.parents[i];
      const int grow = p.grow != nullptr ? p.grow[i] : p.grow_all;
      int len = 0, copy = 0;
      if (from < -1 || from >= p.R || grow < 0 || grow > p.max_grow) {
        bad = true;
      } else if (from >= 0) {
        len = p.lens[from];
        if (len < 0 || len > static_cast<long long>(p.M) * P) {
          bad = true;
          len = 0;
        } else if (len % P != 0) {
          const int page = p.table[static_cast<long long>(from) * p.M + len / P];
          const bool sole = page >= 0 && page < p.pool.num_pages && p.pool.refs[page] == 1;
          copy = !(first[from] == i && sole);
        }
      }
      const long long end = static_cast<long long>(len) + (bad ? 0 : grow);
      if (end > room || end > 0x7fffffffll) bad = true;
      need = bad ? 0 : copy + (end + P - 1) / P - (len + P - 1) / P;
      p.row_copy[i] = copy;
    }
    long long all;
    const long long s = block_scan<kScanThreads>(need, part, &all);
    if (i < p.N) p.row_first[i] = static_cast<int>(min(base + s, 0x7fffffffll));  // (more than a pool has: the call is void)
    base += all;
  }
  for (int r = threadIdx.x; r < p.R; r += kScanThreads) {
    int kept = 0;
    if (first[r] != 0x7fffffff) kept = p.row_copy[first[r]] == 0 ? 1 : 0;
    p.keeps[r] = kept;  // whether the row's begun page (if it has one) stays with its first child
  }
  if (bad) void_call = 1;
  __syncthreads();
  if (threadIdx.x == 0) {
    *p.need = base;
    *p.bad_plan = void_call;
  }
}

// CTA 0 plans the rows, the others take chunks of the pool and rows of the table.
__global__ void __launch_bounds__(kScanThreads) fork_scan_kernel(const __grid_constant__ ForkParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ int part[32];
  if (blockIdx.x == 0) {
    plan_rows(p);
    return;
  }
  const int cta = blockIdx.x - 1, ctas = gridDim.x - 1;
  const bool bad = rows_are_bad(p, cta, ctas);
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) p.bad_rows[cta] = any;
  for (int c = cta; c < p.pool.chunks; c += ctas) scan_chunk(p.pool, c, part);
}

__global__ void __launch_bounds__(kScanThreads) pool_scan_kernel(const __grid_constant__ PoolParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ int part[32];
  for (int c = blockIdx.x; c < p.chunks; c += gridDim.x) scan_chunk(p, c, part);
}

// 16-byte pieces [from, to) of the rows of page src to page dst, by kN threads of which this is `me`; four in flight each.
template <int kN>
__device__ __forceinline__ void copy_pieces(const CacheRows& kv, long long src, long long dst, int from, int to, int me) {
  const int per_row = kv.row_bytes / 16;
  const uint8_t* a = kv.data + src * kv.page_size * kv.row_stride;
  uint8_t* b = kv.data + dst * kv.page_size * kv.row_stride;
  const int pad = static_cast<int>(kv.row_stride) - kv.row_bytes;
  for (int i = from + me; i < to; i += 4 * kN) {
    uint4 v[4];
    long long off[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = i + j * kN;
      off[j] = static_cast<long long>(at) * 16 + (pad != 0 ? static_cast<long long>(at / per_row) * pad : 0);
      if (at < to) v[j] = *reinterpret_cast<const uint4*>(a + off[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j * kN < to) *reinterpret_cast<uint4*>(b + off[j]) = v[j];
  }
}

// CTA (x, y): row x of the rows to come (y = 0: its table, counts and slots; every y its share of the copy), then, for
// x >= N, a row of the old table, whose pages' counts lose it.
__global__ void __launch_bounds__(kThreads) fork_apply_kernel(const __grid_constant__ ForkParams p) {
  __shared__ int sums[kPoolMaxChunks + 1];
  __shared__ int part[32];
  __shared__ int children;
  const int tid = threadIdx.x;
  const int P = p.page_size;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blockIdx.y != 0 && (blockIdx.x >= static_cast<unsigned>(p.N) || p.row_copy[blockIdx.x] == 0)) return;
  chunk_sums<kThreads>(p.pool.counts, p.pool.chunks, sums, part);
  int bad = *p.bad_plan != 0;
  for (int i = tid; i < p.scan_ctas; i += kThreads) bad |= p.bad_rows[i] != 0;
  bad = __syncthreads_or(bad);
  const bool short_of = !bad && *p.need > sums[p.pool.chunks];
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0 && (bad || short_of))
    atomicOr(p.status, bad ? SVT_DEV_ERR_INDEX_RANGE : SVT_DEV_ERR_NO_PAGES);
  const bool off = bad || short_of;
  if (blockIdx.x >= static_cast<unsigned>(p.N)) {
    // the old row r: its whole pages are held by as many rows as name it in place of it, its begun page by the one that keeps it
    const int r = blockIdx.x - p.N;
    if (off) return;
    if (tid == 0) children = 0;
    __syncthreads();
    int c = 0;
    for (int i = tid; i < p.N; i += kThreads) c += p.parents[i] == r;
    c = __reduce_add_sync(0xffffffffu, c);
    if ((tid & 31) == 0 && c != 0) atomicAdd(&children, c);
    __syncthreads();
    const int len = p.lens[r], full = len / P;
    const int change = children - 1;
    const int32_t* row = p.table + static_cast<long long>(r) * p.M;
    if (change != 0)
      for (int j = tid; j < full; j += kThreads) atomicAdd(p.pool.refs_out + row[j], change);
    if (tid == 0 && len % P != 0 && p.keeps[r] == 0) atomicAdd(p.pool.refs_out + row[full], -1);
    return;
  }
  const PageMap map{p.pool.bits, p.pool.word_before, sums, p.pool.chunk_pages, p.pool.chunks, p.pool.num_pages};
  const int i = blockIdx.x;
  int32_t* out = p.table_out + static_cast<long long>(i) * p.M_out;
  int32_t* slots = p.slots + static_cast<long long>(i) * p.max_grow;
  if (off) {
    if (blockIdx.y != 0) return;
    for (int j = tid; j < p.M_out; j += kThreads) out[j] = -1;
    for (int j = tid; j < p.max_grow; j += kThreads) slots[j] = -1;
    if (tid == 0) p.lens_out[i] = 0;
    return;
  }
  const int from = p.parents[i];
  const int grow = p.grow != nullptr ? p.grow[i] : p.grow_all;
  const int len = from >= 0 ? p.lens[from] : 0;
  const int copy = p.row_copy[i], begin = p.row_first[i];
  const int full = len / P, held = (len + P - 1) / P, after = static_cast<int>((static_cast<long long>(len) + grow + P - 1) / P);
  const int32_t* old = p.table + static_cast<long long>(from) * p.M;
  if (blockIdx.y == 0) {
    // (a row's new pages follow one another among the free ones, not in the pool: each thread looks its own up)
    auto page_at = [&](int j) -> int {
      if (j >= after) return -1;
      if (j >= held) return static_cast<int>(map.at<true>(begin + copy + (j - held)));
      if (j == full && copy) return static_cast<int>(map.at<true>(begin));
      return old[j];
    };
    for (int j = tid; j < p.M_out; j += kThreads) {
      const int page = page_at(j);
      out[j] = page;
      if (page >= 0 && (j >= held || (j == full && copy))) p.pool.refs_out[page] = 1;
    }
    for (int j = tid; j < p.max_grow; j += kThreads) {
      int slot = -1;
      if (j < grow) slot = page_at((len + j) / P) * P + (len + j) % P;
      slots[j] = slot;
    }
    if (tid == 0) p.lens_out[i] = len + grow;
  }
  if (copy) {
    const int pieces = len % P * (p.kv.row_bytes / 16);
    const long long share = blockIdx.y, shares = gridDim.y;
    copy_pieces<kThreads>(p.kv, old[full], map.at<true>(begin), static_cast<int>(pieces * share / shares),
                          static_cast<int>(pieces * (share + 1) / shares), tid);
  }
}

constexpr int kMovePieces = 512;  // 8 KB

// All threads of the grid: pages, then table entries; warps: the moves.
__global__ void __launch_bounds__(kThreads) compact_apply_kernel(const __grid_constant__ CompactParams p) {
  __shared__ int sums[kPoolMaxChunks + 1];
  __shared__ int part[32];
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  chunk_sums<kThreads>(p.pool.counts, p.pool.chunks, sums, part);
  const PageMap map{p.pool.bits, p.pool.word_before, sums, p.pool.chunk_pages, p.pool.chunks, p.pool.num_pages};
  const long long n = p.pool.num_pages;
  const long long live = n - sums[p.pool.chunks];
  // the live pages from `live` on take the free ones below, in order
  const long long stay = live < n ? map.before<false>(live) : live;
  const long long moves = live - stay;
  auto is_free = [&](long long q) { return (p.pool.bits[q >> 5] >> (q & 31)) & 1u; };
  const long long threads = static_cast<long long>(gridDim.x) * kThreads;
  const long long me = static_cast<long long>(blockIdx.x) * kThreads + tid;
  for (long long q = me; q < n; q += threads) {
    int to = -1;
    if (!is_free(q)) {
      if (q < live) {
        to = static_cast<int>(q);
      } else {
        const long long k = map.before<false>(q) - stay;
        to = static_cast<int>(map.at<true>(k));
        const int r = p.pool.refs[q];  // one thread moves the count: in place, no other touches either
        p.pool.refs_out[to] = r;
        p.pool.refs_out[q] = 0;
      }
    } else if (q >= live) {
      p.pool.refs_out[q] = 0;
    }
    if (p.mapping != nullptr) p.mapping[q] = to;
    // (a page that stays has its count copied by the first kernel, or in place)
  }
  int err = 0;
  for (long long e = me; e < p.entries; e += threads) {
    const int page = p.table[e];
    int to = -1;
    if (page >= 0) {
      if (page >= n || is_free(page)) {
        err = 1;
      } else {
        to = page < live ? page : static_cast<int>(map.at<true>(map.before<false>(page) - stay));
      }
    }
    p.table_out[e] = to;
  }
  if (__syncthreads_or(err) && tid == 0) atomicOr(p.status, SVT_DEV_ERR_INDEX_RANGE);
  // a warp takes a part of a page: enough of them in flight to hide the searches
  const int pieces = p.kv.page_size * (p.kv.row_bytes / 16);
  const int parts = (pieces + kMovePieces - 1) / kMovePieces;
  for (long long k = me >> 5; k < moves * parts; k += threads >> 5) {
    const long long mv = k / parts;
    const int from = static_cast<int>(k - mv * parts) * kMovePieces;
    copy_pieces<32>(p.kv, map.at<false>(stay + mv), map.at<true>(mv), from, min(pieces, from + kMovePieces), tid & 31);
  }
}

cudaError_t launch_behind(void (*kernel)(ForkParams), dim3 grid, const ForkParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

// Chunks of the pool: at most kPoolMaxChunks of a multiple of the scan's 1024 pages.
void plan_pool(PoolParams& p) {
  long long pages = kScanThreads;
  while ((p.num_pages + pages - 1) / pages > kPoolMaxChunks) pages *= 2;
  p.chunk_pages = static_cast<int>(pages);
  p.chunks = static_cast<int>((p.num_pages + pages - 1) / pages);
}

int fork_scan_ctas(const PoolParams& p, int R, int sms) {
  return std::max(1, std::min(std::max(p.chunks, R), sms - 1));
}

cudaError_t launch_fork(const ForkParams& p, cudaStream_t stream) {
  const size_t smem = static_cast<size_t>(p.R) * 4;
  cudaError_t e = cudaSuccess;
  if (smem > 40000) {  // (always the largest: a call in another thread may set it at the same time)
    e = cudaFuncSetAttribute(fork_scan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kForkMaxRows);
    if (e != cudaSuccess) return e;
  }
  fork_scan_kernel<<<p.scan_ctas + 1, kScanThreads, smem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (p.N + p.R == 0) return cudaSuccess;
  return launch_behind(fork_apply_kernel, dim3(p.N + p.R, p.shares), p, stream);
}

cudaError_t launch_compact(const CompactParams& p, int sms, cudaStream_t stream) {
  pool_scan_kernel<<<std::min(p.pool.chunks, sms), kScanThreads, 0, stream>>>(p.pool);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(sms) * 8);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, compact_apply_kernel, p);
}

}  // namespace svt
