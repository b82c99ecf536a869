// C ABI of the operators that continue a prompt several ways: attention over shared prefixes, beam search's selection, and
// the pages' forking, freeing and compacting. As everywhere in the library, every check comes before anything is enqueued,
// and nothing allocates device memory or waits for a stream.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "internal.h"

namespace {

using svt::set_last_error;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t round_up(size_t x, size_t a = 256) { return (x + a - 1) / a * a; }

svt_status cuda_fail(cudaError_t e, const char* what) {
  return set_last_error(SVT_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Of the current device; known ones are kept.
int sm_count() {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (dev < kDevices && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) return 1;
  if (dev < kDevices) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

// Takes the parts of a workspace one after another, behind its status header.
struct Carver {
  char* base;
  size_t at = svt::kStatusBytes;
  template <typename T>
  void take(T*& p, size_t n) {
    if (base != nullptr) p = reinterpret_cast<T*>(base + at);
    at += round_up(n * sizeof(T));
  }
};

void set_prefix_plan(svt::SharedPrefixParams& p) {
  p.max_row_tiles = static_cast<int>(static_cast<long long>(p.T) * p.H / 128 + p.groups);
  p.max_pairs = std::min(std::max(1, svt::shared_prefix_pairs()), svt::kMaxPairs);
  p.min_tiles = 1;
}
size_t carve_prefix(svt::SharedPrefixParams& p, void* ws) {
  Carver c{static_cast<char*>(ws)};
  c.take(p.plan, 1);
  c.take(p.token_len, p.T);
  c.take(p.own_before, p.T + 1ull);
  c.take(p.group_tile, p.groups);
  c.take(p.row_tiles, p.max_row_tiles);
  c.take(p.tile_first, p.max_row_tiles + 1ull);
  c.take(p.cost_first, p.max_row_tiles);
  c.take(p.pairs, p.max_pairs);
  c.take(p.part_lse, 2ull * p.max_pairs * 128);
  c.take(p.part_scale, 2ull * p.max_pairs * 128 * 4);
  c.take(p.part_o, 2ull * p.max_pairs * 128 * svt::kVdim);
  return c.at;
}

size_t carve_beam(svt::BeamParams& p, void* ws) {
  Carver c{static_cast<char*>(ws)};
  const size_t slices = static_cast<size_t>(p.B) * p.W * p.slices;
  c.take(p.part_sum, slices);
  c.take(p.part_max, slices);
  c.take(p.part_keys, slices * p.K);
  return c.at;
}

void carve_pool(svt::PoolParams& p, Carver& c) {
  const size_t words = (static_cast<size_t>(p.num_pages) + 31) / 32;
  c.take(p.bits, words);
  c.take(p.word_before, words);
  c.take(p.counts, p.chunks);
}
size_t carve_fork(svt::ForkParams& p, void* ws) {
  Carver c{static_cast<char*>(ws)};
  carve_pool(p.pool, c);
  c.take(p.need, 1);
  c.take(p.bad_plan, 1);
  c.take(p.bad_rows, p.scan_ctas);
  c.take(p.row_copy, p.N);
  c.take(p.row_first, p.N);
  c.take(p.keeps, p.R);
  return c.at;
}
size_t carve_compact(svt::CompactParams& p, void* ws) {
  Carver c{static_cast<char*>(ws)};
  carve_pool(p.pool, c);
  return c.at;
}

constexpr long long kMaxTokens = 1 << 30;  // of a table's row

svt_status check_pool(const svt_kv_cache* kv, const int32_t* refs, const int32_t* refs_out, svt::PoolParams& pool,
                      svt::CacheRows& rows) {
  long long row_stride = 0;
  const svt_status st = svt::check_kv_cache(kv, &row_stride);
  if (st != SVT_OK) return st;
  if (refs == nullptr || refs_out == nullptr)
    return set_last_error(SVT_ERR_INVALID_ARG, "refs and refs_out must not be null");
  rows = {static_cast<uint8_t*>(const_cast<void*>(kv->data)), row_stride,
          kv->dtype == SVT_KV_BF16 ? svt::kRowBytesBf16 : svt::kRowBytesFp8, kv->page_size};
  // a page's 16-byte pieces are counted in 32 bits
  if (static_cast<long long>(kv->page_size) * row_stride >= (1ll << 31))
    return set_last_error(SVT_ERR_UNSUPPORTED, "a page must have less than 2^31 bytes");
  pool.refs = refs;
  pool.refs_out = refs_out == refs ? const_cast<int32_t*>(refs) : const_cast<int32_t*>(refs_out);
  pool.copy_refs = refs_out != refs;
  pool.num_pages = kv->num_pages;
  svt::plan_pool(pool);
  return SVT_OK;
}

}  // namespace

extern "C" {

size_t svt_mla_decode_shared_prefix_workspace_size(int32_t T, int32_t H, int32_t num_groups) {
  if (T < 0 || H <= 0 || H > 128 || num_groups < 0 || static_cast<long long>(T) * H >= (1ll << 30) ||
      num_groups > (1 << 24))
    return svt::kStatusBytes;  // refused
  svt::SharedPrefixParams p{};
  p.T = T;
  p.H = H;
  p.groups = num_groups;
  set_prefix_plan(p);
  return carve_prefix(p, nullptr);
}

svt_status svt_mla_decode_shared_prefix(const void* q_bf16, int32_t T, int32_t H, const svt_kv_cache* kv,
                                        const int32_t* block_table, int32_t num_reqs, int32_t max_blocks,
                                        const int32_t* req_of_token, const int32_t* lens, const int32_t* group_start,
                                        const int32_t* prefix_lens, int32_t num_groups, float softmax_scale,
                                        void* out_bf16, float* lse, void* ws, size_t ws_bytes, svt_stream_t stream) {
  if (T < 0 || num_groups < 0) return set_last_error(SVT_ERR_INVALID_ARG, "T and num_groups must be >= 0");
  if (H <= 0) return set_last_error(SVT_ERR_INVALID_ARG, "H must be > 0");
  if (H > 128) return set_last_error(SVT_ERR_UNSUPPORTED, "at most 128 heads, got %d", H);
  if (!std::isfinite(softmax_scale)) return set_last_error(SVT_ERR_INVALID_ARG, "softmax_scale must be finite");
  if (static_cast<long long>(T) * H >= (1ll << 30) || num_groups > (1 << 24))
    return set_last_error(SVT_ERR_UNSUPPORTED, "T * H must be below 2^30 and num_groups at most 2^24");
  long long row_stride = 0;
  svt_status st = svt::check_kv_cache(kv, &row_stride);
  if (st != SVT_OK) return st;
  if (T > 0 && num_groups > 0) {
    if (block_table == nullptr || num_reqs <= 0 || max_blocks <= 0)
      return set_last_error(SVT_ERR_INVALID_ARG, "block_table must not be null, num_reqs and max_blocks must be > 0");
    if (max_blocks * static_cast<long long>(kv->page_size) > kMaxTokens)
      return set_last_error(SVT_ERR_UNSUPPORTED, "max_blocks * page_size must be at most 2^30");
    // the pieces of a row tile, its queries' own and the prefix's, are counted in 32 bits
    const long long pieces = max_blocks * static_cast<long long>(kv->page_size) / svt::kListPiece + 2;
    if ((std::min(T, (126 + H) / H + 1) + 1) * pieces >= (1ll << 31) - 8)
      return set_last_error(SVT_ERR_UNSUPPORTED, "the tables of the queries of 128 rows must have fewer than 2^35 positions");
    if (req_of_token == nullptr && num_reqs < T)
      return set_last_error(SVT_ERR_INVALID_ARG, "without req_of_token every query needs a row of block_table");
    if (q_bf16 == nullptr || out_bf16 == nullptr || lens == nullptr || group_start == nullptr || prefix_lens == nullptr)
      return set_last_error(SVT_ERR_INVALID_ARG, "q, out, lens, group_start and prefix_lens must not be null");
    if (!aligned(q_bf16, 16) || !aligned(out_bf16, 16))
      return set_last_error(SVT_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  }
  if (T == 0 || num_groups == 0) return SVT_OK;
  svt::SharedPrefixParams p{};
  p.T = T;
  p.H = H;
  p.groups = num_groups;
  set_prefix_plan(p);
  st = svt::check_workspace(ws, ws_bytes, carve_prefix(p, ws));
  if (st != SVT_OK) return st;
  p.q = static_cast<const uint16_t*>(q_bf16);
  p.kv = static_cast<const uint8_t*>(kv->data);
  p.row_stride = row_stride;
  p.num_pages = kv->num_pages;
  p.num_slots = kv->num_pages * static_cast<long long>(kv->page_size);
  p.block_table = block_table;
  p.req_of_token = req_of_token;
  p.lens = lens;
  p.group_start = group_start;
  p.prefix_lens = prefix_lens;
  p.num_reqs = num_reqs;
  p.max_blocks = max_blocks;
  p.page_size = kv->page_size;
  p.pieces = kv->dtype == SVT_KV_BF16 && kv->page_size % svt::kListPiece == 0;
  // (of two for a tile of the prefix. Own rows by TMA in pieces, measured for shares by 1, 1.5 and 2 tiles: 64 x 64 x 8192 69, 67
  // and 67 us, 128 x 64 x 32768 383, 382 and 388. Where threads load all tiles, these cost alike: an e4m3 cache 5 x 24 x 16 x 12007
  // 99 us (by 2: 110), bf16 with pages of 24 rows 64 x 64 x 8192 228 us (by 1.5: 237), 5 x 24 x 16 x 12007 124 (130))
  p.own_cost = p.pieces ? 3 : 2;
  p.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (kv->page_size == 1 << i) p.page_shift = i;
  p.row_bytes = kv->dtype == SVT_KV_BF16 ? svt::kRowBytesBf16 : svt::kRowBytesFp8;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.out = static_cast<uint16_t*>(out_bf16);
  p.lse = lse;
  p.status = static_cast<int*>(ws);
  svt::debug_fault_state(&p.fault, &p.wait_limit_ns);
  if (svt::shared_prefix_pairs() <= 0) return set_last_error(SVT_ERR_CUDA, "no pair of CTAs fits the device");
  if (!svt::encode_shared_prefix_maps(p, kv->dtype == SVT_KV_BF16)) return set_last_error(SVT_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  const cudaError_t e =
      svt::launch_shared_prefix(p, kv->dtype == SVT_KV_FP8_E4M3, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "svt_mla_decode_shared_prefix");
  return SVT_OK;
}

size_t svt_beam_select_workspace_size(int32_t B, int32_t W, int32_t V, int32_t K) {
  if (B < 0 || W <= 0 || W > svt::kBeamMaxW || V <= 0 || K <= 0 || K > svt::kBeamMaxK) return svt::kStatusBytes;  // refused
  svt::BeamParams p{};
  p.B = B;
  p.W = W;
  p.V = V;
  p.K = K;
  svt::plan_beam(p, sm_count());
  return carve_beam(p, nullptr);
}

svt_status svt_beam_select(const void* logits, svt_dtype dtype, int32_t B, int32_t W, int32_t V, int64_t stride_b,
                           int64_t stride_w, const float* scores, const uint8_t* finished, int32_t end_token, int32_t K,
                           float* out_scores, int32_t* parents, int32_t* tokens, void* ws, size_t ws_bytes,
                           svt_stream_t stream) {
  if (dtype != SVT_BF16 && dtype != SVT_F32)
    return set_last_error(SVT_ERR_UNSUPPORTED, "unknown dtype %d", static_cast<int>(dtype));
  if (B < 0) return set_last_error(SVT_ERR_INVALID_ARG, "B must be >= 0");
  if (W <= 0 || V <= 0 || K <= 0) return set_last_error(SVT_ERR_INVALID_ARG, "W, V and K must be > 0");
  if (W > svt::kBeamMaxW || K > svt::kBeamMaxK || W * K > svt::kBeamMaxWK)
    return set_last_error(SVT_ERR_UNSUPPORTED, "at most %d beams and %d candidates, W * K at most %d", svt::kBeamMaxW,
                          svt::kBeamMaxK, svt::kBeamMaxWK);
  if (static_cast<long long>(W) * V >= (1ll << 31) || static_cast<long long>(B) * W >= (1ll << 24))
    return set_last_error(SVT_ERR_UNSUPPORTED, "W * V must be below 2^31 and B * W below 2^24");
  if (finished != nullptr && (end_token < 0 || end_token >= V))
    return set_last_error(SVT_ERR_INVALID_ARG, "end_token %d is no token of %d", end_token, V);
  svt::BeamParams p{};
  p.logits = logits;
  p.stride_b = stride_b;
  p.stride_w = stride_w;
  p.scores = scores;
  p.finished = finished;
  p.B = B;
  p.W = W;
  p.V = V;
  p.K = K;
  p.end_token = end_token;
  p.out_scores = out_scores;
  p.parents = parents;
  p.tokens = tokens;
  if (B == 0) return SVT_OK;
  if (logits == nullptr || scores == nullptr || out_scores == nullptr || parents == nullptr || tokens == nullptr)
    return set_last_error(SVT_ERR_INVALID_ARG, "logits, scores, out_scores, parents and tokens must not be null");
  if (!aligned(logits, dtype == SVT_F32 ? 4 : 2))
    return set_last_error(SVT_ERR_INVALID_ARG, "logits must be aligned to their elements");
  svt::plan_beam(p, sm_count());
  const svt_status st = svt::check_workspace(ws, ws_bytes, carve_beam(p, ws));
  if (st != SVT_OK) return st;
  const cudaError_t e = svt::launch_beam(p, dtype == SVT_F32, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "svt_beam_select");
  return SVT_OK;
}

size_t svt_fork_pages_workspace_size(int64_t num_pages, int32_t num_rows, int32_t num_new_rows) {
  if (num_pages <= 0 || num_pages >= (1ll << 31) || num_rows < 0 || num_rows > svt::kForkMaxRows || num_new_rows < 0 ||
      num_new_rows > svt::kForkMaxRows)
    return svt::kStatusBytes;  // refused
  svt::ForkParams p{};
  p.pool.num_pages = num_pages;
  svt::plan_pool(p.pool);
  p.R = num_rows;
  p.N = num_new_rows;
  p.scan_ctas = svt::fork_scan_ctas(p.pool, num_rows, sm_count());
  return carve_fork(p, nullptr);
}

svt_status svt_fork_pages(const svt_kv_cache* kv, const int32_t* refs, int32_t* refs_out, const int32_t* block_table,
                          int32_t num_rows, int32_t max_blocks, const int32_t* seq_lens, const int32_t* parents,
                          int32_t num_new_rows, const int32_t* grow, int32_t grow_all, int32_t max_grow,
                          int32_t* block_table_out, int32_t max_blocks_out, int32_t* seq_lens_out, int32_t* slots,
                          void* ws, size_t ws_bytes, svt_stream_t stream) {
  svt::ForkParams p{};
  svt_status st = check_pool(kv, refs, refs_out, p.pool, p.kv);
  if (st != SVT_OK) return st;
  if (num_rows < 0 || num_new_rows < 0 || max_blocks < 0 || max_blocks_out < 0)
    return set_last_error(SVT_ERR_INVALID_ARG, "num_rows, num_new_rows and both max_blocks must be >= 0");
  if (num_rows > svt::kForkMaxRows || num_new_rows > svt::kForkMaxRows)
    return set_last_error(SVT_ERR_UNSUPPORTED, "at most %d rows", svt::kForkMaxRows);
  if (max_blocks * static_cast<long long>(kv->page_size) > kMaxTokens ||
      max_blocks_out * static_cast<long long>(kv->page_size) > kMaxTokens)
    return set_last_error(SVT_ERR_UNSUPPORTED, "max_blocks * page_size must be at most 2^30");
  if (max_grow < 0 || (grow == nullptr && (grow_all < 0 || grow_all > max_grow)))
    return set_last_error(SVT_ERR_INVALID_ARG, "grow must be between 0 and max_grow");
  if (max_grow > kMaxTokens) return set_last_error(SVT_ERR_UNSUPPORTED, "max_grow must be at most 2^30");
  if (num_rows > 0 && (seq_lens == nullptr || (max_blocks > 0 && block_table == nullptr)))
    return set_last_error(SVT_ERR_INVALID_ARG, "block_table and seq_lens must not be null");
  if (num_new_rows > 0 && (parents == nullptr || seq_lens_out == nullptr ||
                           (max_blocks_out > 0 && block_table_out == nullptr) || (max_grow > 0 && slots == nullptr)))
    return set_last_error(SVT_ERR_INVALID_ARG, "parents, block_table_out, seq_lens_out and slots must not be null");
  const size_t in_bytes = 4ull * num_rows * max_blocks, out_bytes = 4ull * num_new_rows * max_blocks_out;
  const char *in = reinterpret_cast<const char*>(block_table), *out = reinterpret_cast<const char*>(block_table_out);
  if (in_bytes > 0 && out_bytes > 0 && in < out + out_bytes && out < in + in_bytes)
    return set_last_error(SVT_ERR_INVALID_ARG, "block_table_out must not overlap block_table");
  if (seq_lens_out != nullptr && seq_lens_out == seq_lens)
    return set_last_error(SVT_ERR_INVALID_ARG, "seq_lens_out must not be seq_lens");
  p.table = block_table;
  p.lens = seq_lens;
  p.parents = parents;
  p.grow = grow;
  p.R = num_rows;
  p.M = max_blocks;
  p.N = num_new_rows;
  p.M_out = max_blocks_out;
  p.page_size = kv->page_size;
  p.grow_all = grow_all;
  p.max_grow = max_grow;
  p.table_out = block_table_out;
  p.lens_out = seq_lens_out;
  p.slots = slots;
  p.scan_ctas = svt::fork_scan_ctas(p.pool, num_rows, sm_count());
  // a copy's share of at most 16 KB for a CTA, while they do not all fill the GPU by themselves
  const long long page_bytes = static_cast<long long>(kv->page_size) * p.kv.row_bytes;
  p.shares = static_cast<int>(std::max(1ll, std::min(8ll, page_bytes / 16384)));
  st = svt::check_workspace(ws, ws_bytes, carve_fork(p, ws));
  if (st != SVT_OK) return st;
  p.status = static_cast<int*>(ws);
  const cudaError_t e = svt::launch_fork(p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "svt_fork_pages");
  return SVT_OK;
}

size_t svt_compact_pages_workspace_size(int64_t num_pages) {
  if (num_pages <= 0 || num_pages >= (1ll << 31)) return svt::kStatusBytes;  // refused
  svt::CompactParams p{};
  p.pool.num_pages = num_pages;
  svt::plan_pool(p.pool);
  return carve_compact(p, nullptr);
}

svt_status svt_compact_pages(const svt_kv_cache* kv, const int32_t* refs, int32_t* refs_out, const int32_t* block_table,
                             int64_t entries, int32_t* block_table_out, int32_t* mapping, void* ws, size_t ws_bytes,
                             svt_stream_t stream) {
  svt::CompactParams p{};
  svt_status st = check_pool(kv, refs, refs_out, p.pool, p.kv);
  if (st != SVT_OK) return st;
  if (entries < 0) return set_last_error(SVT_ERR_INVALID_ARG, "entries must be >= 0");
  if (entries > 0 && (block_table == nullptr || block_table_out == nullptr))
    return set_last_error(SVT_ERR_INVALID_ARG, "block_table and block_table_out must not be null");
  p.table = block_table;
  p.table_out = block_table_out;
  p.entries = entries;
  p.mapping = mapping;
  st = svt::check_workspace(ws, ws_bytes, carve_compact(p, ws));
  if (st != SVT_OK) return st;
  p.status = static_cast<int*>(ws);
  const cudaError_t e = svt::launch_compact(p, sm_count(), reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "svt_compact_pages");
  return SVT_OK;
}

}  // extern "C"
