// C ABI of the operators around the attention: rotary positions, cache writes, the attention's
// backward pass and the indexer's distillation loss. As everywhere in the library, every check
// comes before anything is enqueued, and nothing allocates device memory or waits for a stream.
#include <atomic>
#include <cmath>
#include <cstring>

#include "internal.h"

namespace {

using svt::set_last_error;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

svt_status cuda_fail(cudaError_t e, const char* what) {
  return set_last_error(SVT_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

constexpr int kMaxCols = 16384;  // H, D: the kernels divide 16-bit item numbers

// A rotation's frequencies and layout.
svt_status check_rotation(const double* freqs, int32_t dim, int32_t layout, float amplitude) {
  if (dim <= 0 || dim % 2 != 0) return set_last_error(SVT_ERR_INVALID_ARG, "dim must be even and > 0, got %d", dim);
  if (dim > 512) return set_last_error(SVT_ERR_UNSUPPORTED, "at most 512 rotated columns, got %d", dim);
  if (layout != SVT_ROPE_INTERLEAVED && layout != SVT_ROPE_HALF)
    return set_last_error(SVT_ERR_INVALID_ARG, "unknown rope layout %d", layout);
  if (!std::isfinite(amplitude)) return set_last_error(SVT_ERR_INVALID_ARG, "amplitude must be finite");
  if (freqs == nullptr || !aligned(freqs, 8))
    return set_last_error(SVT_ERR_INVALID_ARG, "freqs must be an 8-byte aligned array");
  return SVT_OK;
}

svt_status check_rows(const void* x, const void* out, int elem, int32_t T, int32_t H, int32_t D, int32_t dim,
                      int32_t offset) {
  if (T < 0 || H < 0) return set_last_error(SVT_ERR_INVALID_ARG, "T and H must be >= 0");
  if (H > kMaxCols || D > kMaxCols) return set_last_error(SVT_ERR_UNSUPPORTED, "H and D must be at most %d", kMaxCols);
  if (static_cast<long long>(T) * H >= (1ll << 31)) return set_last_error(SVT_ERR_UNSUPPORTED, "T * H must be below 2^31");
  if (offset < 0 || D < dim || offset > D - dim)
    return set_last_error(SVT_ERR_INVALID_ARG, "columns %d .. %d are outside the %d columns of a row", offset,
                          offset + dim - 1, D);
  if (T > 0 && H > 0) {
    if (x == nullptr || out == nullptr) return set_last_error(SVT_ERR_INVALID_ARG, "x and out must not be null");
    if (!aligned(x, elem) || !aligned(out, elem))
      return set_last_error(SVT_ERR_INVALID_ARG, "x and out must be aligned to their elements");
  }
  return SVT_OK;
}

// Whether rows [T, H] of D elements at these strides may hold two rows in one place.
bool rows_overlap(int32_t T, int32_t H, int32_t D, int64_t st, int64_t sh) {
  const int64_t at = st < 0 ? -st : st, ah = sh < 0 ? -sh : sh;
  if (H > 1 && ah < D) return true;
  if (T > 1 && at < D) return true;
  if (T > 1 && H > 1) {  // one dimension has to step over all of the other
    if (at >= ah ? at < ah * (H - 1) + D : ah < at * (T - 1) + D) return true;
  }
  return false;
}

// Of the current device; asked for two or three times by a backward call, so known ones are kept.
int sm_count() {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < kDevices && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < kDevices) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

// Workspace: status header | slots | list reaches | (lse, delta) | cut row-sets' dq | cache rows' sums.
struct BackwardWs {
  size_t slots, live_len, stats, part, acc, end;
};
BackwardWs backward_ws(const svt::BackwardParams& p) {
  BackwardWs w;
  w.slots = svt::kStatusBytes;
  w.live_len = w.slots + round_up(static_cast<size_t>(p.T) * p.K * 4, 256);
  w.stats = w.live_len + round_up(static_cast<size_t>(p.T) * p.chunks * 4, 256);
  w.part = w.stats + round_up(static_cast<size_t>(p.T) * p.H * 8, 256);
  w.acc = w.part + 2ull * p.num_ctas * 64 * svt::kRow * 4;
  w.end = w.acc + round_up(static_cast<size_t>(p.num_slots) * svt::kRow * 4, 256);
  return w;
}

}  // namespace

extern "C" {

svt_status svt_rope_frequencies(int32_t dim, double base, const svt_rope_scaling* scaling, double* freqs) {
  if (dim <= 0 || dim % 2 != 0 || dim > 512)
    return set_last_error(SVT_ERR_INVALID_ARG, "dim must be even, in 2 .. 512, got %d", dim);
  if (!(base > 0.0) || !std::isfinite(base)) return set_last_error(SVT_ERR_INVALID_ARG, "base must be finite and > 0");
  if (freqs == nullptr) return set_last_error(SVT_ERR_INVALID_ARG, "freqs must not be null");
  const svt_rope_scaling none = {SVT_ROPE_SCALE_NONE, 1.0, 0.0, 0.0, 0.0};
  const svt_rope_scaling& s = scaling ? *scaling : none;
  if (s.kind < SVT_ROPE_SCALE_NONE || s.kind > SVT_ROPE_SCALE_BY_WAVELENGTH)
    return set_last_error(SVT_ERR_INVALID_ARG, "unknown rope scaling %d", static_cast<int>(s.kind));
  if (s.kind != SVT_ROPE_SCALE_NONE && !(s.factor > 0.0 && std::isfinite(s.factor)))
    return set_last_error(SVT_ERR_INVALID_ARG, "the scaling factor must be finite and > 0");
  const bool bands = s.kind == SVT_ROPE_SCALE_BY_PARTS || s.kind == SVT_ROPE_SCALE_BY_WAVELENGTH;
  if (bands && !(s.original_len > 0.0 && s.slow > 0.0 && s.fast > s.slow && std::isfinite(s.fast) &&
                 std::isfinite(s.original_len)))
    return set_last_error(SVT_ERR_INVALID_ARG, "this scaling needs original_len > 0 and fast > slow > 0");
  if (s.kind == SVT_ROPE_SCALE_BY_PARTS && base == 1.0)
    return set_last_error(SVT_ERR_INVALID_ARG, "scaling by parts needs a base other than 1");
  const double two_pi = 6.283185307179586476925;
  double lo = 0.0, hi = 0.0;
  if (s.kind == SVT_ROPE_SCALE_BY_PARTS) {
    // the (fractional) pair index that makes `turns` full turns over the original length
    auto pair_of = [&](double turns) {
      return dim * std::log(s.original_len / (turns * two_pi)) / (2.0 * std::log(base));
    };
    lo = std::fmax(std::floor(pair_of(s.fast)), 0.0);
    hi = std::fmin(std::ceil(pair_of(s.slow)), dim - 1.0);
  }
  for (int i = 0; i < dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / dim);
    double r = f;
    if (s.kind == SVT_ROPE_SCALE_LINEAR) {
      r = f / s.factor;
    } else if (s.kind == SVT_ROPE_SCALE_BY_PARTS) {
      const double ramp = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 1e-3), 0.0), 1.0);
      r = f / s.factor * ramp + f * (1.0 - ramp);
    } else if (s.kind == SVT_ROPE_SCALE_BY_WAVELENGTH) {
      const double turns = s.original_len * f / two_pi;  // over the original length
      const double keep = std::fmin(std::fmax((turns - s.slow) / (s.fast - s.slow), 0.0), 1.0);
      r = f / s.factor * (1.0 - keep) + f * keep;
    }
    freqs[i] = r;
  }
  return SVT_OK;
}

svt_status svt_rope(const void* x, void* out, svt_dtype dtype, int32_t T, int32_t H, int32_t D, int64_t x_stride_t,
                    int64_t x_stride_h, int64_t out_stride_t, int64_t out_stride_h, const int32_t* positions,
                    const double* freqs, int32_t dim, int32_t offset, svt_rope_layout layout, float amplitude,
                    int32_t inverse, svt_stream_t stream) {
  if (dtype != SVT_BF16 && dtype != SVT_F32)
    return set_last_error(SVT_ERR_UNSUPPORTED, "unknown dtype %d", static_cast<int>(dtype));
  svt_status st = check_rotation(freqs, dim, layout, amplitude);
  if (st != SVT_OK) return st;
  st = check_rows(x, out, dtype == SVT_F32 ? 4 : 2, T, H, D, dim, offset);
  if (st != SVT_OK) return st;
  if (T == 0 || H == 0) return SVT_OK;
  if (positions == nullptr) return set_last_error(SVT_ERR_INVALID_ARG, "positions must not be null");
  if (rows_overlap(T, H, D, out_stride_t, out_stride_h))
    return set_last_error(SVT_ERR_INVALID_ARG, "rows of out overlap");
  if (x == out && (x_stride_t != out_stride_t || x_stride_h != out_stride_h) && (T > 1 || H > 1))
    return set_last_error(SVT_ERR_INVALID_ARG, "a rotation in place needs equal strides");
  svt::RopeParams p{};
  p.x = x;
  p.out = out;
  p.T = T;
  p.H = H;
  p.D = D;
  p.dim = dim;
  p.offset = offset;
  p.x_stride_t = x_stride_t;
  p.x_stride_h = x_stride_h;
  p.out_stride_t = out_stride_t;
  p.out_stride_h = out_stride_h;
  p.positions = positions;
  p.freqs = freqs;
  p.amplitude = amplitude;
  p.sign = inverse ? -1.f : 1.f;
  const cudaError_t e =
      svt::launch_rope(p, dtype == SVT_F32, layout == SVT_ROPE_HALF, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "svt_rope");
  return SVT_OK;
}

svt_status svt_rope_append(const void* latent_bf16, int64_t latent_stride, const void* k_rope_bf16,
                           int64_t k_rope_stride, const int32_t* positions, const int32_t* slots, int32_t T,
                           const svt_kv_cache* kv, const double* freqs, svt_rope_layout layout, float amplitude,
                           const void* q_rope_bf16, int32_t H, int64_t q_stride_t, int64_t q_stride_h, void* q_out_bf16,
                           int64_t q_out_stride_t, int64_t q_out_stride_h, void* ws, size_t ws_bytes,
                           svt_stream_t stream) {
  constexpr int kDim = svt::kRow - svt::kVdim;
  svt_status st = check_rotation(freqs, kDim, layout, amplitude);
  if (st != SVT_OK) return st;
  const bool with_q = q_rope_bf16 != nullptr || q_out_bf16 != nullptr;
  st = check_rows(q_rope_bf16, q_out_bf16, 2, T, with_q ? H : 0, kDim, kDim, 0);
  if (st != SVT_OK) return st;
  if (T > (1 << 30)) return set_last_error(SVT_ERR_UNSUPPORTED, "T must be at most 2^30");
  long long row_stride = 0;
  st = svt::check_kv_cache(kv, &row_stride);
  if (st != SVT_OK) return st;
  st = svt::check_workspace(ws, ws_bytes, svt::kStatusBytes);
  if (st != SVT_OK) return st;
  if (T == 0) return SVT_OK;
  if (latent_bf16 == nullptr || k_rope_bf16 == nullptr || positions == nullptr || slots == nullptr)
    return set_last_error(SVT_ERR_INVALID_ARG, "latent, k_rope, positions and slots must not be null");
  if (!aligned(latent_bf16, 16) || (T > 1 && latent_stride % 8 != 0))
    return set_last_error(SVT_ERR_INVALID_ARG, "latent rows must start on 16-byte boundaries");
  if (!aligned(k_rope_bf16, 2)) return set_last_error(SVT_ERR_INVALID_ARG, "k_rope must be 2-byte aligned");
  if (with_q && H > 0) {
    if (rows_overlap(T, H, kDim, q_out_stride_t, q_out_stride_h))
      return set_last_error(SVT_ERR_INVALID_ARG, "rows of q_out overlap");
    if (q_rope_bf16 == q_out_bf16 && (q_stride_t != q_out_stride_t || q_stride_h != q_out_stride_h))
      return set_last_error(SVT_ERR_INVALID_ARG, "a rotation in place needs equal strides");
  }
  svt::AppendParams p{};
  p.latent = static_cast<const uint16_t*>(latent_bf16);
  p.latent_stride = latent_stride;
  p.k_rope = static_cast<const uint16_t*>(k_rope_bf16);
  p.k_rope_stride = k_rope_stride;
  p.positions = positions;
  p.slots = slots;
  p.freqs = freqs;
  p.amplitude = amplitude;
  p.kv = static_cast<uint8_t*>(const_cast<void*>(kv->data));
  p.row_stride = row_stride;
  p.num_slots = kv->num_pages * static_cast<long long>(kv->page_size);
  p.T = T;
  p.status = static_cast<int*>(ws);
  svt::RopeParams q{};
  q.x = q_rope_bf16;
  q.out = q_out_bf16;
  q.T = T;
  q.H = with_q ? H : 0;
  q.D = q.dim = kDim;
  q.x_stride_t = q_stride_t;
  q.x_stride_h = q_stride_h;
  q.out_stride_t = q_out_stride_t;
  q.out_stride_h = q_out_stride_h;
  q.positions = positions;
  q.freqs = freqs;
  q.amplitude = amplitude;
  q.sign = 1.f;
  const cudaError_t e = svt::launch_append(p, q, kv->dtype == SVT_KV_FP8_E4M3, layout == SVT_ROPE_HALF,
                                           reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "svt_rope_append");
  return SVT_OK;
}

size_t svt_sparse_mla_backward_workspace_size(int32_t T, int32_t H, int32_t K, int64_t num_slots) {
  if (T < 0 || H < 0 || H > 128 || K < 0 || K > (1 << 30) || num_slots < 0) return svt::kStatusBytes;  // refused
  svt::BackwardParams p{};
  p.T = T;
  p.H = H;
  p.K = K;
  p.num_slots = num_slots;
  svt::plan_backward(p, sm_count());
  return backward_ws(p).end;
}

svt_status svt_sparse_mla_backward(const void* q_bf16, int32_t T, int32_t H, const svt_kv_cache* kv,
                                   const int32_t* block_table, int32_t num_reqs, int32_t max_blocks,
                                   const int32_t* req_of_token, const int32_t* seq_lens, const int32_t* topk, int32_t K,
                                   const int32_t* topk_len, float softmax_scale, const void* out_bf16, const float* lse,
                                   const void* dout_bf16, const float* dlse, void* dq_bf16, void* dkv_bf16,
                                   float* weights, void* ws, size_t ws_bytes, svt_stream_t stream) {
  if (T < 0 || K < 0) return set_last_error(SVT_ERR_INVALID_ARG, "T and K must be >= 0");
  if (H <= 0) return set_last_error(SVT_ERR_INVALID_ARG, "H must be > 0");
  if (H > 128) return set_last_error(SVT_ERR_UNSUPPORTED, "backward supports at most 128 heads, got %d", H);
  if (!std::isfinite(softmax_scale)) return set_last_error(SVT_ERR_INVALID_ARG, "softmax_scale must be finite");
  long long row_stride = 0;
  svt_status st = svt::check_kv_cache(kv, &row_stride);
  if (st != SVT_OK) return st;
  if (kv->dtype != SVT_KV_BF16) return set_last_error(SVT_ERR_UNSUPPORTED, "backward takes a bf16 cache");
  if (block_table != nullptr && (num_reqs <= 0 || max_blocks <= 0))
    return set_last_error(SVT_ERR_INVALID_ARG, "num_reqs and max_blocks must be > 0 with a block table");
  const long long num_slots = kv->num_pages * static_cast<long long>(kv->page_size);
  if (static_cast<long long>(T) * H >= (1ll << 30) || static_cast<long long>(T) * K >= (1ll << 40) ||
      K > (1 << 30))
    return set_last_error(SVT_ERR_UNSUPPORTED, "T * H and K must be below 2^30 and T * K below 2^40");
  svt::BackwardParams p{};
  p.T = T;
  p.H = H;
  p.K = K;
  p.num_slots = num_slots;
  svt::plan_backward(p, sm_count());
  const BackwardWs w = backward_ws(p);
  if (dkv_bf16 == nullptr || !aligned(dkv_bf16, 16))
    return set_last_error(SVT_ERR_INVALID_ARG, "dkv must be a 16-byte aligned array");
  if (T > 0) {
    if (q_bf16 == nullptr || out_bf16 == nullptr || lse == nullptr || dout_bf16 == nullptr || dq_bf16 == nullptr)
      return set_last_error(SVT_ERR_INVALID_ARG, "q, out, lse, dout and dq must not be null");
    if (!aligned(q_bf16, 16) || !aligned(out_bf16, 16) || !aligned(dout_bf16, 16) || !aligned(dq_bf16, 16))
      return set_last_error(SVT_ERR_INVALID_ARG, "q, out, dout and dq must be 16-byte aligned");
    if (K > 0 && topk == nullptr) return set_last_error(SVT_ERR_INVALID_ARG, "topk must not be null");
  }
  // the last check: a call that is refused for anything else is refused before its workspace is made
  st = svt::check_workspace(ws, ws_bytes, w.end);
  if (st != SVT_OK) return st;
  p.q = static_cast<const uint16_t*>(q_bf16);
  p.out = static_cast<const uint16_t*>(out_bf16);
  p.dout = static_cast<const uint16_t*>(dout_bf16);
  p.lse = lse;
  p.dlse = dlse;
  p.kv = static_cast<const uint8_t*>(kv->data);
  p.row_stride = row_stride;
  p.scale = softmax_scale;
  p.dq = static_cast<uint16_t*>(dq_bf16);
  p.dkv = static_cast<uint16_t*>(dkv_bf16);
  p.weights = weights;
  char* base = static_cast<char*>(ws);
  p.slots = reinterpret_cast<int32_t*>(base + w.slots);
  p.live_len = reinterpret_cast<int32_t*>(base + w.live_len);
  p.stats = reinterpret_cast<float2*>(base + w.stats);
  p.dq_part = reinterpret_cast<float*>(base + w.part);
  p.dkv_acc = reinterpret_cast<float*>(base + w.acc);
  p.status = static_cast<int*>(ws);
  svt::debug_fault_state(&p.fault, &p.wait_limit_ns);
  const svt::ListParams lists{topk,     topk_len,      req_of_token, block_table, num_reqs, max_blocks,
                              seq_lens, kv->page_size, kv->num_pages};
  const cudaError_t e = svt::launch_backward(p, lists, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "svt_sparse_mla_backward");
  return SVT_OK;
}

svt_status svt_distill_topk(const void* scores, svt_dtype dtype, int32_t T, int32_t N, int64_t stride,
                            const int32_t* lens, const int32_t* topk, const float* teacher, int32_t K,
                            svt_teacher_kind kind, svt_distill_scope scope, float temperature, const float* row_weight,
                            float* loss, void* dscores, int64_t dstride, svt_stream_t stream) {
  if (dtype != SVT_BF16 && dtype != SVT_F32)
    return set_last_error(SVT_ERR_UNSUPPORTED, "unknown dtype %d", static_cast<int>(dtype));
  const int elem = dtype == SVT_F32 ? 4 : 2;
  if (T < 0 || N < 0) return set_last_error(SVT_ERR_INVALID_ARG, "T and N must be >= 0");
  if (K < 1) return set_last_error(SVT_ERR_INVALID_ARG, "K must be >= 1");
  if (N > (1 << 30) || K > (1 << 30) || T > (1 << 27))
    return set_last_error(SVT_ERR_UNSUPPORTED, "N and K are limited to 2^30, T to 2^27");
  if (kind != SVT_TEACHER_WEIGHTS && kind != SVT_TEACHER_LOGITS)
    return set_last_error(SVT_ERR_INVALID_ARG, "unknown teacher kind %d", static_cast<int>(kind));
  if (scope != SVT_DISTILL_CANDIDATES && scope != SVT_DISTILL_LISTED)
    return set_last_error(SVT_ERR_INVALID_ARG, "unknown scope %d", static_cast<int>(scope));
  if (!std::isfinite(temperature) || !(temperature >= 1e-6f) || temperature > 1e6f)
    return set_last_error(SVT_ERR_INVALID_ARG, "temperature must be between 1e-6 and 1e6");
  if (T > 1 && (stride < N || (dscores != nullptr && dstride < N)))
    return set_last_error(SVT_ERR_INVALID_ARG, "row strides must be at least N");
  if (T == 0) return SVT_OK;
  if (loss == nullptr && dscores == nullptr)
    return set_last_error(SVT_ERR_INVALID_ARG, "loss and dscores are both null");
  if ((N > 0 && scores == nullptr) || topk == nullptr || teacher == nullptr)
    return set_last_error(SVT_ERR_INVALID_ARG, "scores, topk and teacher must not be null");
  if (!aligned(scores, elem) || !aligned(dscores, elem))
    return set_last_error(SVT_ERR_INVALID_ARG, "scores and dscores must be aligned to their elements");
  if (dscores != nullptr && dscores == scores)
    return set_last_error(SVT_ERR_INVALID_ARG, "dscores must not be scores");
  svt::DistillParams p{};
  p.scores = scores;
  p.stride = stride;
  p.lens = lens;
  p.idx = topk;
  p.teacher = teacher;
  p.T = T;
  p.N = N;
  p.K = K;
  p.logits = kind == SVT_TEACHER_LOGITS;
  p.inv_tau = 1.f / temperature;
  p.row_weight = row_weight;
  p.loss = loss;
  p.dscores = dscores;
  p.dstride = dstride;
  auto vec_ok = [&](const void* q, int64_t s) { return aligned(q, 16) && (T == 1 || (s * elem) % 16 == 0); };
  p.vec = vec_ok(scores, stride) && (dscores == nullptr || vec_ok(dscores, dstride));
  const cudaError_t e = svt::launch_distill(p, dtype == SVT_F32, scope == SVT_DISTILL_CANDIDATES,
                                            reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "svt_distill_topk");
  return SVT_OK;
}

}  // extern "C"
