// The C ABI of include/tl.h: argument validation, the per-device status word
// and the kernel launches. Validation happens before any CUDA call, so argument
// errors return without touching the device (and work without a GPU).
#include "tl_internal.cuh"

#include <atomic>
#include <mutex>

#include "kv_append.cuh"
#include "lora.cuh"
#include "paged_attention.cuh"
#include "tree.cuh"
#include "tree_attention.cuh"

namespace {

__device__ int g_status_word;

constexpr int kMaxDevices = 64;
int* g_status_ptr[kMaxDevices];
std::mutex g_status_mu;

// Device address of this device's status word (resolved once per device).
int status_ptr(int** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return TL_ECUDA;
  std::lock_guard<std::mutex> lk(g_status_mu);
  if (g_status_ptr[dev] == nullptr) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_status_word) != cudaSuccess) return TL_ECUDA;
    g_status_ptr[dev] = static_cast<int*>(p);
  }
  *out = g_status_ptr[dev];
  return TL_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_nk(int N, int K) {
  if (N < 0 || K <= 0) return TL_EINVAL;
  if (K % tl::kBlock != 0 || K > tl::kMaxK) return TL_EUNSUPPORTED;
  if (N % 128 != 0) return TL_EUNSUPPORTED;
  return TL_OK;
}

int check_linear(const void* packed, const void* qT, const void* sw, const void* xq,
                 const void* sx, int M, int N, int K, const void* y, int y_dtype,
                 const void* acc_dbg) {
  if (M < 0) return TL_EINVAL;
  int r = check_nk(N, K);
  if (r != TL_OK) return r;
  if (y_dtype != TL_BF16 && y_dtype != TL_F32) return TL_EINVAL;
  if (M == 0 || N == 0) return TL_OK;
  if (!packed || !qT || !sw || !xq || !sx || !y) return TL_EINVAL;
  if (!aligned16(packed) || !aligned16(qT) || !aligned16(sw) || !aligned16(xq) ||
      !aligned16(sx) || !aligned16(y) || (acc_dbg && !aligned16(acc_dbg)))
    return TL_EINVAL;
  return TL_OK;
}

cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

// SMs of the current device (looked up once per device).
int num_sms(int* out) {
  static std::atomic<int> sms[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return TL_ECUDA;
  int n = sms[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return TL_ECUDA;
    sms[dev].store(n, std::memory_order_relaxed);
  }
  *out = n;
  return TL_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// rows of `width` elements, `ld` apart, that are read or written as 16-byte vectors of 16-bit elements
int check_rows(int64_t ld, int64_t width, int64_t rows, int elems16) {
  if (rows <= 1) return TL_OK;
  if (ld < 0) return TL_EINVAL;
  return ld % elems16 == 0 && ld >= width ? TL_OK : TL_EUNSUPPORTED;
}

int check_cache(const tl_kv_cache* c) {
  if (c == nullptr || c->kv_heads <= 0 || c->head_dim <= 0 || c->page_size <= 0 || c->num_pages < 0) return TL_EINVAL;
  if (c->dtype != TL_BF16 && c->dtype != TL_F16 && c->dtype != TL_F8E4M3) return TL_EINVAL;
  const bool f8 = c->dtype == TL_F8E4M3;
  if (f8 != (c->k_scale != nullptr) || f8 != (c->v_scale != nullptr)) return TL_EINVAL;
  if (!aligned4(c->k_scale) || !aligned4(c->v_scale) || !aligned16(c->k) || !aligned16(c->v)) return TL_EINVAL;
  if (c->num_pages > 0 && (c->k == nullptr || c->v == nullptr)) return TL_EINVAL;
  const int64_t step = f8 ? 16 : 8;
  if (c->page_stride <= 0 || c->head_stride <= 0 || c->token_stride <= 0) return TL_EINVAL;
  if (c->page_stride % step || c->head_stride % step || c->token_stride % step) return TL_EUNSUPPORTED;
  if (c->kv_heads > 1024) return TL_EUNSUPPORTED;
  return TL_OK;
}

bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

// Places of a request's pages; keys and a tile more stay in an int.
int tree_capacity(int max_pages, int page_size) {
  const int64_t most = static_cast<int64_t>(max_pages) * page_size, limit = 0x7FFF0000;
  return static_cast<int>(most < limit ? most : limit);
}

// What the calls on drafted trees share.
int check_trees(const int32_t* starts, int B, int T, const int32_t* lens, const int32_t* pages, int max_pages, int64_t ldp) {
  if (B < 0 || T < 0 || max_pages < 0) return TL_EINVAL;
  if (B == 0 && T == 0) return TL_OK;
  if (!starts || !aligned4(starts) || !aligned4(lens) || !aligned4(pages)) return TL_EINVAL;
  if (B > 0 && (!lens || (max_pages > 0 && !pages))) return TL_EINVAL;
  if (B > 1 && ldp < max_pages) return TL_EINVAL;
  return TL_OK;
}

// Query heads are taken in groups of 8, 16 or 32, columns of the MMA: the fewest that hold the heads of one
// key-value head, at most 16 for head_dim 256, whose output fills the registers.
int attention_columns(int group, int dim) {
  return group <= 8 ? 1 : group <= 16 || dim == 256 ? 2 : 4;
}

int check_attention_shape(int B, int q_heads, int kv_heads, int head_dim) {
  if (B < 0 || q_heads <= 0 || kv_heads <= 0 || head_dim <= 0) return TL_EINVAL;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return TL_EUNSUPPORTED;
  if (q_heads % kv_heads != 0 || q_heads / kv_heads > 128 || q_heads > 1024) return TL_EUNSUPPORTED;
  return TL_OK;
}

// A wait that nothing ends: phase 0 of a fresh mbarrier with no arrival. The
// bounded wait gives up after limit_ns and records TL_ETIMEOUT, the path every
// kernel of the library takes when one of its waits runs out.
__global__ void wait_selftest_kernel(int* status, unsigned long long limit_ns) {
  __shared__ __align__(8) uint64_t bar;
  if (threadIdx.x == 0) {
    tl::mbar_init(tl::smem_u32(&bar), 1);
    tl::fence_barrier_init();
  }
  __syncthreads();
  if (threadIdx.x == 0 && !tl::mbar_wait(tl::smem_u32(&bar), 0, nullptr, limit_ns))
    tl::set_status(status, TL_ETIMEOUT);
}

}  // namespace

extern "C" {

const char* tl_strerror(int status) {
  switch (status) {
    case TL_OK: return "TL_OK";
    case TL_EINVAL: return "TL_EINVAL: invalid argument (NULL, negative size, misaligned, bad dtype)";
    case TL_EUNSUPPORTED: return "TL_EUNSUPPORTED: unsupported shape";
    case TL_ECUDA: return "TL_ECUDA: CUDA runtime or launch error";
    case TL_ETIMEOUT: return "TL_ETIMEOUT: a bounded device-side wait gave up";
    case TL_EDATA: return "TL_EDATA: input data out of range";
    case TL_ENOSPACE: return "TL_ENOSPACE: size exceeds the provided capacity";
    default: return "unknown tl_status";
  }
}

int tl_version(void) { return 10100; }

int tl_packed_sizes(int N, int K, size_t* packed_bytes, size_t* qT_bytes, size_t* sw_bytes) {
  const int r = check_nk(N, K);
  if (r != TL_OK) return r;
  if (packed_bytes) *packed_bytes = static_cast<size_t>(N) * K / 4;
  if (qT_bytes) *qT_bytes = static_cast<size_t>(K / tl::kGroup) * N;
  if (sw_bytes) *sw_bytes = static_cast<size_t>(N) * 4;
  return TL_OK;
}

int tl_pack_weights(const int8_t* codes, const uint16_t* s, int N, int K, uint8_t* packed,
                    int8_t* qT, float* sw, void* stream) {
  int r = check_nk(N, K);
  if (r != TL_OK) return r;
  if (N == 0) return TL_OK;
  if (!codes || !s || !packed || !qT || !sw) return TL_EINVAL;
  if (!aligned16(codes) || !aligned16(s) || !aligned16(packed) || !aligned16(qT) || !aligned16(sw))
    return TL_EINVAL;
  int* status = nullptr;
  if ((r = status_ptr(&status)) != TL_OK) return r;
  return tl::launch_pack(codes, s, N, K, reinterpret_cast<uint32_t*>(packed), qT, sw, status,
                         as_stream(stream)) == cudaSuccess
             ? TL_OK
             : TL_ECUDA;
}

int tl_rotate_quant_act(const uint16_t* x, int M, int K, const int8_t* signs, void* xq,
                        int xq_dtype, float* sx, void* stream) {
  if (M < 0 || K <= 0) return TL_EINVAL;
  if (K % tl::kBlock != 0 || K > tl::kMaxK) return TL_EUNSUPPORTED;
  if (xq_dtype != TL_I8 && xq_dtype != TL_F16) return TL_EINVAL;
  if (M == 0) return TL_OK;
  if (!x || !xq || !sx) return TL_EINVAL;
  if (!aligned16(x) || !aligned16(xq) || !aligned16(sx) || (signs && !aligned16(signs)))
    return TL_EINVAL;
  return tl::launch_rotate_quant(x, M, K, signs, xq, xq_dtype, sx, as_stream(stream)) == cudaSuccess
             ? TL_OK
             : TL_ECUDA;
}

int tl_prefill_workspace_size(int M, int N, int K, size_t* bytes) {
  if (bytes == nullptr || M < 0) return TL_EINVAL;
  const int r = check_nk(N, K);
  if (r != TL_OK) return r;
  *bytes = 0;
  if (M == 0 || N == 0) return TL_OK;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return TL_ECUDA;
  *bytes = tl::prefill_workspace_bytes(M, N, K, sms);
  return TL_OK;
}

int tl_linear_prefill(const uint8_t* packed, const int8_t* qT, const float* sw,
                      const uint16_t* xq, const float* sx, int M, int N, int K, void* y,
                      int y_dtype, int32_t* acc_dbg, void* workspace, size_t ws_bytes,
                      void* stream) {
  int r = check_linear(packed, qT, sw, xq, sx, M, N, K, y, y_dtype, acc_dbg);
  if (r != TL_OK || M == 0 || N == 0) return r;
  if (workspace && !aligned16(workspace)) return TL_EINVAL;
  int* status = nullptr;
  if ((r = status_ptr(&status)) != TL_OK) return r;
  tl::PrefillArgs a{packed, qT, sw, xq, sx, M, N, K, y, y_dtype, acc_dbg, workspace, ws_bytes, false};
  cudaError_t ce;
  return tl::launch_prefill(a, status, as_stream(stream), &ce);
}

int tl_linear_prefill_noalloc(const uint8_t* packed, const int8_t* qT, const float* sw,
                              const uint16_t* xq, const float* sx, int M, int N, int K, void* y,
                              int y_dtype, int32_t* acc_dbg, void* stream) {
  int r = check_linear(packed, qT, sw, xq, sx, M, N, K, y, y_dtype, acc_dbg);
  if (r != TL_OK || M == 0 || N == 0) return r;
  size_t need = 0;
  if ((r = tl_prefill_workspace_size(M, N, K, &need)) != TL_OK) return r;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return TL_ECUDA;
  // with fewer tiles than SMs the split is the point: refuse what does not fit;
  // with more, a split without room runs every tile whole
  if (need > tl::kNoAllocScratchBytes && tl::prefill_split_required(M, N, sms)) return TL_ENOSPACE;
  int* status = nullptr;
  if ((r = status_ptr(&status)) != TL_OK) return r;
  void* scratch = nullptr;
  if ((r = tl::prefill_noalloc_scratch(&scratch)) != TL_OK) return r;
  tl::PrefillArgs a{packed, qT, sw, xq, sx, M, N, K, y, y_dtype, acc_dbg, scratch,
                    tl::kNoAllocScratchBytes, true};
  cudaError_t ce;
  return tl::launch_prefill(a, status, as_stream(stream), &ce);
}

int tl_linear_decode(const uint8_t* packed, const int8_t* qT, const float* sw, const int8_t* xq,
                     const float* sx, int M, int N, int K, void* y, int y_dtype,
                     int32_t* acc_dbg, void* stream) {
  int r = check_linear(packed, qT, sw, xq, sx, M, N, K, y, y_dtype, acc_dbg);
  if (r != TL_OK) return r;
  if (M > tl::kMaxDecodeM) return TL_EUNSUPPORTED;
  if (M == 0 || N == 0) return TL_OK;
  return tl::launch_decode(reinterpret_cast<const uint32_t*>(packed), qT, sw, xq, sx, M, N, K, y,
                           y_dtype, acc_dbg, as_stream(stream)) == cudaSuccess
             ? TL_OK
             : TL_ECUDA;
}

int tl_linear_decode_tc(const uint8_t* packed, const int8_t* qT, const float* sw,
                        const uint16_t* xq, const float* sx, int M, int N, int K, void* y,
                        int y_dtype, int32_t* acc_dbg, void* stream) {
  int r = check_linear(packed, qT, sw, xq, sx, M, N, K, y, y_dtype, acc_dbg);
  if (r != TL_OK) return r;
  if (M > tl::kMaxDecodeM) return TL_EUNSUPPORTED;
  if (M == 0 || N == 0) return TL_OK;
  int* status = nullptr;
  if ((r = status_ptr(&status)) != TL_OK) return r;
  return tl::launch_decode_tc(packed, qT, sw, xq, sx, M, N, K, y, y_dtype, acc_dbg, status,
                              as_stream(stream)) == cudaSuccess
             ? TL_OK
             : TL_ECUDA;
}

int tl_linear_decode_fused(const uint8_t* packed, const int8_t* qT, const float* sw,
                           const uint16_t* x, const int8_t* signs, int M, int N, int K, void* y,
                           int y_dtype, int32_t* acc_dbg, int8_t* xq_out, float* sx_out,
                           void* stream) {
  int r = check_linear(packed, qT, sw, x, sw, M, N, K, y, y_dtype, acc_dbg);
  if (r != TL_OK) return r;
  if (M > 16 || (M == 1 && K > tl::kMaxFusedDecodeK)) return TL_EUNSUPPORTED;
  if (M == 0 || N == 0) return TL_OK;
  if ((signs && !aligned16(signs)) || (xq_out && !aligned16(xq_out)) || (sx_out && !aligned16(sx_out)))
    return TL_EINVAL;
  if (M == 1)
    return tl::launch_decode_fused(reinterpret_cast<const uint32_t*>(packed), qT, sw, x, signs, N,
                                   K, y, y_dtype, acc_dbg, xq_out, sx_out,
                                   as_stream(stream)) == cudaSuccess
               ? TL_OK
               : TL_ECUDA;
  bool supported = false;
  const cudaError_t e = tl::launch_decode_fused_m(reinterpret_cast<const uint32_t*>(packed), qT, sw,
                                                  x, signs, M, N, K, y, y_dtype, acc_dbg, xq_out,
                                                  sx_out, as_stream(stream), &supported);
  if (!supported) return TL_EUNSUPPORTED;
  return e == cudaSuccess ? TL_OK : TL_ECUDA;
}

int tl_rotate_act(const uint16_t* x, int M, int K, const int8_t* signs, float* xr, void* stream) {
  if (M < 0 || K <= 0) return TL_EINVAL;
  if (K % tl::kBlock != 0 || K > tl::kMaxK) return TL_EUNSUPPORTED;
  if (M == 0) return TL_OK;
  if (!x || !xr) return TL_EINVAL;
  if (!aligned16(x) || !aligned16(xr) || (signs && !aligned16(signs))) return TL_EINVAL;
  return tl::launch_rotate(x, M, K, signs, xr, as_stream(stream)) == cudaSuccess ? TL_OK : TL_ECUDA;
}

int tl_linear_decode_f32act(const uint8_t* packed, const uint16_t* s, const float* xr, int M, int N,
                            int K, void* y, int y_dtype, void* stream) {
  if (M < 0) return TL_EINVAL;
  int r = check_nk(N, K);
  if (r != TL_OK) return r;
  if (y_dtype != TL_BF16 && y_dtype != TL_F32) return TL_EINVAL;
  if (M > tl::kMaxF32ActM || static_cast<long long>(M) * K > tl::kMaxF32ActMK) return TL_EUNSUPPORTED;
  if (M == 0 || N == 0) return TL_OK;
  if (!packed || !s || !xr || !y) return TL_EINVAL;
  if (!aligned16(packed) || !aligned16(s) || !aligned16(xr) || !aligned16(y)) return TL_EINVAL;
  return tl::launch_decode_f32act(packed, s, xr, M, N, K, y, y_dtype, as_stream(stream)) == cudaSuccess
             ? TL_OK
             : TL_ECUDA;
}

int tl_codec_quant(const uint16_t* x, int R, int H, int8_t* q, float* scale, void* stream) {
  if (R < 0 || H <= 0) return TL_EINVAL;
  if (H % tl::kGroup != 0) return TL_EUNSUPPORTED;
  if (R == 0) return TL_OK;
  if (!x || !q || !scale) return TL_EINVAL;
  if (!aligned16(x) || !aligned16(q) || !aligned16(scale)) return TL_EINVAL;
  return tl::launch_codec_quant(x, R, H, q, scale, as_stream(stream)) == cudaSuccess ? TL_OK
                                                                                      : TL_ECUDA;
}

int tl_codec_dequant_add(const uint16_t* own, const int8_t* q_peers, const float* scale_peers,
                         int npeers, int R, int H, uint16_t* out, void* stream) {
  if (R < 0 || H <= 0 || npeers < 0) return TL_EINVAL;
  if (H % tl::kGroup != 0 || npeers > tl::kMaxCodecPeers) return TL_EUNSUPPORTED;
  if (R == 0) return TL_OK;
  if (!own || !out || (npeers > 0 && (!q_peers || !scale_peers))) return TL_EINVAL;
  if (!aligned16(own) || !aligned16(out) || (npeers > 0 && (!aligned16(q_peers) || !aligned16(scale_peers))))
    return TL_EINVAL;
  return tl::launch_codec_dequant_add(own, q_peers, scale_peers, npeers, R, H, out,
                                      as_stream(stream)) == cudaSuccess
             ? TL_OK
             : TL_ECUDA;
}

int tl_kv_append(const tl_kv_cache* cache, const void* q, const void* k, const void* v, int dtype,
                 int T, int q_heads, int64_t ldq, int64_t ldk, int64_t ldv, void* q_out,
                 int64_t ldqo, const float* cos_sin, int max_pos, int rot_dim, int interleaved,
                 const int32_t* positions, const int64_t* slots, void* stream) {
  return tl_kv_append_norm(cache, q, k, v, dtype, T, q_heads, ldq, ldk, ldv, q_out, ldqo, nullptr, nullptr, 1.f, cos_sin, max_pos,
                           rot_dim, interleaved, positions, slots, stream);
}

int tl_kv_append_norm(const tl_kv_cache* cache, const void* q, const void* k, const void* v,
                      int dtype, int T, int q_heads, int64_t ldq, int64_t ldk, int64_t ldv,
                      void* q_out, int64_t ldqo, const float* q_norm, const float* k_norm,
                      float eps, const float* cos_sin, int max_pos, int rot_dim, int interleaved,
                      const int32_t* positions, const int64_t* slots, void* stream) {
  int r = check_cache(cache);
  if (r != TL_OK) return r;
  if (T < 0 || q_heads < 0 || rot_dim < 0 || max_pos < 0 || (interleaved != 0 && interleaved != 1)) return TL_EINVAL;
  if (dtype != TL_BF16 && dtype != TL_F16) return TL_EINVAL;
  if (cache->dtype != TL_F8E4M3 && cache->dtype != dtype) return TL_EINVAL;
  if (!(eps > 0.f) || !(eps - eps == 0.f)) return TL_EINVAL;
  const int d = cache->head_dim;
  if (d % 16 != 0 || d > 512 || q_heads > 1024 || rot_dim % 16 != 0 || rot_dim > d) return TL_EUNSUPPORTED;
  if (q == nullptr) q_heads = 0;
  if (T == 0) return TL_OK;
  if (!k || !v || !slots || (q_heads > 0 && !q_out)) return TL_EINVAL;
  if (rot_dim > 0 && (!cos_sin || !positions)) return TL_EINVAL;
  if (!aligned16(k) || !aligned16(v) || !aligned16(q) || (q_heads > 0 && !aligned16(q_out)) || !aligned16(cos_sin) ||
      !aligned16(q_norm) || !aligned16(k_norm) || !aligned4(positions) || (reinterpret_cast<uintptr_t>(slots) & 7u) != 0)
    return TL_EINVAL;
  const int64_t wq = static_cast<int64_t>(q_heads) * d, wk = static_cast<int64_t>(cache->kv_heads) * d;
  if ((r = check_rows(ldk, wk, T, 8)) != TL_OK || (r = check_rows(ldv, wk, T, 8)) != TL_OK) return r;
  if (q_heads > 0 && ((r = check_rows(ldq, wq, T, 8)) != TL_OK || (r = check_rows(ldqo, wq, T, 8)) != TL_OK)) return r;
  if (q_heads > 0 && q == q_out && T > 1 && ldq != ldqo) return TL_EINVAL;      // in place, but the rows lie elsewhere
  int sms = 0;
  int* status = nullptr;
  if ((r = num_sms(&sms)) != TL_OK || (r = status_ptr(&status)) != TL_OK) return r;
  tl::AppendParams p{};
  p.ck = cache->k, p.cv = cache->v, p.k_scale = cache->k_scale, p.v_scale = cache->v_scale;
  p.page_stride = cache->page_stride, p.head_stride = cache->head_stride, p.token_stride = cache->token_stride;
  p.num_slots = static_cast<int64_t>(cache->num_pages) * cache->page_size;
  p.q = static_cast<const uint16_t*>(q), p.k = static_cast<const uint16_t*>(k), p.v = static_cast<const uint16_t*>(v);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.ldq = ldq, p.ldk = ldk, p.ldv = ldv, p.ldqo = ldqo;
  p.cos_sin = cos_sin, p.positions = positions, p.slots = slots, p.status = status;
  p.q_heads = q_heads, p.kv_heads = cache->kv_heads, p.dim = d, p.page_size = cache->page_size;
  p.rot = rot_dim, p.max_pos = max_pos, p.interleaved = interleaved;
  p.q_norm = q_heads > 0 ? q_norm : nullptr, p.k_norm = k_norm, p.eps = eps;
  return tl::launch_kv_append(p, T, dtype == TL_BF16, cache->dtype == TL_F8E4M3, sms, as_stream(stream)) == cudaSuccess
             ? TL_OK
             : TL_ECUDA;
}

int tl_paged_attention_workspace_size(int B, int q_heads, int kv_heads, int head_dim, size_t* bytes) {
  if (bytes == nullptr) return TL_EINVAL;
  int r = check_attention_shape(B, q_heads, kv_heads, head_dim);
  if (r != TL_OK) return r;
  *bytes = 0;
  if (B == 0) return TL_OK;
  int sms = 0;
  if ((r = num_sms(&sms)) != TL_OK) return r;
  const long long grid = sms * tl::kAttnMaxBlocksPerSm < tl::kAttnMaxGrid ? sms * tl::kAttnMaxBlocksPerSm : tl::kAttnMaxGrid;
  const int heads = 8 * attention_columns(q_heads / kv_heads, head_dim);
  *bytes = tl::kAttnLevels * tl::kAttnMaxGrid * sizeof(int) + 2 * grid * tl::attn_partial_floats(heads, head_dim) * sizeof(float);
  return TL_OK;
}

int tl_paged_attention(const tl_kv_cache* cache, const void* q, int dtype, int B, int q_heads,
                       int64_t ldq, const int32_t* pages, int max_pages, int64_t ldp,
                       const int32_t* lens, float scale, int window, void* out, int64_t ldo,
                       float* lse, void* workspace, size_t ws_bytes, void* stream) {
  int r = check_cache(cache);
  if (r != TL_OK) return r;
  if (max_pages < 0 || window < 0 || !(scale - scale == 0.f)) return TL_EINVAL;
  if (dtype != TL_BF16 && dtype != TL_F16) return TL_EINVAL;
  if (cache->dtype != TL_F8E4M3 && cache->dtype != dtype) return TL_EINVAL;
  if ((r = check_attention_shape(B, q_heads, cache->kv_heads, cache->head_dim)) != TL_OK) return r;
  if (B == 0) return TL_OK;
  if (!q || !out || !lens || !workspace || (max_pages > 0 && !pages)) return TL_EINVAL;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || !aligned4(lens) || !aligned4(pages) || !aligned4(lse))
    return TL_EINVAL;
  const int64_t wq = static_cast<int64_t>(q_heads) * cache->head_dim;
  if ((r = check_rows(ldq, wq, B, 8)) != TL_OK || (r = check_rows(ldo, wq, B, 8)) != TL_OK) return r;
  if (B > 1 && ldp < max_pages) return TL_EINVAL;
  size_t need = 0;
  if ((r = tl_paged_attention_workspace_size(B, q_heads, cache->kv_heads, cache->head_dim, &need)) != TL_OK) return r;
  if (ws_bytes < need) return TL_ENOSPACE;
  int sms = 0;
  int* status = nullptr;
  if ((r = num_sms(&sms)) != TL_OK || (r = status_ptr(&status)) != TL_OK) return r;
  const int bytes = cache->dtype == TL_F8E4M3 ? 1 : 2;
  tl::AttnParams p{};
  p.k = static_cast<const uint8_t*>(cache->k), p.v = static_cast<const uint8_t*>(cache->v);
  p.k_scale = cache->k_scale, p.v_scale = cache->v_scale;
  p.page_stride = cache->page_stride * bytes, p.head_stride = cache->head_stride * bytes, p.token_stride = cache->token_stride * bytes;
  p.num_pages = cache->num_pages;
  p.page = tl::FastDiv::make(static_cast<uint32_t>(cache->page_size));
  p.q = static_cast<const uint16_t*>(q), p.out = static_cast<uint16_t*>(out), p.ldq = ldq, p.ldo = ldo;
  p.pages = pages, p.ldp = ldp, p.lens = lens, p.lse = lse;
  const int64_t most = static_cast<int64_t>(max_pages) * cache->page_size, limit = 0x7FFF0000;   // keys + a tile stay in an int
  p.max_len = static_cast<int>(most < limit ? most : limit);
  p.scale_log2 = scale * tl::kLog2e;
  p.B = B, p.q_heads = q_heads, p.kv_heads = cache->kv_heads, p.group = q_heads / cache->kv_heads, p.window = window;
  p.q_bf16 = dtype == TL_BF16;
  p.runs16 = cache->page_size % 16 == 0;
  const int columns = attention_columns(p.group, cache->head_dim);
  p.groups_per_kv = (p.group + 8 * columns - 1) / (8 * columns);
  p.counters = static_cast<int*>(workspace);
  p.partials = reinterpret_cast<float*>(static_cast<char*>(workspace) + tl::kAttnLevels * tl::kAttnMaxGrid * sizeof(int));
  p.status = status;
  const cudaStream_t st = as_stream(stream);
  const cudaError_t e = cache->dtype == TL_BF16  ? tl::launch_attn_bf16(p, cache->head_dim, columns, sms, st)
                        : cache->dtype == TL_F16 ? tl::launch_attn_f16(p, cache->head_dim, columns, sms, st)
                                                 : tl::launch_attn_f8(p, cache->head_dim, columns, sms, st);
  return e == cudaSuccess ? TL_OK : TL_ECUDA;
}

int tl_tree_plan(const int32_t* parents, const int32_t* starts, int B, int T, const int32_t* lens,
                 const int32_t* pages, int max_pages, int64_t ldp, int page_size, int num_pages,
                 int64_t* masks, int32_t* positions, int64_t* slots, void* stream) {
  if (B < 0 || T < 0 || page_size <= 0 || num_pages < 0) return TL_EINVAL;
  int r = check_trees(starts, B, T, lens, pages, max_pages, ldp);
  if (r != TL_OK || T == 0) return r;
  if (!parents || !masks || !positions || !slots) return TL_EINVAL;
  if (!aligned4(parents) || !aligned8(masks) || !aligned4(positions) || !aligned8(slots)) return TL_EINVAL;
  int* status = nullptr;
  if ((r = status_ptr(&status)) != TL_OK) return r;
  const tl::TreePlanParams p{parents, starts, lens, pages, ldp, masks, positions, slots, status, B, T, page_size, num_pages,
                             tree_capacity(max_pages, page_size)};
  return tl::launch_tree_plan(p, as_stream(stream)) == cudaSuccess ? TL_OK : TL_ECUDA;
}

int tl_tree_attention_workspace_size(int B, int T, int q_heads, int kv_heads, int head_dim, size_t* bytes) {
  if (bytes == nullptr || T < 0) return TL_EINVAL;
  int r = check_attention_shape(B, q_heads, kv_heads, head_dim);
  if (r != TL_OK) return r;
  *bytes = 0;
  if (B == 0 || T == 0) return TL_OK;
  int sms = 0;
  if ((r = num_sms(&sms)) != TL_OK) return r;
  const long long all = static_cast<long long>(sms) * tl::tree_blocks_per_sm(head_dim);
  const long long grid = all < tl::kTreeMaxGrid ? all : tl::kTreeMaxGrid;
  *bytes = tl::kTreeMaxGrid * sizeof(tl::TreeCut) + 2 * grid * tl::tree_partial_floats(head_dim) * sizeof(float);
  return TL_OK;
}

int tl_tree_attention(const tl_kv_cache* cache, const void* q, int dtype, int B, int T, int q_heads,
                      int64_t ldq, const int64_t* masks, const int32_t* starts,
                      const int32_t* pages, int max_pages, int64_t ldp, const int32_t* lens,
                      float scale, int window, int sinks, void* out, int64_t ldo, float* lse,
                      void* workspace, size_t ws_bytes, void* stream) {
  int r = check_cache(cache);
  if (r != TL_OK) return r;
  if (T < 0 || window < 0 || sinks < 0 || (window == 0 && sinks != 0) || !(scale - scale == 0.f)) return TL_EINVAL;
  if (dtype != TL_BF16 && dtype != TL_F16) return TL_EINVAL;
  if (cache->dtype != TL_F8E4M3 && cache->dtype != dtype) return TL_EINVAL;
  if ((r = check_attention_shape(B, q_heads, cache->kv_heads, cache->head_dim)) != TL_OK) return r;
  if (window > 0 && window < TL_TREE_NODES) return TL_EUNSUPPORTED;
  if ((r = check_trees(starts, B, T, lens, pages, max_pages, ldp)) != TL_OK || T == 0 || B == 0) return r;
  if (!q || !out || !masks || !workspace) return TL_EINVAL;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || !aligned8(masks) || !aligned4(lse)) return TL_EINVAL;
  const int64_t wq = static_cast<int64_t>(q_heads) * cache->head_dim;
  if ((r = check_rows(ldq, wq, T, 8)) != TL_OK || (r = check_rows(ldo, wq, T, 8)) != TL_OK) return r;
  size_t need = 0;
  if ((r = tl_tree_attention_workspace_size(B, T, q_heads, cache->kv_heads, cache->head_dim, &need)) != TL_OK) return r;
  if (ws_bytes < need) return TL_ENOSPACE;
  int sms = 0;
  int* status = nullptr;
  if ((r = num_sms(&sms)) != TL_OK || (r = status_ptr(&status)) != TL_OK) return r;
  const int bytes = cache->dtype == TL_F8E4M3 ? 1 : 2;
  tl::TreeAttnParams p{};
  p.k = static_cast<const uint8_t*>(cache->k), p.v = static_cast<const uint8_t*>(cache->v);
  p.k_scale = cache->k_scale, p.v_scale = cache->v_scale;
  p.page_stride = cache->page_stride * bytes, p.head_stride = cache->head_stride * bytes, p.token_stride = cache->token_stride * bytes;
  p.num_pages = cache->num_pages;
  p.page = tl::FastDiv::make(static_cast<uint32_t>(cache->page_size));
  p.group = q_heads / cache->kv_heads;
  p.group_div = tl::FastDiv::make(static_cast<uint32_t>(p.group));
  p.q = static_cast<const uint16_t*>(q), p.out = static_cast<uint16_t*>(out), p.ldq = ldq, p.ldo = ldo;
  p.masks = masks, p.starts = starts, p.lens = lens, p.pages = pages, p.ldp = ldp, p.lse = lse;
  p.scale_log2 = scale * tl::kLog2e;
  p.B = B, p.T = T, p.q_heads = q_heads, p.kv_heads = cache->kv_heads, p.window = window, p.sinks = sinks;
  p.q_bf16 = dtype == TL_BF16;
  p.runs16 = cache->page_size % 16 == 0;
  p.capacity = tree_capacity(max_pages, cache->page_size);
  p.cuts = static_cast<tl::TreeCut*>(workspace);
  p.partials = reinterpret_cast<float*>(static_cast<char*>(workspace) + tl::kTreeMaxGrid * sizeof(tl::TreeCut));
  p.status = status;
  const cudaStream_t st = as_stream(stream);
  const cudaError_t e = cache->dtype == TL_BF16  ? tl::launch_tree_attn_bf16(p, cache->head_dim, sms, st)
                        : cache->dtype == TL_F16 ? tl::launch_tree_attn_f16(p, cache->head_dim, sms, st)
                                                 : tl::launch_tree_attn_f8(p, cache->head_dim, sms, st);
  return e == cudaSuccess ? TL_OK : TL_ECUDA;
}

int tl_verify_tree(const float* target, int64_t ldt, const float* draft, int64_t ldd, int vocab,
                   const int32_t* tokens, const int32_t* parents, const int32_t* starts, int B,
                   int T, const float* uniform, int32_t* path, int32_t* counts, int32_t* next,
                   void* stream) {
  if (B < 0 || T < 0 || vocab <= 0) return TL_EINVAL;
  if (vocab > (1 << 24)) return TL_EUNSUPPORTED;
  if (B == 0 && T == 0) return TL_OK;
  if (!starts || (B > 0 && (!counts || !next)) || (T > 0 && (!target || !tokens || !parents || !uniform || !path))) return TL_EINVAL;
  for (const void* x : {static_cast<const void*>(target), static_cast<const void*>(draft), static_cast<const void*>(tokens),
                        static_cast<const void*>(parents), static_cast<const void*>(starts), static_cast<const void*>(uniform),
                        static_cast<const void*>(path), static_cast<const void*>(counts), static_cast<const void*>(next)})
    if (!aligned4(x)) return TL_EINVAL;
  int r;
  if ((r = check_rows(ldt, vocab, T, 1)) != TL_OK || (draft != nullptr && (r = check_rows(ldd, vocab, T, 1)) != TL_OK)) return r;
  if (B == 0)                                          // all rows are padding
    return cudaMemsetAsync(path, 0xFF, static_cast<size_t>(T) * sizeof(int32_t), as_stream(stream)) == cudaSuccess ? TL_OK : TL_ECUDA;
  int sms = 0;
  int* status = nullptr;
  if ((r = num_sms(&sms)) != TL_OK || (r = status_ptr(&status)) != TL_OK) return r;
  const tl::VerifyParams p{target, draft, ldt, ldd, tokens, parents, starts, uniform, path, counts, next, status, vocab, B, T};
  return tl::launch_verify_tree(p, sms, as_stream(stream)) == cudaSuccess ? TL_OK : TL_ECUDA;
}

int tl_kv_compact(const tl_kv_cache* cache, const int32_t* path, const int32_t* counts,
                  const int32_t* starts, int B, int T, const int32_t* pages, int max_pages,
                  int64_t ldp, const int32_t* lens, void* stream) {
  int r = check_cache(cache);
  if (r != TL_OK) return r;
  if (T < 0) return TL_EINVAL;
  const int d = cache->head_dim;
  if (d % 16 != 0 || d > 512) return TL_EUNSUPPORTED;
  if ((r = check_trees(starts, B, T, lens, pages, max_pages, ldp)) != TL_OK || B == 0 || T == 0) return r;
  if (!path || !counts || !aligned4(path) || !aligned4(counts)) return TL_EINVAL;
  int* status = nullptr;
  if ((r = status_ptr(&status)) != TL_OK) return r;
  const int bytes = cache->dtype == TL_F8E4M3 ? 1 : 2;
  tl::CompactParams p{};
  p.k = static_cast<uint8_t*>(cache->k), p.v = static_cast<uint8_t*>(cache->v);
  p.page_stride = cache->page_stride * bytes, p.head_stride = cache->head_stride * bytes, p.token_stride = cache->token_stride * bytes;
  p.path = path, p.counts = counts, p.starts = starts, p.lens = lens, p.pages = pages, p.ldp = ldp, p.status = status;
  p.B = B, p.T = T, p.page_size = cache->page_size, p.num_pages = cache->num_pages;
  p.capacity = tree_capacity(max_pages, cache->page_size);
  p.kv_heads = cache->kv_heads, p.row = d * bytes / 16;
  return tl::launch_kv_compact(p, as_stream(stream)) == cudaSuccess ? TL_OK : TL_ECUDA;
}

int tl_lora_plan_size(int M, int n_adapters, size_t* bytes) {
  if (bytes == nullptr || M < 0 || n_adapters < 0) return TL_EINVAL;
  if (M > tl::kLoraMaxM || n_adapters > tl::kLoraMaxAdapters) return TL_EUNSUPPORTED;
  *bytes = M == 0 ? 0 : tl::lora_plan_bytes(M, n_adapters);
  return TL_OK;
}

int tl_lora_plan(const int32_t* ids, int M, int n_adapters, void* plan, size_t plan_bytes, void* stream) {
  size_t need = 0;
  int r = tl_lora_plan_size(M, n_adapters, &need);
  if (r != TL_OK || M == 0) return r;
  if (!ids || !plan || !aligned4(ids) || !aligned16(plan)) return TL_EINVAL;
  if (plan_bytes < need) return TL_ENOSPACE;
  int* status = nullptr;
  if ((r = status_ptr(&status)) != TL_OK) return r;
  return tl::launch_lora_plan(ids, M, n_adapters, plan, status, as_stream(stream)) == cudaSuccess ? TL_OK : TL_ECUDA;
}

int tl_lora_apply(const void* x, int64_t ldx, const void* A, const void* B, const float* scale,
                  int dtype, int n_adapters, int rank, const void* plan, int M, int N, int K,
                  const void* base, int64_t ldb, void* y, int64_t ldy, int y_dtype, void* stream) {
  if (n_adapters < 0 || M < 0 || N < 0 || K <= 0 || rank <= 0) return TL_EINVAL;
  if (dtype != TL_BF16 && dtype != TL_F16) return TL_EINVAL;
  if (y_dtype != TL_BF16 && y_dtype != TL_F16 && y_dtype != TL_F32) return TL_EINVAL;
  if (M > tl::kLoraMaxM || rank > tl::kLoraMaxRank || rank % 8 != 0) return TL_EUNSUPPORTED;
  if (n_adapters > tl::kLoraMaxAdapters || N % 8 != 0 || K % 8 != 0 || N > (1 << 22)) return TL_EUNSUPPORTED;
  if (M == 0 || N == 0) return TL_OK;
  if (!x || !plan || !base || !y || (n_adapters > 0 && (!A || !B || !scale))) return TL_EINVAL;
  if (!aligned16(x) || !aligned16(A) || !aligned16(B) || !aligned4(scale) || !aligned16(plan) || !aligned16(base) ||
      !aligned16(y))
    return TL_EINVAL;
  int r;
  if ((r = check_rows(ldx, K, M, 8)) != TL_OK || (r = check_rows(ldb, N, M, 8)) != TL_OK || (r = check_rows(ldy, N, M, 8)) != TL_OK)
    return r;
  if (base == y && M > 1 && ldb != ldy) return TL_EINVAL;
  int sms = 0;
  int* status = nullptr;
  if ((r = num_sms(&sms)) != TL_OK || (r = status_ptr(&status)) != TL_OK) return r;
  tl::LoraParams p{};
  p.x = static_cast<const uint16_t*>(x), p.A = static_cast<const uint16_t*>(A), p.B = static_cast<const uint16_t*>(B);
  p.scale = scale;
  p.plan = static_cast<const tl::LoraPlanHeader*>(plan);
  p.items = reinterpret_cast<const tl::LoraItem*>(p.plan + 1);
  p.base = base, p.y = y, p.ldx = ldx, p.ldb = ldb, p.ldy = ldy;
  p.M = M, p.N = N, p.K = K, p.rank = rank, p.n_adapters = n_adapters, p.y_dtype = y_dtype;
  p.copy_bare = base != y;
  p.status = status;
  return tl::launch_lora_apply(p, dtype == TL_BF16, sms, as_stream(stream)) == cudaSuccess ? TL_OK : TL_ECUDA;
}

int tl_selftest_wait_timeout(unsigned int limit_us, void* stream) {
  if (limit_us == 0 || limit_us > 100000) return TL_EINVAL;
  int* status = nullptr;
  const int r = status_ptr(&status);
  if (r != TL_OK) return r;
  wait_selftest_kernel<<<1, 32, 0, as_stream(stream)>>>(status, 1000ull * limit_us);
  return cudaGetLastError() == cudaSuccess ? TL_OK : TL_ECUDA;
}

int tl_get_status(void* stream) {
  int* status = nullptr;
  int r = status_ptr(&status);
  if (r != TL_OK) return r;
  if (cudaStreamSynchronize(as_stream(stream)) != cudaSuccess) return TL_ECUDA;
  int v = 0;
  if (cudaMemcpy(&v, status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return TL_ECUDA;
  const int zero = 0;
  if (cudaMemcpy(status, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess)
    return TL_ECUDA;
  return v;
}

}  // extern "C"
