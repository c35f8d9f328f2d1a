// C ABI of libhpa: argument checks, task map sizing, TMA descriptor set-up
// and kernel launches.  See include/hpa.h for the contract of every call.
#include <cudaTypedefs.h>

#include <climits>
#include <cmath>
#include <cstring>
#include <mutex>

#include "hpa_internal.cuh"

namespace hpa {

namespace {
thread_local int g_last_cuda_error = 0;  // what hpa_last_cuda_error() reports, per thread
}  // namespace

int cuda_fail(cudaError_t e) {
  g_last_cuda_error = static_cast<int>(e);
  return HPA_ERR_CUDA;
}

int last_cuda_error() { return g_last_cuda_error; }

}  // namespace hpa

namespace {

using hpa::cuda_fail;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Whether [a, a + na) and [b, b + nb) share a byte (null pointers share none).
bool overlap(const void *a, uint64_t na, const void *b, uint64_t nb) {
  const uint64_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && (x < y ? y - x < na : x - y < nb);
}

constexpr int32_t kMaxB = 1 << 24;
constexpr int32_t kMaxC = 1 << 20;

int64_t taskmap_words(int64_t B, int64_t C, int64_t s_cap) {
  return hpa::TaskMapLayout::make(B, C).words(s_cap);
}

// ---- TMA descriptors for a KV pool: 3-D view (d, token-in-page, page*Hkv + head)
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

struct MapKey {
  const void *ptr;
  int64_t rows;
  int kv_dtype;
  bool operator==(const MapKey &o) const {
    return ptr == o.ptr && rows == o.rows && kv_dtype == o.kv_dtype;
  }
};

std::mutex g_map_mu;
constexpr int kMapCache = 8;
MapKey g_map_keys[kMapCache];
CUtensorMap g_maps[kMapCache];
int g_map_next = 0, g_map_used = 0;

int pool_map(const void *pool, int64_t num_pages, int Hkv, int kv_dtype, CUtensorMap *out) {
  const int64_t zdim = num_pages * Hkv;
  const MapKey key{pool, zdim, kv_dtype};
  {
    std::lock_guard<std::mutex> lk(g_map_mu);
    for (int i = 0; i < g_map_used; ++i)
      if (g_map_keys[i] == key) {
        *out = g_maps[i];
        return HPA_OK;
      }
  }
  auto fn = encode_fn();
  if (!fn) return cuda_fail(cudaErrorNotSupported);
  const int es = kv_dtype == HPA_KV_BF16 ? 2 : 1;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(hpa::HEAD_DIM),
                              static_cast<cuuint64_t>(hpa::PAGE), static_cast<cuuint64_t>(zdim)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(hpa::HEAD_DIM * es),
                                 static_cast<cuuint64_t>(hpa::HEAD_DIM * es * hpa::PAGE)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / es), static_cast<cuuint32_t>(hpa::PAGE),
                             1u};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  CUtensorMap m;
  CUresult r = fn(&m,
                  kv_dtype == HPA_KV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                          : CU_TENSOR_MAP_DATA_TYPE_UINT8,
                  3, const_cast<void *>(pool), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return HPA_ERR_INVALID;
  std::lock_guard<std::mutex> lk(g_map_mu);
  g_map_keys[g_map_next] = key;
  g_maps[g_map_next] = m;
  g_map_next = (g_map_next + 1) % kMapCache;
  if (g_map_used < kMapCache) ++g_map_used;
  *out = m;
  return HPA_OK;
}

int check_plan_args(const int32_t *seq_lens, int32_t B, int32_t tile, int64_t C,
                    const void *tm, size_t bytes, int64_t s_cap) {
  if (!seq_lens || !tm) return HPA_ERR_INVALID;
  if (B < 1 || B > kMaxB || C < 1 || C > kMaxC) return HPA_ERR_INVALID;
  if (tile < hpa::PAGE || tile % hpa::PAGE != 0) return HPA_ERR_INVALID;
  if (!aligned(tm, 16)) return HPA_ERR_ALIGN;
  if (bytes < static_cast<size_t>(taskmap_words(B, C, s_cap)) * 4) return HPA_ERR_WORKSPACE;
  return HPA_OK;
}

}  // namespace

extern "C" {

size_t hpa_taskmap_bytes(int32_t B, int32_t num_ctas) {
  if (B < 1 || B > kMaxB || num_ctas < 1 || num_ctas > kMaxC) return 0;
  return static_cast<size_t>(taskmap_words(B, num_ctas, int64_t(B) + num_ctas - 1)) * 4;
}

int32_t hpa_max_segments(int32_t B, int32_t num_ctas) {
  if (B < 1 || B > kMaxB || num_ctas < 1 || num_ctas > kMaxC) return 0;
  return B + num_ctas - 1;
}

int32_t hpa_static_num_ctas(int32_t B, int32_t splits) {
  if (B < 1 || B > kMaxB || splits < 1 || int64_t(B) * splits > kMaxC) return 0;
  return B * splits;
}

size_t hpa_static_taskmap_bytes(int32_t B, int32_t splits) {
  const int32_t C = hpa_static_num_ctas(B, splits);
  if (C == 0) return 0;
  return static_cast<size_t>(taskmap_words(B, C, C)) * 4;
}

int32_t hpa_default_num_ctas_mma(int32_t Hq, int32_t Hkv, int32_t q_len, int32_t kv_dtype) {
  if (Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || q_len < 1 ||
      (kv_dtype != HPA_KV_BF16 && kv_dtype != HPA_KV_E4M3))
    return -1;
  int dev = 0, sms = 0, per_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) {
    cuda_fail(e);
    return -1;
  }
  if (hpa::attn_ctas_per_sm(kv_dtype, q_len, &per_sm) != 0 || per_sm < 1) return -1;
  // one CTA per (partition, KV head, group of up to 16 query rows)
  const int groups = ((Hq / Hkv) * q_len + hpa::MAX_ROWS - 1) / hpa::MAX_ROWS;
  const int c = sms * per_sm / (Hkv * groups);
  return c < 1 ? 1 : c;
}

int hpa_plan(const int32_t *seq_lens_dev, int32_t B, int32_t tile, int32_t num_ctas,
             void *taskmap_dev, size_t taskmap_bytes, hpa_stream_t stream) {
  const int64_t s_cap = int64_t(B) + num_ctas - 1;
  int rc = check_plan_args(seq_lens_dev, B, tile, num_ctas, taskmap_dev, taskmap_bytes, s_cap);
  if (rc != HPA_OK) return rc;
  cudaError_t e = hpa::launch_plan(seq_lens_dev, B, tile, num_ctas, 0, 0,
                                   static_cast<int32_t *>(taskmap_dev), s_cap,
                                   reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HPA_OK : cuda_fail(e);
}

int hpa_plan_weighted(const int32_t *seq_lens_dev, int32_t B, int32_t tile, int32_t num_ctas,
                      void *taskmap_dev, size_t taskmap_bytes, hpa_stream_t stream) {
  const int64_t s_cap = int64_t(B) + num_ctas - 1;
  int rc = check_plan_args(seq_lens_dev, B, tile, num_ctas, taskmap_dev, taskmap_bytes, s_cap);
  if (rc != HPA_OK) return rc;
  if (hpa::plan_stage_bytes(B, num_ctas, 2) > hpa::kPlanStageLimit) return HPA_ERR_UNSUPPORTED;
  cudaError_t e = hpa::launch_plan(seq_lens_dev, B, tile, num_ctas, 2, 0,
                                   static_cast<int32_t *>(taskmap_dev), s_cap,
                                   reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HPA_OK : cuda_fail(e);
}

int hpa_plan_static(const int32_t *seq_lens_dev, int32_t B, int32_t tile, int32_t splits,
                    void *taskmap_dev, size_t taskmap_bytes, hpa_stream_t stream) {
  const int32_t C = hpa_static_num_ctas(B, splits);
  if (C == 0) return HPA_ERR_INVALID;
  int rc = check_plan_args(seq_lens_dev, B, tile, C, taskmap_dev, taskmap_bytes, C);
  if (rc != HPA_OK) return rc;
  cudaError_t e = hpa::launch_plan(seq_lens_dev, B, tile, C, 1, splits,
                                   static_cast<int32_t *>(taskmap_dev), C,
                                   reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HPA_OK : cuda_fail(e);
}

int hpa_plan_window(const int32_t *seq_lens_dev, int32_t B, int32_t q_len, int32_t window,
                    int32_t sinks, int32_t tile, int32_t num_ctas, void *taskmap_dev,
                    size_t taskmap_bytes, hpa_stream_t stream) {
  const int64_t s_cap = int64_t(B) + num_ctas - 1;
  if (q_len < 1 || window < 1 || sinks < 0) return HPA_ERR_INVALID;
  int rc = check_plan_args(seq_lens_dev, B, tile, num_ctas, taskmap_dev, taskmap_bytes, s_cap);
  if (rc != HPA_OK) return rc;
  cudaError_t e = hpa::launch_plan(seq_lens_dev, B, tile, num_ctas, hpa::KIND_WINDOW, 0,
                                   static_cast<int32_t *>(taskmap_dev), s_cap,
                                   reinterpret_cast<cudaStream_t>(stream),
                                   hpa::PlanWindow{window, sinks, q_len});
  return e == cudaSuccess ? HPA_OK : cuda_fail(e);
}

static int decode_attn_impl(const void *q_dev, const void *k_pool_dev, const void *v_pool_dev,
                            int32_t kv_dtype, const float *k_scale_dev,
                            const float *v_scale_dev, int64_t num_pages,
                            const int32_t *page_indptr_dev, const int32_t *page_indices_dev,
                            int32_t page_size, int32_t B, int32_t q_len, int32_t Hq, int32_t Hkv,
                            int32_t d, float sm_scale, void *taskmap_dev, int32_t num_ctas,
                            float *partial_o_dev, float *partial_lse_dev, uint64_t *trace_dev,
                            void *out_dev, float *out_lse_dev, int32_t *arrivals_dev,
                            hpa_stream_t stream, bool tc = false, bool all_heads = false,
                            bool window = false) {
  if (!q_dev || !k_pool_dev || !v_pool_dev || !page_indptr_dev || !page_indices_dev ||
      !taskmap_dev || !partial_o_dev || !partial_lse_dev)
    return HPA_ERR_INVALID;
  const bool e2m1 = kv_dtype == HPA_KV_E2M1;
  if (kv_dtype != HPA_KV_BF16 && kv_dtype != HPA_KV_E4M3 && !e2m1) return HPA_ERR_INVALID;
  if (kv_dtype != HPA_KV_BF16 && (!k_scale_dev || !v_scale_dev)) return HPA_ERR_INVALID;
  if (e2m1 && (tc || all_heads || trace_dev || out_dev)) return HPA_ERR_UNSUPPORTED;
  if (B < 1 || B > kMaxB || num_ctas < 1 || num_ctas > kMaxC || q_len < 1 || Hq < 1 ||
      Hkv < 1 || Hkv > 65535 || num_pages < 1 || !std::isfinite(sm_scale))
    return HPA_ERR_INVALID;
  if (d != hpa::HEAD_DIM || page_size != hpa::PAGE || Hq % Hkv != 0 ||
      int64_t(Hq / Hkv) * q_len > hpa::MAX_ROWS_TOTAL)
    return HPA_ERR_UNSUPPORTED;
  if (num_pages * Hkv > INT_MAX) return HPA_ERR_UNSUPPORTED;
  if (!aligned(q_dev, 16) || !aligned(k_pool_dev, 16) || !aligned(v_pool_dev, 16) ||
      !aligned(taskmap_dev, 16) || !aligned(partial_o_dev, 16) || !aligned(partial_lse_dev, 4))
    return HPA_ERR_ALIGN;
  CUtensorMap tmk, tmv;
  if (!e2m1) {  // 4-bit pages are whole blocks of memory and need no tensor map
    int rc = pool_map(k_pool_dev, num_pages, Hkv, kv_dtype, &tmk);
    if (rc == HPA_OK) rc = pool_map(v_pool_dev, num_pages, Hkv, kv_dtype, &tmv);
    if (rc != HPA_OK) return rc;
  }
  hpa::AttnParams p;
  p.q = static_cast<const __nv_bfloat16 *>(q_dev);
  p.tm = static_cast<int32_t *>(taskmap_dev);
  p.page_indptr = page_indptr_dev;
  p.page_indices = page_indices_dev;
  p.k_scale = k_scale_dev;
  p.v_scale = v_scale_dev;
  p.partial_o = partial_o_dev;
  p.partial_lse = partial_lse_dev;
  p.trace = reinterpret_cast<unsigned long long *>(trace_dev);
  p.out = static_cast<__nv_bfloat16 *>(out_dev);
  p.out_lse = out_lse_dev;
  p.arrivals = arrivals_dev;
  p.num_pages = num_pages;
  p.lay = hpa::TaskMapLayout::make(B, num_ctas);
  p.B = B;
  p.C = num_ctas;
  p.q_len = q_len;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.rows = p.G * q_len;
  const int groups = (p.rows + hpa::MAX_ROWS - 1) / hpa::MAX_ROWS;
  p.group = e2m1     ? hpa::attn_e2m1_group(p.rows)
            : window ? (p.rows + groups - 1) / groups
                     : hpa::MAX_ROWS;
  p.heads_per_cta = all_heads ? Hkv : 1;
  p.window = window;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  cudaError_t e =
      e2m1 ? hpa::launch_decode_attn_e2m1(p, k_pool_dev, v_pool_dev,
                                          reinterpret_cast<cudaStream_t>(stream))
      : tc ? hpa::launch_decode_attn_tc(p, tmk, tmv, kv_dtype,
                                        reinterpret_cast<cudaStream_t>(stream))
           : hpa::launch_decode_attn(p, tmk, tmv, kv_dtype,
                                     reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HPA_OK : cuda_fail(e);
}

int hpa_decode_attn_tc(const void *q_dev, const void *k_pool_dev, const void *v_pool_dev,
                       int32_t kv_dtype, const float *k_scale_dev, const float *v_scale_dev,
                       int64_t num_pages, const int32_t *page_indptr_dev,
                       const int32_t *page_indices_dev, int32_t page_size, int32_t B,
                       int32_t q_len, int32_t Hq, int32_t Hkv, int32_t d, float sm_scale,
                       void *taskmap_dev, int32_t num_ctas, float *partial_o_dev,
                       float *partial_lse_dev, hpa_stream_t stream) {
  return decode_attn_impl(q_dev, k_pool_dev, v_pool_dev, kv_dtype, k_scale_dev, v_scale_dev,
                          num_pages, page_indptr_dev, page_indices_dev, page_size, B, q_len, Hq,
                          Hkv, d, sm_scale, taskmap_dev, num_ctas, partial_o_dev,
                          partial_lse_dev, nullptr, nullptr, nullptr, nullptr, stream, true);
}

int32_t hpa_default_num_ctas_tc(int32_t Hq, int32_t Hkv, int32_t q_len, int32_t kv_dtype) {
  if (Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || q_len < 1 ||
      int64_t(Hq / Hkv) * q_len > hpa::MAX_ROWS_TOTAL ||
      (kv_dtype != HPA_KV_BF16 && kv_dtype != HPA_KV_E4M3))
    return -1;
  int dev = 0, sms = 0, per_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) {
    cuda_fail(e);
    return -1;
  }
  if (hpa::attn_tc_ctas_per_sm(kv_dtype, (Hq / Hkv) * q_len, &per_sm) != 0 || per_sm < 1)
    return -1;
  const int c = sms * per_sm / Hkv;
  return c < 1 ? 1 : c;
}

int hpa_decode_attn_mma(const void *q_dev, const void *k_pool_dev, const void *v_pool_dev,
                        int32_t kv_dtype, const float *k_scale_dev, const float *v_scale_dev,
                        int64_t num_pages, const int32_t *page_indptr_dev,
                        const int32_t *page_indices_dev, int32_t page_size, int32_t B,
                        int32_t q_len, int32_t Hq, int32_t Hkv, int32_t d, float sm_scale,
                        void *taskmap_dev, int32_t num_ctas, float *partial_o_dev,
                        float *partial_lse_dev, hpa_stream_t stream) {
  if (kv_dtype == HPA_KV_E2M1) return HPA_ERR_UNSUPPORTED;  // a kernel of the wider types
  return decode_attn_impl(q_dev, k_pool_dev, v_pool_dev, kv_dtype, k_scale_dev, v_scale_dev,
                          num_pages, page_indptr_dev, page_indices_dev, page_size, B, q_len, Hq,
                          Hkv, d, sm_scale, taskmap_dev, num_ctas, partial_o_dev,
                          partial_lse_dev, nullptr, nullptr, nullptr, nullptr, stream);
}

int hpa_decode_attn_window(const void *q_dev, const void *k_pool_dev, const void *v_pool_dev,
                           int32_t kv_dtype, const float *k_scale_dev, const float *v_scale_dev,
                           int64_t num_pages, const int32_t *page_indptr_dev,
                           const int32_t *page_indices_dev, int32_t page_size, int32_t B,
                           int32_t q_len, int32_t Hq, int32_t Hkv, int32_t d, float sm_scale,
                           void *taskmap_dev, int32_t num_ctas, float *partial_o_dev,
                           float *partial_lse_dev, hpa_stream_t stream) {
  return decode_attn_impl(q_dev, k_pool_dev, v_pool_dev, kv_dtype, k_scale_dev, v_scale_dev,
                          num_pages, page_indptr_dev, page_indices_dev, page_size, B, q_len, Hq,
                          Hkv, d, sm_scale, taskmap_dev, num_ctas, partial_o_dev,
                          partial_lse_dev, nullptr, nullptr, nullptr, nullptr, stream, false,
                          false, true);
}

// More than 16 query rows per KV head (MTP with several draft tokens) go to the
// tcgen05 kernel, which takes all rows in one pass over the keys.
// (4-bit pages choose by rows in their own launch.)
static bool routes_to_tc(int32_t Hq, int32_t Hkv, int32_t q_len, int32_t kv_dtype) {
  return kv_dtype != HPA_KV_E2M1 && Hkv >= 1 && Hq % Hkv == 0 &&
         int64_t(Hq / Hkv) * q_len > hpa::MAX_ROWS;
}

// Partitions per KV head that fill the device once with the kernel of 4-bit pages.
static int32_t default_num_ctas_e2m1(int32_t Hq, int32_t Hkv, int32_t q_len) {
  if (Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || q_len < 1 ||
      int64_t(Hq / Hkv) * q_len > hpa::MAX_ROWS_TOTAL)
    return -1;
  int dev = 0, sms = 0, per_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) {
    cuda_fail(e);
    return -1;
  }
  const int rows = (Hq / Hkv) * q_len, group = hpa::attn_e2m1_group(rows);
  if (hpa::attn_e2m1_ctas_per_sm(rows, &per_sm) != 0 || per_sm < 1) return -1;
  const int c = sms * per_sm / (Hkv * ((rows + group - 1) / group));
  return c < 1 ? 1 : c;
}

int32_t hpa_default_num_ctas_window(int32_t Hq, int32_t Hkv, int32_t q_len, int32_t kv_dtype) {
  if (kv_dtype == HPA_KV_E2M1) return default_num_ctas_e2m1(Hq, Hkv, q_len);
  return hpa_default_num_ctas_mma(Hq, Hkv, q_len, kv_dtype);
}

int hpa_decode_attn(const void *q_dev, const void *k_pool_dev, const void *v_pool_dev,
                    int32_t kv_dtype, const float *k_scale_dev, const float *v_scale_dev,
                    int64_t num_pages, const int32_t *page_indptr_dev,
                    const int32_t *page_indices_dev, int32_t page_size, int32_t B,
                    int32_t q_len, int32_t Hq, int32_t Hkv, int32_t d, float sm_scale,
                    void *taskmap_dev, int32_t num_ctas, float *partial_o_dev,
                    float *partial_lse_dev, hpa_stream_t stream) {
  return decode_attn_impl(q_dev, k_pool_dev, v_pool_dev, kv_dtype, k_scale_dev, v_scale_dev,
                          num_pages, page_indptr_dev, page_indices_dev, page_size, B, q_len, Hq,
                          Hkv, d, sm_scale, taskmap_dev, num_ctas, partial_o_dev,
                          partial_lse_dev, nullptr, nullptr, nullptr, nullptr, stream,
                          routes_to_tc(Hq, Hkv, q_len, kv_dtype));
}

int32_t hpa_default_num_ctas(int32_t Hq, int32_t Hkv, int32_t q_len, int32_t kv_dtype) {
  if (kv_dtype == HPA_KV_E2M1) return default_num_ctas_e2m1(Hq, Hkv, q_len);
  return routes_to_tc(Hq, Hkv, q_len, kv_dtype)
             ? hpa_default_num_ctas_tc(Hq, Hkv, q_len, kv_dtype)
             : hpa_default_num_ctas_mma(Hq, Hkv, q_len, kv_dtype);
}

int hpa_decode_attn_traced(const void *q_dev, const void *k_pool_dev, const void *v_pool_dev,
                           int32_t kv_dtype, const float *k_scale_dev, const float *v_scale_dev,
                           int64_t num_pages, const int32_t *page_indptr_dev,
                           const int32_t *page_indices_dev, int32_t page_size, int32_t B,
                           int32_t q_len, int32_t Hq, int32_t Hkv, int32_t d, float sm_scale,
                           void *taskmap_dev, int32_t num_ctas, float *partial_o_dev,
                           float *partial_lse_dev, uint64_t *trace_dev, hpa_stream_t stream) {
  if (!trace_dev) return HPA_ERR_INVALID;
  if (!aligned(trace_dev, 8)) return HPA_ERR_ALIGN;
  return decode_attn_impl(q_dev, k_pool_dev, v_pool_dev, kv_dtype, k_scale_dev, v_scale_dev,
                          num_pages, page_indptr_dev, page_indices_dev, page_size, B, q_len, Hq,
                          Hkv, d, sm_scale, taskmap_dev, num_ctas, partial_o_dev,
                          partial_lse_dev, trace_dev, nullptr, nullptr, nullptr, stream,
                          routes_to_tc(Hq, Hkv, q_len, kv_dtype));
}

int hpa_decode_attn_allheads(const void *q_dev, const void *k_pool_dev, const void *v_pool_dev,
                             int32_t kv_dtype, const float *k_scale_dev,
                             const float *v_scale_dev, int64_t num_pages,
                             const int32_t *page_indptr_dev, const int32_t *page_indices_dev,
                             int32_t page_size, int32_t B, int32_t q_len, int32_t Hq,
                             int32_t Hkv, int32_t d, float sm_scale, void *taskmap_dev,
                             int32_t num_ctas, float *partial_o_dev, float *partial_lse_dev,
                             uint64_t *trace_dev, hpa_stream_t stream) {
  if (trace_dev && !aligned(trace_dev, 8)) return HPA_ERR_ALIGN;
  return decode_attn_impl(q_dev, k_pool_dev, v_pool_dev, kv_dtype, k_scale_dev, v_scale_dev,
                          num_pages, page_indptr_dev, page_indices_dev, page_size, B, q_len, Hq,
                          Hkv, d, sm_scale, taskmap_dev, num_ctas, partial_o_dev,
                          partial_lse_dev, trace_dev, nullptr, nullptr, nullptr, stream, false,
                          true);
}

int32_t hpa_default_num_ctas_allheads(int32_t Hq, int32_t Hkv, int32_t q_len, int32_t kv_dtype) {
  const int32_t per_head = hpa_default_num_ctas_mma(Hq, Hkv, q_len, kv_dtype);
  if (per_head <= 0) return per_head;
  int dev = 0, sms = 0, per_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) {
    cuda_fail(e);
    return -1;
  }
  if (hpa::attn_ctas_per_sm(kv_dtype, q_len, &per_sm) != 0 || per_sm < 1) return -1;
  // one CTA per (partition, group of up to 16 query rows), each walking every KV head
  const int groups = ((Hq / Hkv) * q_len + hpa::MAX_ROWS - 1) / hpa::MAX_ROWS;
  const int c = sms * per_sm / groups;
  return c < 1 ? 1 : c;
}

size_t hpa_arrivals_elems(int32_t B, int32_t Hq, int32_t Hkv, int32_t q_len) {
  if (B < 1 || B > kMaxB || Hkv < 1 || Hkv > 65535 || Hq < Hkv || Hq % Hkv || q_len < 1)
    return 0;
  const int64_t groups = (int64_t(Hq / Hkv) * q_len + hpa::MAX_ROWS - 1) / hpa::MAX_ROWS;
  return static_cast<size_t>(B) * Hkv * groups;
}

int hpa_decode_attn_fused(const void *q_dev, const void *k_pool_dev, const void *v_pool_dev,
                          int32_t kv_dtype, const float *k_scale_dev, const float *v_scale_dev,
                          int64_t num_pages, const int32_t *page_indptr_dev,
                          const int32_t *page_indices_dev, int32_t page_size, int32_t B,
                          int32_t q_len, int32_t Hq, int32_t Hkv, int32_t d, float sm_scale,
                          void *taskmap_dev, int32_t num_ctas, float *partial_o_dev,
                          float *partial_lse_dev, void *out_dev, float *out_lse_dev,
                          int32_t *arrivals_dev, hpa_stream_t stream) {
  if (!out_dev || !arrivals_dev) return HPA_ERR_INVALID;
  if (!aligned(out_dev, 8) || !aligned(arrivals_dev, 4)) return HPA_ERR_ALIGN;
  return decode_attn_impl(q_dev, k_pool_dev, v_pool_dev, kv_dtype, k_scale_dev, v_scale_dev,
                          num_pages, page_indptr_dev, page_indices_dev, page_size, B, q_len, Hq,
                          Hkv, d, sm_scale, taskmap_dev, num_ctas, partial_o_dev,
                          partial_lse_dev, nullptr, out_dev, out_lse_dev, arrivals_dev, stream);
}

int hpa_combine(const float *partial_o_dev, const float *partial_lse_dev, void *taskmap_dev,
                int32_t B, int32_t num_ctas, int32_t q_len, int32_t Hq, int32_t d,
                void *out_dev, float *out_lse_dev, hpa_stream_t stream) {
  if (!partial_o_dev || !partial_lse_dev || !taskmap_dev || !out_dev) return HPA_ERR_INVALID;
  if (B < 1 || B > kMaxB || num_ctas < 1 || num_ctas > kMaxC || q_len < 1 || Hq < 1)
    return HPA_ERR_INVALID;
  if (d != hpa::HEAD_DIM) return HPA_ERR_UNSUPPORTED;
  if (int64_t(B) * q_len * Hq > INT_MAX) return HPA_ERR_UNSUPPORTED;  // one block per row
  if (!aligned(partial_o_dev, 16) || !aligned(out_dev, 8) || !aligned(taskmap_dev, 16))
    return HPA_ERR_ALIGN;
  cudaError_t e = hpa::launch_combine(partial_o_dev, partial_lse_dev,
                                      static_cast<int32_t *>(taskmap_dev), B, num_ctas, q_len,
                                      Hq, static_cast<__nv_bfloat16 *>(out_dev), out_lse_dev,
                                      reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HPA_OK : cuda_fail(e);
}

int hpa_selftest_wait_timeout(int32_t *status_dev, int64_t limit_ns, hpa_stream_t stream) {
  if (!status_dev) return HPA_ERR_INVALID;
  if (limit_ns < 1000 || limit_ns > 5000000000ll) return HPA_ERR_INVALID;
  if (!aligned(status_dev, 4)) return HPA_ERR_ALIGN;
  cudaError_t e = hpa::launch_selftest_wait(status_dev, limit_ns,
                                            reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HPA_OK : cuda_fail(e);
}

static int store_kv_impl(const void *k_new_dev, const void *v_new_dev,
                         const int32_t *seq_lens_dev, const int32_t *page_indptr_dev,
                         const int32_t *page_indices_dev, int64_t num_pages, int32_t page_size,
                         const float *cos_sin_dev, int32_t max_pos, const float *norm_w_dev,
                         float eps, int32_t use_hadamard, int32_t kv_dtype,
                         const float *k_scale_dev, const float *v_scale_dev, void *k_pool_dev,
                         void *v_pool_dev, int32_t B, int32_t q_len, int32_t Hkv, int32_t d,
                         int32_t *status_dev, const int32_t *text_pos_dev,
                         hpa_stream_t stream) {
  if (!k_new_dev || !v_new_dev || !seq_lens_dev || !page_indptr_dev || !page_indices_dev ||
      !cos_sin_dev || !norm_w_dev || !k_pool_dev || !v_pool_dev)
    return HPA_ERR_INVALID;
  if (kv_dtype != HPA_KV_BF16 && kv_dtype != HPA_KV_E4M3) return HPA_ERR_INVALID;
  if (kv_dtype == HPA_KV_E4M3 && (!k_scale_dev || !v_scale_dev)) return HPA_ERR_INVALID;
  if (B < 1 || B > kMaxB || q_len < 1 || Hkv < 1 || Hkv > 65535 || num_pages < 1 ||
      max_pos < 1 || !(eps >= 0.f) || !std::isfinite(eps))
    return HPA_ERR_INVALID;
  if (d != hpa::HEAD_DIM || page_size != hpa::PAGE) return HPA_ERR_UNSUPPORTED;
  if (int64_t(B) * q_len * Hkv > (int64_t(1) << 34)) return HPA_ERR_UNSUPPORTED;
  if (!aligned(k_new_dev, 16) || !aligned(v_new_dev, 16) || !aligned(cos_sin_dev, 16) ||
      !aligned(norm_w_dev, 16) || !aligned(k_pool_dev, 16) || !aligned(v_pool_dev, 16) ||
      (status_dev && !aligned(status_dev, 4)))
    return HPA_ERR_ALIGN;
  hpa::StoreKvParams p;
  p.k_new = static_cast<const __nv_bfloat16 *>(k_new_dev);
  p.v_new = static_cast<const __nv_bfloat16 *>(v_new_dev);
  p.seq_lens = seq_lens_dev;
  p.page_indptr = page_indptr_dev;
  p.page_indices = page_indices_dev;
  p.num_pages = num_pages;
  p.cos_sin = cos_sin_dev;
  p.max_pos = max_pos;
  p.norm_w = norm_w_dev;
  p.eps = eps;
  p.use_hadamard = use_hadamard != 0;
  p.kv_dtype = kv_dtype;
  p.k_scale = k_scale_dev;
  p.v_scale = v_scale_dev;
  p.k_pool = k_pool_dev;
  p.v_pool = v_pool_dev;
  p.B = B;
  p.q_len = q_len;
  p.Hkv = Hkv;
  p.status = status_dev;
  p.text_pos = text_pos_dev;
  cudaError_t e = hpa::launch_store_kv(p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HPA_OK : cuda_fail(e);
}

int hpa_store_kv(const void *k_new_dev, const void *v_new_dev, const int32_t *seq_lens_dev,
                 const int32_t *page_indptr_dev, const int32_t *page_indices_dev,
                 int64_t num_pages, int32_t page_size, const float *cos_sin_dev, int32_t max_pos,
                 const float *norm_w_dev, float eps, int32_t use_hadamard, int32_t kv_dtype,
                 const float *k_scale_dev, const float *v_scale_dev, void *k_pool_dev,
                 void *v_pool_dev, int32_t B, int32_t q_len, int32_t Hkv, int32_t d,
                 int32_t *status_dev, hpa_stream_t stream) {
  return store_kv_impl(k_new_dev, v_new_dev, seq_lens_dev, page_indptr_dev, page_indices_dev,
                       num_pages, page_size, cos_sin_dev, max_pos, norm_w_dev, eps, use_hadamard,
                       kv_dtype, k_scale_dev, v_scale_dev, k_pool_dev, v_pool_dev, B, q_len, Hkv, d,
                       status_dev, nullptr, stream);
}

int hpa_store_kv_at(const void *k_new_dev, const void *v_new_dev, const int32_t *seq_lens_dev,
                    const int32_t *text_pos_dev, const int32_t *page_indptr_dev,
                    const int32_t *page_indices_dev, int64_t num_pages, int32_t page_size,
                    const float *cos_sin_dev, int32_t max_pos, const float *norm_w_dev, float eps,
                    int32_t use_hadamard, int32_t kv_dtype, const float *k_scale_dev,
                    const float *v_scale_dev, void *k_pool_dev, void *v_pool_dev, int32_t B,
                    int32_t q_len, int32_t Hkv, int32_t d, int32_t *status_dev,
                    hpa_stream_t stream) {
  if (!text_pos_dev) return HPA_ERR_INVALID;
  return store_kv_impl(k_new_dev, v_new_dev, seq_lens_dev, page_indptr_dev, page_indices_dev,
                       num_pages, page_size, cos_sin_dev, max_pos, norm_w_dev, eps, use_hadamard,
                       kv_dtype, k_scale_dev, v_scale_dev, k_pool_dev, v_pool_dev, B, q_len, Hkv, d,
                       status_dev, text_pos_dev, stream);
}

int hpa_store_qkv(const void *q_dev, int64_t q_stride, const void *k_dev, int64_t k_stride,
                  const void *v_dev, int64_t v_stride, int32_t num_tokens, int32_t Hq, int32_t Hkv,
                  int32_t d, const int32_t *positions_dev, const int64_t *slots_dev,
                  const float *cos_sin_dev, int32_t max_pos, int32_t rot_dim,
                  const float *q_norm_dev, const float *k_norm_dev, float eps, int32_t flags,
                  void *q_out_dev, int64_t q_out_stride, int32_t kv_dtype,
                  const float *k_scale_dev, const float *v_scale_dev, void *k_pool_dev,
                  void *v_pool_dev, int64_t num_pages, int32_t page_size, int32_t *status_dev,
                  hpa_stream_t stream) {
  constexpr int32_t kFlags = HPA_QKV_NORM_AFTER | HPA_QKV_INTERLEAVED | HPA_QKV_HADAMARD;
  const bool has_q = q_dev != nullptr, has_kv = k_dev != nullptr;
  if ((k_dev == nullptr) != (v_dev == nullptr) || (!has_q && !has_kv)) return HPA_ERR_INVALID;
  if (!positions_dev || !slots_dev || (rot_dim != 0 && !cos_sin_dev) || (has_q && !q_out_dev) ||
      (has_kv && (!k_pool_dev || !v_pool_dev)))
    return HPA_ERR_INVALID;
  if (kv_dtype != HPA_KV_BF16 && kv_dtype != HPA_KV_E4M3 && kv_dtype != HPA_KV_E2M1)
    return HPA_ERR_INVALID;
  if (has_kv && kv_dtype != HPA_KV_BF16 && (!k_scale_dev || !v_scale_dev)) return HPA_ERR_INVALID;
  if (num_tokens < 0 || (has_q && Hq < 1) || (has_kv && Hkv < 1) || Hq > 65535 || Hkv > 65535 ||
      num_pages < 1 || (rot_dim != 0 && max_pos < 1) || !(eps >= 0.f) || !std::isfinite(eps) ||
      (flags & ~kFlags) != 0)
    return HPA_ERR_INVALID;
  if (d != hpa::HEAD_DIM || page_size != hpa::PAGE || num_pages * 64 > (int64_t(1) << 40) ||
      (rot_dim != 0 && rot_dim != 16 && rot_dim != 32 && rot_dim != 64 && rot_dim != 128))
    return HPA_ERR_UNSUPPORTED;
  if (has_kv && num_pages > INT_MAX / Hkv) return HPA_ERR_UNSUPPORTED;
  if (num_pages > INT_MAX) return HPA_ERR_UNSUPPORTED;
  // tokens apart by at least their heads, rows on 16-byte boundaries
  if ((has_q && (q_stride < int64_t(Hq) * d || q_out_stride < int64_t(Hq) * d)) ||
      (has_kv && (k_stride < int64_t(Hkv) * d || v_stride < int64_t(Hkv) * d)))
    return HPA_ERR_INVALID;
  if ((has_q && (q_stride % 8 || q_out_stride % 8 || !aligned(q_dev, 16) ||
                 !aligned(q_out_dev, 16))) ||
      (has_kv && (k_stride % 8 || v_stride % 8 || !aligned(k_dev, 16) || !aligned(v_dev, 16) ||
                  !aligned(k_pool_dev, 16) || !aligned(v_pool_dev, 16))) ||
      !aligned(positions_dev, 4) || !aligned(slots_dev, 8) || !aligned(cos_sin_dev, 16) ||
      !aligned(q_norm_dev, 4) || !aligned(k_norm_dev, 4) || !aligned(k_scale_dev, 4) ||
      !aligned(v_scale_dev, 4) || !aligned(status_dev, 4))
    return HPA_ERR_ALIGN;
  if (num_tokens == 0) return HPA_OK;
  // what the call writes lies apart from what it reads, but for queries in place
  const auto span = [&](int64_t stride, int32_t heads) {  // from the first row to the last's end
    return 2ull * (stride * (num_tokens - 1) + int64_t(heads) * d);
  };
  const uint64_t q_out_bytes = has_q ? span(q_out_stride, Hq) : 0;
  if (has_q && (q_dev != q_out_dev || (q_stride != q_out_stride && num_tokens > 1)) &&
      overlap(q_dev, span(q_stride, Hq), q_out_dev, q_out_bytes))
    return HPA_ERR_INVALID;
  const auto meets_q_out = [&](const void *x, int64_t stride) {  // keys or values
    if (!overlap(x, span(stride, Hkv), q_out_dev, q_out_bytes)) return false;
    if (num_tokens == 1 || stride != q_out_stride) return true;
    const int64_t apart = (static_cast<const char *>(x) - static_cast<char *>(q_out_dev)) / 2;
    const int64_t column = (apart % stride + stride) % stride;  // in a token's packed row
    return column < int64_t(Hq) * d || column + int64_t(Hkv) * d > stride;
  };
  if (has_q && has_kv && (meets_q_out(k_dev, k_stride) || meets_q_out(v_dev, v_stride)))
    return HPA_ERR_INVALID;
  if (has_kv) {
    const uint64_t unit = kv_dtype == HPA_KV_E2M1   ? hpa::E2M1_UNIT
                          : kv_dtype == HPA_KV_E4M3 ? hpa::PAGE * hpa::HEAD_DIM
                                                    : hpa::PAGE * hpa::HEAD_DIM * 2;
    const uint64_t bytes = unit * num_pages * Hkv;
    if (overlap(k_pool_dev, bytes, v_pool_dev, bytes)) return HPA_ERR_INVALID;
    for (const void *pool : {k_pool_dev, v_pool_dev})
      if (overlap(pool, bytes, k_dev, span(k_stride, Hkv)) ||
          overlap(pool, bytes, v_dev, span(v_stride, Hkv)) ||
          (has_q && (overlap(pool, bytes, q_dev, span(q_stride, Hq)) ||
                     overlap(pool, bytes, q_out_dev, q_out_bytes))))
        return HPA_ERR_INVALID;
  }
  hpa::StoreQkvParams p;
  p.q = static_cast<const __nv_bfloat16 *>(q_dev);
  p.k = static_cast<const __nv_bfloat16 *>(k_dev);
  p.v = static_cast<const __nv_bfloat16 *>(v_dev);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out_stride = q_out_stride;
  p.num_tokens = num_tokens;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.positions = positions_dev;
  p.slots = slots_dev;
  p.cos_sin = cos_sin_dev;
  p.max_pos = max_pos;
  p.rot_dim = rot_dim;
  p.q_norm = q_norm_dev;
  p.k_norm = k_norm_dev;
  p.eps = eps;
  p.norm_after = (flags & HPA_QKV_NORM_AFTER) != 0;
  p.interleaved = (flags & HPA_QKV_INTERLEAVED) != 0;
  p.use_hadamard = (flags & HPA_QKV_HADAMARD) != 0;
  p.q_out = static_cast<__nv_bfloat16 *>(q_out_dev);
  p.kv_dtype = kv_dtype;
  p.k_scale = k_scale_dev;
  p.v_scale = v_scale_dev;
  p.k_pool = k_pool_dev;
  p.v_pool = v_pool_dev;
  p.num_pages = num_pages;
  p.status = status_dev;
  cudaError_t e = hpa::launch_store_qkv(p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HPA_OK : cuda_fail(e);
}

size_t hpa_assign_pages_workspace(int32_t B, int32_t num_rows) {
  if (B < 1 || B > kMaxB || num_rows < 1) return 0;
  return static_cast<size_t>(hpa::assign_workspace_words(B, num_rows)) * 4;
}

int hpa_assign_pages(const int32_t *seq_lens_dev, const int32_t *new_tokens_dev,
                     const int32_t *rows_dev, const int32_t *pos_offset_dev, int32_t B,
                     int32_t num_rows, int32_t *table_dev, int32_t table_stride,
                     const int32_t *held_in_dev, int32_t *held_out_dev, int32_t *free_pages_dev,
                     const int32_t *free_count_in_dev, int32_t *free_count_out_dev,
                     int32_t num_pages, int32_t page_size, int32_t *page_indptr_dev,
                     int32_t *page_indices_dev, int32_t indices_cap, int64_t *slots_dev,
                     int32_t *positions_dev, int32_t max_tokens, void *workspace_dev,
                     size_t workspace_bytes, int32_t *status_dev, hpa_stream_t stream) {
  if (!seq_lens_dev || !table_dev || !held_in_dev || !held_out_dev || !free_pages_dev ||
      !free_count_in_dev || !free_count_out_dev || !page_indptr_dev || !page_indices_dev ||
      !workspace_dev)
    return HPA_ERR_INVALID;
  if (new_tokens_dev && (!slots_dev || !positions_dev)) return HPA_ERR_INVALID;
  if (B < 1 || B > kMaxB || num_rows < 1 || table_stride < 1 || num_pages < 1 || indices_cap < 0 ||
      (new_tokens_dev && max_tokens < 0))
    return HPA_ERR_INVALID;
  if (!rows_dev && B > num_rows) return HPA_ERR_INVALID;
  if (page_size != hpa::PAGE) return HPA_ERR_UNSUPPORTED;
  if (!aligned(workspace_dev, 16) || !aligned(slots_dev, 8)) return HPA_ERR_ALIGN;
  const int32_t *const words[] = {
      seq_lens_dev,      new_tokens_dev,     rows_dev,        pos_offset_dev,   table_dev,
      held_in_dev,       held_out_dev,       free_pages_dev,  page_indices_dev, page_indptr_dev,
      free_count_in_dev, free_count_out_dev, positions_dev,   status_dev};
  for (const int32_t *p : words)
    if (!aligned(p, 4)) return HPA_ERR_ALIGN;
  if (workspace_bytes < hpa_assign_pages_workspace(B, num_rows)) return HPA_ERR_WORKSPACE;
  // the arrays that the call writes lie apart from each other and from what it reads; the state
  // may be updated in place
  struct Range {
    const void *p;
    uint64_t bytes;
  };
  const uint64_t b4 = 4ull * B;
  const Range written[] = {{table_dev, 4ull * num_rows * table_stride},
                           {free_pages_dev, 4ull * num_pages},
                           {page_indptr_dev, b4 + 4},
                           {page_indices_dev, 4ull * indices_cap},
                           {new_tokens_dev ? slots_dev : nullptr, 8ull * max_tokens},
                           {new_tokens_dev ? positions_dev : nullptr, 4ull * max_tokens},
                           {held_out_dev, 4ull * num_rows},
                           {free_count_out_dev, 4},
                           {workspace_dev, workspace_bytes}};
  const Range read[] = {{seq_lens_dev, b4}, {new_tokens_dev, b4}, {rows_dev, b4},
                        {pos_offset_dev, b4}};
  constexpr int kWritten = sizeof(written) / sizeof(written[0]);
  for (int i = 0; i < kWritten; ++i) {
    for (const Range &r : read)
      if (overlap(written[i].p, written[i].bytes, r.p, r.bytes)) return HPA_ERR_INVALID;
    for (int j = 0; j < i; ++j)
      if (overlap(written[i].p, written[i].bytes, written[j].p, written[j].bytes))
        return HPA_ERR_INVALID;
    if (held_in_dev != held_out_dev || written[i].p != held_out_dev)
      if (overlap(written[i].p, written[i].bytes, held_in_dev, 4ull * num_rows))
        return HPA_ERR_INVALID;
    if (free_count_in_dev != free_count_out_dev || written[i].p != free_count_out_dev)
      if (overlap(written[i].p, written[i].bytes, free_count_in_dev, 4)) return HPA_ERR_INVALID;
  }
  hpa::AssignParams p;
  p.seq_lens = seq_lens_dev;
  p.new_tokens = new_tokens_dev;
  p.rows = rows_dev;
  p.pos_offset = pos_offset_dev;
  p.B = B;
  p.num_rows = num_rows;
  p.table = table_dev;
  p.stride = table_stride;
  p.held_in = held_in_dev;
  p.held_out = held_out_dev;
  p.free_pages = free_pages_dev;
  p.free_in = free_count_in_dev;
  p.free_out = free_count_out_dev;
  p.num_pages = num_pages;
  p.page_indptr = page_indptr_dev;
  p.page_indices = page_indices_dev;
  p.indices_cap = indices_cap;
  p.slots = slots_dev;
  p.positions = positions_dev;
  p.max_tokens = new_tokens_dev ? max_tokens : 0;
  p.ws = static_cast<int32_t *>(workspace_dev);
  p.status = status_dev;
  cudaError_t e = hpa::launch_assign_pages(p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HPA_OK : cuda_fail(e);
}

int hpa_key_weights(const void *q_dev, const float *lse_dev, const void *k_pool_dev,
                    int32_t kv_dtype, const float *k_scale_dev, int64_t num_pages,
                    const int32_t *page_indptr_dev, const int32_t *page_indices_dev,
                    int32_t page_size, int32_t B, int32_t q_len, int32_t Hq, int32_t Hkv,
                    int32_t d, float sm_scale, float decay, void *taskmap_dev, int32_t num_ctas,
                    const float *acc_in_dev, float *acc_out_dev, hpa_stream_t stream) {
  if (!q_dev || !lse_dev || !k_pool_dev || !page_indptr_dev || !page_indices_dev ||
      !taskmap_dev || !acc_out_dev)
    return HPA_ERR_INVALID;
  if (kv_dtype != HPA_KV_BF16 && kv_dtype != HPA_KV_E4M3) return HPA_ERR_INVALID;
  if (kv_dtype == HPA_KV_E4M3 && !k_scale_dev) return HPA_ERR_INVALID;
  if (B < 1 || B > kMaxB || num_ctas < 1 || num_ctas > kMaxC || q_len < 1 || Hq < 1 ||
      Hkv < 1 || Hkv > 65535 || num_pages < 1 || !std::isfinite(sm_scale) ||
      !std::isfinite(decay) || decay < 0.f)
    return HPA_ERR_INVALID;
  if (d != hpa::HEAD_DIM || page_size != hpa::PAGE || Hq % Hkv != 0 ||
      int64_t(Hq / Hkv) * q_len > hpa::MAX_ROWS_TOTAL)
    return HPA_ERR_UNSUPPORTED;
  if (num_pages * Hkv > INT_MAX) return HPA_ERR_UNSUPPORTED;
  if (!aligned(q_dev, 16) || !aligned(k_pool_dev, 16) || !aligned(taskmap_dev, 16) ||
      !aligned(acc_in_dev, 16) || !aligned(acc_out_dev, 16) || !aligned(lse_dev, 4) ||
      !aligned(k_scale_dev, 4) || !aligned(page_indptr_dev, 4) || !aligned(page_indices_dev, 4))
    return HPA_ERR_ALIGN;
  const uint64_t acc_bytes = static_cast<uint64_t>(num_pages) * Hkv * hpa::PAGE * 4;
  if (acc_in_dev != acc_out_dev && overlap(acc_in_dev, acc_bytes, acc_out_dev, acc_bytes))
    return HPA_ERR_INVALID;
  CUtensorMap tmk;
  const int rc = pool_map(k_pool_dev, num_pages, Hkv, kv_dtype, &tmk);
  if (rc != HPA_OK) return rc;
  hpa::KeyWeightsParams p;
  p.q = static_cast<const __nv_bfloat16 *>(q_dev);
  p.lse = lse_dev;
  p.tm = static_cast<int32_t *>(taskmap_dev);
  p.page_indptr = page_indptr_dev;
  p.page_indices = page_indices_dev;
  p.k_scale = k_scale_dev;
  p.acc_in = decay == 0.f ? nullptr : acc_in_dev;  // nothing of it would be left
  p.acc_out = acc_out_dev;
  p.num_pages = num_pages;
  p.lay = hpa::TaskMapLayout::make(B, num_ctas);
  p.B = B;
  p.C = num_ctas;
  p.q_len = q_len;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.rows = p.G * q_len;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  p.decay = decay;
  cudaError_t e =
      hpa::launch_key_weights(p, tmk, kv_dtype, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HPA_OK : cuda_fail(e);
}

static int evict_params(const float *acc_dev, const int32_t *seq_lens_dev,
                        const int32_t *page_indptr_dev, const int32_t *page_indices_dev,
                        int64_t num_pages, int32_t page_size, const int32_t *budgets_dev,
                        int32_t sinks, int32_t recent, int32_t B, int32_t Hkv, int32_t *kept_dev,
                        int64_t kept_stride, int32_t *new_lens_dev, int32_t *status_dev,
                        hpa::EvictParams *p) {
  if (!acc_dev || !seq_lens_dev || !page_indptr_dev || !page_indices_dev || !budgets_dev ||
      !kept_dev || !new_lens_dev)
    return HPA_ERR_INVALID;
  if (B < 1 || B > kMaxB || Hkv < 1 || Hkv > 65535 || num_pages < 1 || sinks < 0 ||
      recent < 0 || kept_stride < 1)
    return HPA_ERR_INVALID;
  if (page_size != hpa::PAGE || int64_t(B) * Hkv > INT_MAX) return HPA_ERR_UNSUPPORTED;
  if (!aligned(acc_dev, 16) || !aligned(kept_dev, 4) || !aligned(new_lens_dev, 4) ||
      !aligned(seq_lens_dev, 4) || !aligned(budgets_dev, 4) || !aligned(page_indptr_dev, 4) ||
      !aligned(page_indices_dev, 4) || (status_dev && !aligned(status_dev, 4)))
    return HPA_ERR_ALIGN;
  // the blocks of a request's other heads may still read what the first one writes
  const uint64_t lens_bytes = static_cast<uint64_t>(B) * 4;
  if (overlap(new_lens_dev, lens_bytes, seq_lens_dev, lens_bytes) ||
      overlap(new_lens_dev, lens_bytes, budgets_dev, lens_bytes))
    return HPA_ERR_INVALID;
  *p = hpa::EvictParams{acc_dev,   seq_lens_dev, page_indptr_dev, page_indices_dev,
                        budgets_dev, num_pages,  sinks,           recent,
                        B,         Hkv,          kept_dev,        kept_stride,
                        new_lens_dev, status_dev,    nullptr,         nullptr};
  return HPA_OK;
}

static int compact_params(void *k_pool_dev, void *v_pool_dev, int32_t kv_dtype, float *acc_dev,
                          int64_t num_pages, const int32_t *page_indptr_dev,
                          const int32_t *page_indices_dev, const int32_t *dst_indptr_dev,
                          const int32_t *dst_indices_dev, int32_t page_size,
                          const int32_t *kept_dev, int64_t kept_stride,
                          const int32_t *new_lens_dev, int32_t B, int32_t Hkv, int32_t d,
                          int32_t *status_dev, hpa::CompactParams *p) {
  if (!k_pool_dev || !v_pool_dev || !page_indptr_dev || !page_indices_dev || !kept_dev ||
      !new_lens_dev || !dst_indptr_dev != !dst_indices_dev)
    return HPA_ERR_INVALID;
  if (kv_dtype != HPA_KV_BF16 && kv_dtype != HPA_KV_E4M3) return HPA_ERR_INVALID;
  if (B < 1 || B > kMaxB || Hkv < 1 || Hkv > 65535 || num_pages < 1 || kept_stride < 1)
    return HPA_ERR_INVALID;
  if (d != hpa::HEAD_DIM || page_size != hpa::PAGE || int64_t(B) * Hkv > INT_MAX)
    return HPA_ERR_UNSUPPORTED;
  if (!aligned(k_pool_dev, 16) || !aligned(v_pool_dev, 16) || !aligned(acc_dev, 4) ||
      !aligned(kept_dev, 4) || !aligned(new_lens_dev, 4) || !aligned(page_indptr_dev, 4) ||
      !aligned(page_indices_dev, 4) || !aligned(dst_indptr_dev, 4) ||
      !aligned(dst_indices_dev, 4) || (status_dev && !aligned(status_dev, 4)))
    return HPA_ERR_ALIGN;
  const int row_bytes = d * (kv_dtype == HPA_KV_BF16 ? 2 : 1);
  const uint64_t bytes = static_cast<uint64_t>(num_pages) * Hkv * hpa::PAGE * row_bytes;
  if (overlap(k_pool_dev, bytes, v_pool_dev, bytes)) return HPA_ERR_INVALID;
  if (dst_indptr_dev == page_indptr_dev && dst_indices_dev == page_indices_dev)
    dst_indptr_dev = dst_indices_dev = nullptr;  // the request's own pages: in place
  *p = hpa::CompactParams{k_pool_dev,     v_pool_dev,      acc_dev,   page_indptr_dev,
                          page_indices_dev, dst_indptr_dev, dst_indices_dev, num_pages,
                          kept_dev,       new_lens_dev,    kept_stride, B,
                          Hkv,            row_bytes,       status_dev};
  return HPA_OK;
}

int hpa_evict_select(const float *acc_dev, const int32_t *seq_lens_dev,
                     const int32_t *page_indptr_dev, const int32_t *page_indices_dev,
                     int64_t num_pages, int32_t page_size, const int32_t *budgets_dev,
                     int32_t sinks, int32_t recent, int32_t B, int32_t Hkv, int32_t *kept_dev,
                     int64_t kept_stride, int32_t *new_lens_dev, int32_t *status_dev,
                     hpa_stream_t stream) {
  hpa::EvictParams p;
  const int rc = evict_params(acc_dev, seq_lens_dev, page_indptr_dev, page_indices_dev, num_pages,
                              page_size, budgets_dev, sinks, recent, B, Hkv, kept_dev, kept_stride,
                              new_lens_dev, status_dev, &p);
  if (rc != HPA_OK) return rc;
  cudaError_t e = hpa::launch_evict_select(p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HPA_OK : cuda_fail(e);
}

int hpa_evict_compact(void *k_pool_dev, void *v_pool_dev, int32_t kv_dtype, float *acc_dev,
                      int64_t num_pages, const int32_t *page_indptr_dev,
                      const int32_t *page_indices_dev, const int32_t *dst_indptr_dev,
                      const int32_t *dst_indices_dev, int32_t page_size, const int32_t *kept_dev,
                      int64_t kept_stride, const int32_t *new_lens_dev, int32_t B, int32_t Hkv,
                      int32_t d, int32_t *status_dev, hpa_stream_t stream) {
  hpa::CompactParams p;
  const int rc = compact_params(k_pool_dev, v_pool_dev, kv_dtype, acc_dev, num_pages,
                                page_indptr_dev, page_indices_dev, dst_indptr_dev,
                                dst_indices_dev, page_size, kept_dev, kept_stride, new_lens_dev, B,
                                Hkv, d, status_dev, &p);
  if (rc != HPA_OK) return rc;
  cudaError_t e = hpa::launch_evict_compact(p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HPA_OK : cuda_fail(e);
}

int hpa_evict(void *k_pool_dev, void *v_pool_dev, int32_t kv_dtype, float *acc_dev,
              int64_t num_pages, const int32_t *seq_lens_dev, const int32_t *page_indptr_dev,
              const int32_t *page_indices_dev, const int32_t *dst_indptr_dev,
              const int32_t *dst_indices_dev, int32_t page_size, const int32_t *budgets_dev,
              int32_t sinks, int32_t recent, int32_t B, int32_t Hkv, int32_t d, int32_t *kept_dev,
              int64_t kept_stride, int32_t *new_lens_dev, int32_t *status_dev,
              hpa_stream_t stream) {
  hpa::EvictParams p;
  hpa::CompactParams mv;
  int rc = evict_params(acc_dev, seq_lens_dev, page_indptr_dev, page_indices_dev, num_pages,
                        page_size, budgets_dev, sinks, recent, B, Hkv, kept_dev, kept_stride,
                        new_lens_dev, status_dev, &p);
  if (rc == HPA_OK)
    rc = compact_params(k_pool_dev, v_pool_dev, kv_dtype, acc_dev, num_pages, page_indptr_dev,
                        page_indices_dev, dst_indptr_dev, dst_indices_dev, page_size, kept_dev,
                        kept_stride, new_lens_dev, B, Hkv, d, status_dev, &mv);
  if (rc != HPA_OK) return rc;
  p.dst_indptr = mv.dst_indptr;
  p.dst_indices = mv.dst_indices;
  cudaError_t e = hpa::launch_evict_select(p, reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaSuccess)
    e = hpa::launch_evict_compact(mv, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HPA_OK : cuda_fail(e);
}

const char *hpa_error_string(int code) {
  switch (code) {
    case HPA_OK: return "ok";
    case HPA_ERR_INVALID: return "invalid argument";
    case HPA_ERR_UNSUPPORTED: return "unsupported shape";
    case HPA_ERR_WORKSPACE: return "task map buffer too small";
    case HPA_ERR_ALIGN: return "misaligned pointer";
    case HPA_ERR_CUDA: return "CUDA runtime error";
    case HPA_ERR_NOALLOC_CAPACITY: return "problem exceeds the fixed no-alloc scratch array";
    default: return "unknown error";
  }
}

int hpa_last_cuda_error(void) { return hpa::last_cuda_error(); }

}  // extern "C"
