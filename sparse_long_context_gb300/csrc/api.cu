// C ABI of libsls: host-side validation, then launch.  Nothing here touches
// device memory or synchronises; a failed check returns before any launch.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "launch.h"
#include "sls.h"

namespace {

thread_local char g_err[512] = "";
std::atomic<unsigned long long> g_stats[sls::kStatCount];

sls_status fail(sls_status code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return code;
}

sls_status ok() {
  g_err[0] = '\0';
  return SLS_OK;
}

sls_status cuda_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return ok();
  return fail(SLS_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool pow2(int v) { return v > 0 && (v & (v - 1)) == 0; }

// a*b*... with overflow detection against int64 and against the int32
// indexing the kernels use for per-row positions.
bool checked_mul(int64_t a, int64_t b, int64_t* out) {
  if (a < 0 || b < 0) return false;
  if (a != 0 && b > INT64_MAX / a) return false;
  *out = a * b;
  return true;
}

sls_status check_desc(const sls_attn_desc* d, sls::Shape* s) {
  if (!d) return fail(SLS_EINVAL, "desc is NULL");
  if (d->batch < 1 || d->num_q_heads < 1 || d->num_kv_heads < 1)
    return fail(SLS_EINVAL, "batch/heads must be >= 1 (B=%d Hq=%d Hkv=%d)", d->batch,
                d->num_q_heads, d->num_kv_heads);
  if (d->num_q_heads % d->num_kv_heads)
    return fail(SLS_EINVAL, "num_q_heads %d not a multiple of num_kv_heads %d", d->num_q_heads,
                d->num_kv_heads);
  const int G = d->num_q_heads / d->num_kv_heads;
  if (G > 8) return fail(SLS_EUNSUPPORTED, "query heads per kv head G=%d > 8", G);
  if (d->head_dim != 64 && d->head_dim != 128)
    return fail(SLS_EUNSUPPORTED, "head_dim %d not in {64, 128}", d->head_dim);
  if (d->dtype != SLS_DTYPE_F32 && d->dtype != SLS_DTYPE_BF16)
    return fail(SLS_EUNSUPPORTED, "dtype %d", d->dtype);
  if (!pow2(d->page_size) || d->page_size > 256)
    return fail(SLS_EINVAL, "page_size %d must be a power of two in [1, 256]", d->page_size);
  if (d->capacity < 1 || d->capacity % d->page_size)
    return fail(SLS_EINVAL, "capacity %d must be >= 1 and a multiple of page_size %d", d->capacity,
                d->page_size);
  if (!(d->scale >= 0.f) || std::isinf(d->scale)) return fail(SLS_EINVAL, "scale must be finite and >= 0");
  if (d->flags & ~(SLS_FLAG_CUDA_CORES | SLS_FLAG_NO_TMA | SLS_FLAG_TEST_WAIT_TIMEOUT))
    return fail(SLS_EINVAL, "unknown flags 0x%x", d->flags);
  // element counts of the caches and of the per-row index space
  int64_t rows, elems;
  if (!checked_mul(d->batch, d->num_kv_heads, &rows) || !checked_mul(rows, d->capacity, &elems) ||
      !checked_mul(elems, d->head_dim, &elems) || rows > INT32_MAX || elems > (int64_t(1) << 48) ||
      (int64_t)d->batch * d->num_q_heads > INT32_MAX)
    return fail(SLS_EOVERFLOW, "cache size overflows");
  s->B = d->batch;
  s->Hq = d->num_q_heads;
  s->Hkv = d->num_kv_heads;
  s->G = G;
  s->D = d->head_dim;
  s->P = d->page_size;
  s->pshift = __builtin_ctz((unsigned)d->page_size);
  s->Cap = d->capacity;
  s->dtype = d->dtype;
  s->flags = d->flags;
  s->scale = d->scale > 0.f ? d->scale : 1.0f / std::sqrt((float)d->head_dim);
  return SLS_OK;
}

}  // namespace

namespace sls {
void stat_add(StatId id) { g_stats[id].fetch_add(1, std::memory_order_relaxed); }
}  // namespace sls

namespace sls {
// Records a failure message for sls_last_error() from another translation unit.
sls_status record_error(sls_status code, const char* msg) { return fail(code, "%s", msg); }
}  // namespace sls

namespace {

#define REQUIRE(ptr)                                     \
  do {                                                   \
    if (!(ptr)) return fail(SLS_EINVAL, "%s is NULL", #ptr); \
  } while (0)

// Tensors the kernels read or write in 16-byte vectors.
#define REQUIRE16(ptr)                                                                      \
  do {                                                                                      \
    if (!(ptr)) return fail(SLS_EINVAL, "%s is NULL", #ptr);                                \
    if (reinterpret_cast<uintptr_t>(ptr) & 15) return fail(SLS_EINVAL, "%s is not 16-byte aligned", #ptr); \
  } while (0)

}  // namespace

extern "C" {

const char* sls_last_error(void) { return g_err; }

int32_t sls_version(void) { return 10000; }

sls_status sls_get_stats(sls_stats* out, int32_t reset) {
  if (!out) return fail(SLS_EINVAL, "out is NULL");
  std::memset(out, 0, sizeof(*out));
  auto take = [&](sls::StatId id) -> uint64_t {
    return reset ? g_stats[id].exchange(0) : g_stats[id].load();
  };
  out->quest_step_one_launch = take(sls::kStatStepOneLaunch);
  out->quest_step_two_launch = take(sls::kStatStepTwoLaunch);
  out->select_pages = take(sls::kStatSelectPages);
  out->select_delta_tensor_cores = take(sls::kStatDeltaTensorCores);
  out->select_delta_cuda_cores = take(sls::kStatDeltaCudaCores);
  out->attend_tma = take(sls::kStatAttendTma);
  out->attend_mma = take(sls::kStatAttendMma);
  out->attend_cuda_cores = take(sls::kStatAttendCudaCores);
  out->attend_stream_k = take(sls::kStatAttendStreamK);
  out->attend_refined = take(sls::kStatAttendRefined);
  out->combine = take(sls::kStatCombine);
  out->metadata = take(sls::kStatMetadata);
  out->recall = take(sls::kStatRecall);
  out->attend_stream_k_tma = take(sls::kStatAttendStreamKTma);
  out->attend_refined_tma = take(sls::kStatAttendRefinedTma);
  if (cudaDeviceSynchronize() != cudaSuccess) return fail(SLS_ECUDA, "device synchronisation failed");
  unsigned long long dense = 0, all_keys = 0;
  sls::take_step_row_stats(&dense, &all_keys, reset != 0);
  out->step_rows_dense = dense;
  out->step_rows_all_keys = all_keys;
  out->select_rows_all_keys = sls::take_select_rows_all_keys(reset != 0);
  return ok();
}

sls_status sls_pipeline_check(void) {
  if (cudaDeviceSynchronize() != cudaSuccess) return fail(SLS_ECUDA, "device synchronisation failed");
  unsigned int timeouts = 0, bad = 0;
  for (auto take : {sls::take_status_attend_cc, sls::take_status_attend_mma, sls::take_status_attend_tma,
                    sls::take_status_attend_refined, sls::take_status_quest_step, sls::take_status_recall,
                    sls::take_status_attend_kv8}) {
    const sls::DeviceStatus st = take();
    timeouts += st.wait_timeouts;
    bad += st.bad_page_ids;
  }
  if (cudaGetLastError() != cudaSuccess) return fail(SLS_ECUDA, "reading the device status words failed");
  if (timeouts)
    return fail(SLS_ETIMEOUT, "%u pipelined CTA(s) gave up waiting for their copies (%u bad page-list entries)",
                timeouts, bad);
  if (bad) return fail(SLS_EDEVICE, "%u page-list entries were neither a page of the pool nor -1 (skipped)", bad);
  return SLS_OK;
}

sls_status sls_pagemeta_build(const sls_attn_desc* desc, const void* k_cache, const int32_t* ctx_len,
                              void* kmin, void* kmax, void* stream) {
  sls::Shape s;
  sls_status r = check_desc(desc, &s);
  if (r) return r;
  REQUIRE16(k_cache); REQUIRE(ctx_len); REQUIRE16(kmin); REQUIRE16(kmax);
  sls::stat_add(sls::kStatMetadata);
  return cuda_status(sls::launch_pagemeta_build(s, k_cache, ctx_len, kmin, kmax, (cudaStream_t)stream),
                     "sls_pagemeta_build");
}

sls_status sls_pagemeta_update(const sls_attn_desc* desc, const void* k_cache, const int32_t* pos,
                               void* kmin, void* kmax, void* stream) {
  sls::Shape s;
  sls_status r = check_desc(desc, &s);
  if (r) return r;
  REQUIRE16(k_cache); REQUIRE(pos); REQUIRE16(kmin); REQUIRE16(kmax);
  sls::stat_add(sls::kStatMetadata);
  return cuda_status(sls::launch_pagemeta_update(s, k_cache, pos, kmin, kmax, (cudaStream_t)stream),
                     "sls_pagemeta_update");
}

static sls_status check_block(const sls::Shape& s, int32_t block) {
  if (!pow2(block) || block < 16 || block > 256)
    return fail(SLS_EINVAL, "block %d must be a power of two in [16, 256]", block);
  if (s.Cap % block) return fail(SLS_EINVAL, "capacity %d not a multiple of block %d", s.Cap, block);
  return SLS_OK;
}

sls_status sls_decode_append(const sls_attn_desc* desc, const void* k_new, const void* v_new, void* k_cache,
                             void* v_cache, void* kmin, void* kmax, int32_t* ctx_len, int32_t* pos_out,
                             void* stream) {
  sls::Shape s;
  sls_status r = check_desc(desc, &s);
  if (r) return r;
  REQUIRE16(k_new); REQUIRE16(v_new); REQUIRE16(k_cache); REQUIRE16(v_cache); REQUIRE(ctx_len);
  if ((kmin == nullptr) != (kmax == nullptr)) return fail(SLS_EINVAL, "kmin and kmax: both or neither");
  if (kmin && s.P == 1) return fail(SLS_EINVAL, "page_size 1: the key cache is its own page metadata (pass NULL)");
  sls::stat_add(sls::kStatMetadata);
  return cuda_status(sls::launch_decode_append(s, k_new, v_new, k_cache, v_cache, kmin, kmax, ctx_len, pos_out,
                                               (cudaStream_t)stream),
                     "sls_decode_append");
}

sls_status sls_thumb_build(const sls_attn_desc* desc, const void* k_cache, const int32_t* ctx_len,
                           int32_t block, uint8_t* codes, void* scales, void* stream) {
  sls::Shape s;
  sls_status r = check_desc(desc, &s);
  if (r) return r;
  if ((r = check_block(s, block))) return r;
  REQUIRE16(k_cache); REQUIRE(ctx_len); REQUIRE16(codes); REQUIRE16(scales);
  sls::stat_add(sls::kStatMetadata);
  return cuda_status(sls::launch_thumb_build(s, k_cache, ctx_len, block, codes, scales, nullptr,
                                             (cudaStream_t)stream),
                     "sls_thumb_build");
}

sls_status sls_thumb_residual_build(const sls_attn_desc* desc, const void* k_cache, const int32_t* ctx_len,
                                    int32_t block, uint8_t* codes, void* scales, int8_t* res, void* stream) {
  sls::Shape s;
  sls_status r = check_desc(desc, &s);
  if (r) return r;
  if ((r = check_block(s, block))) return r;
  REQUIRE16(k_cache); REQUIRE(ctx_len); REQUIRE16(codes); REQUIRE16(scales); REQUIRE16(res);
  sls::stat_add(sls::kStatMetadata);
  return cuda_status(sls::launch_thumb_build(s, k_cache, ctx_len, block, codes, scales, res, (cudaStream_t)stream),
                     "sls_thumb_residual_build");
}

sls_status sls_thumb_update(const sls_attn_desc* desc, const void* k_cache, const int32_t* pos,
                            int32_t block, uint8_t* codes, void* scales, void* stream) {
  sls::Shape s;
  sls_status r = check_desc(desc, &s);
  if (r) return r;
  if ((r = check_block(s, block))) return r;
  REQUIRE16(k_cache); REQUIRE(pos); REQUIRE16(codes); REQUIRE16(scales);
  sls::stat_add(sls::kStatMetadata);
  return cuda_status(sls::launch_thumb_update(s, k_cache, pos, block, codes, scales, nullptr,
                                              (cudaStream_t)stream),
                     "sls_thumb_update");
}

sls_status sls_thumb_residual_update(const sls_attn_desc* desc, const void* k_cache, const int32_t* pos,
                                     int32_t block, uint8_t* codes, void* scales, int8_t* res, void* stream) {
  sls::Shape s;
  sls_status r = check_desc(desc, &s);
  if (r) return r;
  if ((r = check_block(s, block))) return r;
  REQUIRE16(k_cache); REQUIRE(pos); REQUIRE16(codes); REQUIRE16(scales); REQUIRE16(res);
  sls::stat_add(sls::kStatMetadata);
  return cuda_status(sls::launch_thumb_update(s, k_cache, pos, block, codes, scales, res, (cudaStream_t)stream),
                     "sls_thumb_residual_update");
}

size_t sls_select_pages_workspace_size(const sls_attn_desc* desc) {
  sls::Shape s;
  if (check_desc(desc, &s)) return 0;
  return sls::select_pages_workspace(s);
}

sls_status sls_select_pages(const sls_attn_desc* desc, const void* q, const void* kmin,
                            const void* kmax, const int32_t* ctx_len, int32_t k,
                            int32_t n_sink_pages, int32_t n_local_tokens, int32_t* page_idx,
                            void* workspace, size_t workspace_bytes, void* stream) {
  sls::Shape s;
  sls_status r = check_desc(desc, &s);
  if (r) return r;
  REQUIRE16(q); REQUIRE16(kmin); REQUIRE16(kmax); REQUIRE(ctx_len); REQUIRE(page_idx);
  const int npcap = s.Cap >> s.pshift;
  if (k < 1 || k > npcap) return fail(SLS_EINVAL, "k=%d must be in [1, Cap/P=%d]", k, npcap);
  if (n_sink_pages < 0 || n_local_tokens < 0)
    return fail(SLS_EINVAL, "n_sink_pages and n_local_tokens must be >= 0");
  const int64_t forced_max =
      (int64_t)n_sink_pages + (n_local_tokens > 0 ? ((int64_t)n_local_tokens + s.P - 1) / s.P + 1 : 0);
  if (forced_max > k)
    return fail(SLS_EINVAL, "budget k=%d cannot hold the forced pages (up to %lld)", k,
                (long long)forced_max);
  if (s.P == 1 && kmin != kmax)
    return fail(SLS_EINVAL, "page_size 1: pass the key cache as both kmin and kmax");
  if (npcap > sls::select_pages_max_pages())
    return fail(SLS_EUNSUPPORTED, "Cap/P=%d pages per row exceeds the supported %d", npcap,
                sls::select_pages_max_pages());
  const size_t need = sls::select_pages_workspace(s);
  if (!workspace || workspace_bytes < need)
    return fail(SLS_EWORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
  sls::stat_add(sls::kStatSelectPages);
  return cuda_status(sls::launch_select_pages(s, q, kmin, kmax, ctx_len, k, n_sink_pages, n_local_tokens,
                                              page_idx, workspace, (cudaStream_t)stream),
                     "sls_select_pages");
}

size_t sls_select_delta_workspace_size(const sls_attn_desc* desc, int32_t block) {
  sls::Shape s;
  if (check_desc(desc, &s) || check_block(s, block)) return 0;
  return sls::select_delta_workspace(s, block);
}

sls_status sls_select_delta(const sls_attn_desc* desc, const void* q, const void* k_cache,
                            const uint8_t* codes, const void* scales, const int32_t* ctx_len,
                            int32_t block, float delta, int32_t* count, int32_t* block_idx,
                            int32_t idx_stride, void* workspace, size_t workspace_bytes,
                            void* stream) {
  sls::Shape s;
  sls_status r = check_desc(desc, &s);
  if (r) return r;
  if ((r = check_block(s, block))) return r;
  REQUIRE16(q); REQUIRE16(k_cache); REQUIRE16(codes); REQUIRE16(scales); REQUIRE(ctx_len);
  REQUIRE(count); REQUIRE(block_idx);
  if (!(delta >= 0.f) || std::isinf(delta)) return fail(SLS_EINVAL, "delta must be finite and >= 0");
  if (idx_stride < s.Cap / block)
    return fail(SLS_EINVAL, "idx_stride %d < Cap/block %d", idx_stride, s.Cap / block);
  const size_t need = sls::select_delta_workspace(s, block);
  if (!workspace || workspace_bytes < need)
    return fail(SLS_EWORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
  return cuda_status(sls::launch_select_delta(s, q, k_cache, codes, scales, ctx_len, block, delta, count,
                                              block_idx, idx_stride, workspace, (cudaStream_t)stream),
                     "sls_select_delta");
}

sls_status sls_sparse_decode_attend(const sls_attn_desc* desc, const void* q, const void* k_cache,
                                    const void* v_cache, const int32_t* page_idx, int32_t idx_stride,
                                    const int32_t* count, int32_t k_fixed, const int32_t* ctx_len,
                                    int32_t num_splits, float* o_part, float* m_part, float* l_part,
                                    void* stream) {
  sls::Shape s;
  sls_status r = check_desc(desc, &s);
  if (r) return r;
  REQUIRE16(q); REQUIRE16(k_cache); REQUIRE16(v_cache); REQUIRE(ctx_len);
  REQUIRE16(o_part); REQUIRE(m_part); REQUIRE(l_part);
  if (num_splits < 1 || num_splits > 1024) return fail(SLS_EINVAL, "num_splits %d not in [1, 1024]", num_splits);
  if (page_idx) {
    if (idx_stride < 1) return fail(SLS_EINVAL, "idx_stride %d < 1", idx_stride);
    if (!count && (k_fixed < 0 || k_fixed > idx_stride))
      return fail(SLS_EINVAL, "k_fixed %d not in [0, idx_stride=%d]", k_fixed, idx_stride);
  }
  int64_t ctas;
  if (!checked_mul((int64_t)s.B * s.Hkv, num_splits, &ctas) || ctas > INT32_MAX)
    return fail(SLS_EOVERFLOW, "grid too large");
  return cuda_status(sls::launch_attend(s, q, k_cache, v_cache, page_idx, idx_stride, count, k_fixed, ctx_len,
                                        num_splits, o_part, m_part, l_part, (cudaStream_t)stream),
                     "sls_sparse_decode_attend");
}

int32_t sls_attend_default_splits(const sls_attn_desc* desc, int32_t max_entries) {
  sls::Shape s;
  if (check_desc(desc, &s) || max_entries < 1) return 1;
  return sls::attend_default_splits(s, max_entries);
}

static size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

size_t sls_attend_combine_workspace_size(const sls_attn_desc* desc, int32_t num_splits) {
  sls::Shape s;
  if (check_desc(desc, &s) || num_splits < 0 || num_splits > 1024) return 0;
  if (num_splits == 0) num_splits = sls::max_auto_splits(s);
  const size_t heads = (size_t)s.B * s.Hq * num_splits;
  return align256((size_t)s.B * s.Hkv * 4) + align256(heads * s.D * 4) + 2 * align256(heads * 4);
}

sls_status sls_sparse_decode_attend_combine(const sls_attn_desc* desc, const void* q, const void* k_cache,
                                            const void* v_cache, const int32_t* page_idx, int32_t idx_stride,
                                            const int32_t* count, int32_t k_fixed, const int32_t* ctx_len,
                                            int32_t num_splits, const float* sink, void* out, float* lse,
                                            void* workspace, size_t workspace_bytes, void* stream) {
  sls::Shape s;
  sls_status r = check_desc(desc, &s);
  if (r) return r;
  REQUIRE16(q); REQUIRE16(k_cache); REQUIRE16(v_cache); REQUIRE(ctx_len); REQUIRE(out);
  if (num_splits < 0 || num_splits > 1024) return fail(SLS_EINVAL, "num_splits %d not in [0, 1024]", num_splits);
  if (page_idx) {
    if (idx_stride < 1) return fail(SLS_EINVAL, "idx_stride %d < 1", idx_stride);
    if (!count && (k_fixed < 0 || k_fixed > idx_stride))
      return fail(SLS_EINVAL, "k_fixed %d not in [0, idx_stride=%d]", k_fixed, idx_stride);
  }
  int64_t ctas;
  if (!checked_mul((int64_t)s.B * s.Hkv, num_splits, &ctas) || ctas > INT32_MAX)
    return fail(SLS_EOVERFLOW, "grid too large");
  const size_t need = sls_attend_combine_workspace_size(desc, num_splits);
  if (!workspace || workspace_bytes < need)
    return fail(SLS_EWORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
  char* w = static_cast<char*>(workspace);
  const size_t heads = (size_t)s.B * s.Hq * (num_splits ? num_splits : sls::max_auto_splits(s));
  sls::FusedCombine f;
  f.tickets = reinterpret_cast<int32_t*>(w);
  w += align256((size_t)s.B * s.Hkv * 4);
  float* o_part = reinterpret_cast<float*>(w);
  w += align256(heads * s.D * 4);
  float* m_part = reinterpret_cast<float*>(w);
  w += align256(heads * 4);
  float* l_part = reinterpret_cast<float*>(w);
  f.sink = sink;
  f.out = out;
  f.lse = lse;
  return cuda_status(sls::launch_attend(s, q, k_cache, v_cache, page_idx, idx_stride, count, k_fixed, ctx_len,
                                        num_splits, o_part, m_part, l_part, (cudaStream_t)stream, &f),
                     "sls_sparse_decode_attend_combine");
}

size_t sls_refined_decode_attend_workspace_size(const sls_attn_desc* desc) {
  sls::Shape s;
  if (check_desc(desc, &s)) return 0;
  return sls::refined_workspace(s);
}

sls_status sls_refined_decode_attend_combine(const sls_attn_desc* desc, const void* q, const void* k_cache,
                                             const void* v_cache, const uint8_t* codes, const void* scales,
                                             const int8_t* res, const int32_t* block_idx, int32_t idx_stride,
                                             const int32_t* count, const int32_t* ctx_len, const float* sink,
                                             void* out, float* lse, void* workspace, size_t workspace_bytes,
                                             void* stream) {
  sls::Shape s;
  sls_status r = check_desc(desc, &s);
  if (r) return r;
  REQUIRE16(q); REQUIRE16(k_cache); REQUIRE16(v_cache); REQUIRE(block_idx); REQUIRE(count); REQUIRE(ctx_len);
  REQUIRE(out);
  if ((codes == nullptr) != (res == nullptr) || (codes == nullptr) != (scales == nullptr))
    return fail(SLS_EINVAL, "codes, scales and res: all or none");
  if (!sls::refined_supported(s))
    return fail(SLS_EUNSUPPORTED,
                "needs bf16, G <= 8, blocks (page_size) of >= 16 tokens and at most 4096 rows (B*Hkv)");
  if (idx_stride < 1) return fail(SLS_EINVAL, "idx_stride %d < 1", idx_stride);
  if (codes) {
    REQUIRE16(codes); REQUIRE16(scales); REQUIRE16(res);
  }
  const size_t need = sls::refined_workspace(s);
  if (!workspace || workspace_bytes < need)
    return fail(SLS_EWORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
  sls::stat_add(codes ? sls::kStatAttendRefined : sls::kStatAttendStreamK);
  return cuda_status(sls::launch_attend_refined(s, q, k_cache, v_cache, codes, scales, res, block_idx, idx_stride,
                                                count, ctx_len, sink, out, lse, workspace, (cudaStream_t)stream),
                     "sls_refined_decode_attend_combine");
}

size_t sls_quest_decode_step_workspace_size(const sls_attn_desc* desc, int32_t k, int32_t num_splits) {
  sls::Shape s;
  if (check_desc(desc, &s) || k < 1 || num_splits < 0 || num_splits > 1024) return 0;
  // what the two-launch path needs (the one-launch kernel uses none of it)
  return align256(sls::select_pages_workspace(s)) + align256((size_t)s.B * s.Hkv * k * 4) +
         sls_attend_combine_workspace_size(desc, num_splits);
}

int32_t sls_quest_decode_step_splits(const sls_attn_desc* desc, int32_t k) {
  sls::Shape s;
  if (check_desc(desc, &s) || k < 1 || k > (s.Cap >> s.pshift) || !sls::quest_step_eligible(s, k)) return 0;
  return sls::quest_step_splits(s, k);
}

sls_status sls_quest_decode_step(const sls_attn_desc* desc, const void* q, const void* k_cache, const void* v_cache,
                                 const void* kmin, const void* kmax, const int32_t* ctx_len, int32_t k,
                                 int32_t n_sink_pages, int32_t n_local_tokens, const float* sink, int32_t* page_idx,
                                 void* out, float* lse, int32_t num_splits, float min_sparsity, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  sls::Shape s;
  sls_status r = check_desc(desc, &s);
  if (r) return r;
  REQUIRE16(q); REQUIRE16(k_cache); REQUIRE16(v_cache); REQUIRE16(kmin); REQUIRE16(kmax); REQUIRE(ctx_len); REQUIRE(out);
  const int npcap = s.Cap >> s.pshift;
  if (k < 1 || k > npcap) return fail(SLS_EINVAL, "k=%d must be in [1, Cap/P=%d]", k, npcap);
  if (n_sink_pages < 0 || n_local_tokens < 0) return fail(SLS_EINVAL, "n_sink_pages and n_local_tokens must be >= 0");
  const int64_t forced_max =
      (int64_t)n_sink_pages + (n_local_tokens > 0 ? ((int64_t)n_local_tokens + s.P - 1) / s.P + 1 : 0);
  if (forced_max > k)
    return fail(SLS_EINVAL, "budget k=%d cannot hold the forced pages (up to %lld)", k, (long long)forced_max);
  if (s.P == 1 && kmin != kmax) return fail(SLS_EINVAL, "page_size 1: pass the key cache as both kmin and kmax");
  if (num_splits < 0 || num_splits > 1024) return fail(SLS_EINVAL, "num_splits %d not in [0, 1024]", num_splits);
  if (!(min_sparsity >= 0.f) || std::isinf(min_sparsity))
    return fail(SLS_EINVAL, "min_sparsity must be finite and >= 0");
  const size_t need = sls_quest_decode_step_workspace_size(desc, k, num_splits);
  if (!workspace || workspace_bytes < need)
    return fail(SLS_EWORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
  bool handled = false;
  cudaError_t e = sls::launch_quest_step(s, q, k_cache, v_cache, kmin, kmax, ctx_len, k, n_sink_pages,
                                         n_local_tokens, sink, page_idx, out, lse, num_splits, min_sparsity,
                                         (cudaStream_t)stream, &handled);
  if (handled) {
    sls::stat_add(sls::kStatStepOneLaunch);
    return cuda_status(e, "sls_quest_decode_step");
  }
  if (min_sparsity > 0.f)
    return fail(SLS_EUNSUPPORTED, "min_sparsity needs the one-launch step (bf16, pages of >= 16 tokens)");
  // two launches: select into page_idx (or the workspace), then attend with the fused combine
  sls::stat_add(sls::kStatStepTwoLaunch);
  if (npcap > sls::select_pages_max_pages())
    return fail(SLS_EUNSUPPORTED, "Cap/P=%d pages per row exceeds the supported %d", npcap,
                sls::select_pages_max_pages());
  char* w = static_cast<char*>(workspace);
  void* sel_ws = w;
  w += align256(sls::select_pages_workspace(s));
  int32_t* list = page_idx ? page_idx : reinterpret_cast<int32_t*>(w);
  w += align256((size_t)s.B * s.Hkv * k * 4);
  e = sls::launch_select_pages(s, q, kmin, kmax, ctx_len, k, n_sink_pages, n_local_tokens, list, sel_ws,
                               (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_status(e, "sls_quest_decode_step (select)");
  const size_t heads = (size_t)s.B * s.Hq * (num_splits ? num_splits : sls::max_auto_splits(s));
  sls::FusedCombine f;
  f.tickets = reinterpret_cast<int32_t*>(w);
  w += align256((size_t)s.B * s.Hkv * 4);
  float* o_part = reinterpret_cast<float*>(w);
  w += align256(heads * s.D * 4);
  float* m_part = reinterpret_cast<float*>(w);
  w += align256(heads * 4);
  float* l_part = reinterpret_cast<float*>(w);
  f.sink = sink;
  f.out = out;
  f.lse = lse;
  return cuda_status(sls::launch_attend(s, q, k_cache, v_cache, list, k, nullptr, k, ctx_len, num_splits, o_part,
                                        m_part, l_part, (cudaStream_t)stream, &f),
                     "sls_quest_decode_step (attend)");
}

size_t sls_selection_recall_workspace_size(const sls_attn_desc* desc) {
  sls::Shape s;
  if (check_desc(desc, &s)) return 0;
  return sls::recall_workspace(s);
}

sls_status sls_selection_recall(const sls_attn_desc* desc, const void* q, const void* k_cache,
                                const int32_t* page_idx, int32_t idx_stride, const int32_t* count, int32_t k_fixed,
                                const int32_t* ctx_len, float* recall, void* workspace, size_t workspace_bytes,
                                void* stream) {
  sls::Shape s;
  sls_status r = check_desc(desc, &s);
  if (r) return r;
  REQUIRE16(q); REQUIRE16(k_cache); REQUIRE(ctx_len); REQUIRE(recall);
  if (page_idx) {
    if (idx_stride < 1) return fail(SLS_EINVAL, "idx_stride %d < 1", idx_stride);
    if (!count && (k_fixed < 0 || k_fixed > idx_stride))
      return fail(SLS_EINVAL, "k_fixed %d not in [0, idx_stride=%d]", k_fixed, idx_stride);
  }
  if (!sls::recall_supported(s)) return fail(SLS_EUNSUPPORTED, "Cap/P above 262144 pages");
  const size_t need = sls::recall_workspace(s);
  if (!workspace || workspace_bytes < need)
    return fail(SLS_EWORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
  sls::stat_add(sls::kStatRecall);
  return cuda_status(sls::launch_recall(s, q, k_cache, page_idx, idx_stride, count, k_fixed, ctx_len, recall,
                                        workspace, (cudaStream_t)stream),
                     "sls_selection_recall");
}

sls_status sls_combine_splits(const sls_attn_desc* desc, const float* o_part, const float* m_part,
                              const float* l_part, int32_t num_splits, const float* sink, void* out,
                              float* lse, void* stream) {
  sls::Shape s;
  sls_status r = check_desc(desc, &s);
  if (r) return r;
  REQUIRE16(o_part); REQUIRE(m_part); REQUIRE(l_part); REQUIRE(out);
  if (num_splits < 1 || num_splits > 1024) return fail(SLS_EINVAL, "num_splits %d not in [1, 1024]", num_splits);
  return cuda_status(sls::launch_combine(s, o_part, m_part, l_part, num_splits, sink, out, lse, (cudaStream_t)stream),
                     "sls_combine_splits");
}

// ---- per-head norm and rotation, the 8-bit cache

sls_status sls_qk_norm_rope(const sls_rope_desc* rope, int32_t num_tokens, const void* q, int64_t q_token_stride,
                            int64_t q_head_stride, const void* k, int64_t k_token_stride, int64_t k_head_stride,
                            const void* q_weight, const void* k_weight, const int32_t* positions, void* q_out,
                            int64_t q_out_token_stride, int64_t q_out_head_stride, void* k_out,
                            int64_t k_out_token_stride, int64_t k_out_head_stride, void* stream) {
  if (!rope) return fail(SLS_EINVAL, "rope is NULL");
  const int Hq = rope->num_q_heads, Hkv = rope->num_kv_heads, D = rope->head_dim, R = rope->rotary_dim;
  if (Hq < 0 || Hkv < 0 || Hq > (1 << 20) || Hkv > (1 << 20) || Hq + Hkv < 1)
    return fail(SLS_EINVAL, "head counts Hq=%d Hkv=%d", Hq, Hkv);
  if (D != 64 && D != 128) return fail(SLS_EUNSUPPORTED, "head_dim %d not in {64, 128}", D);
  if (rope->dtype != SLS_DTYPE_F32 && rope->dtype != SLS_DTYPE_BF16)
    return fail(SLS_EUNSUPPORTED, "dtype %d", rope->dtype);
  if (R < 0 || R > D || R % 16) return fail(SLS_EUNSUPPORTED, "rotary_dim %d not a multiple of 16 in [0, %d]", R, D);
  if (rope->interleaved != 0 && rope->interleaved != 1) return fail(SLS_EINVAL, "interleaved must be 0 or 1");
  if (!(rope->eps >= 0.f) || std::isinf(rope->eps)) return fail(SLS_EINVAL, "eps must be finite and >= 0");
  if (!rope->inv_freq && (!(rope->theta > 0.0) || std::isinf(rope->theta)))
    return fail(SLS_EINVAL, "theta must be finite and > 0");
  if (num_tokens < 0) return fail(SLS_EINVAL, "num_tokens %d < 0", num_tokens);
  const int vec = rope->dtype == SLS_DTYPE_F32 ? 4 : 8;
  sls::RopeArgs a = {};
  auto side = [&](const char* name, int heads, const void* in, int64_t it, int64_t ih, const void* w, void* out,
                  int64_t ot, int64_t oh) -> sls_status {
    if (!in || !out) return fail(SLS_EINVAL, "%s or its output is NULL", name);
    if (((uintptr_t)in | (uintptr_t)out | (uintptr_t)w) & 15)
      return fail(SLS_EINVAL, "%s, its weight and its output must be 16-byte aligned", name);
    const int64_t lim = INT32_MAX;  // tokens * stride stays within 62 bits
    if (it < 0 || ih < 0 || ot < 0 || oh < 0 || it > lim || ih > lim || ot > lim || oh > lim || it % vec || ih % vec ||
        ot % vec || oh % vec)
      return fail(SLS_EINVAL, "strides of %s must be multiples of %d elements in [0, 2^31)", name, vec);
    // no two output vectors overlap: one of the two axes steps past the whole extent of the other
    const bool one_t = num_tokens == 1, one_h = heads == 1;
    const bool t_out = (one_h || oh >= D) && (one_t || ot >= (heads - 1) * oh + D);
    const bool h_out = (one_t || ot >= D) && (one_h || oh >= (num_tokens - 1) * ot + D);
    if (!t_out && !h_out) return fail(SLS_EINVAL, "output vectors of %s overlap", name);
    return SLS_OK;
  };
  if (num_tokens == 0) return ok();
  sls_status r;
  REQUIRE(positions);
  if (Hq && (r = side("q", Hq, q, q_token_stride, q_head_stride, q_weight, q_out, q_out_token_stride, q_out_head_stride)))
    return r;
  if (Hkv && (r = side("k", Hkv, k, k_token_stride, k_head_stride, k_weight, k_out, k_out_token_stride,
                       k_out_head_stride)))
    return r;
  // The frequencies of theta, kept from call to call by their value: R / 2
  // calls of pow are half of a small call's time on the host.
  thread_local double known_theta = 0.0;
  thread_local int known_R = 0;
  thread_local uint64_t known[64];
  if (!rope->inv_freq && rope->theta == known_theta && R == known_R) {
    std::memcpy(a.freq, known, sizeof(known));
  } else {
    for (int i = 0; i < R / 2; ++i) {
      const double f = rope->inv_freq ? rope->inv_freq[i] : std::pow(rope->theta, -2.0 * i / R);
      if (!std::isfinite(f)) return fail(SLS_EINVAL, "frequency %d is not finite", i);
      const double turns = f / 6.283185307179586476925286766559;
      double frac = turns - std::floor(turns);  // in [0, 1]
      if (frac >= 1.0) frac = 0.0;
      a.freq[i] = (uint64_t)std::ldexp(frac, 64);
    }
    if (!rope->inv_freq) {
      known_theta = rope->theta;
      known_R = R;
      std::memcpy(known, a.freq, sizeof(known));
    }
  }
  a.q = q; a.k = k; a.wq = q_weight; a.wk = k_weight; a.qo = q_out; a.ko = k_out; a.pos = positions;
  a.q_t = q_token_stride; a.q_h = q_head_stride; a.k_t = k_token_stride; a.k_h = k_head_stride;
  a.qo_t = q_out_token_stride; a.qo_h = q_out_head_stride; a.ko_t = k_out_token_stride; a.ko_h = k_out_head_stride;
  a.N = num_tokens; a.Hq = Hq; a.Hkv = Hkv; a.D = D; a.R = R;
  a.interleaved = rope->interleaved; a.dtype = rope->dtype; a.eps = rope->eps;
  sls::stat_add(sls::kStatMetadata);
  return cuda_status(sls::launch_qk_norm_rope(a, (cudaStream_t)stream), "sls_qk_norm_rope");
}

// Whether two ranges of device memory share a byte (a null range shares none).
static bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && na > 0 && nb > 0 && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

static sls_status check_kv8(const sls::Shape& s, const sls_kv8_cache* c, int capacity, const char* name, sls::Kv8* out) {
  if (!c) return fail(SLS_EINVAL, "%s is NULL", name);
  if (s.dtype != SLS_DTYPE_BF16) return fail(SLS_EUNSUPPORTED, "the 8-bit cache takes bf16 descriptors only");
  if (c->format != SLS_KV8_INT8 && c->format != SLS_KV8_E4M3)
    return fail(SLS_EUNSUPPORTED, "%s format %d", name, c->format);
  if (!pow2(c->block) || c->block < 16 || c->block > 256)
    return fail(SLS_EINVAL, "%s block %d must be a power of two in [16, 256]", name, c->block);
  if (capacity < c->block || capacity % c->block)
    return fail(SLS_EINVAL, "%s capacity %d not a multiple of its block %d", name, capacity, c->block);
  if (capacity > (1 << 30)) return fail(SLS_EUNSUPPORTED, "%s capacity %d above 2^30", name, capacity);
  if (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales || !c->k_tail || !c->v_tail)
    return fail(SLS_EINVAL, "%s has a NULL pointer", name);
  if (((uintptr_t)c->k_codes | (uintptr_t)c->v_codes | (uintptr_t)c->k_tail | (uintptr_t)c->v_tail) & 15)
    return fail(SLS_EINVAL, "%s codes and tails must be 16-byte aligned", name);
  if (((uintptr_t)c->k_scales | (uintptr_t)c->v_scales) & 3)
    return fail(SLS_EINVAL, "%s scales must be 4-byte aligned", name);
  *out = sls::Kv8{c->format, c->block, __builtin_ctz((unsigned)c->block), c->k_codes, c->v_codes,
                  c->k_scales, c->v_scales, c->k_tail, c->v_tail};
  return SLS_OK;
}

// Memory that a call reads or writes, and its bytes.
struct Span {
  const void* p;
  int64_t n;
};
static Span at(const void* p, int64_t n) { return Span{p, n}; }

// A cache's buffers, for `rows` rows of `capacity` tokens of D channels.
struct CacheSpans {
  Span s[6];
};
static CacheSpans spans_of(const sls::Kv8& c, int64_t rows, int64_t capacity, int D) {
  const int64_t t = rows * capacity;
  return {{at(c.kc, t * D), at(c.vc, t * D), at(c.ks, t / c.block * 4), at(c.vs, t / c.block * 4),
           at(c.kt, rows * c.block * D * 2), at(c.vt, rows * c.block * D * 2)}};
}

// The buffers a cache is made of are six pieces of memory.
static sls_status check_apart(const CacheSpans& c, const char* name) {
  for (int i = 0; i < 6; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(c.s[i].p, c.s[i].n, c.s[j].p, c.s[j].n)) return fail(SLS_EINVAL, "%s has buffers that share memory", name);
  return SLS_OK;
}

sls_status sls_kv8_append(const sls_attn_desc* desc, const sls_kv8_cache* cache, const void* k_new,
                          int64_t k_seq_stride, int64_t k_token_stride, int64_t k_head_stride, const void* v_new,
                          int64_t v_seq_stride, int64_t v_token_stride, int64_t v_head_stride, int32_t max_new,
                          const int32_t* new_len, void* kmin, void* kmax, float* mass, const int32_t* ctx_len,
                          int32_t* ctx_out, int32_t* pos_out, void* stream) {
  sls::Shape s;
  sls::Kv8 c;
  sls_status r = check_desc(desc, &s);
  if (r || (r = check_kv8(s, cache, s.Cap, "cache", &c))) return r;
  REQUIRE(ctx_len); REQUIRE(ctx_out);
  if (max_new < 0) return fail(SLS_EINVAL, "max_new %d < 0", max_new);
  if (max_new > 0) {
    REQUIRE16(k_new); REQUIRE16(v_new);
  }
  for (int64_t st : {k_seq_stride, k_token_stride, k_head_stride, v_seq_stride, v_token_stride, v_head_stride})
    if (st < 0 || st > (int64_t(1) << 40) || st % 8)
      return fail(SLS_EINVAL, "strides of the new tokens must be multiples of 8 elements in [0, 2^40]");
  const int64_t n4 = (int64_t)s.B * 4;
  if ((ctx_out != ctx_len && overlap(ctx_out, n4, ctx_len, n4)) || overlap(ctx_out, n4, new_len, n4) ||
      overlap(pos_out, n4, ctx_len, n4) || overlap(pos_out, n4, new_len, n4) || overlap(pos_out, n4, ctx_out, n4))
    return fail(SLS_EINVAL, "ctx_out must be ctx_len itself or memory of its own, and pos_out memory of its own");
  if ((kmin == nullptr) != (kmax == nullptr)) return fail(SLS_EINVAL, "kmin and kmax: both or neither");
  if (kmin) {
    REQUIRE16(kmin); REQUIRE16(kmax);
    if (s.P == 1) return fail(SLS_EINVAL, "page_size 1: an 8-bit cache has no page summaries of single keys (pass NULL)");
  }
  const int64_t units = (int64_t)(max_new / c.block) + 2;
  int64_t ctas;
  if (!checked_mul((int64_t)s.B * s.Hkv * 2, units, &ctas) || ctas > INT32_MAX)
    return fail(SLS_EOVERFLOW, "grid too large");
  const int64_t rows = (int64_t)s.B * s.Hkv, meta = rows * (s.Cap >> s.pshift) * s.D * 2;
  const CacheSpans cs = spans_of(c, rows, s.Cap, s.D);
  if ((r = check_apart(cs, "cache"))) return r;
  // what is written besides: memory of its own, and none of the cache's
  const Span to[] = {at(kmin, meta), at(kmax, meta), at(mass, rows * (s.Cap / c.block) * 4), at(ctx_out, n4), at(pos_out, n4)};
  for (const Span& x : {at(ctx_len, n4), at(new_len, n4)}) {
    for (const Span& y : cs.s)
      if (overlap(x.p, x.n, y.p, y.n)) return fail(SLS_EINVAL, "the lengths share memory with the cache");
    for (int i = 0; i < 3; ++i)
      if (overlap(x.p, x.n, to[i].p, to[i].n)) return fail(SLS_EINVAL, "the lengths share memory with an output");
  }
  for (int i = 0; i < 5; ++i) {
    for (const Span& x : cs.s)
      if (overlap(to[i].p, to[i].n, x.p, x.n)) return fail(SLS_EINVAL, "an output shares memory with the cache");
    for (int j = 0; j < i; ++j)
      if (overlap(to[i].p, to[i].n, to[j].p, to[j].n)) return fail(SLS_EINVAL, "two outputs share memory");
  }
  sls::Kv8New n = {k_new, v_new, k_seq_stride, k_token_stride, k_head_stride,
                   v_seq_stride, v_token_stride, v_head_stride, max_new, new_len};
  sls::stat_add(sls::kStatMetadata);
  return cuda_status(sls::launch_kv8_append(s, c, n, kmin, kmax, mass, ctx_len, ctx_out, pos_out, (cudaStream_t)stream),
                     "sls_kv8_append");
}

size_t sls_kv8_decode_attend_workspace_size(const sls_attn_desc* desc, const sls_kv8_cache* cache, int32_t with_mass) {
  sls::Shape s;
  sls::Kv8 c;
  if (check_desc(desc, &s) || check_kv8(s, cache, s.Cap, "cache", &c) || !sls::kv8_attend_supported(s)) return 0;
  return sls::kv8_attend_workspace(s, c, with_mass != 0);
}

sls_status sls_kv8_decode_attend(const sls_attn_desc* desc, const sls_kv8_cache* cache, const void* q,
                                 const int32_t* page_idx, int32_t idx_stride, const int32_t* count, int32_t k_fixed,
                                 const int32_t* ctx_len, const float* sink, void* out, float* lse,
                                 const float* mass_in, float* mass_out, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  sls::Shape s;
  sls::Kv8 c;
  sls_status r = check_desc(desc, &s);
  if (r || (r = check_kv8(s, cache, s.Cap, "cache", &c))) return r;
  if (s.flags & ~SLS_FLAG_TEST_WAIT_TIMEOUT)
    return fail(SLS_EUNSUPPORTED, "the 8-bit cache has one attend kernel: flags 0x%x", s.flags);
  if (!sls::kv8_attend_supported(s))
    return fail(SLS_EUNSUPPORTED, "at most 4096 rows (B*Hkv) and 2^31 - 1 cache slots in all");
  REQUIRE16(q); REQUIRE(ctx_len); REQUIRE16(out);
  if (page_idx) {
    if (s.P < 16) return fail(SLS_EUNSUPPORTED, "page lists need pages of >= 16 tokens (P=%d)", s.P);
    if (idx_stride < 1) return fail(SLS_EINVAL, "idx_stride %d < 1", idx_stride);
    if ((int64_t)idx_stride * s.P > INT32_MAX || (int64_t)s.B * s.Hkv * idx_stride * (s.P / 16) > (1 << 30))
      return fail(SLS_EOVERFLOW, "idx_stride %d pages of %d tokens", idx_stride, s.P);
    if (!count && (k_fixed < 0 || k_fixed > idx_stride))
      return fail(SLS_EINVAL, "k_fixed %d not in [0, idx_stride=%d]", k_fixed, idx_stride);
    if (mass_out) return fail(SLS_EUNSUPPORTED, "weight sums need dense attention (page_idx NULL)");
  }
  if (mass_in && !mass_out) return fail(SLS_EINVAL, "mass_in without mass_out");
  const int64_t sums = (int64_t)s.B * s.Hkv * (s.Cap / c.block) * 4, heads = (int64_t)s.B * s.Hq;
  if (mass_in != mass_out && overlap(mass_in, sums, mass_out, sums))
    return fail(SLS_EINVAL, "mass_out must be mass_in itself or memory of its own");
  if (overlap(q, heads * s.D * 2, out, heads * s.D * 2)) return fail(SLS_EINVAL, "out shares memory with q");
  const size_t need = sls::kv8_attend_workspace(s, c, mass_out != nullptr);
  if (!workspace || workspace_bytes < need)
    return fail(SLS_EWORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
  REQUIRE16(workspace);
  const int64_t rows = (int64_t)s.B * s.Hkv, n4 = (int64_t)s.B * 4;
  const CacheSpans cs = spans_of(c, rows, s.Cap, s.D);
  if ((r = check_apart(cs, "cache"))) return r;
  // what is written: memory of its own, and none of what is read (but for mass_in, above)
  const Span to[] = {at(out, heads * s.D * 2), at(lse, heads * 4), at(mass_out, sums), at(workspace, (int64_t)need)};
  const Span in[] = {at(q, heads * s.D * 2), at(ctx_len, n4), at(page_idx, rows * idx_stride * 4), at(count, rows * 4),
                     at(sink, (int64_t)s.Hq * 4), at(mass_in == mass_out ? nullptr : mass_in, sums)};
  for (int i = 0; i < 4; ++i) {
    for (const Span& x : cs.s)
      if (overlap(to[i].p, to[i].n, x.p, x.n)) return fail(SLS_EINVAL, "an output or the workspace shares memory with the cache");
    for (const Span& x : in)
      if (overlap(to[i].p, to[i].n, x.p, x.n)) return fail(SLS_EINVAL, "an output or the workspace shares memory with an input");
    for (int j = 0; j < i; ++j)
      if (overlap(to[i].p, to[i].n, to[j].p, to[j].n)) return fail(SLS_EINVAL, "two outputs (or one and the workspace) share memory");
  }
  return cuda_status(sls::launch_kv8_attend(s, c, q, page_idx, idx_stride, count, k_fixed, ctx_len, sink, out, lse,
                                            mass_in, mass_out, workspace, (cudaStream_t)stream),
                     "sls_kv8_decode_attend");
}

sls_status sls_kv8_evict(const sls_attn_desc* desc, const sls_kv8_cache* src, int32_t dst_capacity,
                         const sls_kv8_cache* dst, int32_t keep, int32_t n_sink_blocks, int32_t n_recent_blocks,
                         const float* mass, float* mass_out, const void* kmin, const void* kmax, void* kmin_out,
                         void* kmax_out, int32_t* kept_idx, const int32_t* ctx_len, int32_t* ctx_out, void* stream) {
  sls::Shape s;
  sls::Kv8Evict e = {};
  sls_status r = check_desc(desc, &s);
  if (r || (r = check_kv8(s, src, s.Cap, "src", &e.src))) return r;
  if (!dst) dst = src;
  if ((r = check_kv8(s, dst, dst_capacity, "dst", &e.dst))) return r;
  REQUIRE(mass); REQUIRE(kept_idx); REQUIRE(ctx_len); REQUIRE(ctx_out);
  if (e.dst.format != e.src.format || e.dst.block != e.src.block)
    return fail(SLS_EINVAL, "src and dst must have the same format and block");
  if (keep < 1 || n_sink_blocks < 0 || n_recent_blocks < 0 || (int64_t)n_sink_blocks + n_recent_blocks > keep)
    return fail(SLS_EINVAL, "keep=%d must be >= 1 and hold n_sink_blocks=%d + n_recent_blocks=%d", keep, n_sink_blocks,
                n_recent_blocks);
  if (((int64_t)keep + 1) * e.src.block > dst_capacity)
    return fail(SLS_EINVAL, "dst capacity %d cannot hold keep=%d blocks of %d and a partial one", dst_capacity, keep,
                e.src.block);
  const bool same = e.dst.kc == e.src.kc;
  const int64_t rows = (int64_t)s.B * s.Hkv;
  int64_t ctas;
  if (!checked_mul(rows, 2 * (int64_t)keep + 128, &ctas) || ctas > INT32_MAX || rows * dst_capacity > (int64_t(1) << 41))
    return fail(SLS_EOVERFLOW, "too many rows");
  if (same) {
    if (e.dst.vc != e.src.vc || e.dst.ks != e.src.ks || e.dst.vs != e.src.vs || e.dst.kt != e.src.kt ||
        e.dst.vt != e.src.vt || dst_capacity != s.Cap || mass_out != mass || kmin_out != kmin ||
        kmax_out != kmax)
      return fail(SLS_EINVAL, "in place every destination must be the source's own buffer and dst_capacity Cap");
  }
  if ((kmin == nullptr) != (kmax == nullptr) || (kmin == nullptr) != (kmin_out == nullptr) ||
      (kmin == nullptr) != (kmax_out == nullptr))
    return fail(SLS_EINVAL, "kmin, kmax and their outputs: all or none");
  if (kmin) {
    REQUIRE16(kmin); REQUIRE16(kmax); REQUIRE16(kmin_out); REQUIRE16(kmax_out);
    if (s.P > e.src.block) return fail(SLS_EUNSUPPORTED, "page summaries move with blocks: page %d > block %d", s.P, e.src.block);
  }
  if (ctx_out != ctx_len && overlap(ctx_out, (int64_t)s.B * 4, ctx_len, (int64_t)s.B * 4))
    return fail(SLS_EINVAL, "ctx_out must be ctx_len itself or memory of its own");
  const int64_t st = rows * s.Cap, dt = rows * dst_capacity, bl = e.src.block, pg = (int64_t)s.D * 2;
  const CacheSpans from = spans_of(e.src, rows, s.Cap, s.D), into = spans_of(e.dst, rows, dst_capacity, s.D);
  const Span in[] = {from.s[0], from.s[1], from.s[2], from.s[3], from.s[4], from.s[5], at(mass, st / bl * 4),
                     at(kmin, st / s.P * pg), at(kmax, st / s.P * pg)};
  const Span to[] = {into.s[0], into.s[1], into.s[2], into.s[3], into.s[4], into.s[5], at(mass_out, dt / bl * 4),
                     at(kmin_out, dt / s.P * pg), at(kmax_out, dt / s.P * pg)};
  if (!same)  // no destination may share memory with what is read
    for (const Span& x : in)
      for (const Span& y : to)
        if (overlap(x.p, x.n, y.p, y.n))
          return fail(SLS_EINVAL, "source and destination share memory without being the same cache");
  // The list and the lengths are read while blocks move (the list's entries as
  // they are): nothing else may lie there.
  const Span own[] = {at(kept_idx, rows * keep * 4), at(ctx_out, (int64_t)s.B * 4), at(ctx_len, (int64_t)s.B * 4)};
  for (int i = 0; i < 9; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(in[i].p, in[i].n, in[j].p, in[j].n) || overlap(to[i].p, to[i].n, to[j].p, to[j].n))
        return fail(SLS_EINVAL, "two buffers of a cache, its sums or page summaries share memory");
    for (const Span& x : own)
      if (overlap(in[i].p, in[i].n, x.p, x.n) || overlap(to[i].p, to[i].n, x.p, x.n))
        return fail(SLS_EINVAL, "kept_idx, ctx_len and ctx_out must be memory of their own");
  }
  if (overlap(own[0].p, own[0].n, own[1].p, own[1].n) || overlap(own[0].p, own[0].n, own[2].p, own[2].n))
    return fail(SLS_EINVAL, "kept_idx must be memory of its own");
  e.cap = s.Cap; e.dcap = dst_capacity; e.keep = keep; e.n_sink = n_sink_blocks; e.n_recent = n_recent_blocks;
  e.in_place = same; e.mass = mass; e.mass_out = mass_out;
  e.kmin = kmin; e.kmax = kmax; e.kmin_out = kmin_out; e.kmax_out = kmax_out;
  e.kept = kept_idx; e.ctx_len = ctx_len; e.ctx_out = ctx_out;
  sls::stat_add(sls::kStatMetadata);
  return cuda_status(sls::launch_kv8_evict(s, e, (cudaStream_t)stream), "sls_kv8_evict");
}

}  // extern "C"
