// C ABI of the 8-bit serving operators: argument checks and launch, as
// api.cpp does for the group-wise products. Every check runs on the host
// before any launch.
#include "api_common.hpp"
#include "kernels.hpp"
#include "kv8_common.hpp"

using namespace qmm_api;

namespace {

constexpr int64_t kCounterBytes = 4 * qmm::kScratchCounters;

int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }
char* past_counters(void* work) { return static_cast<char*>(work) + kCounterBytes; }

qmm_status check_float(const char* tag, qmm_dtype dt) {
  if (dt != QMM_F16 && dt != QMM_BF16)
    return fail(QMM_E_DTYPE, "%s: only float16 and bfloat16 are supported (got dtype %d)", tag,
                (int)dt);
  return QMM_OK;
}

qmm_status check_work(const char* tag, const void* work, int64_t have, int64_t need) {
  if (need > 0 && !work) return fail(QMM_E_NULL, "%s: work must be non-NULL", tag);
  if (have < need)
    return fail(QMM_E_ARG, "%s: work holds %lld bytes, %lld are needed", tag, (long long)have,
                (long long)need);
  if (!aligned(work, 16)) return fail(QMM_E_ALIGN, "%s: work must be 16-byte aligned", tag);
  return QMM_OK;
}

qmm_status check_i8_sizes(const char* tag, int64_t M, int64_t N, int64_t K) {
  if (M < 1 || N < 1 || M > kI32 || N > kI32)
    return fail(QMM_E_SHAPE, "%s: M (%lld) and N (%lld) must be in [1, 2^31)", tag, (long long)M,
                (long long)N);
  if (K < 16 || K % 16 != 0 || K >= (1 << 17))
    return fail(QMM_E_SHAPE,
                "%s: K (%lld) must be a multiple of 16 below 2^17 (pad with zeros; the sums stay "
                "exact in 32 bits)",
                tag, (long long)K);
  if (M * N > ((int64_t)1 << 40)) return fail(QMM_E_SHAPE, "%s: problem too large", tag);
  const int64_t grid = ((M + 127) / 128) * ((N + 127) / 128);
  if (grid > kI32) return fail(QMM_E_SHAPE, "%s: problem too large", tag);
  return QMM_OK;
}

qmm_status check_i8_rows(const char* tag, const void* x, int64_t ldx, int64_t K) {
  if (!aligned(x, 16)) return fail(QMM_E_ALIGN, "%s: x must be 16-byte aligned", tag);
  if (ldx < K || ldx % 8 != 0)
    return fail(QMM_E_SHAPE, "%s: the row stride of x (%lld) must be a multiple of 8, not below K",
                tag, (long long)ldx);
  return QMM_OK;
}

qmm_status check_cache(const char* tag, const qmm_kv8_cache* c, qmm::Kv8* out) {
  if (!c || !c->k || !c->v || !c->k_scales || !c->v_scales)
    return fail(QMM_E_NULL, "%s: the cache and its four arrays must be non-NULL", tag);
  if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64)
    return fail(QMM_E_SHAPE, "%s: page_tokens must be 16, 32 or 64 (got %d)", tag, c->page_tokens);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return fail(QMM_E_SHAPE, "%s: head_dim must be 64, 128 or 256 (got %d)", tag, c->head_dim);
  if (c->heads < 1 || c->heads > 1024)
    return fail(QMM_E_SHAPE, "%s: heads (%d) must be in [1, 1024]", tag, c->heads);
  if (c->pages < 1 || c->pages > (1 << 28))
    return fail(QMM_E_SHAPE, "%s: pages (%lld) must be in [1, 2^28]", tag, (long long)c->pages);
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scales, 4) ||
      !aligned(c->v_scales, 4))
    return fail(QMM_E_ALIGN, "%s: k and v must be 16-byte aligned, the scales 4-byte", tag);
  *out = {c->k, c->v, c->k_scales, c->v_scales, (int)c->pages, c->heads,
          c->page_tokens == 16 ? 4 : c->page_tokens == 32 ? 5 : 6, c->head_dim};
  return QMM_OK;
}

qmm_status check_rows(const char* tag, const char* name, const void* p, int64_t ld, int64_t width) {
  if (!aligned(p, 16)) return fail(QMM_E_ALIGN, "%s: %s must be 16-byte aligned", tag, name);
  if (ld < width || ld % 8 != 0)
    return fail(QMM_E_SHAPE,
                "%s: the token stride of %s (%lld) must be a multiple of 8, not below %lld", tag,
                name, (long long)ld, (long long)width);
  return QMM_OK;
}

qmm_status check_batch(const char* tag, int64_t T, int64_t S, int64_t W) {
  if (T < 1 || T > (1 << 24) || S < 1 || S > 65535 || W < 1 || W > (1 << 24))
    return fail(QMM_E_SHAPE,
                "%s: tokens (%lld) must be in [1, 2^24], sequences (%lld) in [1, 65535], table "
                "columns (%lld) in [1, 2^24]",
                tag, (long long)T, (long long)S, (long long)W);
  return QMM_OK;
}

bool aligned4(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned(p, 4)) return false;
  return true;
}
bool any_null(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!p) return true;
  return false;
}

// what the calls of the attention have in common; `work` and `go` are the
// mask's own
template <class Work, class Go>
qmm_status attention(const char* tag, const qmm_kv8_cache* cache, const void* q, int64_t ldq,
                     qmm_dtype dt, int64_t T, int64_t q_heads, const int32_t* table,
                     const int32_t* lens, const int32_t* cu, int64_t S, int64_t W, void* out,
                     float* lse, void* work, int64_t work_bytes, void* stream, Work need_of,
                     Go go) {
  if (qmm_status s = check_stream(tag, stream)) return s;
  qmm::Kv8 c;
  if (qmm_status s = check_cache(tag, cache, &c)) return s;
  if (any_null({q, table, lens, cu, out}))
    return fail(QMM_E_NULL, "%s: q, table, lens, cu and out must be non-NULL", tag);
  if (qmm_status s = check_float(tag, dt)) return s;
  if (qmm_status s = check_batch(tag, T, S, W)) return s;
  if (q_heads < c.heads || q_heads % c.heads != 0 || q_heads > 65535)
    return fail(QMM_E_SHAPE, "%s: q_heads (%lld) must be a multiple of the cache's heads (%d)", tag,
                (long long)q_heads, c.heads);
  if (T * q_heads > kI32) return fail(QMM_E_SHAPE, "%s: problem too large", tag);
  if (qmm_status s = check_rows(tag, "q", q, ldq, q_heads * c.dim)) return s;
  if (!aligned4({table, lens, cu, lse}) || !aligned(out, 16))
    return fail(QMM_E_ALIGN, "%s: out must be 16-byte aligned, table, lens, cu and lse 4-byte", tag);
  const int64_t need = need_of(c);
  if (qmm_status s = check_work(tag, work, work_bytes, need > 0 ? kCounterBytes + need : 0)) return s;
  return launched(go(c, work ? reinterpret_cast<float*>(past_counters(work)) : nullptr), tag);
}

}  // namespace

extern "C" {

qmm_status qmm_i8_quantize(const void* x, int64_t ldx, qmm_dtype dt, int64_t rows, int64_t K,
                           int8_t* codes, float* scales, void* stream) {
  const char* tag = "qmm_i8_quantize";
  if (qmm_status s = check_stream(tag, stream)) return s;
  if (any_null({x, codes, scales}))
    return fail(QMM_E_NULL, "%s: x, codes and scales must be non-NULL", tag);
  if (qmm_status s = check_float(tag, dt)) return s;
  if (qmm_status s = check_i8_sizes(tag, rows, 1, K)) return s;
  if (qmm_status s = check_i8_rows(tag, x, ldx, K)) return s;
  if (!aligned(codes, 16) || !aligned(scales, 4))
    return fail(QMM_E_ALIGN, "%s: codes must be 16-byte aligned, scales 4-byte", tag);
  return launched(qmm::launch_i8_quantize((int)dt, x, ldx, rows, K, codes, scales,
                                          (hipStream_t)stream),
                  tag);
}

int64_t qmm_i8_t_work(int64_t M, int64_t N, int64_t K) {
  if (M < 1 || N < 1 || K < 16) return 0;
  const int64_t b = qmm::i8_plan(M, N, K).ws_bytes;
  return b > 0 ? kCounterBytes + b : 0;
}

int64_t qmm_i8_linear_work(int64_t M, int64_t N, int64_t K) {
  if (M < 1 || N < 1 || K < 16 || qmm::i8_fused(M, K)) return 0;
  return kCounterBytes + up16(M * K) + up16(4 * M) + qmm::i8_plan(M, N, K).ws_bytes;
}

static qmm_status i8_common(const char* tag, const int8_t* wq, const float* sw, const void* bias,
                            qmm_dtype dt, int64_t M, int64_t N, int64_t K, const void* y) {
  if (any_null({wq, sw, y})) return fail(QMM_E_NULL, "%s: wq, sw and y must be non-NULL", tag);
  if (qmm_status s = check_float(tag, dt)) return s;
  if (qmm_status s = check_i8_sizes(tag, M, N, K)) return s;
  if (!aligned(wq, 16) || !aligned(y, 16) || !aligned(sw, 4) || !aligned(bias, 2))
    return fail(QMM_E_ALIGN, "%s: wq and y must be 16-byte aligned, sw 4-byte, bias 2-byte", tag);
  return QMM_OK;
}

qmm_status qmm_i8_t(const int8_t* xq, const float* sx, const int8_t* wq, const float* sw,
                    const void* bias, qmm_dtype dt, int64_t M, int64_t N, int64_t K, void* y,
                    void* work, int64_t work_bytes, void* stream) {
  const char* tag = "qmm_i8_t";
  if (qmm_status s = check_stream(tag, stream)) return s;
  if (any_null({xq, sx})) return fail(QMM_E_NULL, "%s: xq and sx must be non-NULL", tag);
  if (qmm_status s = i8_common(tag, wq, sw, bias, dt, M, N, K, y)) return s;
  if (!aligned(xq, 16) || !aligned(sx, 4))
    return fail(QMM_E_ALIGN, "%s: xq must be 16-byte aligned, sx 4-byte", tag);
  if (qmm_status s = check_work(tag, work, work_bytes, qmm_i8_t_work(M, N, K))) return s;
  return launched(qmm::launch_i8_t((int)dt, xq, sx, wq, sw, bias, M, N, K, y,
                                   static_cast<unsigned*>(work),
                                   work ? reinterpret_cast<int*>(past_counters(work)) : nullptr,
                                   (hipStream_t)stream),
                  tag);
}

qmm_status qmm_i8_linear(const void* x, int64_t ldx, const int8_t* wq, const float* sw,
                         const void* bias, qmm_dtype dt, int64_t M, int64_t N, int64_t K, void* y,
                         void* work, int64_t work_bytes, void* stream) {
  const char* tag = "qmm_i8_linear";
  if (qmm_status s = check_stream(tag, stream)) return s;
  if (!x) return fail(QMM_E_NULL, "%s: x must be non-NULL", tag);
  if (qmm_status s = i8_common(tag, wq, sw, bias, dt, M, N, K, y)) return s;
  if (qmm_status s = check_i8_rows(tag, x, ldx, K)) return s;
  if (qmm_status s = check_work(tag, work, work_bytes, qmm_i8_linear_work(M, N, K))) return s;
  if (qmm::i8_fused(M, K))
    return launched(qmm::launch_i8_fused((int)dt, x, ldx, wq, sw, bias, M, N, K, y,
                                         (hipStream_t)stream),
                    tag);
  char* p = past_counters(work);
  int8_t* xq = reinterpret_cast<int8_t*>(p);
  float* sx = reinterpret_cast<float*>(p + up16(M * K));
  int* ws = reinterpret_cast<int*>(p + up16(M * K) + up16(4 * M));
  const hipStream_t st = (hipStream_t)stream;
  hipError_t e = qmm::launch_i8_quantize((int)dt, x, ldx, M, K, xq, sx, st);
  if (e == hipSuccess)
    e = qmm::launch_i8_t((int)dt, xq, sx, wq, sw, bias, M, N, K, y, static_cast<unsigned*>(work),
                         ws, st);
  return launched(e, tag);
}

qmm_status qmm_kv8_append(const qmm_kv8_cache* cache, const void* k, int64_t ldk, const void* v,
                          int64_t ldv, qmm_dtype dt, int64_t T, const int32_t* table,
                          const int32_t* lens, const int32_t* cu, int64_t S, int64_t W,
                          void* stream) {
  const char* tag = "qmm_kv8_append";
  if (qmm_status s = check_stream(tag, stream)) return s;
  qmm::Kv8 c;
  if (qmm_status s = check_cache(tag, cache, &c)) return s;
  if (any_null({k, v, table, lens, cu}))
    return fail(QMM_E_NULL, "%s: k, v, table, lens and cu must be non-NULL", tag);
  if (qmm_status s = check_float(tag, dt)) return s;
  if (qmm_status s = check_batch(tag, T, S, W)) return s;
  const int64_t width = (int64_t)c.heads * c.dim;
  if (qmm_status s = check_rows(tag, "k", k, ldk, width)) return s;
  if (qmm_status s = check_rows(tag, "v", v, ldv, width)) return s;
  if (!aligned4({table, lens, cu}))
    return fail(QMM_E_ALIGN, "%s: table, lens and cu must be 4-byte aligned", tag);
  return launched(qmm::launch_kv8_append(c, (int)dt, k, ldk, v, ldv, T, table, lens, cu, S, W,
                                         (hipStream_t)stream),
                  tag);
}

qmm_status qmm_kv8_read(const qmm_kv8_cache* cache, const int32_t* pages, int64_t n, qmm_dtype dt,
                        void* k, void* v, void* stream) {
  const char* tag = "qmm_kv8_read";
  if (qmm_status s = check_stream(tag, stream)) return s;
  qmm::Kv8 c;
  if (qmm_status s = check_cache(tag, cache, &c)) return s;
  if (any_null({pages, k, v}))
    return fail(QMM_E_NULL, "%s: pages, k and v must be non-NULL", tag);
  if (qmm_status s = check_float(tag, dt)) return s;
  if (n < 1 || n > kI32) return fail(QMM_E_SHAPE, "%s: n (%lld) must be in [1, 2^31)", tag, (long long)n);
  if (!aligned(pages, 4) || !aligned(k, 16) || !aligned(v, 16))
    return fail(QMM_E_ALIGN, "%s: k and v must be 16-byte aligned, pages 4-byte", tag);
  return launched(qmm::launch_kv8_read(c, (int)dt, pages, n, k, v, (hipStream_t)stream), tag);
}

int64_t qmm_kv8_attention_work(const qmm_kv8_cache* cache, int64_t T, int64_t q_heads, int64_t S,
                               int64_t W) {
  qmm::Kv8 c;
  if (check_cache("qmm_kv8_attention_work", cache, &c) ||
      check_batch("qmm_kv8_attention_work", T, S, W) || q_heads < c.heads)
    return 0;
  const int64_t b = qmm::kv8_attention_work(c, T, q_heads, S, W);
  return b > 0 ? kCounterBytes + b : 0;
}

qmm_status qmm_kv8_attention(const qmm_kv8_cache* cache, const void* q, int64_t ldq, qmm_dtype dt,
                             int64_t T, int64_t q_heads, const int32_t* table, const int32_t* lens,
                             const int32_t* cu, int64_t S, int64_t W, float scale, void* out,
                             float* lse, void* work, int64_t work_bytes, void* stream) {
  return attention(
      "qmm_kv8_attention", cache, q, ldq, dt, T, q_heads, table, lens, cu, S, W, out, lse, work,
      work_bytes, stream,
      [&](const qmm::Kv8& c) { return qmm::kv8_attention_work(c, T, q_heads, S, W); },
      [&](const qmm::Kv8& c, float* ws) {
        return qmm::launch_kv8_attention(c, (int)dt, q, ldq, T, q_heads, table, lens, cu, S, W,
                                         scale, out, lse, ws, (hipStream_t)stream);
      });
}

// positions stay below 2^30, so that a longer window or more sinks see no more
static int64_t cap30(int64_t n) { return n < ((int64_t)1 << 30) ? n : (int64_t)1 << 30; }

int64_t qmm_kv8_attention_window_work(const qmm_kv8_cache* cache, int64_t T, int64_t q_heads,
                                      int64_t S, int64_t W, int64_t window, int64_t sinks) {
  qmm::Kv8 c;
  if (check_cache("qmm_kv8_attention_window_work", cache, &c) ||
      check_batch("qmm_kv8_attention_window_work", T, S, W) || q_heads < c.heads || window < 1 ||
      sinks < 0)
    return 0;
  const int64_t b = qmm::kv8_attention_window_work(c, T, q_heads, S, W, cap30(window), cap30(sinks));
  return b > 0 ? kCounterBytes + b : 0;
}

qmm_status qmm_kv8_attention_window(const qmm_kv8_cache* cache, const void* q, int64_t ldq,
                                    qmm_dtype dt, int64_t T, int64_t q_heads, const int32_t* table,
                                    const int32_t* lens, const int32_t* cu, int64_t S, int64_t W,
                                    int64_t window, int64_t sinks, float scale, void* out, float* lse,
                                    void* work, int64_t work_bytes, void* stream) {
  const char* tag = "qmm_kv8_attention_window";
  if (window < 1 || sinks < 0)
    return fail(QMM_E_ARG, "%s: window (%lld) must be at least 1 and sinks (%lld) at least 0", tag,
                (long long)window, (long long)sinks);
  const int64_t w = cap30(window), n = cap30(sinks);
  return attention(
      tag, cache, q, ldq, dt, T, q_heads, table, lens, cu, S, W, out, lse, work, work_bytes, stream,
      [&](const qmm::Kv8& c) { return qmm::kv8_attention_window_work(c, T, q_heads, S, W, w, n); },
      [&](const qmm::Kv8& c, float* ws) {
        return qmm::launch_kv8_attention_window(c, (int)dt, q, ldq, T, q_heads, table, lens, cu, S,
                                                W, w, n, scale, out, lse, ws, (hipStream_t)stream);
      });
}

int64_t qmm_kv8_attention_tree_work(const qmm_kv8_cache* cache, int64_t T, int64_t q_heads, int64_t S,
                                    int64_t W) {
  qmm::Kv8 c;
  if (check_cache("qmm_kv8_attention_tree_work", cache, &c) ||
      check_batch("qmm_kv8_attention_tree_work", T, S, W) || q_heads < c.heads)
    return 0;
  const int64_t b = qmm::kv8_attention_tree_work(c, T, q_heads, S, W);
  return b > 0 ? kCounterBytes + b : 0;
}

qmm_status qmm_kv8_attention_tree(const qmm_kv8_cache* cache, const void* q, int64_t ldq,
                                  qmm_dtype dt, int64_t T, int64_t q_heads, const int32_t* table,
                                  const int32_t* lens, const int32_t* cu, int64_t S, int64_t W,
                                  const int32_t* parent, float scale, void* out, float* lse,
                                  void* work, int64_t work_bytes, void* stream) {
  const char* tag = "qmm_kv8_attention_tree";
  if (!parent) return fail(QMM_E_NULL, "%s: parent must be non-NULL", tag);
  if (!aligned(parent, 4)) return fail(QMM_E_ALIGN, "%s: parent must be 4-byte aligned", tag);
  return attention(
      tag, cache, q, ldq, dt, T, q_heads, table, lens, cu, S, W, out, lse, work, work_bytes, stream,
      [&](const qmm::Kv8& c) { return qmm::kv8_attention_tree_work(c, T, q_heads, S, W); },
      [&](const qmm::Kv8& c, float* ws) {
        return qmm::launch_kv8_attention_tree(c, (int)dt, q, ldq, T, q_heads, table, lens, cu, S, W,
                                              parent, scale, out, lse, ws, (hipStream_t)stream);
      });
}

int64_t qmm_kv8_pages_work(int64_t pages) {
  return pages < 1 ? 0 : kCounterBytes + qmm::kv8_pages_work(pages);
}

qmm_status qmm_kv8_update(const qmm_kv8_cache* cache, const int32_t* ref, const int32_t* table,
                          const int32_t* lens, const int32_t* parent, const int32_t* new_lens,
                          int64_t S, int64_t W, int32_t* ref_out, int32_t* table_out,
                          int32_t* shortage, void* work, int64_t work_bytes, void* stream) {
  const char* tag = "qmm_kv8_update";
  if (qmm_status s = check_stream(tag, stream)) return s;
  qmm::Kv8 c;
  if (qmm_status s = check_cache(tag, cache, &c)) return s;
  if (any_null({ref, table, lens, parent, new_lens, ref_out, table_out, shortage}))
    return fail(QMM_E_NULL, "%s: every array must be non-NULL", tag);
  if (qmm_status s = check_batch(tag, 1, S, W)) return s;
  if (ref_out == ref || table_out == table)
    return fail(QMM_E_ARG, "%s: the new counts and table must be arrays of their own", tag);
  if (!aligned4({ref, table, lens, parent, new_lens, ref_out, table_out, shortage}))
    return fail(QMM_E_ALIGN, "%s: arrays must be 4-byte aligned", tag);
  if (qmm_status s = check_work(tag, work, work_bytes, qmm_kv8_pages_work(c.pages))) return s;
  return launched(qmm::launch_kv8_update(c, ref, table, lens, parent, new_lens, S, W, ref_out,
                                         table_out, shortage,
                                         reinterpret_cast<int32_t*>(past_counters(work)),
                                         (hipStream_t)stream),
                  tag);
}

qmm_status qmm_kv8_compact(const qmm_kv8_cache* cache, const int32_t* ref, const int32_t* table,
                           int64_t S, int64_t W, int32_t* ref_out, int32_t* table_out,
                           int32_t* remap, int32_t* used, void* work, int64_t work_bytes,
                           void* stream) {
  const char* tag = "qmm_kv8_compact";
  if (qmm_status s = check_stream(tag, stream)) return s;
  qmm::Kv8 c;
  if (qmm_status s = check_cache(tag, cache, &c)) return s;
  if (any_null({ref, table, ref_out, table_out, remap, used}))
    return fail(QMM_E_NULL, "%s: every array must be non-NULL", tag);
  if (qmm_status s = check_batch(tag, 1, S, W)) return s;
  if (ref_out == ref) return fail(QMM_E_ARG, "%s: the new counts must be an array of their own", tag);
  if (!aligned4({ref, table, ref_out, table_out, remap, used}))
    return fail(QMM_E_ALIGN, "%s: arrays must be 4-byte aligned", tag);
  if (qmm_status s = check_work(tag, work, work_bytes, qmm_kv8_pages_work(c.pages))) return s;
  return launched(qmm::launch_kv8_compact(c, ref, table, S, W, ref_out, table_out, remap, used,
                                          reinterpret_cast<int32_t*>(past_counters(work)),
                                          (hipStream_t)stream),
                  tag);
}

qmm_status qmm_kv8_copy(const qmm_kv8_cache* to, const int32_t* dst, const qmm_kv8_cache* from,
                        const int32_t* src, int64_t n, void* stream) {
  const char* tag = "qmm_kv8_copy";
  if (qmm_status s = check_stream(tag, stream)) return s;
  qmm::Kv8 a, b;
  if (qmm_status s = check_cache(tag, to, &a)) return s;
  if (qmm_status s = check_cache(tag, from, &b)) return s;
  if (any_null({dst, src})) return fail(QMM_E_NULL, "%s: dst and src must be non-NULL", tag);
  if (a.heads != b.heads || a.bt_log2 != b.bt_log2 || a.dim != b.dim)
    return fail(QMM_E_SHAPE, "%s: the caches' pages differ in shape", tag);
  if (n < 1 || n > kI32) return fail(QMM_E_SHAPE, "%s: n (%lld) must be in [1, 2^31)", tag, (long long)n);
  if (!aligned4({dst, src})) return fail(QMM_E_ALIGN, "%s: dst and src must be 4-byte aligned", tag);
  return launched(qmm::launch_kv8_copy(a, b, dst, src, n, (hipStream_t)stream), tag);
}

qmm_status qmm_qk_norm_rope(const void* q, int64_t ldq, const void* k, int64_t ldk, qmm_dtype dt,
                            int64_t T, int64_t q_heads, int64_t k_heads, int64_t head_dim,
                            const int32_t* positions, const float* inv_freq, int64_t rot_dim,
                            int interleaved, const void* q_weight, const void* k_weight, float eps,
                            void* q_out, int64_t ldqo, void* k_out, int64_t ldko, void* stream) {
  const char* tag = "qmm_qk_norm_rope";
  if (qmm_status s = check_stream(tag, stream)) return s;
  if (any_null({q, k, positions, inv_freq, q_out, k_out}))
    return fail(QMM_E_NULL, "%s: q, k, positions, inv_freq, q_out and k_out must be non-NULL", tag);
  if (qmm_status s = check_float(tag, dt)) return s;
  if (T < 1 || T > (1 << 24))
    return fail(QMM_E_SHAPE, "%s: tokens (%lld) must be in [1, 2^24]", tag, (long long)T);
  if (q_heads < 1 || k_heads < 1 || q_heads > 65535 || k_heads > 65535)
    return fail(QMM_E_SHAPE, "%s: q_heads (%lld) and k_heads (%lld) must be in [1, 65535]", tag,
                (long long)q_heads, (long long)k_heads);
  if (head_dim < 8 || head_dim > 512 || head_dim % 8 != 0 || rot_dim < 8 || rot_dim > head_dim ||
      rot_dim % 8 != 0)
    return fail(QMM_E_SHAPE,
                "%s: head_dim (%lld) must be a multiple of 8 up to 512, rot_dim (%lld) one up to "
                "head_dim",
                tag, (long long)head_dim, (long long)rot_dim);
  if (T * (q_heads + k_heads) > kI32) return fail(QMM_E_SHAPE, "%s: problem too large", tag);
  const int64_t wide_q = q_heads * head_dim, wide_k = k_heads * head_dim;
  if (qmm_status s = check_rows(tag, "q", q, ldq, wide_q)) return s;
  if (qmm_status s = check_rows(tag, "k", k, ldk, wide_k)) return s;
  if (qmm_status s = check_rows(tag, "q_out", q_out, ldqo, wide_q)) return s;
  if (qmm_status s = check_rows(tag, "k_out", k_out, ldko, wide_k)) return s;
  if (!aligned(inv_freq, 16) || !aligned(q_weight, 16) || !aligned(k_weight, 16) ||
      !aligned(positions, 4))
    return fail(QMM_E_ALIGN, "%s: inv_freq and weights must be 16-byte aligned, positions 4-byte",
                tag);
  if (!(eps >= 0.0f)) return fail(QMM_E_ARG, "%s: eps must not be negative", tag);
  if ((q_out == q && ldqo != ldq) || (k_out == k && ldko != ldk) || q_out == k || k_out == q ||
      q_out == k_out)
    return fail(QMM_E_ARG,
                "%s: an output may be its own input with the same stride, and no other array", tag);
  return launched(qmm::launch_qk_norm_rope((int)dt, q, ldq, k, ldk, T, q_heads, k_heads, head_dim,
                                           positions, inv_freq, rot_dim, interleaved != 0, q_weight,
                                           k_weight, eps, q_out, ldqo, k_out, ldko,
                                           (hipStream_t)stream),
                  tag);
}

static bool logprobs_sizes(qmm_dtype dt, int64_t M, int64_t V, int64_t top) {
  return (dt == QMM_F16 || dt == QMM_BF16 || dt == QMM_F32) && M >= 1 && M <= (1 << 23) && V >= 1 &&
         V <= (1 << 30) && top >= 0 && top <= 64 && top <= V;
}

int64_t qmm_logprobs_work(qmm_dtype dt, int64_t M, int64_t V, int64_t top) {
  if (!logprobs_sizes(dt, M, V, top)) return 0;
  const int64_t b = qmm::logprobs_work((int)dt, M, V, top);
  return b > 0 ? kCounterBytes + b : 0;
}

qmm_status qmm_logprobs(const void* logits, int64_t ld, qmm_dtype dt, int64_t M, int64_t V,
                        const int32_t* tokens, int64_t top, float* logprob, float* entropy,
                        int32_t* top_ids, float* top_logprobs, void* work, int64_t work_bytes,
                        void* stream) {
  const char* tag = "qmm_logprobs";
  if (qmm_status s = check_stream(tag, stream)) return s;
  if (any_null({logits, tokens, logprob, entropy}) || (top > 0 && any_null({top_ids, top_logprobs})))
    return fail(QMM_E_NULL,
                "%s: logits, tokens, logprob and entropy (with top > 0 also top_ids and "
                "top_logprobs) must be non-NULL",
                tag);
  if (dt != QMM_F16 && dt != QMM_BF16 && dt != QMM_F32)
    return fail(QMM_E_DTYPE, "%s: only float16, bfloat16 and float32 are supported (got dtype %d)",
                tag, (int)dt);
  if (!logprobs_sizes(dt, M, V, top))
    return fail(QMM_E_SHAPE,
                "%s: rows (%lld) must be in [1, 2^23], V (%lld) in [1, 2^30], top (%lld) in [0, 64] "
                "and at most V",
                tag, (long long)M, (long long)V, (long long)top);
  if (ld < V)
    return fail(QMM_E_SHAPE, "%s: the row stride (%lld) must not be below V", tag, (long long)ld);
  if (!aligned(logits, elem_bytes(dt)) ||
      !aligned4({tokens, logprob, entropy, top_ids, top_logprobs}))
    return fail(QMM_E_ALIGN, "%s: logits must be aligned to their type, the others 4-byte", tag);
  if (qmm_status s = check_work(tag, work, work_bytes, qmm_logprobs_work(dt, M, V, top))) return s;
  return launched(qmm::launch_logprobs((int)dt, logits, ld, M, V, tokens, top, logprob, entropy,
                                       top_ids, top_logprobs, work ? past_counters(work) : nullptr,
                                       (hipStream_t)stream),
                  tag);
}

}  // extern "C"
