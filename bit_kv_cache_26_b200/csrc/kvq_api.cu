// C-ABI entry points of libkvq (declared in include/kvq.h): host-side argument
// validation, workspace sizing and kernel launches.  No exception crosses the
// ABI; nothing here allocates device memory.
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "kvq_common.cuh"
#include "kvq_internal.h"

namespace {

thread_local char g_err[512] = "";

kvq_status fail(kvq_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return st;
}

kvq_status cuda_fail(cudaError_t e, const char* where) {
  return fail(KVQ_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

int num_sms() {
  static std::atomic<int> known[64];  // per device, asked once
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) != cudaSuccess) return sms;
  const bool kept = dev >= 0 && dev < 64;
  if (kept && known[dev].load(std::memory_order_relaxed) > 0) return known[dev].load(std::memory_order_relaxed);
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) return 148;
  if (kept) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

// Whether two of the n x m rows of 128 elements at i * si + j * sj share an element.
bool rows_overlap(int64_t n, int64_t si, int64_t m, int64_t sj) {
  if ((n > 1 && si < 128) || (m > 1 && sj < 128)) return true;
  if (n == 1 || m == 1) return false;
  if (si >= 128 && (si - 128) / sj >= m - 1) return false;  // all of one dimension within a step of the other, as usual
  if (sj >= 128 && (sj - 128) / si >= n - 1) return false;
  for (int64_t j = 1; j < m; ++j) {  // the multiples of si on both sides of j * sj
    const int64_t i = j * (sj / si) + j * (sj % si) / si, over = j * (sj % si) % si;
    if ((i < n && over < 128) || (i + 1 < n && si - over < 128)) return true;
  }
  return false;
}

kvq_status check_cache(const kvq_cache* c) {
  if (!c) return fail(KVQ_ERR_INVALID_ARG, "cache is NULL");
  if (c->head_dim != 128) return fail(KVQ_ERR_UNSUPPORTED, "head_dim %d unsupported (only 128)", c->head_dim);
  if (c->group != 32) return fail(KVQ_ERR_UNSUPPORTED, "group %d unsupported (only 32)", c->group);
  if (c->bits != 2 && c->bits != 4) return fail(KVQ_ERR_UNSUPPORTED, "bits %d unsupported (2 or 4)", c->bits);
  if (c->num_patterns < 1 || c->num_patterns > 255)
    return fail(KVQ_ERR_UNSUPPORTED, "num_patterns %d outside 1..255", c->num_patterns);
  if (c->dtype != KVQ_F16 && c->dtype != KVQ_BF16) return fail(KVQ_ERR_UNSUPPORTED, "dtype %d", c->dtype);
  if (c->transform != KVQ_TX_NONE && c->transform != KVQ_TX_HADAMARD_VARNORM)
    return fail(KVQ_ERR_UNSUPPORTED, "transform %d", c->transform);
  if (!(c->v_rho >= 0.0f) || !(c->v_rho < INFINITY))
    return fail(KVQ_ERR_INVALID_ARG, "v_rho must be finite and >= 0 (0 = adaptive threshold off)");
  if (c->reserved != 0) return fail(KVQ_ERR_INVALID_ARG, "reserved field must be 0");
  if (c->pattern_window_len < 0) return fail(KVQ_ERR_INVALID_ARG, "pattern_window_len %d < 0", c->pattern_window_len);
  if (c->pattern_window_len > 0 && (!c->pattern_counts || !c->pattern_window))
    return fail(KVQ_ERR_INVALID_ARG, "pattern insertion needs pattern_counts and pattern_window");
  if (c->num_seqs < 0 || c->num_kv_heads < 1 || c->num_sets < 1 || c->max_pages_per_seq < 0 || c->num_pages < 0)
    return fail(KVQ_ERR_INVALID_ARG, "negative or zero size in cache (seqs %d heads %d sets %d pages %d/%d)",
                c->num_seqs, c->num_kv_heads, c->num_sets, c->max_pages_per_seq, c->num_pages);
  // sequences and KV heads index the z and y dimensions of the launch grids
  if (c->num_seqs > 65535 || c->num_kv_heads > 65535)
    return fail(KVQ_ERR_CAPACITY, "%d sequences / %d KV heads exceed the 65535 the launch grids allow", c->num_seqs,
                c->num_kv_heads);
  if (c->num_seqs > 0) {
    if (!c->page_pool || !c->page_table || !c->seq_len || !c->k_tail || !c->k_patterns || !c->v_patterns ||
        !c->status)
      return fail(KVQ_ERR_INVALID_ARG, "a required cache pointer is NULL");
    if (!aligned(c->page_pool, 256)) return fail(KVQ_ERR_INVALID_ARG, "page_pool must be 256-byte aligned");
    if (!aligned(c->k_tail, 16) || !aligned(c->k_patterns, 16) || !aligned(c->v_patterns, 16))
      return fail(KVQ_ERR_INVALID_ARG, "k_tail / patterns must be 16-byte aligned");
    if (c->transform && (!c->k_colscale || !c->v_colscale))
      return fail(KVQ_ERR_INVALID_ARG, "transform enabled but colscale pointers are NULL");
  }
  return KVQ_OK;
}

}  // namespace

extern "C" {

const char* kvq_last_error(void) { return g_err; }

const char* kvq_version(void) { return "kvq 0.1 (sm_100a)"; }

float kvq_v_rho_star(int32_t head_dim, double alpha) {
  if (!(alpha > 0.0) || !(alpha < 0.5) || head_dim < 1) return 0.0f;
  // z = Phi^-1(1 - alpha) by bisection on the upper tail 0.5 erfc(z / sqrt 2)
  double lo = 0.0, hi = 40.0;
  for (int it = 0; it < 200; ++it) {
    const double mid = 0.5 * (lo + hi);
    (0.5 * erfc(mid / sqrt(2.0)) > alpha ? lo : hi) = mid;
  }
  const double z = 0.5 * (lo + hi);
  // Eq. 10 with equality, u = rho^2, k = 2 z / sqrt(5 d): (1 - k^2) u^2 - 2 u + (1 - k^2) = 0
  const double k = 2.0 * z / sqrt(5.0 * head_dim), a = 1.0 - k * k;
  if (!(a > 0.0)) return 0.0f;
  const double u = (1.0 - sqrt(1.0 - a * a)) / a;
  return (float)sqrt(u);
}

size_t kvq_subblock_bytes(int32_t bits, int32_t transform) {
  if (bits != 2 && bits != 4) return 0;
  return (size_t)kvq::subblock_bytes_of(bits, transform ? 1 : 0);
}

size_t kvq_page_bytes(const kvq_cache* c) {
  if (!c || c->num_kv_heads < 1) return 0;
  size_t s = kvq_subblock_bytes(c->bits, c->transform);
  return s * (size_t)c->num_kv_heads;
}

size_t kvq_mine_workspace_bytes(int64_t n, int32_t num_sets, int32_t num_kv_heads, int32_t P, int32_t transform) {
  if (n < 0 || num_sets < 0 || num_kv_heads < 0 || P < 1) return 0;
  return kvq::mine_workspace(n, num_sets, num_kv_heads, P, transform ? 1 : 0);
}

kvq_status kvq_mine_patterns(const void* x, int32_t dtype, int64_t n, int32_t num_sets, int32_t num_kv_heads,
                             int64_t tok_stride, int64_t head_stride, int64_t set_stride, int32_t P,
                             int32_t iters, int32_t transform, float* patterns_out, float* colscale_out,
                             int32_t* assign_out, void* ws, size_t ws_bytes, kvq_stream_t stream) {
  g_err[0] = 0;
  if (dtype != KVQ_F16 && dtype != KVQ_BF16) return fail(KVQ_ERR_UNSUPPORTED, "dtype %d", dtype);
  if (transform != KVQ_TX_NONE && transform != KVQ_TX_HADAMARD_VARNORM)
    return fail(KVQ_ERR_UNSUPPORTED, "transform %d", transform);
  if (P < 1 || P > 255) return fail(KVQ_ERR_UNSUPPORTED, "P %d outside 1..255", P);
  if (num_sets < 0 || num_kv_heads < 0 || iters < 0 || n < 0)
    return fail(KVQ_ERR_INVALID_ARG, "negative size (n %lld sets %d heads %d iters %d)", (long long)n, num_sets,
                num_kv_heads, iters);
  if (num_sets == 0 || num_kv_heads == 0) return KVQ_OK;
  if (n < P) return fail(KVQ_ERR_INVALID_ARG, "n = %lld tokens is fewer than P = %d patterns", (long long)n, P);
  if (n > (int64_t)1 << 31) return fail(KVQ_ERR_CAPACITY, "n = %lld exceeds 2^31", (long long)n);
  // (set, KV head) problems index the y / z dimension of the mining grids
  if ((int64_t)num_sets * num_kv_heads > 65535)
    return fail(KVQ_ERR_CAPACITY, "%d sets x %d KV heads exceed the 65535 problems the launch grids allow", num_sets,
                num_kv_heads);
  if (!x || !patterns_out) return fail(KVQ_ERR_INVALID_ARG, "x / patterns_out is NULL");
  if (transform && !colscale_out) return fail(KVQ_ERR_INVALID_ARG, "transform needs colscale_out");
  if (tok_stride < 0 || head_stride < 0 || set_stride < 0)
    return fail(KVQ_ERR_INVALID_ARG, "negative stride");
  if (!aligned(x, 16) || tok_stride % 8 || head_stride % 8 || set_stride % 8)
    return fail(KVQ_ERR_INVALID_ARG, "x must be 16-byte aligned and its strides multiples of 8 elements");
  size_t need = kvq::mine_workspace(n, num_sets, num_kv_heads, P, transform);
  if (ws_bytes < need || (!ws && need))
    return fail(KVQ_ERR_WORKSPACE, "mine workspace %zu < %zu bytes", ws_bytes, need);
  if (!aligned(ws, 256)) return fail(KVQ_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if ((size_t)P * 128 * sizeof(float) > 200 * 1024) return fail(KVQ_ERR_UNSUPPORTED, "P too large");
  kvq::MineArgs a{x, dtype, n, num_sets, num_kv_heads, tok_stride, head_stride, set_stride, P, iters, transform,
                  patterns_out, colscale_out, assign_out};
  cudaError_t e = kvq::launch_mine(a, ws, ws_bytes, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kvq_mine_patterns");
  return KVQ_OK;
}

size_t kvq_append_workspace_bytes(const kvq_cache* cache, int32_t n_new) {
  (void)n_new;
  if (!cache || cache->num_kv_heads < 1 || cache->num_sets < 1 || cache->num_patterns < 1) return 0;
  return kvq::append_workspace(kvq::make_geom(*cache));
}

kvq_status kvq_quantize_append(const kvq_cache* cache, const void* k_new, const void* v_new, int32_t n_new,
                               void* ws, size_t ws_bytes, kvq_stream_t stream) {
  g_err[0] = 0;
  kvq_status s = check_cache(cache);
  if (s != KVQ_OK) return s;
  if (n_new < 0) return fail(KVQ_ERR_INVALID_ARG, "n_new %d < 0", n_new);
  if (n_new == 0 || cache->num_seqs == 0) return KVQ_OK;
  if ((int64_t)n_new > (int64_t)cache->max_pages_per_seq * 32)
    return fail(KVQ_ERR_CAPACITY, "n_new %d exceeds the page table capacity %d", n_new,
                cache->max_pages_per_seq * 32);
  if (!k_new || !v_new) return fail(KVQ_ERR_INVALID_ARG, "k_new / v_new is NULL");
  if (!aligned(k_new, 16) || !aligned(v_new, 16)) return fail(KVQ_ERR_INVALID_ARG, "k_new / v_new must be 16-byte aligned");
  kvq::Geom g = kvq::make_geom(*cache);
  const size_t need = kvq::append_workspace(g);
  if (ws_bytes < need || !ws) return fail(KVQ_ERR_WORKSPACE, "append workspace %zu < %zu bytes", ws_bytes, need);
  if (!aligned(ws, 256)) return fail(KVQ_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  cudaError_t e = kvq::launch_append(g, k_new, v_new, n_new, ws, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kvq_quantize_append");
  return KVQ_OK;
}

size_t kvq_decode_workspace_bytes(const kvq_cache* cache, int32_t num_q_heads) {
  if (!cache || num_q_heads < 1 || cache->num_kv_heads < 1) return 0;
  kvq::Geom g = kvq::make_geom(*cache);
  return kvq::decode_workspace(g, num_q_heads, kvq::decode_num_splits(g, num_q_heads, num_sms()));
}

kvq_status kvq_decode_attention(const kvq_cache* cache, const void* q, int32_t num_q_heads, float sm_scale,
                                float* out, void* ws, size_t ws_bytes, kvq_stream_t stream) {
  g_err[0] = 0;
  kvq_status s = check_cache(cache);
  if (s != KVQ_OK) return s;
  if (num_q_heads < 1 || num_q_heads % cache->num_kv_heads)
    return fail(KVQ_ERR_UNSUPPORTED, "num_q_heads %d is not a multiple of num_kv_heads %d", num_q_heads,
                cache->num_kv_heads);
  if (num_q_heads / cache->num_kv_heads > 16)
    return fail(KVQ_ERR_UNSUPPORTED, "more than 16 query heads per KV head");
  if (cache->num_seqs == 0) return KVQ_OK;
  if (!q || !out) return fail(KVQ_ERR_INVALID_ARG, "q / out is NULL");
  if (!aligned(q, 16) || !aligned(out, 16)) return fail(KVQ_ERR_INVALID_ARG, "q / out must be 16-byte aligned");
  if (!(sm_scale > 0.0f)) return fail(KVQ_ERR_INVALID_ARG, "sm_scale must be positive");
  kvq::Geom g = kvq::make_geom(*cache);
  int nsplit = kvq::decode_num_splits(g, num_q_heads, num_sms());
  size_t need = kvq::decode_workspace(g, num_q_heads, nsplit);
  if (ws_bytes < need || !ws) return fail(KVQ_ERR_WORKSPACE, "decode workspace %zu < %zu bytes", ws_bytes, need);
  if (!aligned(ws, 256)) return fail(KVQ_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  cudaError_t e = kvq::launch_decode(g, q, num_q_heads, sm_scale, out, ws, nsplit, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kvq_decode_attention");
  return KVQ_OK;
}

size_t kvq_step_workspace_bytes(const kvq_cache* cache, int32_t num_q_heads) {
  if (!cache || num_q_heads < 1 || cache->num_kv_heads < 1) return 0;
  kvq::Geom g = kvq::make_geom(*cache);
  return kvq::step_workspace(g, num_q_heads, kvq::decode_num_splits(g, num_q_heads, num_sms()));
}

kvq_status kvq_decode_step(const kvq_cache* cache, const void* k_new, const void* v_new, const void* q,
                           int32_t num_q_heads, float sm_scale, float* out, void* ws, size_t ws_bytes,
                           kvq_stream_t stream) {
  g_err[0] = 0;
  kvq_status s = check_cache(cache);
  if (s != KVQ_OK) return s;
  if (num_q_heads < 1 || num_q_heads % cache->num_kv_heads)
    return fail(KVQ_ERR_UNSUPPORTED, "num_q_heads %d is not a multiple of num_kv_heads %d", num_q_heads,
                cache->num_kv_heads);
  if (num_q_heads / cache->num_kv_heads > 16)
    return fail(KVQ_ERR_UNSUPPORTED, "more than 16 query heads per KV head");
  if (cache->num_seqs == 0) return KVQ_OK;
  if (!q || !out || !k_new || !v_new) return fail(KVQ_ERR_INVALID_ARG, "q / out / k_new / v_new is NULL");
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_new, 16) || !aligned(v_new, 16))
    return fail(KVQ_ERR_INVALID_ARG, "q / out / k_new / v_new must be 16-byte aligned");
  if (!(sm_scale > 0.0f)) return fail(KVQ_ERR_INVALID_ARG, "sm_scale must be positive");
  if (cache->max_pages_per_seq < 1) return fail(KVQ_ERR_CAPACITY, "the page table has no column");
  kvq::Geom g = kvq::make_geom(*cache);
  const int nsplit = kvq::decode_num_splits(g, num_q_heads, num_sms());
  const size_t need = kvq::step_workspace(g, num_q_heads, nsplit);
  if (ws_bytes < need || !ws) return fail(KVQ_ERR_WORKSPACE, "step workspace %zu < %zu bytes", ws_bytes, need);
  if (!aligned(ws, 256)) return fail(KVQ_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  cudaError_t e = kvq::launch_decode_step(g, k_new, v_new, q, num_q_heads, sm_scale, out, ws, nsplit, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kvq_decode_step");
  return KVQ_OK;
}

kvq_status kvq_norm_rope(const kvq_rows* q, const kvq_rows* k, const kvq_rows* v, int32_t dtype, int64_t num_tokens,
                         const int32_t* positions, const float* inv_freq, int32_t rot_dim, int32_t interleaved,
                         float eps, kvq_stream_t stream) {
  g_err[0] = 0;
  if (dtype != KVQ_F16 && dtype != KVQ_BF16) return fail(KVQ_ERR_UNSUPPORTED, "dtype %d", dtype);
  if (rot_dim < 0 || rot_dim > 128 || rot_dim % 16)
    return fail(KVQ_ERR_UNSUPPORTED, "rot_dim %d is not a multiple of 16 in 0..128", rot_dim);
  if (num_tokens < 0) return fail(KVQ_ERR_INVALID_ARG, "num_tokens %lld < 0", (long long)num_tokens);
  if (num_tokens > INT32_MAX) return fail(KVQ_ERR_CAPACITY, "num_tokens %lld exceeds the launch grid", (long long)num_tokens);
  if (!(eps >= 0.0f)) return fail(KVQ_ERR_INVALID_ARG, "eps must be >= 0");
  const kvq_rows* rows[3] = {q, k, v};
  kvq::RopeArgs a{};
  int64_t heads = 0;
  for (int i = 0; i < 3; ++i) {
    const kvq_rows* r = rows[i];
    if (!r || r->heads == 0) continue;
    if (r->reserved != 0) return fail(KVQ_ERR_INVALID_ARG, "reserved field must be 0");
    if (r->heads < 0) return fail(KVQ_ERR_INVALID_ARG, "negative head count %d", r->heads);
    heads += r->heads;
    if (num_tokens == 0) continue;
    if (!r->in || !r->out) return fail(KVQ_ERR_INVALID_ARG, "rows without an in or out pointer");
    if (!aligned(r->in, 16) || !aligned(r->out, 16) || (r->weight && !aligned(r->weight, 16)))
      return fail(KVQ_ERR_INVALID_ARG, "rows and weights must be 16-byte aligned");
    if (r->in_tok_stride % 8 || r->in_head_stride % 8 || r->out_tok_stride % 8 || r->out_head_stride % 8 ||
        r->in_tok_stride < 0 || r->in_head_stride < 0 || r->out_tok_stride < 0 || r->out_head_stride < 0)
      return fail(KVQ_ERR_INVALID_ARG, "strides must be multiples of 8 elements, not negative");
    if (i == 2 && r->weight) return fail(KVQ_ERR_INVALID_ARG, "values take no weight");
    a.rows[i] = {r->in, r->out, r->weight, r->heads, r->in_tok_stride, r->in_head_stride, r->out_tok_stride,
                 r->out_head_stride};
  }
  if (num_tokens == 0 || heads == 0) return KVQ_OK;
  if (heads > 65535) return fail(KVQ_ERR_CAPACITY, "%lld heads in all exceed 65535", (long long)heads);
  for (const kvq::RopeRows& r : a.rows)
    if (r.heads > 0 && rows_overlap(num_tokens, r.out_tok, r.heads, r.out_head))
      return fail(KVQ_ERR_INVALID_ARG, "output rows overlap (strides %lld, %lld)", (long long)r.out_tok, (long long)r.out_head);
  const bool turned = a.rows[0].heads + a.rows[1].heads > 0 && rot_dim > 0;
  if (turned && (!positions || !inv_freq)) return fail(KVQ_ERR_INVALID_ARG, "positions / inv_freq is NULL");
  a.pos = positions;
  a.inv_freq = inv_freq;
  a.tokens = num_tokens;
  a.rot = turned ? rot_dim : 0;
  a.eps = eps;
  cudaError_t e = kvq::launch_norm_rope(a, dtype, interleaved != 0, num_sms(), (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kvq_norm_rope");
  return KVQ_OK;
}

size_t kvq_plan_workspace_bytes(const kvq_cache* cache) {
  if (!cache || cache->num_seqs < 0) return 0;
  return kvq::plan_workspace(kvq::make_geom(*cache));
}

kvq_status kvq_plan_pages(const kvq_cache* cache, const int32_t* new_len, const int32_t* free_pages,
                          int32_t free_capacity, const int32_t* free_count, int32_t* free_left, int32_t* cu_new,
                          int64_t* slot_map, int32_t* positions, int32_t* seq_ids, int64_t max_tokens, void* ws,
                          size_t ws_bytes, kvq_stream_t stream) {
  g_err[0] = 0;
  kvq_status s = check_cache(cache);
  if (s != KVQ_OK) return s;
  if (cache->num_seqs == 0) return KVQ_OK;
  if (free_capacity < 0 || max_tokens < 0)
    return fail(KVQ_ERR_INVALID_ARG, "negative size (free_capacity %d max_tokens %lld)", free_capacity,
                (long long)max_tokens);
  if (max_tokens > INT32_MAX - 8192) return fail(KVQ_ERR_CAPACITY, "max_tokens %lld exceeds 2^31 - 8192", (long long)max_tokens);
  if (!new_len || !free_count || !free_left || !cu_new || (free_capacity > 0 && !free_pages) ||
      (max_tokens > 0 && (!slot_map || !positions || !seq_ids)))
    return fail(KVQ_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned(slot_map, 16) || !aligned(positions, 16) || !aligned(seq_ids, 16))
    return fail(KVQ_ERR_INVALID_ARG, "slot_map / positions / seq_ids must be 16-byte aligned");
  kvq::Geom g = kvq::make_geom(*cache);
  const size_t need = kvq::plan_workspace(g);
  if (ws_bytes < need || !ws) return fail(KVQ_ERR_WORKSPACE, "plan workspace %zu < %zu bytes", ws_bytes, need);
  if (!aligned(ws, 4)) return fail(KVQ_ERR_INVALID_ARG, "workspace must be 4-byte aligned");
  kvq::PlanArgs a{new_len,  free_pages, free_capacity, free_count, free_left, cu_new,
                  slot_map, positions,  seq_ids,       max_tokens, (int32_t*)ws};
  cudaError_t e = kvq::launch_plan(g, a, num_sms(), (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kvq_plan_pages");
  return KVQ_OK;
}

kvq_status kvq_page_bounds(const kvq_cache* cache, const void* k_new, int32_t n_new, void* bounds,
                           kvq_stream_t stream) {
  g_err[0] = 0;
  kvq_status s = check_cache(cache);
  if (s != KVQ_OK) return s;
  if (n_new < 0) return fail(KVQ_ERR_INVALID_ARG, "n_new %d < 0", n_new);
  if (n_new == 0 || cache->num_seqs == 0) return KVQ_OK;
  if ((int64_t)n_new > (int64_t)cache->max_pages_per_seq * 32)
    return fail(KVQ_ERR_CAPACITY, "n_new %d exceeds the page table capacity %lld", n_new,
                (long long)cache->max_pages_per_seq * 32);
  if (!k_new || !bounds) return fail(KVQ_ERR_INVALID_ARG, "k_new / bounds is NULL");
  if (!aligned(k_new, 16) || !aligned(bounds, 16))
    return fail(KVQ_ERR_INVALID_ARG, "k_new / bounds must be 16-byte aligned");
  cudaError_t e = kvq::launch_page_bounds(kvq::make_geom(*cache), k_new, n_new, bounds, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kvq_page_bounds");
  return KVQ_OK;
}

static kvq_status check_q_heads(const kvq_cache* cache, int32_t num_q_heads) {
  if (num_q_heads < 1 || num_q_heads % cache->num_kv_heads)
    return fail(KVQ_ERR_UNSUPPORTED, "num_q_heads %d is not a multiple of num_kv_heads %d", num_q_heads,
                cache->num_kv_heads);
  if (num_q_heads / cache->num_kv_heads > 16)
    return fail(KVQ_ERR_UNSUPPORTED, "more than 16 query heads per KV head");
  return KVQ_OK;
}

size_t kvq_select_workspace_bytes(const kvq_cache* cache) {
  if (!cache || cache->num_seqs < 0 || cache->num_kv_heads < 1 || cache->max_pages_per_seq < 0) return 0;
  return kvq::select_workspace(kvq::make_geom(*cache));
}

kvq_status kvq_select_pages(const kvq_cache* cache, const void* q, int32_t num_q_heads, const void* bounds,
                            int32_t budget, int32_t sink, int32_t recent, int32_t* page_list, int32_t* list_len,
                            void* ws, size_t ws_bytes, kvq_stream_t stream) {
  g_err[0] = 0;
  kvq_status s = check_cache(cache);
  if (s == KVQ_OK) s = check_q_heads(cache, num_q_heads);
  if (s != KVQ_OK) return s;
  if (sink < 0 || recent < 1 || (int64_t)sink + recent > budget)
    return fail(KVQ_ERR_INVALID_ARG, "budget %d, sink %d, recent %d: needs sink >= 0, recent >= 1, sink + recent <= budget",
                budget, sink, recent);
  if (cache->num_seqs == 0) return KVQ_OK;
  if (!q || !bounds || !page_list || !list_len) return fail(KVQ_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned(q, 16) || !aligned(bounds, 16)) return fail(KVQ_ERR_INVALID_ARG, "q / bounds must be 16-byte aligned");
  kvq::Geom g = kvq::make_geom(*cache);
  const size_t need = kvq::select_workspace(g);
  if (ws_bytes < need || !ws) return fail(KVQ_ERR_WORKSPACE, "select workspace %zu < %zu bytes", ws_bytes, need);
  if (!aligned(ws, 256)) return fail(KVQ_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  kvq::SelectArgs a{};
  a.q = (const uint16_t*)q;
  a.Gq = num_q_heads / cache->num_kv_heads;
  a.bounds = (const uint16_t*)bounds;
  a.budget = budget;
  a.sink = sink;
  a.recent = recent;
  a.list = page_list;
  a.list_len = list_len;
  cudaError_t e = kvq::launch_select(g, a, ws, num_sms(), (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kvq_select_pages");
  return KVQ_OK;
}

size_t kvq_decode_pages_workspace_bytes(const kvq_cache* cache, int32_t num_q_heads, int32_t budget) {
  if (!cache || num_q_heads < 1 || cache->num_kv_heads < 1 || cache->num_seqs < 0 || budget < 1) return 0;
  kvq::Geom g = kvq::make_geom(*cache);
  return kvq::decode_pages_workspace(g, num_q_heads, kvq::decode_pages_most_splits(g, num_q_heads / cache->num_kv_heads, budget, num_sms()));
}

kvq_status kvq_decode_attention_pages(const kvq_cache* cache, const void* q, int32_t num_q_heads, float sm_scale,
                                      const int32_t* page_list, const int32_t* list_len, int32_t budget, void* out,
                                      void* ws, size_t ws_bytes, kvq_stream_t stream) {
  g_err[0] = 0;
  kvq_status s = check_cache(cache);
  if (s == KVQ_OK) s = check_q_heads(cache, num_q_heads);
  if (s != KVQ_OK) return s;
  if (budget < 1) return fail(KVQ_ERR_INVALID_ARG, "budget %d < 1", budget);
  if (!(sm_scale > 0.0f) || !(sm_scale < INFINITY)) return fail(KVQ_ERR_INVALID_ARG, "sm_scale must be positive and finite");
  if (cache->num_seqs == 0) return KVQ_OK;
  if (!q || !out || !page_list || !list_len) return fail(KVQ_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned(q, 16) || !aligned(out, 16)) return fail(KVQ_ERR_INVALID_ARG, "q / out must be 16-byte aligned");
  kvq::Geom g = kvq::make_geom(*cache);
  kvq::PagesArgs a{};
  a.q = (const uint16_t*)q;
  a.Hq = num_q_heads;
  a.Gq = num_q_heads / cache->num_kv_heads;
  a.scale_log2 = sm_scale * 1.4426950408889634f;
  a.list = page_list;
  a.list_len = list_len;
  a.budget = budget;
  a.nsplit = kvq::decode_pages_splits(g, a.Gq, budget, num_sms());
  a.out = (uint16_t*)out;
  const size_t need = kvq::decode_pages_need(g, num_q_heads, a.nsplit);
  if (ws_bytes < need || !ws) return fail(KVQ_ERR_WORKSPACE, "decode workspace %zu < %zu bytes", ws_bytes, need);
  if (!aligned(ws, 256)) return fail(KVQ_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  cudaError_t e = kvq::launch_decode_pages(g, a, ws, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kvq_decode_attention_pages");
  return KVQ_OK;
}

kvq_status kvq_dequantize(const kvq_cache* cache, int32_t seq, int32_t seq_len_host, int32_t start, int32_t count,
                          float* k_out, float* v_out, kvq_stream_t stream) {
  g_err[0] = 0;
  kvq_status s = check_cache(cache);
  if (s != KVQ_OK) return s;
  if (seq < 0 || seq >= cache->num_seqs) return fail(KVQ_ERR_INVALID_ARG, "seq %d out of range", seq);
  if (start < 0 || count < 0 || (int64_t)start + count > seq_len_host)
    return fail(KVQ_ERR_INVALID_ARG, "token range [%d, %d) outside the sequence length %d", start, start + count,
                seq_len_host);
  if ((int64_t)seq_len_host > (int64_t)cache->max_pages_per_seq * 32)
    return fail(KVQ_ERR_CAPACITY, "seq_len_host %d exceeds the page table", seq_len_host);
  if (count == 0) return KVQ_OK;
  kvq::Geom g = kvq::make_geom(*cache);
  cudaError_t e = kvq::launch_dequant(g, seq, start, count, k_out, v_out, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kvq_dequantize");
  return KVQ_OK;
}

kvq_status kvq_mine_read_status(const void* ws, int32_t* bits_out, kvq_stream_t stream) {
  g_err[0] = 0;
  if (!ws || !bits_out) return fail(KVQ_ERR_INVALID_ARG, "NULL argument");
  cudaStream_t st = (cudaStream_t)stream;
  int32_t v = 0;
  cudaError_t e = cudaMemcpyAsync(&v, ws, sizeof(int32_t), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(e, "kvq_mine_read_status");
  *bits_out = v;
  if (v) return fail(KVQ_ERR_DEVICE, "mining status bits 0x%x", v);
  return KVQ_OK;
}

kvq_status kvq_read_status(const kvq_cache* cache, int32_t* bits_out, int32_t clear, kvq_stream_t stream) {
  g_err[0] = 0;
  if (!cache || !cache->status || !bits_out) return fail(KVQ_ERR_INVALID_ARG, "NULL argument");
  cudaStream_t st = (cudaStream_t)stream;
  int32_t v = 0;
  cudaError_t e = cudaMemcpyAsync(&v, cache->status, sizeof(int32_t), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(e, "kvq_read_status");
  if (clear) {
    e = cudaMemsetAsync(cache->status, 0, sizeof(int32_t), st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return cuda_fail(e, "kvq_read_status (clear)");
  }
  *bits_out = v;
  if (v) return fail(KVQ_ERR_DEVICE, "device status bits 0x%x", v);
  return KVQ_OK;
}

// ---- allocation-free decode: the split partials in a file-scope device array ----------
namespace {
__device__ __align__(256) uint8_t g_decode_scratch[KVQ_DECODE_STATIC_SCRATCH_BYTES];
constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_addr[kMaxDevices];  // per device, resolved on first use
}  // namespace

kvq_status kvq_decode_attention_static(const kvq_cache* cache, const void* q, int32_t num_q_heads, float sm_scale,
                                       float* out, kvq_stream_t stream) {
  g_err[0] = 0;
  kvq_status s = check_cache(cache);
  if (s != KVQ_OK) return s;
  if (num_q_heads < 1 || num_q_heads % cache->num_kv_heads)
    return fail(KVQ_ERR_UNSUPPORTED, "num_q_heads %d is not a multiple of num_kv_heads %d", num_q_heads,
                cache->num_kv_heads);
  if (num_q_heads / cache->num_kv_heads > 16)
    return fail(KVQ_ERR_UNSUPPORTED, "more than 16 query heads per KV head");
  if (cache->num_seqs == 0) return KVQ_OK;
  if (!q || !out) return fail(KVQ_ERR_INVALID_ARG, "q / out is NULL");
  if (!aligned(q, 16) || !aligned(out, 16)) return fail(KVQ_ERR_INVALID_ARG, "q / out must be 16-byte aligned");
  if (!(sm_scale > 0.0f)) return fail(KVQ_ERR_INVALID_ARG, "sm_scale must be positive");
  kvq::Geom g = kvq::make_geom(*cache);
  const int nsplit = kvq::decode_num_splits(g, num_q_heads, num_sms());
  const size_t need = kvq::decode_workspace(g, num_q_heads, nsplit);
  if (need > KVQ_DECODE_STATIC_SCRATCH_BYTES)
    return fail(KVQ_ERR_WORKSPACE, "decode partials need %zu bytes; the static scratch holds %zu", need,
                (size_t)KVQ_DECODE_STATIC_SCRATCH_BYTES);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "kvq_decode_attention_static (cudaGetDevice)");
  if (dev < 0 || dev >= kMaxDevices) return fail(KVQ_ERR_UNSUPPORTED, "device %d beyond %d", dev, kMaxDevices);
  void* ws;
  {
    std::lock_guard<std::mutex> lk(g_scratch_mu);
    if (!g_scratch_addr[dev]) {
      e = cudaGetSymbolAddress(&g_scratch_addr[dev], g_decode_scratch);
      if (e != cudaSuccess) {
        g_scratch_addr[dev] = nullptr;
        return cuda_fail(e, "kvq_decode_attention_static (cudaGetSymbolAddress)");
      }
    }
    ws = g_scratch_addr[dev];
  }
  e = kvq::launch_decode(g, q, num_q_heads, sm_scale, out, ws, nsplit, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kvq_decode_attention_static");
  return KVQ_OK;
}

}  // extern "C"
