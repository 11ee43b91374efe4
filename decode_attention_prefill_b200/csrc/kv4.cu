// kv4.cu -- the entry points of the 4-bit paged cache and of the norm with rotation
// (include/pnmix.h): host-side validation and launches.  No entry point allocates, frees or
// synchronises (except pnmix_kv4_read_error, a synchronous read by definition).
#include <math.h>
#include <string.h>

#include "kv4_launch.cuh"

namespace pnmix {
namespace kv4 {
namespace {

constexpr uint32_t kWaitLimit = 1u << 22;   // try_wait rounds of a staging wait

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

pnmix_status cuda_status(cudaError_t e) { return e == cudaSuccess ? PNMIX_OK : PNMIX_ERR_CUDA; }

pnmix_status check_config(const pnmix_kv4_config* c, Geo* g) {
  if (!c || c->n_q_heads <= 0 || c->n_kv_heads <= 0 || c->n_q_heads % c->n_kv_heads) return PNMIX_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return PNMIX_ERR_UNSUPPORTED;
  if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128)
    return PNMIX_ERR_UNSUPPORTED;
  if (c->n_q_heads > 4096 || c->n_q_heads / c->n_kv_heads > 128) return PNMIX_ERR_UNSUPPORTED;
  if (!(c->softmax_scale <= 0.f) && !isfinite(c->softmax_scale)) return PNMIX_ERR_INVALID_ARG;
  *g = Geo{};
  g->Hq = c->n_q_heads;
  g->Hkv = c->n_kv_heads;
  g->G = g->Hq / g->Hkv;
  g->D = c->head_dim;
  g->page_shift = c->page_tokens == 16 ? 4 : c->page_tokens == 32 ? 5 : c->page_tokens == 64 ? 6 : 7;
  g->scale = c->softmax_scale > 0.f ? c->softmax_scale : 1.0f / sqrtf(static_cast<float>(g->D));
  g->wait_limit = kWaitLimit;
  g->skip_seq = -1;
  return PNMIX_OK;
}

size_t pages_bytes(const Geo& g, int n_pages) {
  return static_cast<size_t>(n_pages) * g.Hkv * (static_cast<size_t>(1) << (g.page_shift - 4)) * block_bytes(g.D);
}

pnmix_status check_cache(const pnmix_kv4_cache* c, Geo* g) {
  if (!c || !c->base || !c->pages || !c->error) return PNMIX_ERR_INVALID_ARG;
  if (c->n_pages <= 0 || c->n_kv_heads != g->Hkv || c->head_dim != g->D || c->page_tokens != 1 << g->page_shift)
    return PNMIX_ERR_INVALID_ARG;
  g->n_pages = c->n_pages;
  g->pages = c->pages;
  g->error = c->error;
  return PNMIX_OK;
}

pnmix_status check_batch(const pnmix_kv4_batch* b, const Geo& g, Batch* out) {
  if (!b || !b->kv_len || !b->page_table) return PNMIX_ERR_INVALID_ARG;
  if (b->batch <= 0 || b->n_tokens < 0 || b->max_pages <= 0) return PNMIX_ERR_INVALID_ARG;
  if (b->batch > kMaxBatch) return PNMIX_ERR_UNSUPPORTED;
  if (static_cast<long long>(b->max_pages) << g.page_shift > 1 << 29) return PNMIX_ERR_UNSUPPORTED;
  if (b->n_tokens > 1 << 28 || static_cast<long long>(b->n_tokens) * g.Hq > 1 << 30) return PNMIX_ERR_UNSUPPORTED;
  // the attention numbers its work in 64 bits, times the CTAs: heads x row tiles x tokens
  const double tiles = static_cast<double>(g.Hkv) * (b->batch + static_cast<double>(b->n_tokens) * g.G / 8);
  if (tiles * (static_cast<double>(static_cast<long long>(b->max_pages) << g.page_shift) + b->n_tokens + 4096) > 0x1p51)
    return PNMIX_ERR_UNSUPPORTED;
  if (b->n_tokens > 0 && (b->max_q < 1 || b->max_q > b->n_tokens)) return PNMIX_ERR_INVALID_ARG;
  if (!b->q_start && b->n_tokens % b->batch) return PNMIX_ERR_INVALID_ARG;
  if (!b->q_start && b->max_q < b->n_tokens / b->batch) return PNMIX_ERR_INVALID_ARG;
  if (!aligned(b->kv_len, 4) || !aligned(b->page_table, 4) || !aligned(b->q_start, 4)) return PNMIX_ERR_ALIGNMENT;
  out->B = b->batch;
  out->n_tokens = b->n_tokens;
  out->max_pages = b->max_pages;
  out->max_q = b->max_q;
  out->uniform = b->q_start ? 0 : b->n_tokens / b->batch;
  out->q_start = b->q_start;
  out->kv_len = b->kv_len;
  out->table = b->page_table;
  return PNMIX_OK;
}

// `writes`: rows must not overlap one another.
pnmix_status check_rows(const pnmix_rows* r, long long tokens, long long heads, long long dim, bool writes) {
  if (!r || !r->data) return PNMIX_ERR_INVALID_ARG;
  if (!aligned(r->data, 16) || r->token_stride % 8 || r->head_stride % 8) return PNMIX_ERR_ALIGNMENT;
  if (r->token_stride < 0 || r->head_stride < 0) return PNMIX_ERR_INVALID_ARG;
  if (writes) {
    const long long ts = r->token_stride, hs = r->head_stride;
    const bool tokens_outer = (heads == 1 || hs >= dim) && (tokens == 1 || ts >= (heads - 1) * hs + dim);
    const bool heads_outer = (tokens == 1 || ts >= dim) && (heads == 1 || hs >= (tokens - 1) * ts + dim);
    if (!tokens_outer && !heads_outer) return PNMIX_ERR_INVALID_ARG;
  }
  return PNMIX_OK;
}

pnmix_status check_rope(const pnmix_rope* r) {
  if (!r) return PNMIX_ERR_INVALID_ARG;
  if (r->head_dim != 64 && r->head_dim != 128 && r->head_dim != 256) return PNMIX_ERR_UNSUPPORTED;
  if (r->rot_dim < 0 || r->rot_dim > r->head_dim || r->rot_dim % 16) return PNMIX_ERR_UNSUPPORTED;
  if (r->n_axes < 1 || r->n_axes > 4) return PNMIX_ERR_UNSUPPORTED;
  if (!(r->eps >= 0.f) || !isfinite(r->eps)) return PNMIX_ERR_INVALID_ARG;
  for (int i = 0; i < r->rot_dim / 2; ++i)
    if (r->axis[i] >= r->n_axes || !isfinite(r->inv_freq[i])) return PNMIX_ERR_INVALID_ARG;
  return PNMIX_OK;
}

#define PNMIX_TRY(x)                                  \
  do {                                                \
    const pnmix_status st_ = (x);                     \
    if (st_ != PNMIX_OK) return st_;                  \
  } while (0)

}  // namespace
}  // namespace kv4
}  // namespace pnmix

using namespace pnmix;
using namespace pnmix::kv4;

extern "C" {

pnmix_status pnmix_norm_rope(const pnmix_rope* rope, int n_tokens, int n_q_heads, int n_k_heads, const pnmix_rows* q,
                             const pnmix_rows* k, const uint16_t* q_weight, const uint16_t* k_weight,
                             const int32_t* positions, const pnmix_rows* q_out, const pnmix_rows* k_out,
                             void* stream) {
  PNMIX_TRY(check_rope(rope));
  if (n_tokens < 0 || n_q_heads < 0 || n_k_heads < 0 || n_q_heads + static_cast<long long>(n_k_heads) < 1)
    return PNMIX_ERR_INVALID_ARG;
  if (static_cast<long long>(n_tokens) * (static_cast<long long>(n_q_heads) + n_k_heads) > 1 << 30)
    return PNMIX_ERR_UNSUPPORTED;
  if (n_tokens == 0) return PNMIX_OK;
  if (!positions) return PNMIX_ERR_INVALID_ARG;
  if (!aligned(positions, 4) || !aligned(q_weight, 16) || !aligned(k_weight, 16)) return PNMIX_ERR_ALIGNMENT;
  const pnmix_rows none = {nullptr, 0, 0};
  if (n_q_heads) {
    PNMIX_TRY(check_rows(q, n_tokens, n_q_heads, rope->head_dim, false));
    PNMIX_TRY(check_rows(q_out, n_tokens, n_q_heads, rope->head_dim, true));
  }
  if (n_k_heads) {
    PNMIX_TRY(check_rows(k, n_tokens, n_k_heads, rope->head_dim, false));
    PNMIX_TRY(check_rows(k_out, n_tokens, n_k_heads, rope->head_dim, true));
  }
  // an output may be its own input; over another tensor it would be read after it was written
  if (n_q_heads && n_k_heads && (q_out->data == k_out->data || q_out->data == k->data || k_out->data == q->data))
    return PNMIX_ERR_INVALID_ARG;
  return cuda_status(launch_norm_rope(*rope, n_tokens, n_q_heads, n_k_heads, n_q_heads ? *q : none,
                                      n_k_heads ? *k : none, n_q_heads ? q_weight : nullptr,
                                      n_k_heads ? k_weight : nullptr, positions, n_q_heads ? *q_out : none,
                                      n_k_heads ? *k_out : none, static_cast<cudaStream_t>(stream)));
}

pnmix_status pnmix_kv4_cache_bytes(const pnmix_kv4_config* cfg, int n_pages, size_t* total_bytes) {
  Geo g;
  PNMIX_TRY(check_config(cfg, &g));
  if (!total_bytes || n_pages <= 0) return PNMIX_ERR_INVALID_ARG;
  *total_bytes = pages_bytes(g, n_pages) + 256;   // a page is a multiple of 256 bytes
  return PNMIX_OK;
}

pnmix_status pnmix_kv4_cache_init(const pnmix_kv4_config* cfg, int n_pages, void* device_base, size_t bytes,
                                  pnmix_kv4_cache* out) {
  if (!out || !device_base) return PNMIX_ERR_INVALID_ARG;
  size_t need = 0;
  PNMIX_TRY(pnmix_kv4_cache_bytes(cfg, n_pages, &need));
  if (!aligned(device_base, 256)) return PNMIX_ERR_ALIGNMENT;
  if (bytes < need) return PNMIX_ERR_CAPACITY;
  memset(out, 0, sizeof(*out));
  out->n_pages = n_pages;
  out->page_tokens = cfg->page_tokens;
  out->n_kv_heads = cfg->n_kv_heads;
  out->head_dim = cfg->head_dim;
  out->pages = static_cast<uint8_t*>(device_base);
  out->error = reinterpret_cast<uint32_t*>(out->pages + need - 256);
  out->base = device_base;
  out->total_bytes = need;
  return PNMIX_OK;
}

pnmix_status pnmix_kv4_cache_reset(const pnmix_kv4_cache* cache, void* stream) {
  if (!cache || !cache->base) return PNMIX_ERR_INVALID_ARG;
  return cuda_status(cudaMemsetAsync(cache->base, 0, cache->total_bytes, static_cast<cudaStream_t>(stream)));
}

pnmix_status pnmix_kv4_append(const pnmix_kv4_config* cfg, const pnmix_kv4_batch* batch, const pnmix_rows* k,
                              const pnmix_rows* v, pnmix_kv4_cache* cache, void* stream) {
  Geo g;
  Batch bt;
  PNMIX_TRY(check_config(cfg, &g));
  PNMIX_TRY(check_cache(cache, &g));
  PNMIX_TRY(check_batch(batch, g, &bt));
  if (bt.n_tokens == 0) return PNMIX_OK;
  PNMIX_TRY(check_rows(k, bt.n_tokens, g.Hkv, g.D, false));
  PNMIX_TRY(check_rows(v, bt.n_tokens, g.Hkv, g.D, false));
  return cuda_status(launch_append(g, bt, *k, *v, static_cast<cudaStream_t>(stream)));
}

pnmix_status pnmix_kv4_append_qkv(const pnmix_kv4_config* cfg, const pnmix_rope* rope, const pnmix_kv4_batch* batch,
                                  const pnmix_rows* q, const pnmix_rows* k, const pnmix_rows* v,
                                  const uint16_t* q_weight, const uint16_t* k_weight, const int32_t* positions,
                                  const pnmix_rows* q_out, pnmix_kv4_cache* cache, void* stream) {
  Geo g;
  Batch bt;
  PNMIX_TRY(check_config(cfg, &g));
  PNMIX_TRY(check_rope(rope));
  if (rope->head_dim != g.D) return PNMIX_ERR_INVALID_ARG;
  PNMIX_TRY(check_cache(cache, &g));
  PNMIX_TRY(check_batch(batch, g, &bt));
  if (bt.n_tokens == 0) return PNMIX_OK;
  if (!positions) return PNMIX_ERR_INVALID_ARG;
  if (!aligned(positions, 4) || !aligned(q_weight, 16) || !aligned(k_weight, 16)) return PNMIX_ERR_ALIGNMENT;
  PNMIX_TRY(check_rows(q, bt.n_tokens, g.Hq, g.D, false));
  PNMIX_TRY(check_rows(k, bt.n_tokens, g.Hkv, g.D, false));
  PNMIX_TRY(check_rows(v, bt.n_tokens, g.Hkv, g.D, false));
  PNMIX_TRY(check_rows(q_out, bt.n_tokens, g.Hq, g.D, true));
  if (q_out->data == k->data || q_out->data == v->data) return PNMIX_ERR_INVALID_ARG;
  return cuda_status(launch_append_qkv(g, bt, *rope, *q, *k, *v, q_weight, k_weight, positions, *q_out,
                                       static_cast<cudaStream_t>(stream)));
}

pnmix_status pnmix_kv4_read(const pnmix_kv4_config* cfg, const pnmix_kv4_batch* batch, const pnmix_kv4_cache* cache,
                            const pnmix_rows* k_out, const pnmix_rows* v_out, void* stream) {
  Geo g;
  Batch bt;
  PNMIX_TRY(check_config(cfg, &g));
  PNMIX_TRY(check_cache(cache, &g));
  PNMIX_TRY(check_batch(batch, g, &bt));
  if (bt.n_tokens == 0) return PNMIX_OK;
  PNMIX_TRY(check_rows(k_out, bt.n_tokens, g.Hkv, g.D, true));
  PNMIX_TRY(check_rows(v_out, bt.n_tokens, g.Hkv, g.D, true));
  if (k_out->data == v_out->data) return PNMIX_ERR_INVALID_ARG;
  return cuda_status(launch_read(g, bt, *k_out, *v_out, static_cast<cudaStream_t>(stream)));
}

size_t pnmix_kv4_workspace_bytes(const pnmix_kv4_config* cfg, const pnmix_kv4_batch* batch) {
  Geo g;
  Batch bt;
  if (check_config(cfg, &g) != PNMIX_OK || check_batch(batch, g, &bt) != PNMIX_OK) return 0;
  return attention_workspace_bytes(g, bt);
}

static pnmix_status attention(Geo g, const pnmix_kv4_batch* batch, const pnmix_rows* q, const pnmix_kv4_cache* cache,
                              const pnmix_rows* out, void* workspace, size_t workspace_bytes, void* stream) {
  Batch bt;
  PNMIX_TRY(check_cache(cache, &g));
  PNMIX_TRY(check_batch(batch, g, &bt));
  if (bt.n_tokens == 0) return PNMIX_OK;
  PNMIX_TRY(check_rows(q, bt.n_tokens, g.Hq, g.D, false));
  PNMIX_TRY(check_rows(out, bt.n_tokens, g.Hq, g.D, true));
  if (!workspace) return PNMIX_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return PNMIX_ERR_ALIGNMENT;
  if (workspace_bytes < attention_workspace_bytes(g, bt)) return PNMIX_ERR_CAPACITY;
  if (q->data == out->data) return PNMIX_ERR_INVALID_ARG;      // rows are read again after some are written
  return cuda_status(launch_attention(g, bt, *q, *out, workspace, static_cast<cudaStream_t>(stream)));
}

pnmix_status pnmix_kv4_attention(const pnmix_kv4_config* cfg, const pnmix_kv4_batch* batch, const pnmix_rows* q,
                                 const pnmix_kv4_cache* cache, const pnmix_rows* out, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  Geo g;
  PNMIX_TRY(check_config(cfg, &g));
  return attention(g, batch, q, cache, out, workspace, workspace_bytes, stream);
}

pnmix_status pnmix_debug_kv4_stall(const pnmix_kv4_config* cfg, const pnmix_kv4_batch* batch, const pnmix_rows* q,
                                   const pnmix_kv4_cache* cache, const pnmix_rows* out, void* workspace,
                                   size_t workspace_bytes, int skip_seq, uint32_t wait_rounds, void* stream) {
  Geo g;
  PNMIX_TRY(check_config(cfg, &g));
  if (!batch || skip_seq < 0 || skip_seq >= batch->batch || wait_rounds < 1) return PNMIX_ERR_INVALID_ARG;
  g.skip_seq = skip_seq;
  g.wait_limit = wait_rounds;
  return attention(g, batch, q, cache, out, workspace, workspace_bytes, stream);
}

pnmix_status pnmix_kv4_read_error(const pnmix_kv4_cache* cache, int clear, uint32_t* host_error) {
  if (!cache || !cache->error || !host_error) return PNMIX_ERR_INVALID_ARG;
  // the calls before may be on streams that the default stream does not wait for, those behind as well
  if (cudaDeviceSynchronize() != cudaSuccess ||
      cudaMemcpy(host_error, cache->error, sizeof(uint32_t), cudaMemcpyDeviceToHost) != cudaSuccess)
    return PNMIX_ERR_CUDA;
  if (clear && (cudaMemset(cache->error, 0, sizeof(uint32_t)) != cudaSuccess ||
                cudaStreamSynchronize(nullptr) != cudaSuccess))
    return PNMIX_ERR_CUDA;
  return *host_error ? PNMIX_ERR_DEVICE : PNMIX_OK;
}

}  // extern "C"
