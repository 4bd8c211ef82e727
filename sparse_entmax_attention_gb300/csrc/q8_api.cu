// q8_api.cu -- the extern "C" entry points of the 8-bit paged cache: argument
// checks and launches.
#include <math.h>

#include "q8.cuh"

namespace ekv {

static int check_q8_config(const entmaxkv_config* c) {
  if (!c) return ENTMAXKV_ERR_INVALID_ARG;
  if (c->num_kv_heads < 1 || c->group < 1 || c->max_seqs < 1 || c->max_pages_per_seq < 1 || c->num_phys_pages < 1)
    return ENTMAXKV_ERR_INVALID_ARG;
  if (c->kv_dtype != ENTMAXKV_I8 && c->kv_dtype != ENTMAXKV_E4M3) return ENTMAXKV_ERR_INVALID_ARG;
  if (c->group > 8 || c->num_kv_heads > 4096) return ENTMAXKV_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128) return ENTMAXKV_ERR_UNSUPPORTED;
  if (c->page_size != 16 && c->page_size != 32) return ENTMAXKV_ERR_UNSUPPORTED;
  if ((long long)c->max_pages_per_seq * c->page_size > 1 << 30) return ENTMAXKV_ERR_UNSUPPORTED;  // (kNoKey)
  return ENTMAXKV_OK;
}

static int check_q8_cache(const entmaxkv_q8_cache* k) {
  if (!k || !k->k_pool || !k->v_pool || !k->k_scale || !k->v_scale || !k->block_table || !k->seq_lens)
    return ENTMAXKV_ERR_INVALID_ARG;
  if (((uintptr_t)k->k_pool | (uintptr_t)k->v_pool) & 15u) return ENTMAXKV_ERR_INVALID_ARG;
  return ENTMAXKV_OK;
}

static int check_batch(const entmaxkv_batch* b) {
  if (!b || b->n_seqs < 0 || b->n_seqs > 65535 || b->total < 0 || b->max_count < 0) return ENTMAXKV_ERR_INVALID_ARG;
  if (b->n_seqs > 0 && (!b->start || !b->count)) return ENTMAXKV_ERR_INVALID_ARG;
  return ENTMAXKV_OK;
}
static bool idle(const entmaxkv_batch* b) { return b->n_seqs == 0 || b->total == 0 || b->max_count == 0; }

static int check_rows(const entmaxkv_rows* r, bool written) {
  if (!r || !r->data || ((uintptr_t)r->data & 15u)) return ENTMAXKV_ERR_INVALID_ARG;
  if (r->token_stride < 0 || r->head_stride < 0 || (r->token_stride & 7) || (r->head_stride & 7))
    return ENTMAXKV_ERR_INVALID_ARG;
  if (written && (r->token_stride == 0 || r->head_stride == 0)) return ENTMAXKV_ERR_INVALID_ARG;
  return ENTMAXKV_OK;
}

static Q8Cache cache_of(const entmaxkv_config* c, const entmaxkv_q8_cache* k) {
  return Q8Cache{c->num_kv_heads, c->group, c->head_dim, c->page_size, c->max_pages_per_seq, c->num_phys_pages,
                 c->max_seqs, static_cast<uint8_t*>(k->k_pool), static_cast<uint8_t*>(k->v_pool), k->k_scale,
                 k->v_scale, k->block_table, k->seq_lens, k->status};
}
static Q8Batch batch_of(const entmaxkv_batch* b) {
  return Q8Batch{b->seq_ids, b->start, b->count, b->n_seqs, b->total, b->max_count};
}
static Q8Rows rows_of(const entmaxkv_rows* r) {
  return Q8Rows{static_cast<__nv_bfloat16*>(r->data), r->token_stride, r->head_stride};
}
static bool streams(const entmaxkv_config* c, int max_count) {
  return (long long)max_count * c->group <= kStreamRows;
}
static int32_t code_of(cudaError_t e) { return e == cudaSuccess ? ENTMAXKV_OK : ENTMAXKV_ERR_CUDA; }

}  // namespace ekv

using namespace ekv;

extern "C" {

static int check_table(const entmaxkv_config* c) {
  if (!c || c->max_seqs < 1 || c->max_pages_per_seq < 1 || c->num_phys_pages < 1) return ENTMAXKV_ERR_INVALID_ARG;
  if (c->page_size != 16 && c->page_size != 32) return ENTMAXKV_ERR_UNSUPPORTED;
  if ((long long)c->max_pages_per_seq * c->page_size > 0x7fffffffLL) return ENTMAXKV_ERR_UNSUPPORTED;
  return ENTMAXKV_OK;
}

int32_t entmaxkv_plan_pages_bounded(const entmaxkv_config* cfg, int32_t* block_table, const int32_t* seq_lens,
                                    uint32_t* status, const int32_t* seq_ids, const int32_t* n_new, int32_t n_seqs,
                                    int32_t total, int32_t max_count, const int32_t* free_pages,
                                    const int32_t* free_count, int32_t* free_count_out, int32_t* lens_out,
                                    int32_t* start, int32_t* count, int32_t* positions, int64_t* slots,
                                    void* stream) {
  const int st = check_table(cfg);
  if (st) return st;
  if (n_seqs < 0 || n_seqs > 65535 || total < 0 || max_count < 0) return ENTMAXKV_ERR_INVALID_ARG;
  if (n_seqs == 0) return ENTMAXKV_OK;
  if (!block_table || !seq_lens || !n_new || !free_pages || !free_count || !free_count_out || !start || !count)
    return ENTMAXKV_ERR_INVALID_ARG;
  return code_of(launch_plan(*cfg, block_table, seq_lens, status, seq_ids, n_new, n_seqs, total,
                             max_count ? max_count : 0x7fffffff, free_pages, free_count, free_count_out, lens_out,
                             start, count, positions, slots, (cudaStream_t)stream));
}

int32_t entmaxkv_plan_pages(const entmaxkv_config* cfg, int32_t* block_table, const int32_t* seq_lens,
                            uint32_t* status, const int32_t* seq_ids, const int32_t* n_new, int32_t n_seqs,
                            int32_t total, const int32_t* free_pages, const int32_t* free_count,
                            int32_t* free_count_out, int32_t* lens_out, int32_t* start, int32_t* count,
                            int32_t* positions, int64_t* slots, void* stream) {
  return entmaxkv_plan_pages_bounded(cfg, block_table, seq_lens, status, seq_ids, n_new, n_seqs, total, 0, free_pages,
                                     free_count, free_count_out, lens_out, start, count, positions, slots, stream);
}

int32_t entmaxkv_release_pages(const entmaxkv_config* cfg, const int32_t* block_table, int32_t* seq_lens,
                               uint32_t* status, const int32_t* seq_ids, int32_t n_seqs, int32_t* free_pages,
                               int32_t* free_count, void* stream) {
  const int st = check_table(cfg);
  if (st) return st;
  if (n_seqs < 0 || n_seqs > 65535) return ENTMAXKV_ERR_INVALID_ARG;
  if (n_seqs == 0) return ENTMAXKV_OK;
  if (!block_table || !seq_lens || !free_pages || !free_count) return ENTMAXKV_ERR_INVALID_ARG;
  return code_of(launch_release(*cfg, block_table, seq_lens, status, seq_ids, n_seqs, free_pages, free_count,
                                (cudaStream_t)stream));
}

int32_t entmaxkv_append_q8(const entmaxkv_config* cfg, const entmaxkv_q8_cache* cache, const entmaxkv_batch* batch,
                           const entmaxkv_rows* k, const entmaxkv_rows* v, void* stream) {
  int st;
  if ((st = check_q8_config(cfg)) || (st = check_q8_cache(cache)) || (st = check_batch(batch))) return st;
  if (idle(batch)) return ENTMAXKV_OK;
  if ((st = check_rows(k, false)) || (st = check_rows(v, false))) return st;
  const int sms = device_sms();
  if (sms < 1) return ENTMAXKV_ERR_CUDA;
  return code_of(launch_append_q8(cache_of(cfg, cache), batch_of(batch), rows_of(k), rows_of(v),
                                  cfg->kv_dtype == ENTMAXKV_I8, sms, (cudaStream_t)stream));
}

int32_t entmaxkv_read_q8(const entmaxkv_config* cfg, const entmaxkv_q8_cache* cache, const entmaxkv_batch* batch,
                         const int32_t* first, const entmaxkv_rows* k, const entmaxkv_rows* v, void* stream) {
  int st;
  if ((st = check_q8_config(cfg)) || (st = check_q8_cache(cache)) || (st = check_batch(batch))) return st;
  if (idle(batch)) return ENTMAXKV_OK;
  if (!first) return ENTMAXKV_ERR_INVALID_ARG;
  if ((st = check_rows(k, true)) || (st = check_rows(v, true))) return st;
  const int sms = device_sms();
  if (sms < 1) return ENTMAXKV_ERR_CUDA;
  return code_of(launch_read_q8(cache_of(cfg, cache), batch_of(batch), first, rows_of(k), rows_of(v),
                                cfg->kv_dtype == ENTMAXKV_I8, sms, (cudaStream_t)stream));
}

static int check_attend(const entmaxkv_config* cfg, int n_seqs, int total, int max_count, float alpha) {
  const int st = check_q8_config(cfg);
  if (st) return st;
  if (n_seqs < 0 || n_seqs > 65535 || total < 0 || max_count < 0) return ENTMAXKV_ERR_INVALID_ARG;
  if (!(alpha >= 1.0f) || !isfinite(alpha)) return ENTMAXKV_ERR_INVALID_ARG;
  if (alpha > 1.0f) {
    // equal scores of n keys lie n^{1−α} above the threshold, which has to be a normal float with room for the solve's
    // bracket; a weight's β-th power, β = 1/(α−1), is good to β·2^-22, which has to be less than a half's 2^-11
    const double a1 = (double)alpha - 1.0, keys = (double)cfg->max_pages_per_seq * cfg->page_size;
    if (a1 < 0x1p-10 || a1 * log2(keys) > 120.0) return ENTMAXKV_ERR_UNSUPPORTED;
  }
  if (alpha > 1.0f && max_count > 1) return ENTMAXKV_ERR_UNSUPPORTED;
  if (!streams(cfg, max_count) && !chunk_counts_fit(*cfg, n_seqs, total)) return ENTMAXKV_ERR_UNSUPPORTED;
  return ENTMAXKV_OK;
}

size_t entmaxkv_attend_q8_workspace(const entmaxkv_config* cfg, int32_t n_seqs, int32_t total, int32_t max_count,
                                    float alpha) {
  if (check_attend(cfg, n_seqs, total, max_count, alpha)) return 0;
  if (alpha > 1.0f) return attend_entmax_bytes(*cfg, n_seqs);
  return streams(cfg, max_count) ? attend_softmax_bytes(*cfg, n_seqs) : attend_chunk_bytes(*cfg, n_seqs, total);
}

static int score_of(const entmaxkv_config* cfg, const entmaxkv_score* score, Q8Score& sc) {
  sc = Q8Score{0.0f, 0.0f, 0.0f, 0, nullptr, nullptr, nullptr};
  if (score) {
    if (!isfinite(score->scale) || score->scale < 0.0f || score->window < 0) return ENTMAXKV_ERR_INVALID_ARG;
    if (score->softcap != 0.0f && !(score->softcap >= 0x1p-60f && score->softcap <= 0x1p60f))
      return ENTMAXKV_ERR_INVALID_ARG;
    sc = Q8Score{score->scale, score->softcap, score->softcap > 0.0f ? 1.0f / score->softcap : 0.0f, score->window,
                 score->slopes, score->prefix, score->first_key};
  }
  if (sc.scale == 0.0f) sc.scale = (float)(1.0 / sqrt((double)cfg->head_dim));
  return ENTMAXKV_OK;
}

// lam null: attention, else the differences of pairs of heads.
static int32_t attend(const entmaxkv_config* cfg, const entmaxkv_q8_cache* cache, const entmaxkv_batch* batch,
                      const entmaxkv_rows* q, const entmaxkv_score* score, float alpha, const float* lam,
                      int64_t lam_stride, const float* gain, float eps, void* workspace, size_t workspace_bytes,
                      const entmaxkv_rows* out, float* tau, void* stream) {
  int st;
  if ((st = check_q8_config(cfg)) || (st = check_q8_cache(cache)) || (st = check_batch(batch))) return st;
  if ((st = check_attend(cfg, batch->n_seqs, batch->total, batch->max_count, alpha))) return st;
  Q8Score sc;
  if ((st = score_of(cfg, score, sc))) return st;
  if (idle(batch)) return ENTMAXKV_OK;
  if ((st = check_rows(q, false)) || (st = check_rows(out, true))) return st;
  if (!workspace || ((uintptr_t)workspace & 255u) ||
      workspace_bytes < entmaxkv_attend_q8_workspace(cfg, batch->n_seqs, batch->total, batch->max_count, alpha))
    return ENTMAXKV_ERR_WORKSPACE_TOO_SMALL;
  const int sms = device_sms();
  if (sms < 1) return ENTMAXKV_ERR_CUDA;
  Q8AttendArgs a{};
  a.c = cache_of(cfg, cache);
  a.b = batch_of(batch);
  a.sc = sc;
  a.q = rows_of(q);
  a.out = rows_of(out);
  a.tau = tau;
  a.lam = lam;
  a.lam_ts = lam_stride;
  a.gain = gain;
  a.eps = eps;
  const bool i8 = cfg->kv_dtype == ENTMAXKV_I8;
  const cudaStream_t s = (cudaStream_t)stream;
  if (alpha > 1.0f) return code_of(launch_attend_entmax(*cfg, a, i8, alpha, workspace, sms, s));
  if (streams(cfg, batch->max_count))
    return code_of(launch_attend_softmax(a, i8, workspace, sms, s));
  return code_of(launch_attend_chunk(a, i8, workspace, sms, s));
}

int32_t entmaxkv_attend_q8(const entmaxkv_config* cfg, const entmaxkv_q8_cache* cache, const entmaxkv_batch* batch,
                           const entmaxkv_rows* q, const entmaxkv_score* score, float alpha, void* workspace,
                           size_t workspace_bytes, const entmaxkv_rows* out, float* tau, void* stream) {
  return attend(cfg, cache, batch, q, score, alpha, nullptr, 0, nullptr, 0.0f, workspace, workspace_bytes, out, tau,
                stream);
}

int32_t entmaxkv_attend_diff_q8(const entmaxkv_config* cfg, const entmaxkv_q8_cache* cache,
                                const entmaxkv_batch* batch, const entmaxkv_rows* q, const entmaxkv_score* score,
                                const float* lam, int64_t lam_stride, const float* gain, float eps, void* workspace,
                                size_t workspace_bytes, const entmaxkv_rows* out, float* tau, void* stream) {
  const int st = check_q8_config(cfg);
  if (st) return st;
  if (cfg->group & 1) return ENTMAXKV_ERR_UNSUPPORTED;
  if (lam_stride < 0 || (gain && !(eps >= 0x1p-100f && isfinite(eps)))) return ENTMAXKV_ERR_INVALID_ARG;
  if (!lam && batch && !idle(batch)) return ENTMAXKV_ERR_INVALID_ARG;
  return attend(cfg, cache, batch, q, score, 1.0f, lam, lam_stride, gain, eps, workspace, workspace_bytes, out, tau,
                stream);
}

static bool weigh_streams(const entmaxkv_config* c, int max_count) {
  return (long long)max_count * c->group <= kWeighRows;
}

size_t entmaxkv_weigh_q8_workspace(const entmaxkv_config* cfg, int32_t n_seqs, int32_t total, int32_t max_count,
                                   float alpha) {
  if (check_attend(cfg, n_seqs, total, max_count, alpha)) return 0;
  return weigh_streams(cfg, max_count) ? 256 : weigh_chunk_bytes(*cfg, n_seqs, total);
}

int32_t entmaxkv_weigh_q8(const entmaxkv_config* cfg, const entmaxkv_q8_cache* cache, const entmaxkv_batch* batch,
                          const entmaxkv_rows* q, const float* tau, const entmaxkv_score* score, float alpha,
                          const float* coef, float decay, const int32_t* fresh, float* weights, void* workspace,
                          size_t workspace_bytes, void* stream) {
  int st;
  if ((st = check_q8_config(cfg)) || (st = check_q8_cache(cache)) || (st = check_batch(batch))) return st;
  if ((st = check_attend(cfg, batch->n_seqs, batch->total, batch->max_count, alpha))) return st;
  Q8Score sc;
  if ((st = score_of(cfg, score, sc))) return st;
  if (!(decay >= 0.0f) || !isfinite(decay)) return ENTMAXKV_ERR_INVALID_ARG;
  if (idle(batch)) return ENTMAXKV_OK;
  if ((st = check_rows(q, false))) return st;
  if (!tau || !weights) return ENTMAXKV_ERR_INVALID_ARG;
  if (!workspace || ((uintptr_t)workspace & 255u) ||
      workspace_bytes < entmaxkv_weigh_q8_workspace(cfg, batch->n_seqs, batch->total, batch->max_count, alpha))
    return ENTMAXKV_ERR_WORKSPACE_TOO_SMALL;
  const int sms = device_sms();
  if (sms < 1) return ENTMAXKV_ERR_CUDA;
  const float a1 = (float)((double)alpha - 1.0);
  const Q8WeighArgs a{cache_of(cfg, cache), batch_of(batch), sc, rows_of(q), tau, coef, fresh, weights, decay, a1,
                      a1 > 0.0f ? (float)(1.0 / ((double)alpha - 1.0)) : 0.0f};
  const bool i8 = cfg->kv_dtype == ENTMAXKV_I8;
  const cudaStream_t s = (cudaStream_t)stream;
  return code_of(weigh_streams(cfg, batch->max_count) ? launch_weigh_stream(a, i8, sms, s)
                                                      : launch_weigh_chunk(a, i8, workspace, sms, s));
}

static int check_evict(const entmaxkv_config* cfg, int32_t n_seqs, int32_t keep) {
  const int st = check_q8_config(cfg);
  if (st) return st;
  if ((long long)cfg->num_phys_pages * cfg->page_size > 0xffffffffLL) return ENTMAXKV_ERR_UNSUPPORTED;  // (EvictArgs::src)
  return n_seqs < 0 || n_seqs > 65535 || keep < 1 || (long long)keep > (long long)cfg->max_pages_per_seq * cfg->page_size
             ? ENTMAXKV_ERR_INVALID_ARG : ENTMAXKV_OK;
}

size_t entmaxkv_evict_q8_workspace(const entmaxkv_config* cfg, int32_t n_seqs, int32_t keep) {
  return check_evict(cfg, n_seqs, keep) ? 0 : evict_bytes(*cfg, n_seqs, keep);
}

int32_t entmaxkv_evict_q8(const entmaxkv_config* cfg, const entmaxkv_q8_cache* cache, const float* weights,
                          const int32_t* seq_ids, const int32_t* count, int32_t n_seqs, int32_t keep, int32_t above,
                          int32_t sinks, int32_t recent, float* weights_out, int32_t* lens_out, int32_t* free_pages,
                          const int32_t* free_count, int32_t* free_count_out, void* workspace, size_t workspace_bytes,
                          void* stream) {
  int st;
  if ((st = check_evict(cfg, n_seqs, keep)) || (st = check_q8_cache(cache))) return st;
  if (above < keep || sinks < 0 || recent < 0 || (long long)sinks + recent > keep) return ENTMAXKV_ERR_INVALID_ARG;
  if (n_seqs == 0) return ENTMAXKV_OK;
  if (!seq_ids || !lens_out || !free_pages || !free_count || !free_count_out) return ENTMAXKV_ERR_INVALID_ARG;
  if (weights ? !weights_out || ((uintptr_t)weights & 15u) : sinks + recent < keep) return ENTMAXKV_ERR_INVALID_ARG;
  if (!workspace || ((uintptr_t)workspace & 255u) || workspace_bytes < evict_bytes(*cfg, n_seqs, keep))
    return ENTMAXKV_ERR_WORKSPACE_TOO_SMALL;
  const int sms = device_sms();
  if (sms < 1) return ENTMAXKV_ERR_CUDA;
  return code_of(launch_evict(cache_of(cfg, cache), seq_ids, count, n_seqs, keep, above, sinks, recent, weights, weights_out,
                              lens_out, free_pages, free_count, free_count_out, cfg->kv_dtype == ENTMAXKV_I8, workspace,
                              sms, (cudaStream_t)stream));
}

}  // extern "C"
