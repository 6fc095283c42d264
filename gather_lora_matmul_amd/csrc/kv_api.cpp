// Entry points of the KV cache in the unified pool (layout, write, read,
// attention, eviction) and of the verification of drafted tokens, chains and
// trees: argument checks, then stream-ordered launches without allocation or
// device wait.
#include <cmath>

#include "kv.h"
#include "runtime.h"

using namespace lora;

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

lora_status hip_status(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(LORA_E_HIP, "%s launch: %s", what, hipGetErrorString(e));
  return LORA_OK;
}

// The cache's geometry in this pool; host-only pools have one too.
lora_status geometry(const lora_pool* p, const lora_kv_desc* d, KvTypes& ty, int32_t& T) {
  if (!p) return fail(LORA_E_ARG, "null pool");
  if (!d) return fail(LORA_E_ARG, "null cache description");
  if (p->act != LORA_F16 && p->act != LORA_BF16)
    return fail(LORA_E_UNSUPPORTED, "KV caches need a pool with 16-bit activations");
  if (d->dtype != p->act && d->dtype != LORA_FP8_E4M3)
    return fail(LORA_E_ARG, "cache dtype %d must be the activation dtype or LORA_FP8_E4M3", d->dtype);
  if (d->n_kv_heads < 1 || d->n_kv_heads > kKvMaxHeads)
    return fail(LORA_E_ARG, "n_kv_heads %d not in [1, %d]", d->n_kv_heads, kKvMaxHeads);
  if (d->head_dim != 64 && d->head_dim != 128)
    return fail(LORA_E_UNSUPPORTED, "head_dim %d (64 and 128 are built)", d->head_dim);
  ty.act = p->act;
  ty.kv = d->dtype;
  ty.D = d->head_dim;
  const int elt = elt_bytes(d->dtype), E = 16 / elt;
  const int64_t t = p->page_bytes / ((int64_t)d->head_dim * elt) / E * E;
  if (t < E) return fail(LORA_E_ARG, "a page of %lld bytes holds fewer than %d tokens of one head",
                         (long long)p->page_bytes, E);
  if (t > (1 << 20)) return fail(LORA_E_UNSUPPORTED, "pages of more than 2^20 tokens");
  T = (int32_t)t;
  return LORA_OK;
}

lora_status batch_sizes(const lora_kv_batch* b, int32_t T) {
  if (!b) return fail(LORA_E_ARG, "null batch");
  if (b->n_seqs < 0 || b->n_seqs > kKvMaxSeqs)
    return fail(LORA_E_ARG, "n_seqs %d not in [0, %d]", b->n_seqs, kKvMaxSeqs);
  if (b->n_tokens < 0 || b->n_tokens > (1 << 24))
    return fail(LORA_E_ARG, "n_tokens %d not in [0, 2^24]", b->n_tokens);
  if (b->max_q_len < 0 || b->max_q_len > b->n_tokens)
    return fail(LORA_E_ARG, "max_q_len %d not in [0, n_tokens]", b->max_q_len);
  if (b->max_blocks < 1 || (int64_t)b->max_blocks * T > (1 << 28))
    return fail(LORA_E_ARG, "max_blocks %d (a sequence holds 1 block to 2^28 tokens)", b->max_blocks);
  return LORA_OK;
}

lora_status view_of(const lora_pool* p, const lora_kv_desc* d, const lora_kv_batch* b, KvTypes& ty,
                    KvView& v) {
  int32_t T = 0;
  lora_status st = geometry(p, d, ty, T);
  if (st) return st;
  st = batch_sizes(b, T);
  if (st) return st;
  if (b->n_seqs > 0 && (!b->q_start_dev || !b->kv_len_dev || !b->table_dev))
    return fail(LORA_E_ARG, "null batch pointer");
  if (((uintptr_t)b->q_start_dev | (uintptr_t)b->kv_len_dev | (uintptr_t)b->table_dev) & 3u)
    return fail(LORA_E_ARG, "batch pointers must be 4-byte aligned");
  if (ty.kv == LORA_FP8_E4M3 && (!d->scales_dev || !aligned16(d->scales_dev)))
    return fail(LORA_E_ARG, "FP8 caches need scales_dev (16-byte aligned)");
  v.pages = p->pages;
  v.scales = ty.kv == LORA_FP8_E4M3 ? d->scales_dev : nullptr;
  v.page_bytes = p->page_bytes;
  v.n_pages = (int32_t)p->n_pages;
  v.T = T;
  div_init(T, v.div_m, v.div_s);
  v.H = d->n_kv_heads;
  v.n_seqs = b->n_seqs;
  v.n_tokens = b->n_tokens;
  v.nb = b->max_blocks;
  v.q_start = b->q_start_dev;
  v.kv_len = b->kv_len_dev;
  v.table = b->table_dev;
  return LORA_OK;
}

// Asked last, so that a host-only pool reports a wrong argument first.
lora_status runnable(const lora_pool* p) {
  if (p->host_only) return fail(LORA_E_STATE, "host-only pool cannot run kernels");
  return LORA_OK;
}

lora_status check_rows(const void* ptr, int64_t ld, int64_t need, const char* what) {
  if (!ptr) return fail(LORA_E_ARG, "null %s", what);
  if (!aligned16(ptr)) return fail(LORA_E_ARG, "%s not 16-byte aligned", what);
  if (ld < need || (ld & 7)) return fail(LORA_E_ARG, "%s: row stride %lld (at least %lld, a multiple of 8)",
                                         what, (long long)ld, (long long)need);
  return LORA_OK;
}

}  // namespace

#define LORA_TRY(expr)          \
  do {                          \
    lora_status _s = (expr);    \
    if (_s != LORA_OK) return _s; \
  } while (0)

extern "C" {

lora_status lora_kv_layout(const lora_pool* p, const lora_kv_desc* d, int32_t* tokens_per_page,
                           int32_t* pages_per_block, size_t* scale_bytes) {
  clear_error();
  KvTypes ty;
  int32_t T = 0;
  LORA_TRY(geometry(p, d, ty, T));
  if (tokens_per_page) *tokens_per_page = T;
  if (pages_per_block) *pages_per_block = 2 * d->n_kv_heads;
  if (scale_bytes) *scale_bytes = ty.kv == LORA_FP8_E4M3 ? (size_t)p->n_pages * (size_t)T : 0;
  return LORA_OK;
}

static lora_status kv_copy(const lora_pool* p, const lora_kv_desc* d, const lora_kv_batch* b,
                           const void* k, const void* v, int64_t ld, bool write, void* stream) {
  KvTypes ty;
  KvView view;
  LORA_TRY(view_of(p, d, b, ty, view));
  if (b->n_seqs == 0 || b->n_tokens == 0) return LORA_OK;
  const int64_t row = (int64_t)d->n_kv_heads * d->head_dim;
  LORA_TRY(check_rows(k, ld, row, "k"));
  LORA_TRY(check_rows(v, ld, row, "v"));
  const int E = 16 / elt_bytes(ty.kv);
  if (((int64_t)b->n_tokens / E + 2 * (int64_t)b->n_seqs) * d->n_kv_heads > INT32_MAX - 8)
    return fail(LORA_E_UNSUPPORTED, "more than 2^31 token groups");
  LORA_TRY(runnable(p));
  if (write)
    return hip_status(launch_kv_write(ty, view, k, v, ld, (hipStream_t)stream), "kv_write");
  return hip_status(launch_kv_read(ty, view, const_cast<void*>(k), const_cast<void*>(v), ld,
                                   (hipStream_t)stream),
                    "kv_read");
}

lora_status lora_kv_write(lora_pool* p, const lora_kv_desc* d, const lora_kv_batch* b,
                          const void* k_dev, const void* v_dev, int64_t ld, void* stream) {
  clear_error();
  return kv_copy(p, d, b, k_dev, v_dev, ld, true, stream);
}

lora_status lora_kv_read(const lora_pool* p, const lora_kv_desc* d, const lora_kv_batch* b,
                         void* k_dev, void* v_dev, int64_t ld, void* stream) {
  clear_error();
  return kv_copy(p, d, b, k_dev, v_dev, ld, false, stream);
}

// What chooses among the kernels: a length of none is as wrong as any other, where there are tokens.
static int32_t longest(const lora_kv_batch* b) { return b->max_q_len < 1 ? 1 : b->max_q_len; }

static lora_status check_scale(float scale, int32_t window) {
  if (!(scale > 0.f) || !std::isfinite(scale * 2.8853900817779268f))   // (f16 over FP8 doubles it)
    return fail(LORA_E_ARG, "scale must be positive and finite");
  if (window < 0) return fail(LORA_E_ARG, "negative window");
  return LORA_OK;
}

static lora_status check_workspace(const void* ws, size_t bytes, size_t need, const char* call) {
  if (!ws || bytes < need)
    return fail(LORA_E_ARG, "workspace of %zu bytes, this call needs %zu (%s)", bytes, need, call);
  if ((uintptr_t)ws & 255u) return fail(LORA_E_ARG, "workspace not 256-byte aligned");
  return LORA_OK;
}

static lora_status check_heads(const lora_kv_desc* d, int32_t n_q_heads, const lora_kv_batch* b) {
  if (n_q_heads < d->n_kv_heads || n_q_heads % d->n_kv_heads)
    return fail(LORA_E_ARG, "n_q_heads %d is no multiple of n_kv_heads %d", n_q_heads, d->n_kv_heads);
  if ((int64_t)b->n_tokens * (n_q_heads / d->n_kv_heads) > (1 << 28))
    return fail(LORA_E_UNSUPPORTED, "more than 2^28 query rows of a head");
  return LORA_OK;
}

lora_status lora_kv_attend_workspace_size(const lora_pool* p, const lora_kv_desc* d,
                                          const lora_kv_batch* b, int32_t n_q_heads, size_t* bytes) {
  clear_error();
  KvTypes ty;
  int32_t T = 0;
  LORA_TRY(geometry(p, d, ty, T));
  LORA_TRY(batch_sizes(b, T));
  if (!bytes) return fail(LORA_E_ARG, "null size");
  LORA_TRY(check_heads(d, n_q_heads, b));
  *bytes = attend_workspace(ty, p->n_cu, n_q_heads / d->n_kv_heads, longest(b), b->n_seqs,
                            d->n_kv_heads);
  return LORA_OK;
}

// The arguments that both forms of the attention have; work: there is something to do.
static lora_status attend_args(const lora_pool* p, const lora_kv_desc* d, const lora_kv_batch* b,
                               const void* q_dev, int64_t q_ld, int32_t n_q_heads, float scale, int32_t window,
                               void* out_dev, int64_t out_ld, float* lse_dev, void* workspace_dev, size_t ws_bytes,
                               KvTypes& ty, AttendArgs& a, bool& work) {
  work = false;
  LORA_TRY(view_of(p, d, b, ty, a.kv));
  LORA_TRY(check_heads(d, n_q_heads, b));
  LORA_TRY(check_scale(scale, window));
  if (b->n_seqs == 0 || b->n_tokens == 0) return LORA_OK;
  if (attend_units(a.kv, n_q_heads / d->n_kv_heads, longest(b)) > INT32_MAX)
    return fail(LORA_E_UNSUPPORTED, "more than 2^31 units of work: split the call's tokens");
  const int64_t row = (int64_t)n_q_heads * d->head_dim;
  LORA_TRY(check_rows(q_dev, q_ld, row, "q"));
  LORA_TRY(check_rows(out_dev, out_ld, row, "out"));
  if ((uintptr_t)lse_dev & 3u) return fail(LORA_E_ARG, "lse not 4-byte aligned");
  LORA_TRY(check_workspace(workspace_dev, ws_bytes,
                           attend_workspace(ty, p->n_cu, n_q_heads / d->n_kv_heads, longest(b), b->n_seqs,
                                            d->n_kv_heads),
                           "lora_kv_attend_workspace_size"));
  a.q = q_dev;
  a.q_ld = q_ld;
  a.out = out_dev;
  a.out_ld = out_ld;
  a.lse = lse_dev;
  a.n_q_heads = n_q_heads;
  a.group = n_q_heads / d->n_kv_heads;
  div_init(a.group < 2 ? 2 : a.group, a.group_m, a.group_s);
  a.max_q_len = longest(b);
  a.two_terms = b->two_terms != 0;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.window = window > (1 << 28) ? 0 : window;   // no position is farther back; keeps differences in 32 bits
  a.ws = (char*)workspace_dev;
  a.n_cu = p->n_cu;
  work = true;
  return LORA_OK;
}

lora_status lora_kv_attend(const lora_pool* p, const lora_kv_desc* d, const lora_kv_batch* b,
                           const void* q_dev, int64_t q_ld, int32_t n_q_heads, float scale,
                           int32_t window, void* out_dev, int64_t out_ld, float* lse_dev,
                           void* workspace_dev, size_t ws_bytes, void* stream) {
  clear_error();
  KvTypes ty;
  AttendArgs a;
  bool work;
  LORA_TRY(attend_args(p, d, b, q_dev, q_ld, n_q_heads, scale, window, out_dev, out_ld, lse_dev, workspace_dev,
                       ws_bytes, ty, a, work));
  if (!work) return LORA_OK;
  LORA_TRY(runnable(p));
  return hip_status(launch_attend(ty, a, (hipStream_t)stream), "kv_attend");
}

static lora_status tree_words(int32_t words) {
  if (words < 1 || words > kTreeTokens / 64)
    return fail(LORA_E_ARG, "words %d not in [1, %d]", words, kTreeTokens / 64);
  return LORA_OK;
}

lora_status lora_kv_tree_build(int32_t n_seqs, int32_t n_tokens, const int32_t* q_start_dev,
                               const int32_t* parent_dev, int32_t words, int32_t window, uint64_t* seen_dev,
                               int32_t* depth_dev, void* stream) {
  clear_error();
  if (n_seqs < 0 || n_seqs > kKvMaxSeqs) return fail(LORA_E_ARG, "n_seqs %d not in [0, %d]", n_seqs, kKvMaxSeqs);
  if (n_tokens < 0 || n_tokens > (1 << 24)) return fail(LORA_E_ARG, "n_tokens %d not in [0, 2^24]", n_tokens);
  LORA_TRY(tree_words(words));
  if (window < 0) return fail(LORA_E_ARG, "negative window");
  if (n_seqs == 0 || n_tokens == 0) return LORA_OK;
  if (!q_start_dev || !parent_dev || !seen_dev || !depth_dev) return fail(LORA_E_ARG, "null device pointer");
  if (((uintptr_t)q_start_dev | (uintptr_t)parent_dev | (uintptr_t)depth_dev) & 3u)
    return fail(LORA_E_ARG, "pointer not 4-byte aligned");
  if ((uintptr_t)seen_dev & 7u) return fail(LORA_E_ARG, "seen not 8-byte aligned");
  TreeBuildArgs a;
  a.n_seqs = n_seqs;
  a.n_tokens = n_tokens;
  a.words = words;
  a.window = window;
  a.q_start = q_start_dev;
  a.parent = parent_dev;
  a.seen = seen_dev;
  a.depth = depth_dev;
  return hip_status(launch_tree_build(a, (hipStream_t)stream), "kv_tree_build");
}

lora_status lora_kv_attend_tree(const lora_pool* p, const lora_kv_desc* d, const lora_kv_batch* b,
                                const lora_kv_tree* tree, const void* q_dev, int64_t q_ld, int32_t n_q_heads,
                                float scale, int32_t window, void* out_dev, int64_t out_ld, float* lse_dev,
                                void* workspace_dev, size_t ws_bytes, void* stream) {
  clear_error();
  KvTypes ty;
  TreeArgs a;
  bool work;
  LORA_TRY(attend_args(p, d, b, q_dev, q_ld, n_q_heads, scale, window, out_dev, out_ld, lse_dev, workspace_dev,
                       ws_bytes, ty, a, work));
  if (!tree) return fail(LORA_E_ARG, "null tree");
  LORA_TRY(tree_words(tree->words));
  if (!work) return LORA_OK;
  if (!tree->seen_dev || ((uintptr_t)tree->seen_dev & 7u)) return fail(LORA_E_ARG, "seen null or not 8-byte aligned");
  if (window > 0 && !tree->depth_dev) return fail(LORA_E_ARG, "a window needs the tokens' depths");
  if ((uintptr_t)tree->depth_dev & 3u) return fail(LORA_E_ARG, "depth not 4-byte aligned");
  LORA_TRY(runnable(p));
  a.seen = tree->seen_dev;
  a.depth = tree->depth_dev;
  a.words = tree->words;
  return hip_status(launch_attend_tree(ty, a, (hipStream_t)stream), "kv_attend_tree");
}

// Weights [n_seqs][n_kv_heads][w_ld] of cached tokens.
static lora_status check_weights(const void* ptr, int64_t w_ld, const char* what) {
  if (!ptr || ((uintptr_t)ptr & 3u)) return fail(LORA_E_ARG, "%s null or not 4-byte aligned", what);
  if (w_ld < 1 || w_ld > (1 << 28)) return fail(LORA_E_ARG, "w_ld %lld not in [1, 2^28]", (long long)w_ld);
  return LORA_OK;
}

lora_status lora_kv_weigh_workspace_size(const lora_pool* p, const lora_kv_desc* d, const lora_kv_batch* b,
                                         int32_t n_q_heads, size_t* bytes) {
  clear_error();
  KvTypes ty;
  int32_t T = 0;
  LORA_TRY(geometry(p, d, ty, T));
  LORA_TRY(batch_sizes(b, T));
  if (!bytes) return fail(LORA_E_ARG, "null size");
  LORA_TRY(check_heads(d, n_q_heads, b));
  *bytes = weigh_workspace(p->n_cu, n_q_heads / d->n_kv_heads, longest(b));
  return LORA_OK;
}

lora_status lora_kv_weigh(const lora_pool* p, const lora_kv_desc* d, const lora_kv_batch* b, const void* q_dev,
                          int64_t q_ld, int32_t n_q_heads, float scale, int32_t window, const float* lse_dev,
                          float decay, const float* before_dev, float* weights_dev, int64_t w_ld,
                          void* workspace_dev, size_t ws_bytes, void* stream) {
  clear_error();
  KvTypes ty;
  WeighArgs a;
  LORA_TRY(view_of(p, d, b, ty, a.kv));
  LORA_TRY(check_heads(d, n_q_heads, b));
  LORA_TRY(check_scale(scale, window));
  if (!(decay >= 0.f) || !(decay <= 1.f)) return fail(LORA_E_ARG, "decay not in [0, 1]");
  if (b->n_seqs == 0) return LORA_OK;
  if (weigh_units(a.kv) > INT32_MAX)
    return fail(LORA_E_UNSUPPORTED, "more than 2^31 tiles of cached tokens: split the call's sequences");
  LORA_TRY(check_weights(weights_dev, w_ld, "weights"));
  if ((uintptr_t)before_dev & 3u) return fail(LORA_E_ARG, "before not 4-byte aligned");
  if (b->n_tokens > 0) {
    LORA_TRY(check_rows(q_dev, q_ld, (int64_t)n_q_heads * d->head_dim, "q"));
    if (!lse_dev || ((uintptr_t)lse_dev & 3u)) return fail(LORA_E_ARG, "lse null or not 4-byte aligned");
  }
  const size_t need = weigh_workspace(p->n_cu, n_q_heads / d->n_kv_heads, longest(b));
  if (need) LORA_TRY(check_workspace(workspace_dev, ws_bytes, need, "lora_kv_weigh_workspace_size"));
  LORA_TRY(runnable(p));
  a.q = q_dev;
  a.q_ld = q_ld;
  a.lse = lse_dev;
  a.before = before_dev;
  a.weights = weights_dev;
  a.w_ld = w_ld;
  a.n_q_heads = n_q_heads;
  a.group = n_q_heads / d->n_kv_heads;
  div_init(a.group < 2 ? 2 : a.group, a.group_m, a.group_s);
  a.max_q_len = longest(b);
  a.scale_log2 = scale * 1.4426950408889634f;
  a.decay = decay;
  a.window = window > (1 << 28) ? 0 : window;
  a.ws = (char*)workspace_dev;
  a.n_cu = p->n_cu;
  return hip_status(launch_weigh(ty, a, (hipStream_t)stream), "kv_weigh");
}

lora_status lora_kv_select_workspace_size(const lora_pool* p, const lora_kv_desc* d, const lora_kv_batch* b,
                                          size_t* bytes) {
  clear_error();
  KvTypes ty;
  int32_t T = 0;
  LORA_TRY(geometry(p, d, ty, T));
  LORA_TRY(batch_sizes(b, T));
  if (!bytes) return fail(LORA_E_ARG, "null size");
  *bytes = select_workspace(b->n_seqs, d->n_kv_heads, (int64_t)b->max_blocks * T);
  return LORA_OK;
}

lora_status lora_kv_select(const lora_pool* p, const lora_kv_desc* d, const lora_kv_batch* b,
                           const float* weights_dev, int64_t w_ld, int32_t budget, int32_t sinks, int32_t recent,
                           int32_t* keep_dev, int64_t keep_ld, int32_t* n_keep_dev, void* workspace_dev,
                           size_t ws_bytes, void* stream) {
  clear_error();
  KvTypes ty;
  SelectArgs a;
  LORA_TRY(view_of(p, d, b, ty, a.kv));
  if (budget < 0 || sinks < 0 || recent < 0 || (int64_t)sinks + recent > budget)
    return fail(LORA_E_ARG, "budget %d, of which %d first and %d latest tokens", budget, sinks, recent);
  if (b->n_seqs == 0) return LORA_OK;
  LORA_TRY(check_weights(weights_dev, w_ld, "weights"));
  if (keep_ld < budget) return fail(LORA_E_ARG, "keep_ld %lld < budget %d", (long long)keep_ld, budget);
  if ((!keep_dev && budget > 0) || ((uintptr_t)keep_dev & 3u) || !n_keep_dev || ((uintptr_t)n_keep_dev & 3u))
    return fail(LORA_E_ARG, "keep or n_keep null or not 4-byte aligned");
  LORA_TRY(check_workspace(workspace_dev, ws_bytes, select_workspace(b->n_seqs, d->n_kv_heads, (int64_t)b->max_blocks * a.kv.T),
                           "lora_kv_select_workspace_size"));
  LORA_TRY(runnable(p));
  a.weights = weights_dev;
  a.w_ld = w_ld;
  a.budget = budget;
  a.sinks = sinks;
  a.recent = recent;
  a.keep = keep_dev;
  a.keep_ld = keep_ld;
  a.n_keep = n_keep_dev;
  a.ws = (char*)workspace_dev;
  return hip_status(launch_select(a, (hipStream_t)stream), "kv_select");
}

lora_status lora_kv_compact(lora_pool* p, const lora_kv_desc* d, const lora_kv_batch* b, const int32_t* keep_dev,
                            int32_t keep_heads, int64_t keep_ld, const int32_t* n_keep_dev, int32_t from_new,
                            float* weights_dev, int64_t w_ld, void* stream) {
  clear_error();
  KvTypes ty;
  CompactArgs a;
  LORA_TRY(view_of(p, d, b, ty, a.kv));
  if (keep_heads != 1 && keep_heads != d->n_kv_heads)
    return fail(LORA_E_ARG, "keep_heads %d is neither 1 nor n_kv_heads", keep_heads);
  if (keep_ld < 0) return fail(LORA_E_ARG, "negative keep_ld");
  if (b->n_seqs == 0 || keep_ld == 0) return LORA_OK;
  if (!keep_dev || ((uintptr_t)keep_dev & 3u) || !n_keep_dev || ((uintptr_t)n_keep_dev & 3u))
    return fail(LORA_E_ARG, "keep or n_keep null or not 4-byte aligned");
  if (weights_dev) LORA_TRY(check_weights(weights_dev, w_ld, "weights"));
  LORA_TRY(runnable(p));
  a.keep = keep_dev;
  a.keep_ld = keep_ld;
  a.keep_heads = keep_heads;
  a.n_keep = n_keep_dev;
  a.from_new = from_new != 0;
  a.weights = weights_dev;
  a.w_ld = w_ld;
  return hip_status(launch_compact(ty, a, (hipStream_t)stream), "kv_compact");
}

static lora_status verify_sizes(int32_t n_seqs, int32_t vocab) {
  if (n_seqs < 0 || n_seqs > 65535) return fail(LORA_E_ARG, "n_seqs %d not in [0, 65535]", n_seqs);
  if (vocab < 1 || vocab > (1 << 18)) return fail(LORA_E_ARG, "vocab %d not in [1, 2^18]", vocab);
  return LORA_OK;
}

lora_status lora_spec_verify_workspace_size(int32_t n_seqs, int32_t vocab, size_t* bytes) {
  clear_error();
  LORA_TRY(verify_sizes(n_seqs, vocab));
  if (!bytes) return fail(LORA_E_ARG, "null size");
  *bytes = verify_workspace(n_seqs, vocab);
  return LORA_OK;
}

lora_status lora_spec_verify(const lora_verify_desc* d, void* workspace_dev, size_t ws_bytes,
                             void* stream) {
  clear_error();
  if (!d) return fail(LORA_E_ARG, "null description");
  LORA_TRY(verify_sizes(d->n_seqs, d->vocab));
  if (d->n_tokens < 0 || d->n_drafts < 0 || d->n_drafts > d->n_tokens)
    return fail(LORA_E_ARG, "n_tokens %d, n_drafts %d", d->n_tokens, d->n_drafts);
  if (d->dtype != LORA_F32 && d->dtype != LORA_F16 && d->dtype != LORA_BF16)
    return fail(LORA_E_ARG, "probabilities of dtype %d", d->dtype);
  if (d->n_seqs == 0) return LORA_OK;
  const uintptr_t elt = (uintptr_t)elt_bytes(d->dtype);
  if (!d->q_start_dev || !d->u_sample_dev || !d->n_out_dev) return fail(LORA_E_ARG, "null device pointer");
  if (d->n_tokens > 0) {
    if (!d->target_dev || !d->tokens_dev) return fail(LORA_E_ARG, "null device pointer");
    if (d->target_ld < d->vocab) return fail(LORA_E_ARG, "target_ld %lld < vocab", (long long)d->target_ld);
  }
  if (d->n_drafts > 0) {
    if (!d->drafted_dev || !d->u_accept_dev) return fail(LORA_E_ARG, "null device pointer");
    if (d->draft_dev && d->draft_ld < d->vocab)
      return fail(LORA_E_ARG, "draft_ld %lld < vocab", (long long)d->draft_ld);
  }
  if (((uintptr_t)d->q_start_dev | (uintptr_t)d->drafted_dev | (uintptr_t)d->u_accept_dev |
       (uintptr_t)d->u_sample_dev | (uintptr_t)d->tokens_dev | (uintptr_t)d->n_out_dev) & 3u)
    return fail(LORA_E_ARG, "pointer not 4-byte aligned");
  if (((uintptr_t)d->target_dev | (uintptr_t)d->draft_dev) & (elt - 1))
    return fail(LORA_E_ARG, "probabilities not aligned to their elements");
  const size_t need = verify_workspace(d->n_seqs, d->vocab);
  if (!workspace_dev || ws_bytes < need)
    return fail(LORA_E_ARG, "workspace of %zu bytes, this call needs %zu (lora_spec_verify_workspace_size)",
                ws_bytes, need);
  if (!aligned16(workspace_dev)) return fail(LORA_E_ARG, "workspace not 16-byte aligned");
  VerifyArgs a;
  a.n_seqs = d->n_seqs;
  a.n_tokens = d->n_tokens;
  a.n_drafts = d->n_drafts;
  a.vocab = d->vocab;
  a.dtype = d->dtype;
  a.target_ld = d->target_ld;
  a.draft_ld = d->draft_ld;
  a.q_start = d->q_start_dev;
  a.drafted = d->drafted_dev;
  a.target = d->target_dev;
  a.draft = d->draft_dev;
  a.u_accept = d->u_accept_dev;
  a.u_sample = d->u_sample_dev;
  a.tokens = d->tokens_dev;
  a.n_out = d->n_out_dev;
  a.ws = (char*)workspace_dev;
  return hip_status(launch_verify(a, (hipStream_t)stream), "spec_verify");
}

lora_status lora_spec_verify_tree_workspace_size(int32_t n_seqs, int32_t vocab, size_t* bytes) {
  clear_error();
  LORA_TRY(verify_sizes(n_seqs, vocab));
  if (!bytes) return fail(LORA_E_ARG, "null size");
  *bytes = tree_verify_workspace(n_seqs, vocab);
  return LORA_OK;
}

lora_status lora_spec_verify_tree(const lora_tree_verify_desc* d, void* workspace_dev, size_t ws_bytes,
                                  void* stream) {
  clear_error();
  if (!d) return fail(LORA_E_ARG, "null description");
  LORA_TRY(verify_sizes(d->n_seqs, d->vocab));
  if (d->n_tokens < 0) return fail(LORA_E_ARG, "n_tokens %d", d->n_tokens);
  if (d->dtype != LORA_F32 && d->dtype != LORA_F16 && d->dtype != LORA_BF16)
    return fail(LORA_E_ARG, "probabilities of dtype %d", d->dtype);
  if (d->path_ld < 1) return fail(LORA_E_ARG, "path_ld %d < 1", d->path_ld);
  if (d->n_seqs == 0) return LORA_OK;
  if (!d->q_start_dev || !d->u_sample_dev || !d->tokens_dev || !d->path_dev || !d->n_out_dev)
    return fail(LORA_E_ARG, "null device pointer");
  if (d->n_tokens > 0) {
    if (!d->parent_dev || !d->drafted_dev || !d->target_dev || !d->u_accept_dev)
      return fail(LORA_E_ARG, "null device pointer");
    if (d->target_ld < d->vocab) return fail(LORA_E_ARG, "target_ld %lld < vocab", (long long)d->target_ld);
  }
  if (((uintptr_t)d->q_start_dev | (uintptr_t)d->parent_dev | (uintptr_t)d->drafted_dev |
       (uintptr_t)d->u_accept_dev | (uintptr_t)d->u_sample_dev | (uintptr_t)d->tokens_dev |
       (uintptr_t)d->path_dev | (uintptr_t)d->n_out_dev) & 3u)
    return fail(LORA_E_ARG, "pointer not 4-byte aligned");
  if ((uintptr_t)d->target_dev & ((uintptr_t)elt_bytes(d->dtype) - 1))
    return fail(LORA_E_ARG, "probabilities not aligned to their elements");
  const size_t need = tree_verify_workspace(d->n_seqs, d->vocab);
  if (!workspace_dev || ws_bytes < need)
    return fail(LORA_E_ARG, "workspace of %zu bytes, this call needs %zu (lora_spec_verify_tree_workspace_size)",
                ws_bytes, need);
  if (!aligned16(workspace_dev)) return fail(LORA_E_ARG, "workspace not 16-byte aligned");
  TreeVerifyArgs a;
  a.n_seqs = d->n_seqs;
  a.n_tokens = d->n_tokens;
  a.vocab = d->vocab;
  a.dtype = d->dtype;
  a.path_ld = d->path_ld;
  a.target_ld = d->target_ld;
  a.q_start = d->q_start_dev;
  a.parent = d->parent_dev;
  a.drafted = d->drafted_dev;
  a.target = d->target_dev;
  a.u_accept = d->u_accept_dev;
  a.u_sample = d->u_sample_dev;
  a.tokens = d->tokens_dev;
  a.path = d->path_dev;
  a.n_out = d->n_out_dev;
  a.ws = (char*)workspace_dev;
  return hip_status(launch_tree_verify(a, (hipStream_t)stream), "spec_verify_tree");
}

}  // extern "C"
