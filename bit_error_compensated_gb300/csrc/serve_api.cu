// serve_api.cu -- host side of the operators of a serving step: argument
// checks and launches (contracts in include/echo.h).
#include <climits>
#include <cmath>
#include <cstring>

#include "matrix_check.h"
#include "serve_common.h"

namespace {
using namespace echo;

constexpr int64_t kMaxTokens = ECHO_BATCH_MAX_TOKENS;

int check_cache(const echo_cache* c) {
  if (c == nullptr) return ECHO_ERR_ARG;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return ECHO_ERR_UNSUPPORTED;
  if (c->bits != 4 && c->bits != 8) return ECHO_ERR_UNSUPPORTED;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128 && c->page_size != 256)
    return ECHO_ERR_UNSUPPORTED;
  if (c->heads < 1 || c->pages < 0) return ECHO_ERR_SHAPE;
  if (c->heads > ECHO_CACHE_MAX_HEADS || c->pages > INT_MAX) return ECHO_ERR_UNSUPPORTED;
  if (c->pages > 0 && (c->codes == nullptr || c->meta == nullptr)) return ECHO_ERR_ARG;
  return on_boundary(c->codes, 16) && on_boundary(c->meta, 16) ? ECHO_OK : ECHO_ERR_ALIGN;
}

bool empty(const echo_batch* b) { return b->sequences == 0 || b->tokens == 0; }

int check_batch(const echo_batch* b, const echo_cache* c) {
  if (b == nullptr) return ECHO_ERR_ARG;
  if (b->sequences < 0 || b->tokens < 0 || b->table_pages < 0) return ECHO_ERR_SHAPE;
  if (b->sequences > kMaxTokens || b->tokens > kMaxTokens || b->table_pages > kMostPlaces / c->page_size)
    return ECHO_ERR_UNSUPPORTED;
  if (empty(b)) return ECHO_OK;
  if (b->sequences > 1 && (b->ld_table < b->table_pages || b->ld_table > kMaxExtent)) return ECHO_ERR_SHAPE;
  if (b->starts == nullptr || b->lengths == nullptr || (b->table == nullptr && b->table_pages > 0)) return ECHO_ERR_ARG;
  return on_boundary(b->starts, 4) && on_boundary(b->lengths, 4) && on_boundary(b->table, 4) ? ECHO_OK : ECHO_ERR_ALIGN;
}

// Values of [tokens][heads][dim]: an output's must not share an element.
int check_heads(const echo_heads* h, int64_t tokens, int64_t heads, int64_t dim, int size, bool output) {
  if (h == nullptr || h->data == nullptr) return ECHO_ERR_ARG;
  if (!on_boundary(h->data, size)) return ECHO_ERR_ALIGN;
  const int64_t ld = tokens > 1 ? h->ld : 0, stride = heads > 1 ? h->head_stride : 0;
  if (ld < 0 || stride < 0 || ld > kMaxExtent || stride > kMaxExtent) return ECHO_ERR_SHAPE;
  if (!output) return ECHO_OK;
  if (heads > 1 && stride < dim) return ECHO_ERR_SHAPE;
  if (tokens > 1 && ld < dim) return ECHO_ERR_SHAPE;
  const bool inner = tokens == 1 || ld >= (heads - 1) * stride + dim;
  const bool outer = heads == 1 || stride >= (tokens - 1) * ld + dim;
  return inner || outer ? ECHO_OK : ECHO_ERR_SHAPE;
}
Region of_heads(const echo_heads* h, int64_t tokens, int64_t heads, int64_t dim, int size) {
  if (h == nullptr || h->data == nullptr) return Region();
  const int64_t ld = tokens > 1 ? h->ld : 0, stride = heads > 1 ? h->head_stride : 0;
  if (stride > ld && tokens > 1) return region(h->data, heads, (tokens - 1) * ld + dim, stride, size);
  return region(h->data, tokens, (heads - 1) * stride + dim, ld, size);
}

int add_cache(const echo_cache* c, Region* r) {
  const int64_t groups = c->pages * 2 * c->heads * c->page_size, row = c->head_dim * c->bits / 8;
  r[0] = region(c->codes, c->pages > 0 ? 1 : 0, groups * row, groups * row, 1);
  r[1] = region(c->meta, c->pages > 0 ? 1 : 0, groups, groups, 4);
  return 2;
}
int add_batch(const echo_batch* b, Region* r) {
  r[0] = region(b->starts, 1, b->sequences + 1, b->sequences + 1, 4);
  r[1] = region(b->lengths, 1, b->sequences, b->sequences, 4);
  r[2] = region(b->table, b->sequences, b->table_pages, b->ld_table, 4);
  return 3;
}
bool clear_of_all(const Region& mine, const Region* r, int n) {
  for (int i = 0; i < n; ++i)
    if (overlaps(mine, r[i])) return false;
  return true;
}

CacheArgs cache_args(const echo_cache* c) {
  CacheArgs a;
  a.codes = static_cast<uint8_t*>(c->codes);
  a.meta = static_cast<uint32_t*>(c->meta);
  a.pages = c->pages;
  a.heads = (int)c->heads;
  a.head_dim = (int)c->head_dim;
  a.bits = (int)c->bits;
  a.page_shift = 0;
  while ((1 << a.page_shift) < c->page_size) ++a.page_shift;
  return a;
}
BatchArgs batch_args(const echo_batch* b) {
  BatchArgs a;
  a.starts = b->starts;
  a.lengths = b->lengths;
  a.table = b->table;
  a.ld_table = b->ld_table;
  a.sequences = (int)b->sequences;
  a.tokens = (int)b->tokens;
  a.table_pages = (int)b->table_pages;
  return a;
}
HeadsArgs heads_args(const echo_heads* h) {
  HeadsArgs a = {nullptr, 0, 0};
  if (h != nullptr) a = {h->data, h->ld, h->head_stride};
  return a;
}

int check_rows(const echo_cache* c, const echo_batch* b, int dtype, const echo_heads* k, const echo_heads* v, bool read) {
  if (!known_dtype(dtype)) return ECHO_ERR_UNSUPPORTED;
  ECHO_TRY(check_cache(c));
  ECHO_TRY(check_batch(b, c));
  if (empty(b)) return ECHO_OK;
  const int size = elem_size(dtype);
  const echo_heads* both[2] = {k, v};
  Region r[7];                           // the cache's two, the batch's three, k and v
  int n = add_cache(c, r);
  if (overlaps(r[0], r[1])) return ECHO_ERR_ARG;
  if (read) n += add_batch(b, r + n);
  for (int i = 0; i < 2; ++i) {
    if (read && (both[i] == nullptr || both[i]->data == nullptr)) continue;
    ECHO_TRY(check_heads(both[i], b->tokens, c->heads, c->head_dim, size, read));
    const Region mine = of_heads(both[i], b->tokens, c->heads, c->head_dim, size);
    if (!clear_of_all(mine, r, n)) return ECHO_ERR_ARG;
    if (read) r[n++] = mine;
  }
  if (!read) {                           // the cache is written: the batch's arrays lie elsewhere
    Region given[3];
    add_batch(b, given);
    for (const Region& g : given)
      if (!clear_of_all(g, r, 2)) return ECHO_ERR_ARG;
  }
  return ECHO_OK;
}

RowsArgs rows_args(const echo_cache* c, const echo_batch* b, const echo_heads* k, const echo_heads* v) {
  return {cache_args(c), batch_args(b), heads_args(k), heads_args(v)};
}

int check_weights(int64_t ranks, int64_t tokens, int64_t channels, int64_t depth, int dtype, int64_t group) {
  ECHO_TRY(check_sizes(ranks, tokens, channels, depth));
  if (!known_dtype(dtype)) return ECHO_ERR_UNSUPPORTED;
  return group == 64 || group == 128 || group == 256 ? ECHO_OK : ECHO_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" {

int echo_cache_append(const echo_cache* cache, const echo_batch* batch, int dtype, const echo_heads* k,
                      const echo_heads* v, void* stream) {
  ECHO_TRY(check_rows(cache, batch, dtype, k, v, false));
  if (empty(batch)) return ECHO_OK;
  ECHO_OPS_CUDA(launch_append(rows_args(cache, batch, k, v), dtype, static_cast<cudaStream_t>(stream)));
  return ECHO_OK;
}

int echo_cache_read(const echo_cache* cache, const echo_batch* batch, int dtype, const echo_heads* k,
                    const echo_heads* v, void* stream) {
  ECHO_TRY(check_rows(cache, batch, dtype, k, v, true));
  if (empty(batch)) return ECHO_OK;
  ECHO_OPS_CUDA(launch_read(rows_args(cache, batch, k, v), dtype, static_cast<cudaStream_t>(stream)));
  return ECHO_OK;
}

static int check_attention_sizes(const echo_cache* cache, const echo_batch* batch, int64_t heads) {
  ECHO_TRY(check_cache(cache));
  ECHO_TRY(check_batch(batch, cache));
  if (heads < 1 || heads % cache->heads != 0) return ECHO_ERR_SHAPE;
  if (heads > INT_MAX / 2 || batch->tokens * heads > INT_MAX / 2) return ECHO_ERR_UNSUPPORTED;
  return ECHO_OK;
}

size_t echo_attention_workspace_bytes(const echo_cache* cache, const echo_batch* batch, int64_t heads) {
  if (check_attention_sizes(cache, batch, heads) != ECHO_OK || empty(batch)) return 0;
  int sms = 0;
  if (device_sms(&sms) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return (size_t)attention_bytes((int)cache->head_dim, sms);
}

int echo_attention(const echo_cache* cache, const echo_batch* batch, int64_t heads, int dtype, const echo_heads* q,
                   const echo_heads* out, float scale, int causal, int64_t window, float* lse, void* workspace,
                   size_t workspace_bytes, void* stream) {
  if (dtype != ECHO_BF16 && dtype != ECHO_F16) return ECHO_ERR_UNSUPPORTED;
  ECHO_TRY(check_attention_sizes(cache, batch, heads));
  if (!std::isfinite(scale) || (causal != 0 && causal != 1) || window < 0 || (window > 0 && !causal)) return ECHO_ERR_ARG;
  if (empty(batch)) return ECHO_OK;
  const int64_t tokens = batch->tokens, dim = cache->head_dim;
  ECHO_TRY(check_heads(q, tokens, heads, dim, 2, false));
  ECHO_TRY(check_heads(out, tokens, heads, dim, 2, true));
  if (!on_boundary(lse, 4)) return ECHO_ERR_ALIGN;
  Region r[9];
  int n = add_cache(cache, r);
  n += add_batch(batch, r + n);
  r[n++] = of_heads(q, tokens, heads, dim, 2);
  for (const Region& w : {of_heads(out, tokens, heads, dim, 2), region(lse, 1, tokens * heads, tokens * heads, 4)}) {
    if (!clear_of_all(w, r, n)) return ECHO_ERR_ARG;
    r[n++] = w;
  }
  int sms = 0;
  ECHO_OPS_CUDA(device_sms(&sms));
  const size_t need = (size_t)attention_bytes((int)dim, sms);
  if (workspace == nullptr || workspace_bytes < need) return ECHO_ERR_TOO_LARGE;
  if (!on_boundary(workspace, 16)) return ECHO_ERR_ALIGN;
  if (!clear_of_all(region(workspace, 1, (int64_t)need, (int64_t)need, 1), r, n)) return ECHO_ERR_ARG;
  AttentionArgs a;
  std::memset(&a, 0, sizeof(a));
  a.cache = cache_args(cache);
  a.batch = batch_args(batch);
  a.q = heads_args(q);
  a.out = heads_args(out);
  a.lse = lse;
  a.heads = (int)heads;
  a.group = (int)(heads / cache->heads);
  a.dtype = dtype;
  a.scale = scale;
  a.causal = causal;
  a.window = window > INT_MAX ? 0 : (int)window;          // no place is beyond that
  a.partial = static_cast<float*>(workspace);
  ECHO_OPS_CUDA(launch_attention(a, sms, static_cast<cudaStream_t>(stream)));
  return ECHO_OK;
}

int echo_quantize_weights(int64_t ranks, int64_t channels, int64_t depth, int dtype, int64_t group,
                          const echo_matrix* w, const echo_matrix* codes, const echo_matrix* meta, void* stream) {
  ECHO_TRY(check_weights(ranks, 0, channels, depth, dtype, group));
  const int size = elem_size(dtype);
  const int64_t bytes = (depth + 1) / 2, groups = (depth + group - 1) / group;
  ECHO_TRY(check_matrix(w, ranks, channels, depth, size, false));
  ECHO_TRY(check_matrix(codes, ranks, channels, bytes, 1, true));
  ECHO_TRY(check_matrix(meta, ranks, channels, groups, 4, true));
  if (channels == 0 || depth == 0) return ECHO_OK;
  Region in[2 * ECHO_MAX_RANKS];
  int n = 0;
  add_regions(w, ranks, channels, depth, size, in, &n);
  if (!clear_of(codes, ranks, channels, bytes, 1, in, n)) return ECHO_ERR_ARG;
  add_regions(codes, ranks, channels, bytes, 1, in, &n);
  if (!clear_of(meta, ranks, channels, groups, 4, in, n)) return ECHO_ERR_ARG;
  WeightsArgs a;
  a.w = w->data; a.ld_w = w->ld; a.rank_w = w->rank_stride;
  a.codes = static_cast<uint8_t*>(codes->data); a.ld_codes = codes->ld; a.rank_codes = codes->rank_stride;
  a.meta = static_cast<uint32_t*>(meta->data); a.ld_meta = meta->ld; a.rank_meta = meta->rank_stride;
  a.ranks = ranks; a.channels = channels; a.depth = depth;
  a.group = (int)group;
  ECHO_OPS_CUDA(launch_quantize_weights(a, dtype, static_cast<cudaStream_t>(stream)));
  return ECHO_OK;
}

int echo_linear_int4(int64_t ranks, int64_t tokens, int64_t channels, int64_t depth, int dtype, int64_t group,
                     const echo_matrix* x, const echo_matrix* codes, const echo_matrix* meta, const echo_matrix* out,
                     void* stream) {
  ECHO_TRY(check_weights(ranks, tokens, channels, depth, dtype, group));
  const int size = elem_size(dtype);
  const int64_t bytes = (depth + 1) / 2, groups = (depth + group - 1) / group;
  ECHO_TRY(check_matrix(x, ranks, tokens, depth, size, false));
  ECHO_TRY(check_matrix(codes, ranks, channels, bytes, 1, false));
  ECHO_TRY(check_matrix(meta, ranks, channels, groups, 4, false));
  ECHO_TRY(check_matrix(out, ranks, tokens, channels, size, true));
  if (tokens == 0 || channels == 0) return ECHO_OK;
  Region in[3 * ECHO_MAX_RANKS];
  int n = 0;
  add_regions(x, ranks, tokens, depth, size, in, &n);
  add_regions(codes, ranks, channels, bytes, 1, in, &n);
  add_regions(meta, ranks, channels, groups, 4, in, &n);
  if (!clear_of(out, ranks, tokens, channels, size, in, n)) return ECHO_ERR_ARG;
  Linear4Args p;
  p.x = x->data; p.ld_x = x->ld; p.rank_x = x->rank_stride;
  p.codes = static_cast<const uint8_t*>(codes->data); p.ld_codes = codes->ld; p.rank_codes = codes->rank_stride;
  p.meta = static_cast<const uint32_t*>(meta->data); p.ld_meta = meta->ld; p.rank_meta = meta->rank_stride;
  p.out = out->data; p.ld_out = out->ld; p.rank_out = out->rank_stride;
  p.ranks = ranks; p.tokens = tokens; p.channels = channels; p.depth = depth;
  p.group = (int)group;
  p.dtype = dtype;
  int sms = 0;
  ECHO_OPS_CUDA(device_sms(&sms));
  // (a launch has 65535 blocks of tokens at the most, of 8 to 32 each)
  constexpr int64_t kTokens = 65535 * 8;
  for (p.tokens = tokens; p.tokens > 0; p.tokens -= kTokens) {
    Linear4Args some = p;
    some.tokens = p.tokens < kTokens ? p.tokens : kTokens;
    ECHO_OPS_CUDA(launch_linear4(some, sms, static_cast<cudaStream_t>(stream)));
    p.x = static_cast<const char*>(p.x) + kTokens * p.ld_x * size;
    p.out = static_cast<char*>(p.out) + kTokens * p.ld_out * size;
  }
  return ECHO_OK;
}

int echo_serving_status(void* stream, int* status) {
  if (status == nullptr) return ECHO_ERR_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const StatusWord words[] = {rows_status(), attn_few_status(), attn_many_status(), weights_status()};
  constexpr int kWords = sizeof(words) / sizeof(words[0]);
  int word[kWords] = {};
  for (int i = 0; i < kWords; ++i) ECHO_OPS_CUDA(words[i].read(&word[i], s));
  ECHO_OPS_CUDA(cudaStreamSynchronize(s));
  int all = 0;
  for (int i = 0; i < kWords; ++i) {
    if (word[i]) ECHO_OPS_CUDA(words[i].clear(word[i], s));
    all |= word[i];
  }
  if (all) ECHO_OPS_CUDA(cudaStreamSynchronize(s));
  *status = all & kGaveUp ? ECHO_ERR_TIMEOUT
            : all & kBadPage ? ECHO_ERR_ARG
            : all & kBadRows ? ECHO_ERR_SHAPE
            : all & kNaNGroup ? ECHO_ERR_OVERFLOW : ECHO_OK;
  return ECHO_OK;
}

}  // extern "C"
