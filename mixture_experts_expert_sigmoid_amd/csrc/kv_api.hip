// Host side of the key-value cache and attention entry points: validation of
// the descriptors, workspace checks and launches. As in api.hip nothing is
// allocated, kept or synchronised.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "kv.h"
#include "launch.h"
#include "moe_mi355x.h"

static_assert(MOE_DEVERR_CACHE_PAGE == moe::kErrPage, "err bit");
static_assert(MOE_DEVERR_CACHE_FULL == moe::kErrFull, "err bit");
static_assert(MOE_DEVERR_CACHE_BUSY == moe::kErrBusy, "err bit");
static_assert(MOE_DEVERR_TREE == moe::kErrTree, "err bit");
static_assert(MOE_TREE_MAX == moe::kTreeMax, "limit");
static_assert(MOE_KV_BF16 == moe::KV_BF16 && MOE_KV_F16 == moe::KV_F16 &&
                  MOE_KV_E4M3 == moe::KV_E4M3,
              "formats");

namespace {

using moe::hip_fail;

constexpr int kMaxLayers = 1024;
constexpr long kMaxTokens = 1L << 28;      // of a table row

int check_cache(const moe_kv_cache* c) {
  if (!c) return MOE_ERR_NULL;
  if (c->fmt < MOE_KV_BF16 || c->fmt > MOE_KV_E4M3) return MOE_ERR_FORMAT;
  if (c->n_pages < 1 || c->page_size < 16 || c->page_size > 4096 || c->page_size % 16 ||
      c->n_heads < 1 || c->n_heads > 1024 ||
      (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256))
    return MOE_ERR_SHAPE;
  const long es = moe::kv_esize(c->fmt), unit = 16 / es;
  for (long s : {c->stride_page, c->stride_head, c->stride_tok})
    if (s < c->head_dim || s > (1L << 46) || s % unit) return MOE_ERR_SHAPE;
  if (c->stride_tok >= (1L << 30) / (16 * es)) return MOE_ERR_SHAPE;
  if (!c->k || !c->v) return MOE_ERR_NULL;
  if ((((uintptr_t)c->k) | ((uintptr_t)c->v)) & 15) return MOE_ERR_PARAM;
  const bool scaled = c->fmt == MOE_KV_E4M3;
  if (scaled && (!c->k_scale || !c->v_scale)) return MOE_ERR_NULL;
  if (!scaled && (c->k_scale || c->v_scale)) return MOE_ERR_PARAM;
  return MOE_OK;
}

int check_table(const moe_kv_table* t, bool refs) {
  if (!t || !t->table || !t->len || (refs && !t->refs)) return MOE_ERR_NULL;
  if (t->n_slots < 1 || t->max_pages < 1 || t->ld < t->max_pages || t->n_pages < 1 ||
      t->page_size < 16 || t->page_size > 4096 || t->page_size % 16 ||
      (long)t->max_pages * t->page_size > kMaxTokens)
    return MOE_ERR_SHAPE;
  return MOE_OK;
}

int check_pair(const moe_kv_cache* c, const moe_kv_table* t) {
  return c->page_size == t->page_size && c->n_pages == t->n_pages ? MOE_OK : MOE_ERR_SHAPE;
}

moe::KvCache dev_cache(const moe_kv_cache* c) {
  const long es = moe::kv_esize(c->fmt);
  return {(char*)c->k, (char*)c->v, c->stride_page * es, c->stride_head * es,
          c->stride_tok * es, c->k_scale, c->v_scale, c->fmt, c->n_pages, c->page_size,
          c->n_heads, c->head_dim};
}

moe::KvTable dev_table(const moe_kv_table* t) {
  return {t->table, t->len, t->refs, t->ld, t->n_slots, t->max_pages, t->n_pages,
          t->page_size, ((1UL << 32) + t->page_size / 16 - 1) / (t->page_size / 16)};
}

bool row_strides_ok(long row, long head, int D) {
  return row >= D && head >= D && row % 8 == 0 && head % 8 == 0 && row < (1L << 46) &&
         head < (1L << 46);
}

// the queries, outputs and scale of an attention call with keys of dk and values
// of dv; rows of q >= 0
int attn_rows(const moe_attn* at, int dk, int dv, long rows, moe::AttnArgs* a) {
  if (!isfinite(at->scale) || at->window < 0 || at->n_first < 0) return MOE_ERR_PARAM;
  if (rows > 0) {
    if (!at->q || !at->out) return MOE_ERR_NULL;
    if (!row_strides_ok(at->q_stride_row, at->q_stride_head, dk) ||
        !row_strides_ok(at->out_stride_row, at->out_stride_head, dv))
      return MOE_ERR_SHAPE;
    if ((((uintptr_t)at->q) | ((uintptr_t)at->out)) & 15) return MOE_ERR_PARAM;
  }
  a->q = (const char*)at->q;
  a->out = (char*)at->out;
  a->q_row = at->q_stride_row * 2;
  a->q_head = at->q_stride_head * 2;
  a->o_row = at->out_stride_row * 2;
  a->o_head = at->out_stride_head * 2;
  a->lse = at->lse;
  a->hq = at->n_heads;
  a->scale = at->scale * 1.44269504088896340736f;
  return MOE_OK;
}

// A window that no context of at most `most` tokens exceeds is none. What is left
// is at most kMaxTokens, so that position - window stays within 32 bits, for rows
// before a sequence's first position too.
void attn_window(const moe_attn* at, long most, moe::AttnArgs* a) {
  a->window = at->window < most ? at->window : 0;
  a->first = a->window ? (int)(at->n_first < most ? at->n_first : most) : 0;
}

// what the calls over a key-value cache ask of their arguments, and the arguments
// of the kernels
int attn_args(const moe_kv_cache* cache, const moe_kv_table* table, const int* slots, long n,
              long rows, const moe_attn* at, int* err_word, moe::AttnArgs* a) {
  int st = check_cache(cache);
  if (st) return st;
  st = check_table(table, false);
  if (st) return st;
  st = check_pair(cache, table);
  if (st) return st;
  if (!at || !err_word) return MOE_ERR_NULL;
  if (at->fmt != MOE_KV_BF16 && at->fmt != MOE_KV_F16) return MOE_ERR_FORMAT;
  if (cache->fmt != MOE_KV_E4M3 && cache->fmt != at->fmt) return MOE_ERR_FORMAT;
  if (n < 0 || n >= (1L << 20) || rows < 0 || at->n_heads < 1 ||
      at->n_heads % cache->n_heads || at->n_heads / cache->n_heads > 64)
    return MOE_ERR_SHAPE;
  if (rows > 0x7FFFFFFFL / at->n_heads) return MOE_ERR_SHAPE;
  *a = moe::AttnArgs{};
  st = attn_rows(at, cache->head_dim, cache->head_dim, rows, a);
  if (st) return st;
  a->c = dev_cache(cache);
  a->t = dev_table(table);
  a->slots = slots;
  a->n = (int)n;
  a->g = at->n_heads / cache->n_heads;
  attn_window(at, (long)table->max_pages * table->page_size, a);
  a->err = err_word;
  return MOE_OK;
}

bool ws_shape_ok(const moe_kv_cache* c, int n_heads) {
  return c && c->n_heads >= 1 && n_heads >= 1 && n_heads % c->n_heads == 0 &&
         n_heads / c->n_heads <= 64 &&
         (c->head_dim == 64 || c->head_dim == 128 || c->head_dim == 256);
}

// the layers' pointers in groups of kCopyLayers; returns a status
int copy_layers(const moe_kv_cache* layers, int n_layers, const moe_kv_table* table,
                moe::CopyLayers* out, int* n_out) {
  if (!layers) return MOE_ERR_NULL;
  if (n_layers < 1 || n_layers > kMaxLayers) return MOE_ERR_SHAPE;
  *n_out = 0;
  for (int i = 0; i < n_layers; ++i) {
    const moe_kv_cache* c = &layers[i];
    int st = check_cache(c);
    if (st) return st;
    if (table) {
      st = check_pair(c, table);
      if (st) return st;
    }
    const moe_kv_cache* f = &layers[0];
    if (c->fmt != f->fmt) return MOE_ERR_FORMAT;
    if (c->n_pages != f->n_pages || c->page_size != f->page_size ||
        c->n_heads != f->n_heads || c->head_dim != f->head_dim ||
        c->stride_page != f->stride_page || c->stride_head != f->stride_head ||
        c->stride_tok != f->stride_tok)
      return MOE_ERR_SHAPE;
    moe::CopyLayers& cl = out[i / moe::kCopyLayers];
    if (i % moe::kCopyLayers == 0) {
      const long es = moe::kv_esize(c->fmt), D = c->head_dim;
      cl.n = 0;
      cl.sp = c->stride_page * es;
      cl.sh = c->stride_head * es;
      cl.st = c->stride_tok * es;
      cl.hkv = c->n_heads;
      cl.ps = c->page_size;
      cl.row_bytes = (int)(D * es);
      cl.linear = (c->stride_tok == D && c->stride_head == D * c->page_size) ||
                  (c->stride_head == D && c->stride_tok == D * c->n_heads);
      ++*n_out;
    }
    cl.p[cl.n++] = (char*)c->k;
    if (c->v != c->k) cl.p[cl.n++] = (char*)c->v;     // (a latent cache has one array)
  }
  return MOE_OK;
}

int check_latent(const moe_latent_cache* c) {
  if (!c) return MOE_ERR_NULL;
  if (c->fmt < MOE_KV_BF16 || c->fmt > MOE_KV_E4M3) return MOE_ERR_FORMAT;
  if (c->n_pages < 1 || c->page_size < 16 || c->page_size > 4096 || c->page_size % 16 ||
      (c->latent_dim != 256 && c->latent_dim != 512) || c->rope_dim != moe::kLatRope)
    return MOE_ERR_SHAPE;
  const long es = moe::kv_esize(c->fmt), unit = 16 / es;
  for (long s : {c->stride_page, c->stride_tok})
    if (s < c->latent_dim + c->rope_dim || s > (1L << 46) || s % unit) return MOE_ERR_SHAPE;
  if (c->stride_tok >= (1L << 30) / (16 * es)) return MOE_ERR_SHAPE;
  if (!c->c) return MOE_ERR_NULL;
  if (((uintptr_t)c->c) & 15) return MOE_ERR_PARAM;
  const bool scaled = c->fmt == MOE_KV_E4M3;
  if (scaled && !c->scale) return MOE_ERR_NULL;
  if (!scaled && c->scale) return MOE_ERR_PARAM;
  return MOE_OK;
}

int check_latent_pair(const moe_latent_cache* c, const moe_kv_table* t) {
  return c->page_size == t->page_size && c->n_pages == t->n_pages ? MOE_OK : MOE_ERR_SHAPE;
}

// D: the latent vector's; one head, keys and values in one array
moe::KvCache dev_latent(const moe_latent_cache* c) {
  const long es = moe::kv_esize(c->fmt);
  return {(char*)c->c, (char*)c->c, c->stride_page * es, 0, c->stride_tok * es, c->scale,
          c->scale, c->fmt, c->n_pages, c->page_size, 1, c->latent_dim};
}

constexpr int kMaxGroups = (kMaxLayers + moe::kCopyLayers - 1) / moe::kCopyLayers;

int done(hipError_t e, const char* where) {
  return e == hipSuccess ? MOE_OK : hip_fail(e, where);
}

}  // namespace

extern "C" {

size_t moe_attn_decode_workspace_size(const moe_kv_cache* cache, long n, int n_heads) {
  if (!ws_shape_ok(cache, n_heads) || n < 0 || n >= (1L << 20)) return 0;
  return moe::decode_ws_bytes(n, n_heads, cache->n_heads, cache->head_dim,
                              cache->fmt == MOE_KV_E4M3);
}

int moe_attn_decode(const moe_kv_cache* cache, const moe_kv_table* table, const int* slots,
                    long n, const moe_attn* attn, int* err_word, void* ws, size_t ws_bytes,
                    void* stream) {
  moe::AttnArgs a;
  int st = attn_args(cache, table, slots, n, n, attn, err_word, &a);
  if (st) return st;
  if (!slots && n > table->n_slots) return MOE_ERR_SHAPE;
  if (n == 0) return MOE_OK;
  const size_t need = moe::decode_ws_bytes(n, a.hq, a.c.hkv, a.c.D, a.c.fmt == moe::KV_E4M3);
  if (!ws || ws_bytes < need || ((uintptr_t)ws & 15)) return MOE_ERR_WORKSPACE;
  a.part = (float*)ws;
  return done(moe::launch_attn_decode(a, attn->fmt, (hipStream_t)stream), "moe_attn_decode");
}

size_t moe_attn_prefill_workspace_size(const moe_kv_cache* cache, long n, long T,
                                       int n_heads) {
  if (!ws_shape_ok(cache, n_heads) || n < 0 || n >= (1L << 20) || T < 0 ||
      T > 0x7FFFFFFFL / n_heads)
    return 0;
  return moe::prefill_ws_bytes(n, T, n_heads, cache->n_heads, cache->head_dim);
}

int moe_attn_prefill(const moe_kv_cache* cache, const moe_kv_table* table, const int* slots,
                     long n, const int* cu_q, long T, const moe_attn* attn, int* err_word,
                     void* ws, size_t ws_bytes, void* stream) {
  moe::AttnArgs a;
  int st = attn_args(cache, table, slots, n, T, attn, err_word, &a);
  if (st) return st;
  if (!slots && n > table->n_slots) return MOE_ERR_SHAPE;
  if (n == 0 && T > 0) return MOE_ERR_SHAPE;
  if (T == 0) return MOE_OK;
  if (!cu_q) return MOE_ERR_NULL;
  const size_t need = moe::prefill_ws_bytes(n, T, a.hq, a.c.hkv, a.c.D);
  if (need > 0 && (!ws || ws_bytes < need || ((uintptr_t)ws & 15))) return MOE_ERR_WORKSPACE;
  a.cu = cu_q;
  a.T = T;
  a.part = (float*)ws;
  return done(moe::launch_attn_prefill(a, attn->fmt, (hipStream_t)stream),
              "moe_attn_prefill");
}

size_t moe_attn_tree_workspace_size(const moe_kv_cache* cache, long n, long T, int n_heads) {
  if (!ws_shape_ok(cache, n_heads) || n < 0 || n >= (1L << 20) || T < 0 ||
      T > 0x7FFFFFFFL / n_heads)
    return 0;
  return moe::tree_ws_bytes(n, T, n_heads, cache->n_heads, cache->head_dim);
}

int moe_attn_tree(const moe_kv_cache* cache, const moe_kv_table* table, const int* slots, long n,
                  const int* cu_q, long T, const int* parent, const moe_attn* attn, int* err_word,
                  void* ws, size_t ws_bytes, void* stream) {
  moe::AttnArgs a;
  int st = attn_args(cache, table, slots, n, T, attn, err_word, &a);
  if (st) return st;
  if (!slots && n > table->n_slots) return MOE_ERR_SHAPE;
  if (n == 0 && T > 0) return MOE_ERR_SHAPE;
  if (T == 0) return MOE_OK;
  if (!cu_q || !parent) return MOE_ERR_NULL;
  const size_t need = moe::tree_ws_bytes(n, T, a.hq, a.c.hkv, a.c.D);
  if (need > 0 && (!ws || ws_bytes < need || ((uintptr_t)ws & 15))) return MOE_ERR_WORKSPACE;
  a.cu = cu_q;
  a.T = T;
  a.parent = parent;
  a.part = (float*)ws;
  return done(moe::launch_attn_tree(a, attn->fmt, (hipStream_t)stream), "moe_attn_tree");
}

int moe_cache_append(const moe_kv_cache* cache, const moe_kv_table* table, const int* slots,
                     const int* start, const int* cu, long n, long T, int fmt, const void* k,
                     long k_stride_row, long k_stride_head, const void* v, long v_stride_row,
                     long v_stride_head, int* err_word, void* stream) {
  int st = check_cache(cache);
  if (st) return st;
  st = check_table(table, false);
  if (st) return st;
  st = check_pair(cache, table);
  if (st) return st;
  if (fmt != MOE_KV_BF16 && fmt != MOE_KV_F16) return MOE_ERR_FORMAT;
  if (cache->fmt != MOE_KV_E4M3 && cache->fmt != fmt) return MOE_ERR_FORMAT;
  if (n < 0 || n >= (1L << 20) || T < 0 || T >= (1L << 31) || (!cu && T != n) ||
      (n == 0 && T > 0) || (!slots && n > table->n_slots))
    return MOE_ERR_SHAPE;
  if (!err_word) return MOE_ERR_NULL;
  if (T == 0) return MOE_OK;
  if (!start || !k || !v) return MOE_ERR_NULL;
  const int D = cache->head_dim;
  if (!row_strides_ok(k_stride_row, k_stride_head, D) ||
      !row_strides_ok(v_stride_row, v_stride_head, D))
    return MOE_ERR_SHAPE;
  if ((((uintptr_t)k) | ((uintptr_t)v)) & 15) return MOE_ERR_PARAM;
  moe::AppendArgs a{dev_cache(cache), dev_table(table), slots, start, cu, (int)n, T,
                    (const char*)k, (const char*)v, k_stride_row * 2, k_stride_head * 2,
                    v_stride_row * 2, v_stride_head * 2, err_word};
  return done(moe::launch_append(a, fmt, (hipStream_t)stream), "moe_cache_append");
}

size_t moe_cache_workspace_size(const moe_kv_table* table, long n) {
  if (!table || table->n_pages < 1 || n < 0 || n >= (1L << 20)) return 0;
  return moe::cache_ws_bytes(table->n_pages, n);
}

int moe_cache_grow(const moe_kv_table* table, const int* slots, const int* n_new, long n,
                   int* start, int* err_word, void* ws, size_t ws_bytes, void* stream) {
  int st = check_table(table, true);
  if (st) return st;
  if (n < 0 || n >= (1L << 20) || (!slots && n > table->n_slots)) return MOE_ERR_SHAPE;
  if (!err_word) return MOE_ERR_NULL;
  if (n == 0) return MOE_OK;
  if (!n_new || !start) return MOE_ERR_NULL;
  if (!ws || ws_bytes < moe::cache_ws_bytes(table->n_pages, n) || ((uintptr_t)ws & 15))
    return MOE_ERR_WORKSPACE;
  return done(moe::launch_cache_grow(dev_table(table), slots, n_new, n, start, err_word, ws,
                                     (hipStream_t)stream),
              "moe_cache_grow");
}

int moe_cache_free(const moe_kv_table* table, const int* slots, long n, int* err_word,
                   void* stream) {
  int st = check_table(table, true);
  if (st) return st;
  if (n < 0 || n >= (1L << 20) || (!slots && n > table->n_slots)) return MOE_ERR_SHAPE;
  if (!err_word) return MOE_ERR_NULL;
  if (n == 0) return MOE_OK;
  return done(moe::launch_cache_free(dev_table(table), slots, n, err_word,
                                     (hipStream_t)stream),
              "moe_cache_free");
}

int moe_cache_trim(const moe_kv_table* table, const int* slots, long n, int window,
                   int n_first, int* err_word, void* stream) {
  int st = check_table(table, true);
  if (st) return st;
  if (n < 0 || n >= (1L << 20) || (!slots && n > table->n_slots)) return MOE_ERR_SHAPE;
  if (window < 1 || n_first < 0) return MOE_ERR_PARAM;
  if (!err_word) return MOE_ERR_NULL;
  if (n == 0) return MOE_OK;
  return done(moe::launch_cache_trim(dev_table(table), slots, n, window, n_first, err_word,
                                     (hipStream_t)stream),
              "moe_cache_trim");
}

int moe_cache_fork(const moe_kv_cache* layers, int n_layers, const moe_kv_table* table,
                   const int* src, const int* dst, long n, int* err_word, void* ws,
                   size_t ws_bytes, void* stream) {
  int st = check_table(table, true);
  if (st) return st;
  moe::CopyLayers cl[kMaxGroups];
  int n_cl = 0;
  st = copy_layers(layers, n_layers, table, cl, &n_cl);
  if (st) return st;
  if (n < 0 || n > 65535) return MOE_ERR_SHAPE;
  if (!err_word) return MOE_ERR_NULL;
  if (n == 0) return MOE_OK;
  if (!src || !dst) return MOE_ERR_NULL;
  if (!ws || ws_bytes < moe::cache_ws_bytes(table->n_pages, n) || ((uintptr_t)ws & 15))
    return MOE_ERR_WORKSPACE;
  return done(moe::launch_cache_fork(cl, n_cl, dev_table(table), src, dst, n, err_word, ws,
                                     (hipStream_t)stream),
              "moe_cache_fork");
}

int moe_cache_keep(const moe_kv_cache* layers, int n_layers, const moe_kv_table* table,
                   const int* slots, const int* n_draft, const int* cu, const int* path,
                   long n_path, long n, int* err_word, void* stream) {
  int st = check_table(table, true);
  if (st) return st;
  moe::CopyLayers cl[kMaxGroups];
  int n_cl = 0;
  st = copy_layers(layers, n_layers, table, cl, &n_cl);
  if (st) return st;
  if (n < 0 || n >= (1L << 20) || n_path < 0 || n_path >= (1L << 31) ||
      (!slots && n > table->n_slots))
    return MOE_ERR_SHAPE;
  if (!err_word) return MOE_ERR_NULL;
  if (n == 0) return MOE_OK;
  if (!n_draft || !cu || (!path && n_path > 0)) return MOE_ERR_NULL;
  const moe::KeepArgs a{dev_table(table), slots, n_draft, cu, path, n_path, 0, err_word};
  return done(moe::launch_cache_keep(cl, n_cl, a, n, (hipStream_t)stream), "moe_cache_keep");
}

int moe_latent_pages(const moe_latent_cache* cache, moe_kv_cache* pages) {
  const int st = check_latent(cache);
  if (st) return st;
  if (!pages) return MOE_ERR_NULL;
  *pages = {cache->fmt, cache->n_pages, cache->page_size,
            (cache->latent_dim + cache->rope_dim) / 64, 64, cache->stride_page, 64,
            cache->stride_tok, cache->c, cache->c, cache->scale, cache->scale};
  return MOE_OK;
}

int moe_latent_append(const moe_latent_cache* cache, const moe_kv_table* table, const int* slots,
                      const int* start, const int* cu, long n, long T, int fmt, const void* c,
                      long c_stride_row, const void* rope, long rope_stride_row, int* err_word,
                      void* stream) {
  int st = check_latent(cache);
  if (st) return st;
  st = check_table(table, false);
  if (st) return st;
  st = check_latent_pair(cache, table);
  if (st) return st;
  if (fmt != MOE_KV_BF16 && fmt != MOE_KV_F16) return MOE_ERR_FORMAT;
  if (cache->fmt != MOE_KV_E4M3 && cache->fmt != fmt) return MOE_ERR_FORMAT;
  if (n < 0 || n >= (1L << 20) || T < 0 || T >= (1L << 31) || (!cu && T != n) ||
      (n == 0 && T > 0) || (!slots && n > table->n_slots))
    return MOE_ERR_SHAPE;
  if (!err_word) return MOE_ERR_NULL;
  if (T == 0) return MOE_OK;
  if (!start || !c || !rope) return MOE_ERR_NULL;
  if (!row_strides_ok(c_stride_row, cache->latent_dim, cache->latent_dim) ||
      !row_strides_ok(rope_stride_row, cache->rope_dim, cache->rope_dim))
    return MOE_ERR_SHAPE;
  if ((((uintptr_t)c) | ((uintptr_t)rope)) & 15) return MOE_ERR_PARAM;
  moe::AppendArgs a{dev_latent(cache), dev_table(table), slots, start, cu, (int)n, T,
                    (const char*)c, (const char*)rope, c_stride_row * 2, 0,
                    rope_stride_row * 2, 0, err_word};
  return done(moe::launch_latent_append(a, fmt, (hipStream_t)stream), "moe_latent_append");
}

size_t moe_attn_latent_prompt_workspace_size(long n, long T, int n_heads) {
  if (n < 0 || n >= (1L << 20) || n_heads < 1 || n_heads > 1024 || T < 0 ||
      T > 0x7FFFFFFFL / n_heads)
    return 0;
  return moe::prefill_ws_bytes(n, T, n_heads, n_heads, moe::kDenseDim);
}

int moe_attn_latent_prompt(const moe_latent_rows* kv, long n, const int* cu_k, long S,
                           const int* cu_q, long T, const moe_attn* at, void* ws,
                           size_t ws_bytes, void* stream) {
  constexpr int D = moe::kDenseDim, DR = moe::kLatRope;
  if (!kv || !at) return MOE_ERR_NULL;
  if (at->fmt != MOE_KV_BF16 && at->fmt != MOE_KV_F16) return MOE_ERR_FORMAT;
  if (n < 0 || n >= (1L << 20) || T < 0 || S < 0 || S > kMaxTokens || at->n_heads < 1 ||
      at->n_heads > 1024 || T > 0x7FFFFFFFL / at->n_heads || (n == 0 && T > 0))
    return MOE_ERR_SHAPE;
  moe::AttnArgs a{};
  const int st = attn_rows(at, D + DR, D, T, &a);
  if (st) return st;
  if (T == 0) return MOE_OK;
  if (!cu_q || !cu_k || (S > 0 && (!kv->k || !kv->k_rope || !kv->v))) return MOE_ERR_NULL;
  if (!row_strides_ok(kv->k_stride_row, kv->k_stride_head, D) ||
      !row_strides_ok(kv->v_stride_row, kv->v_stride_head, D) ||
      !row_strides_ok(kv->rope_stride_row, DR, DR))
    return MOE_ERR_SHAPE;
  for (long s : {kv->k_stride_row, kv->v_stride_row, kv->rope_stride_row})
    if (s >= (1L << 30) / 32) return MOE_ERR_SHAPE;
  if ((((uintptr_t)kv->k) | ((uintptr_t)kv->k_rope) | ((uintptr_t)kv->v)) & 15)
    return MOE_ERR_PARAM;
  const size_t need = moe::prefill_ws_bytes(n, T, at->n_heads, at->n_heads, D);
  if (need > 0 && (!ws || ws_bytes < need || ((uintptr_t)ws & 15))) return MOE_ERR_WORKSPACE;
  a.c.k = (char*)kv->k;
  a.c.v = (char*)kv->v;
  a.c.st = kv->k_stride_row * 2;
  a.c.sh = kv->k_stride_head * 2;
  a.v_row = kv->v_stride_row * 2;
  a.v_head = kv->v_stride_head * 2;
  a.kr = (const char*)kv->k_rope;
  a.kr_row = kv->rope_stride_row * 2;
  a.c.fmt = at->fmt;
  a.c.hkv = at->n_heads;
  a.c.D = D;
  a.g = 1;
  // (no table; contexts are at most the rows there are)
  a.t.ps = 16;
  a.t.max_pages = (int)((S + 15) / 16);
  attn_window(at, S, &a);
  a.n = (int)n;
  a.cu = cu_q;
  a.cu_k = cu_k;
  a.S = S;
  a.T = T;
  a.part = (float*)ws;
  return done(moe::launch_attn_dense(a, at->fmt, (hipStream_t)stream), "moe_attn_latent_prompt");
}

size_t moe_attn_latent_workspace_size(const moe_latent_cache* cache, long n, long T,
                                      int n_heads) {
  if (!cache || (cache->latent_dim != 256 && cache->latent_dim != 512) || n < 0 ||
      n >= (1L << 20) || n_heads < 1 || n_heads > 1024 || T < 0 || T > 0x7FFFFFFFL / n_heads)
    return 0;
  return moe::latent_ws_bytes(cache->latent_dim);
}

int moe_attn_latent(const moe_latent_cache* cache, const moe_kv_table* table, const int* slots,
                    long n, const int* cu_q, long T, const int* parent, const moe_attn* at,
                    int* err_word, void* ws, size_t ws_bytes, void* stream) {
  int st = check_latent(cache);
  if (st) return st;
  st = check_table(table, false);
  if (st) return st;
  st = check_latent_pair(cache, table);
  if (st) return st;
  if (!at || !err_word) return MOE_ERR_NULL;
  if (at->fmt != MOE_KV_BF16 && at->fmt != MOE_KV_F16) return MOE_ERR_FORMAT;
  if (cache->fmt != MOE_KV_E4M3 && cache->fmt != at->fmt) return MOE_ERR_FORMAT;
  if (n < 0 || n >= (1L << 20) || T < 0 || at->n_heads < 1 || at->n_heads > 1024 ||
      T > 0x7FFFFFFFL / at->n_heads || (!cu_q && T != n) || (n == 0 && T > 0) ||
      (!slots && n > table->n_slots))
    return MOE_ERR_SHAPE;
  moe::AttnArgs a{};
  st = attn_rows(at, cache->latent_dim + cache->rope_dim, cache->latent_dim, T, &a);
  if (st) return st;
  if (T == 0) return MOE_OK;
  const size_t need = moe::latent_ws_bytes(cache->latent_dim);
  if (!ws || ws_bytes < need || ((uintptr_t)ws & 15)) return MOE_ERR_WORKSPACE;
  a.c = dev_latent(cache);
  a.t = dev_table(table);
  attn_window(at, (long)table->max_pages * table->page_size, &a);
  a.slots = slots;
  a.n = (int)n;
  a.g = at->n_heads;
  a.err = err_word;
  a.cu = cu_q;
  a.T = T;
  a.parent = parent;
  a.part = (float*)ws;
  return done(moe::launch_attn_latent(a, at->fmt, (hipStream_t)stream), "moe_attn_latent");
}

int moe_cache_compact(const moe_kv_cache* layers, int n_layers, const moe_kv_table* table,
                      int* n_used, int* err_word, void* ws, size_t ws_bytes, void* stream) {
  int st = check_table(table, true);
  if (st) return st;
  moe::CopyLayers cl[kMaxGroups];
  int n_cl = 0;
  st = copy_layers(layers, n_layers, table, cl, &n_cl);
  if (st) return st;
  if (!err_word) return MOE_ERR_NULL;
  if (!ws || ws_bytes < moe::cache_ws_bytes(table->n_pages, 0) || ((uintptr_t)ws & 15))
    return MOE_ERR_WORKSPACE;
  return done(moe::launch_cache_compact(cl, n_cl, dev_table(table), n_used, ws,
                                        (hipStream_t)stream),
              "moe_cache_compact");
}

int moe_cache_copy_pages(const moe_kv_cache* layers, int n_layers, const int* src,
                         const int* dst, long n, int* err_word, void* stream) {
  moe::CopyLayers cl[kMaxGroups];
  int n_cl = 0;
  int st = copy_layers(layers, n_layers, nullptr, cl, &n_cl);
  if (st) return st;
  if (n < 0 || n >= (1L << 31)) return MOE_ERR_SHAPE;
  if (!err_word) return MOE_ERR_NULL;
  if (n == 0) return MOE_OK;
  if (!src || !dst) return MOE_ERR_NULL;
  return done(moe::launch_cache_copy(cl, n_cl, src, dst, n, layers[0].n_pages, err_word,
                                     (hipStream_t)stream),
              "moe_cache_copy_pages");
}

}  // extern "C"
