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

// what both attention calls ask of their arguments, and the arguments of the
// kernels; rows of q > 0
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
  if (!isfinite(at->scale) || at->window < 0 || at->n_first < 0) return MOE_ERR_PARAM;
  if (rows > 0) {
    if (!at->q || !at->out) return MOE_ERR_NULL;
    if (!row_strides_ok(at->q_stride_row, at->q_stride_head, cache->head_dim) ||
        !row_strides_ok(at->out_stride_row, at->out_stride_head, cache->head_dim))
      return MOE_ERR_SHAPE;
    if ((((uintptr_t)at->q) | ((uintptr_t)at->out)) & 15) return MOE_ERR_PARAM;
  }
  *a = moe::AttnArgs{};
  a->c = dev_cache(cache);
  a->t = dev_table(table);
  a->slots = slots;
  a->n = (int)n;
  a->q = (const char*)at->q;
  a->out = (char*)at->out;
  a->q_row = at->q_stride_row * 2;
  a->q_head = at->q_stride_head * 2;
  a->o_row = at->out_stride_row * 2;
  a->o_head = at->out_stride_head * 2;
  a->lse = at->lse;
  a->hq = at->n_heads;
  a->g = at->n_heads / cache->n_heads;
  a->scale = at->scale * 1.44269504088896340736f;
  // A window that no context of this table exceeds is none. What is left is at
  // most kMaxTokens, so that position - window stays within 32 bits, for rows
  // before a sequence's first position too.
  const long most = (long)table->max_pages * table->page_size;
  a->window = at->window < most ? at->window : 0;
  a->first = a->window ? (int)(at->n_first < most ? at->n_first : most) : 0;
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
    cl.p[cl.n++] = (char*)c->v;
  }
  return MOE_OK;
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
