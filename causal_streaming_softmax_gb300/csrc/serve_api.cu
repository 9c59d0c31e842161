// serve_api.cu - the C ABI of the packed and paged calls: host-side admission
// checks and dispatch to the kernel launchers.
#include <math.h>

#include "serve_internal.h"

namespace css {
namespace {

// A stride is read only where its dimension is longer than one; there it keeps
// every row 16-byte aligned and rows apart.  2^38 elements keep a byte stride
// below the 2^40 that a tensor map takes.
bool fix_stride(int64_t* s, int64_t dim) {
  if (dim <= 1) {
    *s = 64;
    return true;
  }
  return *s >= 64 && *s % 8 == 0 && *s < (1ll << 38);
}

// No two head rows of an output share an element.
bool rows_apart(int64_t t, int64_t h, int64_t tokens, int64_t heads) {
  return (h >= 64 && (tokens <= 1 || t >= (heads - 1) * h + 64)) ||
         (t >= 64 && (heads <= 1 || h >= (tokens - 1) * t + 64));
}

int softmax_scale(float scale, float* c) {
  if (!(scale > 0.0f) || !isfinite(scale)) return ATTN_ERR_SHAPE;
  *c = static_cast<float>(static_cast<double>(scale) / 0.69314718055994530942);
  return ATTN_OK;
}

int validate_heads(int heads, int kv_heads, int head_dim, int dtype) {
  if (heads < 1 || heads > 65535 || kv_heads < 1 || heads % kv_heads != 0) return ATTN_ERR_SHAPE;
  if (heads / kv_heads > 128 || head_dim != 64) return ATTN_ERR_SHAPE;
  if (dtype != ATTN_F16 && dtype != ATTN_BF16) return ATTN_ERR_SHAPE;
  return ATTN_OK;
}

// The part of a paged shape that every call reads.
int validate_paged(const attn_paged_shape* s, PagedDims* d) {
  if (!s) return ATTN_ERR_NULL;
  if (s->batch < 1 || s->batch > kMaxPagedBatch || s->tokens < 0 || s->tokens > (1 << 30))
    return ATTN_ERR_SHAPE;
  int shift = 3;
  while (shift < 10 && (1 << shift) != s->page_size) ++shift;
  if ((1 << shift) != s->page_size) return ATTN_ERR_SHAPE;
  if (s->num_pages < 1 || ((int64_t)s->num_pages << shift) > 0x7fffffffLL) return ATTN_ERR_SHAPE;
  if (s->table_width < 1 || ((int64_t)s->table_width << shift) > 0x7fffffffLL)
    return ATTN_ERR_SHAPE;
  *d = PagedDims{};
  d->batch = s->batch;
  d->tokens = s->tokens;
  d->pages = s->num_pages;
  d->width = s->table_width;
  d->shift = shift;
  return ATTN_OK;
}

int validate_attend(const attn_paged_shape* s, PagedDims* d) {
  int rc = validate_paged(s, d);
  if (rc != ATTN_OK) return rc;
  if ((rc = validate_heads(s->heads, s->kv_heads, s->head_dim, s->dtype)) != ATTN_OK) return rc;
  if (s->max_new < 1 || s->max_new > (1 << 30)) return ATTN_ERR_SHAPE;
  d->H = s->heads;
  d->Hkv = s->kv_heads;
  d->G = s->heads / s->kv_heads;
  d->max_new = s->max_new;
  d->bf16 = s->dtype == ATTN_BF16;
  return softmax_scale(s->scale, &d->c);
}

// No two rows of a pool share an element: each stride, in rising order, is past
// the extent of the dimensions before it.
bool pool_apart(const PoolArg& p, int64_t pages, int64_t heads, int64_t rows) {
  int64_t st[3] = {p.r, p.h, p.pg}, n[3] = {rows, heads, pages};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if ((n[i] <= 1 && n[j] > 1) || (n[j] > 1 && st[j] < st[i])) {
        const int64_t a = st[i], b = n[i];
        st[i] = st[j], n[i] = n[j];
        st[j] = a, n[j] = b;
      }
  int64_t extent = 64;
  for (int i = 0; i < 3 && n[i] > 1; ++i) {
    if (st[i] < extent) return false;
    extent += (n[i] - 1) * st[i];
  }
  return true;
}

int pools(const attn_paged_shape* s, const void* kc, const void* vc, PoolArg* k, PoolArg* v) {
  *k = PoolArg{const_cast<void*>(kc), s->kc_page, s->kc_head, s->kc_row};
  *v = PoolArg{const_cast<void*>(vc), s->vc_page, s->vc_head, s->vc_row};
  for (PoolArg* p : {k, v}) {
    int64_t pg = p->pg, h = p->h, r = p->r;
    if (!fix_stride(&pg, s->num_pages) || !fix_stride(&h, s->kv_heads) ||
        !fix_stride(&r, s->page_size))
      return ATTN_ERR_SHAPE;
    p->pg = pg, p->h = h, p->r = r;
  }
  return ATTN_OK;
}

// A stride of a 4-bit pool, in bytes.
bool fix_stride4(int64_t* s, int64_t dim, int64_t page) {
  if (dim <= 1) {
    *s = page;
    return true;
  }
  return *s >= page && *s % 16 == 0 && *s < (1ll << 40);
}

int pools4(const attn_paged_shape* s, int shift, const void* kc, const void* vc, PoolArg* k,
           PoolArg* v) {
  *k = PoolArg{const_cast<void*>(kc), s->kc_page, s->kc_head, 0};
  *v = PoolArg{const_cast<void*>(vc), s->vc_page, s->vc_head, 0};
  const int64_t page = 36ll << shift;
  for (PoolArg* p : {k, v}) {
    int64_t pg = p->pg, h = p->h;
    if (!fix_stride4(&pg, s->num_pages, page) || !fix_stride4(&h, s->kv_heads, page))
      return ATTN_ERR_SHAPE;
    // no two pages of a head share a byte
    if (s->num_pages > 1 && s->kv_heads > 1 && pg < (s->kv_heads - 1) * h + page &&
        h < (s->num_pages - 1) * pg + page)
      return ATTN_ERR_SHAPE;
    p->pg = pg, p->h = h;
  }
  return ATTN_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

// attn_paged_append and attn_paged_append4.
int append(const attn_paged_shape* s, bool four, const void* q, const void* k, const void* v,
           const float* cos_tab, const float* sin_tab, int32_t angles, const int32_t* slots,
           const int32_t* cu, const int32_t* lens, void* q_out, void* k_cache, void* v_cache,
           void* stream) {
  PagedDims d;
  int rc = validate_paged(s, &d);
  if (rc != ATTN_OK) return rc;
  const bool rotate = !four || cos_tab || sin_tab;
  if ((rc = validate_heads(rotate ? s->heads : s->kv_heads, s->kv_heads, s->head_dim,
                           s->dtype)) != ATTN_OK)
    return rc;
  d.Hkv = s->kv_heads;
  d.H = rotate ? s->heads : 0;
  d.bf16 = s->dtype == ATTN_BF16;
  int64_t st[8] = {s->k_token, s->k_head, s->v_token, s->v_head,
                   s->q_token, s->q_head, s->o_token, s->o_head};
  for (int i = 0; i < (rotate ? 8 : 4); ++i)
    if (!fix_stride(&st[i], (i & 1) ? (i > 3 ? s->heads : s->kv_heads) : s->tokens))
      return ATTN_ERR_SHAPE;
  if (rotate && (angles < 1 || !rows_apart(st[6], st[7], s->tokens, s->heads)))
    return ATTN_ERR_SHAPE;
  AppendArgs a{};
  if (four) {
    if ((rc = pools4(s, d.shift, k_cache, v_cache, &a.kc, &a.vc)) != ATTN_OK) return rc;
  } else {
    if ((rc = pools(s, k_cache, v_cache, &a.kc, &a.vc)) != ATTN_OK) return rc;
    if (!pool_apart(a.kc, d.pages, d.Hkv, 1 << d.shift) ||
        !pool_apart(a.vc, d.pages, d.Hkv, 1 << d.shift))
      return ATTN_ERR_SHAPE;
  }
  if (s->tokens == 0) return ATTN_OK;
  if (!k || !v || !slots || !k_cache || !v_cache) return ATTN_ERR_NULL;
  if (rotate && (!q || !cos_tab || !sin_tab || !cu || !lens || !q_out)) return ATTN_ERR_NULL;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned4(slots))
    return ATTN_ERR_ALIGN;
  if (rotate && (!aligned16(q) || !aligned16(q_out) || !aligned16(cos_tab) ||
                 !aligned16(sin_tab) || !aligned4(cu) || !aligned4(lens)))
    return ATTN_ERR_ALIGN;
  // q is turned in place row by row, or lies elsewhere
  if (rotate && q == q_out && (st[4] != st[6] || st[5] != st[7])) return ATTN_ERR_SHAPE;
  DevCtx ctx;
  if ((rc = device_context(&ctx)) != ATTN_OK) return rc;
  a.k = RowsArg{const_cast<void*>(k), st[0], st[1]};
  a.v = RowsArg{const_cast<void*>(v), st[2], st[3]};
  a.q = RowsArg{const_cast<void*>(q), st[4], st[5]};
  a.q_out = RowsArg{q_out, st[6], st[7]};
  a.cos_tab = cos_tab, a.sin_tab = sin_tab;
  a.angles = angles;
  a.slots = slots, a.cu = cu, a.lens = lens;
  return launch_paged_append(d, ctx, a, rotate, four, static_cast<cudaStream_t>(stream));
}

// attn_paged_fwd and attn_paged_fwd4.
int attend(const attn_paged_shape* s, bool four, const void* q, const void* k_cache,
           const void* v_cache, const int32_t* table, const int32_t* cu, const int32_t* lens,
           void* ws, size_t ws_bytes, void* o, float* lse, void* stream) {
  PagedDims d;
  int rc = validate_attend(s, &d);
  if (rc != ATTN_OK) return rc;
  int64_t st[4] = {s->q_token, s->q_head, s->o_token, s->o_head};
  for (int i = 0; i < 4; ++i)
    if (!fix_stride(&st[i], (i & 1) ? s->heads : s->tokens)) return ATTN_ERR_SHAPE;
  if (!rows_apart(st[2], st[3], s->tokens, s->heads)) return ATTN_ERR_SHAPE;
  PoolArg kc, vc;
  rc = four ? pools4(s, d.shift, k_cache, v_cache, &kc, &vc) : pools(s, k_cache, v_cache, &kc, &vc);
  if (rc != ATTN_OK) return rc;
  if (s->tokens == 0) return ATTN_OK;
  if (!q || !k_cache || !v_cache || !table || !cu || !lens || !ws || !o) return ATTN_ERR_NULL;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(ws) ||
      !aligned16(o) || !aligned16(lse) || (reinterpret_cast<uintptr_t>(table) & 3) ||
      (reinterpret_cast<uintptr_t>(cu) & 3) || (reinterpret_cast<uintptr_t>(lens) & 3))
    return ATTN_ERR_ALIGN;
  if (ws_bytes < paged_workspace_bytes(d)) return ATTN_ERR_WORKSPACE;
  DevCtx ctx;
  if ((rc = device_context(&ctx)) != ATTN_OK) return rc;
  return launch_paged_fwd(d, ctx, RowsArg{const_cast<void*>(q), st[0], st[1]}, kc, vc, table, cu,
                          lens, ws, four, RowsArg{o, st[2], st[3]}, lse,
                          static_cast<cudaStream_t>(stream));
}

}  // namespace
}  // namespace css

using namespace css;

extern "C" {

int attn_packed_fwd(const attn_packed_shape* s, const void* q, const void* k, const void* v,
                    const int32_t* cu, void* o, float* lse, void* stream) {
  if (!s) return ATTN_ERR_NULL;
  if (s->tokens < 0 || s->tokens > (1 << 30) || s->batch < 1 || s->batch > 65535)
    return ATTN_ERR_SHAPE;
  if (s->causal != 0 && s->causal != 1) return ATTN_ERR_SHAPE;
  int rc = validate_heads(s->heads, s->kv_heads, s->head_dim, s->dtype);
  if (rc != ATTN_OK) return rc;
  PackedDims d{s->tokens, s->batch, s->heads, s->kv_heads, s->heads / s->kv_heads, s->causal,
               s->dtype == ATTN_BF16, 0.f};
  if ((rc = softmax_scale(s->scale, &d.c)) != ATTN_OK) return rc;
  int64_t st[8] = {s->q_token, s->q_head, s->k_token, s->k_head,
                   s->v_token, s->v_head, s->o_token, s->o_head};
  for (int i = 0; i < 8; ++i)
    if (!fix_stride(&st[i], (i & 1) ? ((i == 1 || i == 7) ? s->heads : s->kv_heads) : s->tokens))
      return ATTN_ERR_SHAPE;
  if (!rows_apart(st[6], st[7], s->tokens, s->heads)) return ATTN_ERR_SHAPE;
  if (s->tokens == 0) return ATTN_OK;
  if (!q || !k || !v || !cu || !o) return ATTN_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse) ||
      (reinterpret_cast<uintptr_t>(cu) & 3))
    return ATTN_ERR_ALIGN;
  DevCtx ctx;
  if ((rc = device_context(&ctx)) != ATTN_OK) return rc;
  return launch_packed_fwd(d, ctx, RowsArg{const_cast<void*>(q), st[0], st[1]},
                           RowsArg{const_cast<void*>(k), st[2], st[3]},
                           RowsArg{const_cast<void*>(v), st[4], st[5]}, cu,
                           RowsArg{o, st[6], st[7]}, lse, static_cast<cudaStream_t>(stream));
}

int attn_paged_plan(const attn_paged_shape* s, const int32_t* cached, const int32_t* fresh,
                    int32_t* ring, const int32_t* state, int32_t* table, int32_t* cu,
                    int32_t* lens, int32_t* slots, int32_t* next, void* stream) {
  PagedDims d;
  int rc = validate_paged(s, &d);
  if (rc != ATTN_OK) return rc;
  if (!cached || !fresh || !ring || !state || !table || !cu || !lens || !next ||
      (!slots && s->tokens > 0))
    return ATTN_ERR_NULL;
  const int64_t B = d.batch;
  const struct {
    const int32_t* p;
    int64_t n;
    bool out;
  } arr[9] = {{cached, B, false},     {fresh, B, false},       {ring, d.pages, true},
              {state, 4, false},      {table, B * d.width, true}, {cu, B + 1, true},
              {lens, B, true},        {slots, d.tokens, true}, {next, 4, true}};
  for (int i = 0; i < 9; ++i) {
    if (reinterpret_cast<uintptr_t>(arr[i].p) & 3) return ATTN_ERR_ALIGN;
    // inputs may overlap one another; an output overlaps nothing
    for (int j = 0; j < i; ++j) {
      const uintptr_t x = reinterpret_cast<uintptr_t>(arr[i].p),
                      y = reinterpret_cast<uintptr_t>(arr[j].p);
      if ((arr[i].out || arr[j].out) && x < y + 4 * arr[j].n && y < x + 4 * arr[i].n)
        return ATTN_ERR_SHAPE;
    }
  }
  DevCtx ctx;
  if ((rc = device_context(&ctx)) != ATTN_OK) return rc;
  return launch_paged_plan(d, ctx, cached, fresh, ring, state, table, cu, lens, slots, next,
                           static_cast<cudaStream_t>(stream));
}

int attn_paged_store(const attn_paged_shape* s, const void* k, const void* v,
                     const int32_t* slots, void* k_cache, void* v_cache, void* stream) {
  PagedDims d;
  int rc = validate_paged(s, &d);
  if (rc != ATTN_OK) return rc;
  if ((rc = validate_heads(s->kv_heads, s->kv_heads, s->head_dim, s->dtype)) != ATTN_OK)
    return rc;
  d.Hkv = s->kv_heads;
  int64_t st[4] = {s->k_token, s->k_head, s->v_token, s->v_head};
  for (int i = 0; i < 4; ++i)
    if (!fix_stride(&st[i], (i & 1) ? s->kv_heads : s->tokens)) return ATTN_ERR_SHAPE;
  PoolArg kc, vc;
  if ((rc = pools(s, k_cache, v_cache, &kc, &vc)) != ATTN_OK) return rc;
  if (!pool_apart(kc, d.pages, d.Hkv, 1 << d.shift) ||
      !pool_apart(vc, d.pages, d.Hkv, 1 << d.shift))
    return ATTN_ERR_SHAPE;
  if (s->tokens == 0) return ATTN_OK;
  if (!k || !v || !slots || !k_cache || !v_cache) return ATTN_ERR_NULL;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(slots) & 3))
    return ATTN_ERR_ALIGN;
  DevCtx ctx;
  if ((rc = device_context(&ctx)) != ATTN_OK) return rc;
  return launch_paged_store(d, ctx, RowsArg{const_cast<void*>(k), st[0], st[1]},
                            RowsArg{const_cast<void*>(v), st[2], st[3]}, slots, kc, vc,
                            static_cast<cudaStream_t>(stream));
}

int attn_paged_append(const attn_paged_shape* s, const void* q, const void* k, const void* v,
                      const float* cos_tab, const float* sin_tab, int32_t angles,
                      const int32_t* slots, const int32_t* cu, const int32_t* lens, void* q_out,
                      void* k_cache, void* v_cache, void* stream) {
  return append(s, false, q, k, v, cos_tab, sin_tab, angles, slots, cu, lens, q_out, k_cache,
                v_cache, stream);
}

int attn_paged_append4(const attn_paged_shape* s, const void* q, const void* k, const void* v,
                       const float* cos_tab, const float* sin_tab, int32_t angles,
                       const int32_t* slots, const int32_t* cu, const int32_t* lens, void* q_out,
                       uint8_t* k_cache, uint8_t* v_cache, void* stream) {
  return append(s, true, q, k, v, cos_tab, sin_tab, angles, slots, cu, lens, q_out, k_cache,
                v_cache, stream);
}

int attn_paged_load4(const attn_paged_shape* s, const int32_t* slots, const uint8_t* k_cache,
                     const uint8_t* v_cache, void* k, void* v, void* stream) {
  PagedDims d;
  int rc = validate_paged(s, &d);
  if (rc != ATTN_OK) return rc;
  if ((rc = validate_heads(s->kv_heads, s->kv_heads, s->head_dim, s->dtype)) != ATTN_OK)
    return rc;
  d.Hkv = s->kv_heads;
  d.bf16 = s->dtype == ATTN_BF16;
  int64_t st[4] = {s->k_token, s->k_head, s->v_token, s->v_head};
  for (int i = 0; i < 4; ++i)
    if (!fix_stride(&st[i], (i & 1) ? s->kv_heads : s->tokens)) return ATTN_ERR_SHAPE;
  if (!rows_apart(st[0], st[1], s->tokens, s->kv_heads) ||
      !rows_apart(st[2], st[3], s->tokens, s->kv_heads))
    return ATTN_ERR_SHAPE;
  PoolArg kc, vc;
  if ((rc = pools4(s, d.shift, k_cache, v_cache, &kc, &vc)) != ATTN_OK) return rc;
  if (s->tokens == 0) return ATTN_OK;
  if (!k || !v || !slots || !k_cache || !v_cache) return ATTN_ERR_NULL;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned4(slots))
    return ATTN_ERR_ALIGN;
  DevCtx ctx;
  if ((rc = device_context(&ctx)) != ATTN_OK) return rc;
  return launch_paged_load4(d, ctx, kc, vc, slots, RowsArg{k, st[0], st[1]},
                            RowsArg{v, st[2], st[3]}, static_cast<cudaStream_t>(stream));
}

size_t attn_paged_workspace_bytes(const attn_paged_shape* s) {
  PagedDims d;
  if (validate_attend(s, &d) != ATTN_OK) return 0;
  return paged_workspace_bytes(d);
}

int attn_paged_fwd(const attn_paged_shape* s, const void* q, const void* k_cache,
                   const void* v_cache, const int32_t* table, const int32_t* cu,
                   const int32_t* lens, void* ws, size_t ws_bytes, void* o, float* lse,
                   void* stream) {
  return attend(s, false, q, k_cache, v_cache, table, cu, lens, ws, ws_bytes, o, lse, stream);
}

int attn_paged_fwd4(const attn_paged_shape* s, const void* q, const uint8_t* k_cache,
                    const uint8_t* v_cache, const int32_t* table, const int32_t* cu,
                    const int32_t* lens, void* ws, size_t ws_bytes, void* o, float* lse,
                    void* stream) {
  return attend(s, true, q, k_cache, v_cache, table, cu, lens, ws, ws_bytes, o, lse, stream);
}

}  // extern "C"
