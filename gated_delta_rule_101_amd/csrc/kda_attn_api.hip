// C ABI of the attention layer's operators: the step's plan, norm and rotation
// of queries and keys, and the 8-bit cache's append and attention.  Host-side
// validation, then the launches on the caller's stream.  Declarations and the
// full contract are in include/kda.h.
#include "kda_attn.h"
#include "kda_check.h"

namespace {

constexpr int64_t INT_LIMIT = (int64_t)1 << 31;

bool valid_page(int page) { return page == 16 || page == 32 || page == 64 || page == 128; }
bool valid_code(kda_code_t c) { return c == KDA_CODE_E4M3 || c == KDA_CODE_INT8; }

// T rows of `width` bytes, `stride` bytes apart.
struct Rows {
    const void *p;
    size_t width, stride;
    int64_t T;
    bool used() const { return width > 0 && T > 0; }
    size_t span() const { return used() ? (size_t)(T - 1) * stride + width : 0; }
};

// Whether two sets of rows share a byte: rows of one larger matrix (the parts of
// a fused projection) lie between each other without touching.
bool touch(const Rows &a, const Rows &b)
{
    if (!a.used() || !b.used() || !a.p || !b.p) return false;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    if (x + a.span() <= y || y + b.span() <= x) return false;
    if (a.stride != b.stride) return true;
    const size_t s = a.stride, d = y >= x ? (y - x) % s : (s - (x - y) % s) % s;
    return d < a.width || d + b.width > s;
}
Rows plain(const void *p, size_t bytes) { return {p, bytes, bytes, 1}; }

kda_status_t check_heads(int64_t T, int Hq, int Hk, int D)
{
    if (T < 0 || Hq < 0 || Hk < 0 || D <= 0 || D % 2) return KDA_ERR_INVALID_ARG;
    if (D > 512 || Hq >= 65536 || Hk >= 65536) return KDA_ERR_UNSUPPORTED;
    if (T >= MAX_COUNT / ((int64_t)D * (Hq + Hk > 0 ? Hq + Hk : 1))) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// What both directions of the norm check: `in` and `out` are rows of queries
// and keys in turn.  An output may be any input of its kind, whole: each head is read
// once, by the lanes that write it.
kda_status_t check_qk(const Rows *in, int ni, const Rows *out, const float *wq, const float *wk, float eps,
                      const int *positions, const float *rotary, int64_t T, int Hq, int Hk, int D, int R, int longest,
                      kda_dtype_t dtype, const Rows *more, int nm)
{
    const size_t e = dsize(dtype);
    if (R < 0 || R > D || R % 2 || longest < 0) return KDA_ERR_INVALID_ARG;
    if (!(eps >= 0.f && eps <= 3.0e38f)) return KDA_ERR_INVALID_ARG;
    if ((R > 0) != (rotary != nullptr) || (rotary && T > 0 && !positions)) return KDA_ERR_INVALID_ARG;
    if (rotary && longest == 0 && T > 0) return KDA_ERR_INVALID_ARG;
    if (((uintptr_t)rotary | (uintptr_t)positions | (uintptr_t)wq | (uintptr_t)wk) & 3) return KDA_ERR_INVALID_ARG;
    const Rows flat[] = {plain(wq, (size_t)D * 4), plain(wk, (size_t)D * 4), plain(positions, (size_t)T * 4),
                         plain(rotary, (size_t)longest * R * 4)};
    const auto row_ok = [&](const Rows &r) {
        return !r.used() || (r.p && !((uintptr_t)r.p & (e - 1)) && r.stride >= r.width && r.stride / e < (size_t)MAX_DIM * 64);
    };
    for (int i = 0; i < ni; ++i)
        if (!row_ok(in[i])) return KDA_ERR_INVALID_ARG;
    for (int i = 0; i < 2; ++i) {
        if (!row_ok(out[i])) return KDA_ERR_INVALID_ARG;
        for (int j = 0; j < ni; ++j) {
            const bool same = (j & 1) == i && out[i].p == in[j].p && out[i].stride == in[j].stride;
            if (!same && touch(out[i], in[j])) return KDA_ERR_INVALID_ARG;
        }
        for (const Rows &f : flat)
            if (touch(out[i], f)) return KDA_ERR_INVALID_ARG;
        for (int j = 0; j < nm; ++j)
            if (touch(out[i], more[j])) return KDA_ERR_INVALID_ARG;
    }
    if (touch(out[0], out[1])) return KDA_ERR_INVALID_ARG;
    for (int i = 0; i < nm; ++i) {
        for (int j = 0; j < ni; ++j)
            if (touch(more[i], in[j])) return KDA_ERR_INVALID_ARG;
        for (const Rows &f : flat)
            if (touch(more[i], f)) return KDA_ERR_INVALID_ARG;
        for (int j = i + 1; j < nm; ++j)
            if (touch(more[i], more[j])) return KDA_ERR_INVALID_ARG;
    }
    return KDA_OK;
}

// The cache's sizes.
kda_status_t check_cache(int Hk, int D, int pages, int page, kda_code_t code, kda_dtype_t dtype)
{
    if (Hk <= 0 || D <= 0 || pages < 0 || page <= 0 || !valid_code(code) || !valid_dtype(dtype)) return KDA_ERR_INVALID_ARG;
    if ((D != 64 && D != 128 && D != 256) || !valid_page(page) || Hk > 32767) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)pages * page >= INT_LIMIT || (int64_t)pages * page >= MAX_COUNT / ((int64_t)Hk * D)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

}  // namespace

extern "C" {

// -------------------------------------------------------------------- plan

kda_status_t kda_cache_plan(const int *cached, const int *added, int *block_table, const int *free_pages,
                            const int *free_count, int *q_start, int *context, int *positions, int *slots,
                            int *free_left, int B, int max_pages, int free_capacity, int tokens, int page, void *stream)
{
    if (B < 0 || max_pages < 0 || free_capacity < 0 || tokens < 0 || page <= 0) return KDA_ERR_INVALID_ARG;
    if (!valid_page(page) || B >= MAX_DIM || (int64_t)max_pages * page >= INT_LIMIT) return KDA_ERR_UNSUPPORTED;
    const size_t n = (size_t)B * 4, table = n * max_pages, rows = (size_t)tokens * 4;
    const Buffer in[] = {{cached, n, true, 4}, {added, n, true, 4}, {free_pages, (size_t)free_capacity * 4, true, 4},
                         {free_count, 4, true, 4}};
    const Buffer out[] = {{block_table, table, true, 4}, {q_start, n + 4, true, 4}, {context, n, true, 4},
                          {positions, rows, true, 4}, {slots, rows, true, 4}, {free_left, 4, true, 4}};
    const kda_status_t ok = check_buffers(in, out);
    if (ok != KDA_OK) return ok;
    kda::PlanArgs a;
    a.cached = cached; a.added = added; a.table = block_table; a.free_pages = free_pages; a.free_count = free_count;
    a.q_start = q_start; a.context = context; a.positions = positions; a.slots = slots; a.free_left = free_left;
    a.B = B; a.per = max_pages; a.capacity = free_capacity; a.tokens = tokens; a.page = page;
    return launched(kda::launch_cache_plan(a, (hipStream_t)stream));
}

// ----------------------------------------------------- query and key norm

kda_status_t kda_qk_norm_rope_fwd(const void *q, const void *k, const float *q_weight, const float *k_weight, float eps,
                                  const int *positions, const float *rotary, void *q_out, void *k_out,
                                  int64_t tokens, int Hq, int Hk, int D, int rotary_dim, int rotary_rows, int neighbours,
                                  int64_t q_stride, int64_t k_stride, int64_t q_out_stride, int64_t k_out_stride,
                                  kda_dtype_t dtype, void *stream)
{
    if (!valid_dtype(dtype)) return KDA_ERR_INVALID_ARG;
    const kda_status_t st = check_heads(tokens, Hq, Hk, D);
    if (st != KDA_OK) return st;
    if (q_stride < 0 || k_stride < 0 || q_out_stride < 0 || k_out_stride < 0) return KDA_ERR_INVALID_ARG;
    const size_t e = dsize(dtype), wq = (size_t)Hq * D * e, wk = (size_t)Hk * D * e;
    const Rows in[] = {{q, wq, (size_t)q_stride * e, tokens}, {k, wk, (size_t)k_stride * e, tokens}};
    const Rows out[] = {{q_out, wq, (size_t)q_out_stride * e, tokens}, {k_out, wk, (size_t)k_out_stride * e, tokens}};
    const kda_status_t ok = check_qk(in, 2, out, q_weight, k_weight, eps, positions, rotary, tokens, Hq, Hk, D,
                                     rotary_dim, rotary_rows, dtype, nullptr, 0);
    if (ok != KDA_OK) return ok;
    if (tokens == 0 || Hq + Hk == 0) return KDA_OK;
    kda::QkNormArgs a;
    a.q = q; a.k = k; a.wq = q_weight; a.wk = k_weight; a.positions = positions; a.rotary = rotary;
    a.q_out = q_out; a.k_out = k_out; a.T = tokens;
    a.q_stride = q_stride; a.k_stride = k_stride; a.qo_stride = q_out_stride; a.ko_stride = k_out_stride;
    a.Hq = Hq; a.Hk = Hk; a.D = D; a.R = rotary_dim; a.longest = rotary_rows; a.eps = eps;
    a.neighbours = neighbours != 0; a.bf16 = dtype == KDA_BF16;
    return launched(kda::launch_qk_norm_fwd(a, (hipStream_t)stream));
}

size_t kda_qk_norm_rope_bwd_workspace_bytes(int64_t tokens, int Hq, int Hk, int D)
{
    if (check_heads(tokens, Hq, Hk, D) != KDA_OK || tokens == 0 || Hq + Hk == 0) return 0;
    return (size_t)kda::qk_norm_bwd_workspace_floats(tokens, Hq, Hk, D) * sizeof(float);
}

kda_status_t kda_qk_norm_rope_bwd(const void *dq_out, const void *dk_out, const void *q, const void *k,
                                  const float *q_weight, const float *k_weight, float eps,
                                  const int *positions, const float *rotary, void *dq, void *dk,
                                  float *dq_weight, float *dk_weight, void *workspace, size_t workspace_bytes,
                                  int64_t tokens, int Hq, int Hk, int D, int rotary_dim, int rotary_rows, int neighbours,
                                  int64_t dq_out_stride, int64_t dk_out_stride, int64_t q_stride, int64_t k_stride,
                                  int64_t dq_stride, int64_t dk_stride, kda_dtype_t dtype, void *stream)
{
    if (!valid_dtype(dtype)) return KDA_ERR_INVALID_ARG;
    const kda_status_t st = check_heads(tokens, Hq, Hk, D);
    if (st != KDA_OK) return st;
    if (q_stride < 0 || k_stride < 0 || dq_stride < 0 || dk_stride < 0 || dq_out_stride < 0 || dk_out_stride < 0)
        return KDA_ERR_INVALID_ARG;
    const bool want = dq_weight || dk_weight;
    const size_t need = want ? kda_qk_norm_rope_bwd_workspace_bytes(tokens, Hq, Hk, D) : 0;
    if (workspace_bytes < need || (need && (!workspace || (uintptr_t)workspace & 15))) return KDA_ERR_INVALID_ARG;
    if (((uintptr_t)dq_weight | (uintptr_t)dk_weight) & 3) return KDA_ERR_INVALID_ARG;
    const size_t e = dsize(dtype), wq = (size_t)Hq * D * e, wk = (size_t)Hk * D * e;
    const Rows in[] = {{dq_out, wq, (size_t)dq_out_stride * e, tokens}, {dk_out, wk, (size_t)dk_out_stride * e, tokens},
                       {q, wq, (size_t)q_stride * e, tokens}, {k, wk, (size_t)k_stride * e, tokens}};
    const Rows out[] = {{dq, wq, (size_t)dq_stride * e, tokens}, {dk, wk, (size_t)dk_stride * e, tokens}};
    const Rows more[] = {plain(dq_weight, (size_t)D * 4), plain(dk_weight, (size_t)D * 4), plain(workspace, need)};
    const kda_status_t ok = check_qk(in, 4, out, q_weight, k_weight, eps, positions, rotary, tokens, Hq, Hk, D,
                                     rotary_dim, rotary_rows, dtype, more, 3);
    if (ok != KDA_OK) return ok;
    const bool some = tokens > 0 && Hq + Hk > 0;
    if (!some && !want) return KDA_OK;
    kda::QkNormArgs a;
    a.gq = dq_out; a.gk = dk_out; a.q = q; a.k = k; a.wq = q_weight; a.wk = k_weight;
    a.positions = positions; a.rotary = rotary; a.q_out = dq; a.k_out = dk;
    a.dwq = dq_weight; a.dwk = dk_weight; a.ws = want && some ? (float *)workspace : nullptr;
    a.T = some ? tokens : 0;
    a.gq_stride = dq_out_stride; a.gk_stride = dk_out_stride; a.q_stride = q_stride; a.k_stride = k_stride;
    a.qo_stride = dq_stride; a.ko_stride = dk_stride;
    a.Hq = Hq; a.Hk = Hk; a.D = D; a.R = rotary_dim; a.longest = rotary_rows; a.eps = eps;
    a.neighbours = neighbours != 0; a.bf16 = dtype == KDA_BF16;
    return launched(kda::launch_qk_norm_bwd(a, (hipStream_t)stream));
}

// ------------------------------------------------------------------ append

kda_status_t kda_cache_append(const void *k, const void *v, const int *slots, void *k_codes, void *v_codes,
                              float *k_scale, float *v_scale, int tokens, int Hk, int D, int pages, int page,
                              int64_t k_stride, int64_t v_stride, kda_code_t code, kda_dtype_t dtype, void *stream)
{
    const kda_status_t st = check_cache(Hk, D, pages, page, code, dtype);
    if (st != KDA_OK) return st;
    if (tokens < 0) return KDA_ERR_INVALID_ARG;
    if (tokens == 0 || pages == 0) return KDA_OK;        // without pages every slot is outside the cache
    const size_t e = dsize(dtype), width = (size_t)Hk * D * e, bytes = (size_t)pages * page * Hk * D;
    const size_t scales = (size_t)pages * Hk * 4;
    const int64_t least = (int64_t)Hk * D;
    if (k_stride < least || v_stride < least || k_stride >= MAX_DIM * 64 || v_stride >= MAX_DIM * 64) return KDA_ERR_INVALID_ARG;
    const Rows rows[] = {{k, width, (size_t)k_stride * e, tokens}, {v, width, (size_t)v_stride * e, tokens}};
    const Buffer in[] = {{k, rows[0].span(), true, e}, {v, rows[1].span(), true, e}, {slots, (size_t)tokens * 4, true, 4}};
    const Buffer out[] = {{k_codes, bytes, true}, {v_codes, bytes, true}, {k_scale, scales, true, 4}, {v_scale, scales, true, 4}};
    const kda_status_t ok = check_buffers(in, out);
    if (ok != KDA_OK) return ok;
    kda::AppendArgs a;
    a.k = k; a.v = v; a.slots = slots; a.k_codes = (uint8_t *)k_codes; a.v_codes = (uint8_t *)v_codes;
    a.k_scale = k_scale; a.v_scale = v_scale; a.k_stride = k_stride; a.v_stride = v_stride;
    a.tokens = tokens; a.Hk = Hk; a.D = D; a.pages = pages; a.page = page;
    a.int8 = code == KDA_CODE_INT8; a.bf16 = dtype == KDA_BF16;
    return launched(kda::launch_cache_append(a, (hipStream_t)stream));
}

// --------------------------------------------------------------- attention

static kda_status_t check_attention(int tokens, int B, int Hq, int Hk, int D, int pages, int page, int max_pages,
                                    int max_queries, kda_code_t code, kda_dtype_t dtype)
{
    const kda_status_t st = check_cache(Hk, D, pages, page, code, dtype);
    if (st != KDA_OK) return st;
    if (tokens < 0 || B < 0 || Hq <= 0 || Hq % Hk || max_pages < 0 || max_queries < 0) return KDA_ERR_INVALID_ARG;
    if (B >= MAX_DIM || tokens >= MAX_DIM || Hq >= 65536 || (int64_t)max_pages * page >= INT_LIMIT - 256) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)tokens * Hq >= INT_LIMIT) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// The longest sequence's rows, as far as the host knows: one at least, and no more than there are.
static int longest_rows(int max_queries, int tokens)
{
    return max_queries < 1 ? 1 : max_queries > tokens ? tokens : max_queries;
}

size_t kda_cache_attention_workspace_bytes(int tokens, int B, int Hq, int Hk, int D, int page, int max_pages,
                                           int max_queries)
{
    if (check_attention(tokens, B, Hq, Hk, D, 0, page, max_pages, max_queries, KDA_CODE_E4M3, KDA_F32) != KDA_OK) return 0;
    if (tokens == 0 || B == 0) return 0;
    return (size_t)kda::cache_attend_workspace_floats(tokens, B, Hq, Hk, D, page, max_pages,
                                                     longest_rows(max_queries, tokens)) * sizeof(float);
}

kda_status_t kda_cache_attention(const void *q, const void *k_codes, const void *v_codes, const float *k_scale,
                                 const float *v_scale, const int *block_table, const int *context, const int *q_start,
                                 void *out, float *lse, void *workspace, size_t workspace_bytes,
                                 int tokens, int B, int Hq, int Hk, int D, int pages, int page, int max_pages,
                                 int max_queries, float scale, kda_code_t code, kda_dtype_t dtype, void *stream)
{
    const kda_status_t st = check_attention(tokens, B, Hq, Hk, D, pages, page, max_pages, max_queries, code, dtype);
    if (st != KDA_OK) return st;
    if (!(scale >= -3.0e38f && scale <= 3.0e38f) || (!q_start && tokens != B)) return KDA_ERR_INVALID_ARG;
    if (tokens == 0 || B == 0) return KDA_OK;
    const size_t need = kda_cache_attention_workspace_bytes(tokens, B, Hq, Hk, D, page, max_pages, max_queries);
    if (workspace_bytes < need) return KDA_ERR_INVALID_ARG;
    const size_t e = dsize(dtype), rows = (size_t)tokens * Hq * D * e, bytes = (size_t)pages * page * Hk * D;
    const size_t scales = (size_t)pages * Hk * 4;
    const Buffer in[] = {{q, rows, true}, {k_codes, bytes, true}, {v_codes, bytes, true}, {k_scale, scales, true, 4},
                         {v_scale, scales, true, 4}, {block_table, (size_t)B * max_pages * 4, true, 4},
                         {context, (size_t)B * 4, true, 4}, {q_start, (size_t)(B + 1) * 4, false, 4}};
    const Buffer out_[] = {{out, rows, true}, {lse, (size_t)tokens * Hq * 4, false, 4}, {workspace, need, true}};
    const kda_status_t ok = check_buffers(in, out_);
    if (ok != KDA_OK) return ok;
    kda::AttendArgs a;
    a.q = q; a.k_codes = (const uint8_t *)k_codes; a.v_codes = (const uint8_t *)v_codes;
    a.k_scale = k_scale; a.v_scale = v_scale; a.table = block_table; a.context = context; a.q_start = q_start;
    a.out = out; a.lse = lse; a.ws = (float *)workspace;
    a.tokens = tokens; a.B = B; a.Hq = Hq; a.Hk = Hk; a.D = D; a.pages = pages; a.page = page;
    a.per = max_pages;                                    // by which kernel and workspace are chosen
    a.room = pages > 0 ? (int64_t)max_pages * page : 0;
    a.most = longest_rows(max_queries, tokens); a.scale = scale;
    a.int8 = code == KDA_CODE_INT8; a.bf16 = dtype == KDA_BF16;
    return launched(kda::launch_cache_attend(a, (hipStream_t)stream));
}

}  // extern "C"
