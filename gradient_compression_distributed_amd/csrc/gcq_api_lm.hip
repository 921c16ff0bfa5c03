// gcq_api_lm.hip -- the C ABI of the language-model operators (declared and
// documented in include/gcq.h): host-side argument checks, then the launch.
#include "gcq.h"
#include "gcq_checks.h"
#include "gcq_lm.h"

namespace {

using gcq::aligned;
using gcq::any_write_overlap;
using gcq::launch_status;
using gcq::range;
using gcq::Range;

bool float_type(int t) { return t == GCQ_F32 || t == GCQ_F16 || t == GCQ_BF16; }

bool index_type(int t) { return t == GCQ_I32 || t == GCQ_I64; }

size_t type_bytes(int t)
{
    return t == GCQ_I64 ? 8 : t == GCQ_F32 || t == GCQ_I32 ? 4 : 2;
}

bool rows_of(size_t rows) { return rows <= GCQ_LM_MAX_ROWS; }

// A matrix of `rows` rows of `cols` elements, `ld` apart: its last element's
// offset stays below GCQ_MAX_ELEMS.
bool shape_ok(size_t rows, size_t cols, size_t ld)
{
    size_t all;
    return ld >= cols && !__builtin_mul_overflow(rows, ld, &all) && all <= GCQ_MAX_ELEMS;
}

Range matrix(const void *p, int type, size_t rows, size_t cols, size_t ld, bool writable)
{
    return range(p, rows && cols ? ((rows - 1) * ld + cols) * type_bytes(type) : 0, writable);
}

bool embed_ok(size_t n, size_t vocab, size_t dim)
{
    return rows_of(n) && vocab >= 1 && vocab <= 0x7FFFFFFFu && dim >= 1 && dim <= GCQ_LM_MAX_DIM;
}

}  // namespace

extern "C" {

int embed_lookup(const void *table, int table_type, size_t vocab, size_t dim, size_t table_ld,
                 const void *tokens, int token_type, size_t n, float scale, void *out,
                 int out_type, size_t out_ld, void *stream)
{
    if (!embed_ok(n, vocab, dim) || !float_type(table_type) || !float_type(out_type) ||
        !index_type(token_type) || !isfinite(scale) || !shape_ok(vocab, dim, table_ld) ||
        !shape_ok(n, dim, out_ld))
        return GCQ_ERR_PARAM;
    if (n == 0)
        return GCQ_OK;
    if (!table || !tokens || !out)
        return GCQ_ERR_NULL;
    if (!aligned(table, type_bytes(table_type)) || !aligned(tokens, type_bytes(token_type)) ||
        !aligned(out, type_bytes(out_type)))
        return GCQ_ERR_ALIGN;
    Range r[] = {matrix(table, table_type, vocab, dim, table_ld, false),
                 range(tokens, n * type_bytes(token_type), false),
                 matrix(out, out_type, n, dim, out_ld, true)};
    if (any_write_overlap(r, r + 3))
        return GCQ_ERR_OVERLAP;
    const gcq::EmbedTable t = {table, table_type, vocab, dim, table_ld};
    return launch_status(gcq::launch_embed_lookup(t, tokens, token_type == GCQ_I64, n, scale, out,
                                                  out_type, out_ld, (hipStream_t)stream));
}

size_t embed_plan_words(size_t n) { return rows_of(n) ? (size_t)gcq::embed_plan_words(n) : 0; }

size_t embed_work_bytes(size_t n, size_t dim)
{
    return rows_of(n) && dim <= GCQ_LM_MAX_DIM ? (size_t)gcq::embed_work_bytes(n, dim) : 0;
}

int embed_sort(const void *tokens, int token_type, size_t n, size_t vocab, uint32_t *plan,
               void *stream)
{
    if (!embed_ok(n, vocab, 1) || !index_type(token_type))
        return GCQ_ERR_PARAM;
    if (n == 0)
        return GCQ_OK;
    if (!tokens || !plan)
        return GCQ_ERR_NULL;
    if (!aligned(tokens, type_bytes(token_type)) || !aligned(plan, 4))
        return GCQ_ERR_ALIGN;
    Range r[] = {range(tokens, n * type_bytes(token_type), false),
                 range(plan, embed_plan_words(n) * 4, true)};
    if (any_write_overlap(r, r + 2))
        return GCQ_ERR_OVERLAP;
    return launch_status(gcq::launch_embed_sort(tokens, token_type == GCQ_I64, n, vocab, plan,
                                                (hipStream_t)stream));
}

namespace {

// The checks and launch that both forms of the gradient share.
int embed_gradient(const void *grad, int grad_type, size_t grad_ld, const uint32_t *plan, size_t n,
                   size_t vocab, size_t dim, float scale, bool add, float *out, size_t out_rows,
                   size_t out_ld, int32_t *ids, int32_t *count, void *work, void *stream)
{
    if (!embed_ok(n, vocab, dim) || !float_type(grad_type) || !isfinite(scale) ||
        !shape_ok(n, dim, grad_ld) || !shape_ok(out_rows, dim, out_ld))
        return GCQ_ERR_PARAM;
    if ((out_rows && !out) || (n && (!grad || !plan || !work)))
        return GCQ_ERR_NULL;
    if (!aligned(grad, type_bytes(grad_type)) || !aligned(plan, 4) || !aligned(out, 4) ||
        !aligned(ids, 4) || !aligned(count, 4) || !aligned(work, 16))
        return GCQ_ERR_ALIGN;
    Range r[] = {matrix(grad, grad_type, n, dim, grad_ld, false),
                 range(plan, embed_plan_words(n) * 4, false),
                 matrix(out, GCQ_F32, out_rows, dim, out_ld, true),
                 range(work, embed_work_bytes(n, dim), true),
                 range(ids, ids ? out_rows * 4 : 0, true),
                 range(count, count ? 4 : 0, true)};
    if (any_write_overlap(r, r + 6))
        return GCQ_ERR_OVERLAP;
    if (n == 0 && add)
        return GCQ_OK;
    gcq::EmbedGrad e = {};
    e.g = grad;
    e.type = grad_type;
    e.ld = grad_ld;
    e.keys = plan;
    e.order = plan + n;
    e.n = n;
    e.vocab = vocab;
    e.dim = dim;
    e.scale = scale;
    e.out = out;
    e.out_ld = out_ld;
    e.ids = ids;
    e.count = count;
    e.add = add;
    gcq::embed_work_layout(e, work);
    return launch_status(gcq::launch_embed_grad(e, (hipStream_t)stream));
}

}  // namespace

int embed_grad(const void *grad, int grad_type, size_t grad_ld, const uint32_t *plan, size_t n,
               size_t vocab, size_t dim, float scale, int accumulate, float *dtable,
               size_t dtable_ld, void *work, void *stream)
{
    return embed_gradient(grad, grad_type, grad_ld, plan, n, vocab, dim, scale, accumulate != 0,
                          dtable, vocab, dtable_ld, nullptr, nullptr, work, stream);
}

int embed_grad_rows(const void *grad, int grad_type, size_t grad_ld, const uint32_t *plan,
                    size_t n, size_t vocab, size_t dim, float scale, int32_t *ids, float *rows,
                    size_t rows_ld, int32_t *count, void *work, void *stream)
{
    if (!count || (n && !ids))
        return GCQ_ERR_NULL;
    return embed_gradient(grad, grad_type, grad_ld, plan, n, vocab, dim, scale, false, rows,
                          n < vocab ? n : vocab, rows_ld, ids, count, work, stream);
}

}  // extern "C"
