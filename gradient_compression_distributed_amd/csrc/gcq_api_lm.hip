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

namespace {

// x and an operand that may take its place element by element.
bool same_matrix(const void *a, size_t a_ld, const void *b, size_t b_ld)
{
    return a && a == b && a_ld == b_ld;
}

// The checks and launch of rms_norm (out: a matrix of `out_type`) and
// rms_norm_q8 (out: codes, one byte each).
int rms(const void *x, int type, size_t rows, size_t dim, size_t x_ld, const void *residual,
        size_t residual_ld, const void *weight, int weight_type, float eps, bool q8, uint32_t group,
        void *out, size_t out_ld, float *scales, void *h, size_t h_ld, float *rstd, void *stream)
{
    if (!rows_of(rows) || dim < 1 || dim > GCQ_LM_MAX_DIM || !float_type(type) ||
        (weight_type != type && weight_type != GCQ_F32) || !(isfinite(eps) && eps >= 0.0f) ||
        !shape_ok(rows, dim, x_ld) || !shape_ok(rows, dim, out_ld) ||
        (residual && !shape_ok(rows, dim, residual_ld)) || (h && !shape_ok(rows, dim, h_ld)) ||
        (h && !residual))
        return GCQ_ERR_PARAM;
    if (q8 && group != 0 && group != 32 && group != 64 && group != 128)
        return GCQ_ERR_PARAM;
    if (rows == 0)
        return GCQ_OK;
    if (!x || !weight || !out || (q8 && !scales))
        return GCQ_ERR_NULL;
    const size_t es = type_bytes(type);
    if (!aligned(x, es) || !aligned(residual, es) || !aligned(weight, type_bytes(weight_type)) ||
        !aligned(out, q8 ? 1 : es) || !aligned(scales, 4) || !aligned(h, es) || !aligned(rstd, 4))
        return GCQ_ERR_ALIGN;
    const size_t parts = group ? (dim + group - 1) / group : 1;
    const bool h_is_x = same_matrix(h, h_ld, x, x_ld);
    const bool h_is_res = same_matrix(h, h_ld, residual, residual_ld);
    Range r[8];
    int n = 0;
    if (!h_is_x)
        r[n++] = matrix(x, type, rows, dim, x_ld, false);
    if (residual && !h_is_res)
        r[n++] = matrix(residual, type, rows, dim, residual_ld, false);
    r[n++] = range(weight, dim * type_bytes(weight_type), false);
    r[n++] = q8 ? range(out, (rows - 1) * out_ld + dim, true)
                : matrix(out, type, rows, dim, out_ld, true);
    if (q8)
        r[n++] = range(scales, rows * parts * 4, true);
    if (h)
        r[n++] = matrix(h, type, rows, dim, h_ld, true);
    if (rstd)
        r[n++] = range(rstd, rows * 4, true);
    if (any_write_overlap(r, r + n))
        return GCQ_ERR_OVERLAP;
    gcq::RmsNorm a = {};
    a.type = type;
    a.w_f32 = weight_type == GCQ_F32;
    a.x = x;
    a.res = residual;
    a.w = weight;
    a.rows = rows;
    a.dim = dim;
    a.x_ld = x_ld;
    a.res_ld = residual_ld;
    a.y_ld = out_ld;
    a.h_ld = h_ld;
    a.eps = eps;
    a.y = q8 ? nullptr : out;
    a.codes = q8 ? (uint8_t *)out : nullptr;
    a.scales = scales;
    a.group = group;
    a.parts = parts;
    a.h = h;
    a.rstd = rstd;
    return launch_status(gcq::launch_rms_norm(a, (hipStream_t)stream));
}

}  // namespace

int rms_norm(const void *x, int type, size_t rows, size_t dim, size_t x_ld, const void *residual,
             size_t residual_ld, const void *weight, int weight_type, float eps, void *y,
             size_t y_ld, void *h, size_t h_ld, float *rstd, void *stream)
{
    return rms(x, type, rows, dim, x_ld, residual, residual_ld, weight, weight_type, eps, false, 0,
               y, y_ld, nullptr, h, h_ld, rstd, stream);
}

int rms_norm_q8(const void *x, int type, size_t rows, size_t dim, size_t x_ld,
                const void *residual, size_t residual_ld, const void *weight, int weight_type,
                float eps, uint32_t group, uint8_t *codes, size_t codes_ld, float *scales, void *h,
                size_t h_ld, float *rstd, void *stream)
{
    return rms(x, type, rows, dim, x_ld, residual, residual_ld, weight, weight_type, eps, true,
               group, codes, codes_ld, scales, h, h_ld, rstd, stream);
}

size_t rms_norm_work_bytes(size_t rows, size_t dim, int type)
{
    if (!rows_of(rows) || dim > GCQ_LM_MAX_DIM || !float_type(type))
        return 0;
    return (size_t)gcq::rms_norm_work_bytes(rows, dim, type);
}

int rms_norm_grad(const void *dy, int type, size_t rows, size_t dim, size_t dy_ld, const void *h,
                  size_t h_ld, const void *weight, int weight_type, const float *rstd,
                  const void *dh, size_t dh_ld, void *dx, size_t dx_ld, float *dweight,
                  int accumulate, void *work, void *stream)
{
    if (!rows_of(rows) || dim < 1 || dim > GCQ_LM_MAX_DIM || !float_type(type) ||
        (weight_type != type && weight_type != GCQ_F32) || !shape_ok(rows, dim, dy_ld) ||
        !shape_ok(rows, dim, h_ld) || !shape_ok(rows, dim, dx_ld) ||
        (dh && !shape_ok(rows, dim, dh_ld)))
        return GCQ_ERR_PARAM;
    if (!dweight || (rows && (!dy || !h || !weight || !rstd || !dx || !work)))
        return GCQ_ERR_NULL;
    const size_t es = type_bytes(type);
    if (!aligned(dy, es) || !aligned(h, es) || !aligned(weight, type_bytes(weight_type)) ||
        !aligned(rstd, 4) || !aligned(dh, es) || !aligned(dx, es) || !aligned(dweight, 4) ||
        !aligned(work, 16))
        return GCQ_ERR_ALIGN;
    Range r[8];
    int n = 0;
    r[n++] = matrix(dy, type, rows, dim, dy_ld, false);
    r[n++] = matrix(h, type, rows, dim, h_ld, false);
    r[n++] = range(weight, rows ? dim * type_bytes(weight_type) : 0, false);
    r[n++] = range(rstd, rows * 4, false);
    if (dh && !same_matrix(dx, dx_ld, dh, dh_ld))
        r[n++] = matrix(dh, type, rows, dim, dh_ld, false);
    r[n++] = matrix(dx, type, rows, dim, dx_ld, true);
    r[n++] = range(dweight, dim * 4, true);
    r[n++] = range(work, gcq::rms_norm_work_bytes(rows, dim, type), true);
    if (any_write_overlap(r, r + n))
        return GCQ_ERR_OVERLAP;
    if (rows == 0 && accumulate)
        return GCQ_OK;
    gcq::RmsGrad a = {};
    a.type = type;
    a.w_f32 = weight_type == GCQ_F32;
    a.dy = dy;
    a.h = h;
    a.w = weight;
    a.dh = dh;
    a.rstd = rstd;
    a.rows = rows;
    a.dim = dim;
    a.dy_ld = dy_ld;
    a.h_ld = h_ld;
    a.dh_ld = dh_ld;
    a.dx_ld = dx_ld;
    a.dx = dx;
    a.dw = dweight;
    a.add = accumulate != 0;
    a.part_w = (float *)work;
    return launch_status(gcq::launch_rms_norm_grad(a, (hipStream_t)stream));
}

namespace {

bool topk_ok(size_t rows, size_t vocab, uint32_t k, int type, int idx_type, int top_type, float t,
             float scale)
{
    return rows_of(rows) && vocab >= 1 && vocab <= GCQ_LM_MAX_DIM && k >= 1 && k <= GCQ_MAX_TOPK &&
           float_type(type) && index_type(idx_type) && (top_type == type || top_type == GCQ_F32) &&
           isfinite(t) && t > 0.0f && isfinite(scale) &&
           // the kernels' factors; an infinite one gives NaN at a row's largest logit
           isfinite(1.44269504f / t) && isfinite(scale / t);
}

// Everything that the three calls share: `lse_in` for the gradient alone,
// `loss` and `lse_out` for the loss, `dz` for a gradient.
int distill(const void *z, int type, size_t rows, size_t vocab, size_t z_ld, const void *idx,
            int idx_type, size_t idx_ld, const void *top, int top_type, size_t top_ld, uint32_t k,
            float temperature, const float *row_scale, float scale, bool loss_wanted,
            bool grad_wanted, const float *lse_in, float *loss, float *lse_out, void *dz,
            size_t dz_ld, void *stream)
{
    if (!topk_ok(rows, vocab, k, type, idx_type, top_type, temperature, scale) ||
        !shape_ok(rows, vocab, z_ld) || !shape_ok(rows, k, idx_ld) || !shape_ok(rows, k, top_ld) ||
        (grad_wanted && !shape_ok(rows, vocab, dz_ld)))
        return GCQ_ERR_PARAM;
    if (rows == 0)
        return GCQ_OK;
    if (!z || !idx || !top || (loss_wanted ? !loss || !lse_out : !lse_in) || (grad_wanted && !dz))
        return GCQ_ERR_NULL;
    const size_t es = type_bytes(type);
    if (!aligned(z, es) || !aligned(idx, type_bytes(idx_type)) ||
        !aligned(top, type_bytes(top_type)) || !aligned(row_scale, 4) || !aligned(lse_in, 4) ||
        !aligned(loss, 4) || !aligned(lse_out, 4) || !aligned(dz, es))
        return GCQ_ERR_ALIGN;
    Range r[8];
    int n = 0;
    if (!grad_wanted || !same_matrix(dz, dz_ld, z, z_ld))
        r[n++] = matrix(z, type, rows, vocab, z_ld, false);
    r[n++] = matrix(idx, idx_type, rows, k, idx_ld, false);
    r[n++] = matrix(top, top_type, rows, k, top_ld, false);
    if (row_scale)
        r[n++] = range(row_scale, rows * 4, false);
    if (loss_wanted) {
        r[n++] = range(loss, rows * 4, true);
        r[n++] = range(lse_out, rows * 4, true);
    } else {
        r[n++] = range(lse_in, rows * 4, false);
    }
    if (grad_wanted)
        r[n++] = matrix(dz, type, rows, vocab, dz_ld, true);
    if (any_write_overlap(r, r + n))
        return GCQ_ERR_OVERLAP;
    gcq::Distill a = {};
    a.type = type;
    a.t_f32 = top_type == GCQ_F32;
    a.idx64 = idx_type == GCQ_I64;
    a.z = z;
    a.idx = idx;
    a.top = top;
    a.rows = rows;
    a.vocab = vocab;
    a.z_ld = z_ld;
    a.idx_ld = idx_ld;
    a.top_ld = top_ld;
    a.dz_ld = dz_ld;
    a.k = k;
    a.temp = temperature;
    a.scale = scale;
    a.row_scale = row_scale;
    a.lse = lse_in;
    a.loss = loss;
    a.lse_out = lse_out;
    a.dz = grad_wanted ? dz : nullptr;
    return launch_status(gcq::launch_distill(a, (hipStream_t)stream));
}

}  // namespace

int distill_loss(const void *logits, int type, size_t rows, size_t vocab, size_t logits_ld,
                 const void *index, int index_type, size_t index_ld, const void *teacher,
                 int teacher_type, size_t teacher_ld, uint32_t k, float temperature,
                 const float *row_scale, float scale, float *loss, float *lse, void *stream)
{
    return distill(logits, type, rows, vocab, logits_ld, index, index_type, index_ld, teacher,
                   teacher_type, teacher_ld, k, temperature, row_scale, scale, true, false, nullptr,
                   loss, lse, nullptr, 0, stream);
}

int distill_grad(const void *logits, int type, size_t rows, size_t vocab, size_t logits_ld,
                 const float *lse, const void *index, int index_type, size_t index_ld,
                 const void *teacher, int teacher_type, size_t teacher_ld, uint32_t k,
                 float temperature, const float *row_scale, float scale, void *dlogits,
                 size_t dlogits_ld, void *stream)
{
    return distill(logits, type, rows, vocab, logits_ld, index, index_type, index_ld, teacher,
                   teacher_type, teacher_ld, k, temperature, row_scale, scale, false, true, lse,
                   nullptr, nullptr, dlogits, dlogits_ld, stream);
}

int distill_loss_grad(const void *logits, int type, size_t rows, size_t vocab, size_t logits_ld,
                      const void *index, int index_type, size_t index_ld, const void *teacher,
                      int teacher_type, size_t teacher_ld, uint32_t k, float temperature,
                      const float *row_scale, float scale, float *loss, float *lse, void *dlogits,
                      size_t dlogits_ld, void *stream)
{
    return distill(logits, type, rows, vocab, logits_ld, index, index_type, index_ld, teacher,
                   teacher_type, teacher_ld, k, temperature, row_scale, scale, true, true, nullptr,
                   loss, lse, dlogits, dlogits_ld, stream);
}

}  // extern "C"
