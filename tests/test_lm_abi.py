"""Refusals of the language-model operators, on the host: the C ABI with fake
device addresses that are never dereferenced, and the binding's own checks."""
import ctypes

import pytest

import gradient_compression_distributed_amd as gcq

OK, E_NULL, E_PARAM, E_ALIGN, E_OVERLAP = 0, -1, -3, -4, -5
A, MB = 0x7F0000000000, 1 << 24
F32, F16, BF16, I32, I64 = range(5)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return gcq.load()


def change(good, **k):
    return {**good, **k}


def refuses(fn, good, cases):
    """Every case (a change of the good arguments) has its status."""
    for k, want in cases:
        got = fn(*change(good, **k).values(), None)
        assert got == want, (k, got, want)


def test_embed_lookup(lib):
    good = dict(table=A, tt=BF16, vocab=100, dim=8, ld=8, tokens=A + MB, kt=I64, n=10, scale=1.0,
                out=A + 2 * MB, ot=BF16, out_ld=8)
    refuses(lib.embed_lookup, good, [
        (dict(vocab=0), E_PARAM), (dict(vocab=1 << 31), E_PARAM), (dict(dim=0), E_PARAM),
        (dict(dim=(1 << 22) + 1, ld=1 << 23, out_ld=1 << 23), E_PARAM), (dict(ld=7), E_PARAM),
        (dict(out_ld=7), E_PARAM), (dict(tt=I32), E_PARAM), (dict(ot=9), E_PARAM),
        (dict(kt=F32), E_PARAM), (dict(n=(1 << 24) + 1), E_PARAM), (dict(scale=NAN), E_PARAM),
        (dict(scale=INF), E_PARAM), (dict(ld=1 << 60), E_PARAM), (dict(table=0), E_NULL),
        (dict(tokens=0), E_NULL), (dict(out=0), E_NULL), (dict(table=A + 1), E_ALIGN),
        (dict(tokens=A + MB + 4), E_ALIGN), (dict(out=A + 2 * MB + 1), E_ALIGN),
        (dict(out=A + 1598), E_OVERLAP), (dict(out=A + MB + 78), E_OVERLAP),
        (dict(n=0, table=0, tokens=0, out=0), OK)])


def test_embed_sort(lib):
    good = dict(tokens=A, kt=I32, n=100, vocab=50, plan=A + MB)
    refuses(lib.embed_sort, good, [
        (dict(vocab=0), E_PARAM), (dict(vocab=1 << 31), E_PARAM), (dict(kt=BF16), E_PARAM),
        (dict(n=(1 << 24) + 1), E_PARAM), (dict(tokens=0), E_NULL), (dict(plan=0), E_NULL),
        (dict(tokens=A + 2), E_ALIGN), (dict(plan=A + MB + 2), E_ALIGN),
        (dict(plan=A + 396), E_OVERLAP), (dict(n=0, tokens=0, plan=0), OK)])
    assert lib.embed_plan_words(0) == 0 and lib.embed_plan_words((1 << 24) + 1) == 0
    assert lib.embed_plan_words(100) >= 200


def test_embed_grad(lib):
    good = dict(grad=A, gt=BF16, ld=8, plan=A + MB, n=100, vocab=50, dim=8, scale=1.0, add=0,
                out=A + 2 * MB, out_ld=8, work=A + 3 * MB)
    refuses(lib.embed_grad, good, [
        (dict(gt=I64), E_PARAM), (dict(ld=7), E_PARAM), (dict(vocab=0), E_PARAM),
        (dict(dim=0), E_PARAM), (dict(scale=NAN), E_PARAM), (dict(out_ld=3), E_PARAM),
        (dict(n=(1 << 24) + 1), E_PARAM), (dict(grad=0), E_NULL), (dict(plan=0), E_NULL),
        (dict(out=0), E_NULL), (dict(work=0), E_NULL), (dict(grad=A + 1), E_ALIGN),
        (dict(plan=A + MB + 1), E_ALIGN), (dict(out=A + 2 * MB + 2), E_ALIGN),
        (dict(work=A + 3 * MB + 8), E_ALIGN), (dict(out=A + 1596), E_OVERLAP),
        (dict(out=A + MB), E_OVERLAP), (dict(work=A + 2 * MB + 1584), E_OVERLAP),
        (dict(work=A + MB), E_OVERLAP), (dict(n=0, add=1, grad=0, plan=0, work=0), OK)])


def test_embed_grad_rows(lib):
    good = dict(grad=A, gt=F32, ld=8, plan=A + MB, n=100, vocab=50, dim=8, scale=1.0,
                ids=A + 4 * MB, rows=A + 2 * MB, rows_ld=8, count=A + 5 * MB, work=A + 3 * MB)
    refuses(lib.embed_grad_rows, good, [
        (dict(ids=0), E_NULL), (dict(count=0), E_NULL), (dict(rows=0), E_NULL),
        (dict(ids=A + 4 * MB + 2), E_ALIGN), (dict(count=A + 5 * MB + 1), E_ALIGN),
        (dict(rows_ld=7), E_PARAM), (dict(ids=A + 2 * MB + 1596), E_OVERLAP),
        (dict(count=A + 4 * MB + 196), E_OVERLAP), (dict(count=A + 396), E_OVERLAP)])
    assert lib.embed_work_bytes(100, 8) >= 4 * 2 * 4 * 8
    assert lib.embed_work_bytes(100, (1 << 22) + 1) == 0


def test_binding_refuses_host_tensors():
    import torch

    t, i = torch.zeros(4, 4), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        gcq.embed_lookup(t, i)
    with pytest.raises(ValueError):
        gcq.embed_sort(i, 4)
    with pytest.raises(TypeError):
        gcq.embed_lookup([1.0], i)
    with pytest.raises(TypeError):
        gcq.embed_sort([1, 2], 4)
    plan = gcq.EmbedPlan(torch.zeros(16, dtype=torch.int32), 4, 4)
    with pytest.raises(ValueError):
        gcq.embed_grad(t, plan)
    with pytest.raises(ValueError):
        gcq.embed_grad_rows(t, plan)


def test_rms_norm(lib):
    good = dict(x=A, t=BF16, rows=10, dim=8, x_ld=8, res=A + MB, res_ld=8, w=A + 2 * MB, wt=F32,
                eps=1e-6, y=A + 3 * MB, y_ld=8, h=A + 4 * MB, h_ld=8, rstd=A + 5 * MB)
    refuses(lib.rms_norm, good, [
        (dict(t=I32), E_PARAM), (dict(wt=F16), E_PARAM), (dict(eps=-1.0), E_PARAM),
        (dict(eps=NAN), E_PARAM), (dict(eps=INF), E_PARAM), (dict(dim=0), E_PARAM),
        (dict(dim=(1 << 22) + 1), E_PARAM), (dict(x_ld=7), E_PARAM), (dict(res_ld=7), E_PARAM),
        (dict(y_ld=7), E_PARAM), (dict(h_ld=7), E_PARAM), (dict(rows=(1 << 24) + 1), E_PARAM),
        (dict(res=0), E_PARAM),                      # h without a residual
        (dict(x=0), E_NULL), (dict(w=0), E_NULL), (dict(y=0), E_NULL), (dict(x=A + 1), E_ALIGN),
        (dict(w=A + 2 * MB + 2), E_ALIGN), (dict(rstd=A + 5 * MB + 2), E_ALIGN),
        (dict(y=A), E_OVERLAP), (dict(y=A + MB + 158), E_OVERLAP), (dict(h=A + 3 * MB), E_OVERLAP),
        (dict(h=A + 2), E_OVERLAP), (dict(h=A, h_ld=9), E_OVERLAP), (dict(rstd=A + 2 * MB), E_OVERLAP),
        (dict(rows=0, x=0, w=0, y=0), OK)])


def test_rms_norm_q8(lib):
    good = dict(x=A, t=F32, rows=10, dim=200, x_ld=200, res=0, res_ld=0, w=A + 2 * MB, wt=F32,
                eps=1e-6, group=64, codes=A + 3 * MB, codes_ld=200, scales=A + 4 * MB, h=0, h_ld=0,
                rstd=A + 5 * MB)
    refuses(lib.rms_norm_q8, good, [
        (dict(group=16), E_PARAM), (dict(group=256), E_PARAM), (dict(group=33), E_PARAM),
        (dict(h=A + 6 * MB, h_ld=200), E_PARAM), (dict(codes_ld=199), E_PARAM),
        (dict(codes=0), E_NULL), (dict(scales=0), E_NULL), (dict(scales=A + 4 * MB + 2), E_ALIGN),
        (dict(scales=A + 3 * MB + 1996), E_OVERLAP), (dict(codes=A + 4 * MB + 156), E_OVERLAP),
        (dict(codes=A + 7996), E_OVERLAP), (dict(rows=0, codes=0, scales=0), OK)])


def test_rms_norm_grad(lib):
    good = dict(dy=A, t=F16, rows=10, dim=8, dy_ld=8, h=A + MB, h_ld=8, w=A + 2 * MB, wt=F16,
                rstd=A + 3 * MB, dh=A + 4 * MB, dh_ld=8, dx=A + 5 * MB, dx_ld=8, dw=A + 6 * MB,
                add=0, work=A + 7 * MB)
    refuses(lib.rms_norm_grad, good, [
        (dict(t=9), E_PARAM), (dict(wt=BF16), E_PARAM), (dict(dh_ld=7), E_PARAM),
        (dict(dx_ld=7), E_PARAM), (dict(dy=0), E_NULL), (dict(h=0), E_NULL), (dict(rstd=0), E_NULL),
        (dict(dx=0), E_NULL), (dict(dw=0), E_NULL), (dict(work=0), E_NULL),
        (dict(dw=A + 6 * MB + 2), E_ALIGN), (dict(work=A + 7 * MB + 8), E_ALIGN),
        (dict(dx=A), E_OVERLAP), (dict(dx=A + MB), E_OVERLAP), (dict(dx=A + 4 * MB, dx_ld=9), E_OVERLAP),
        (dict(dw=A + 2 * MB), E_OVERLAP), (dict(work=A + 6 * MB), E_OVERLAP),
        (dict(rows=0, add=1, dy=0, h=0, w=0, rstd=0, dx=0, work=0), OK)])
    # a row of sums per workgroup, which 16 rows of up to 256 columns share
    assert lib.rms_norm_work_bytes(10, 8, F16) == 8 * 4
    assert lib.rms_norm_work_bytes(33, 256, F16) == 3 * 256 * 4
    assert lib.rms_norm_work_bytes(10, 8, I32) == 0


def test_binding_refuses_host_tensors_rms():
    import torch

    x, w = torch.zeros(4, 4), torch.zeros(4)
    for call in (lambda: gcq.rms_norm(x, w, 1e-6), lambda: gcq.rms_norm_q8(x, w, 1e-6),
                 lambda: gcq.rms_norm_grad(x, x, w, w)):
        with pytest.raises(ValueError):
            call()


def test_distill(lib):
    head = dict(z=A, t=BF16, rows=4, vocab=100, z_ld=100)
    tail = dict(idx=A + MB, it=I64, idx_ld=8, top=A + 2 * MB, tt=BF16, top_ld=8, k=8, T=2.0,
                rs=A + 3 * MB, scale=1.0)
    out = dict(loss=A + 4 * MB, lse=A + 5 * MB)
    dz = dict(dz=A + 6 * MB, dz_ld=100)
    shared = [
        (dict(t=I32), E_PARAM), (dict(rows=(1 << 24) + 1), E_PARAM), (dict(vocab=0), E_PARAM),
        (dict(vocab=(1 << 22) + 1, z_ld=1 << 23), E_PARAM), (dict(z_ld=99), E_PARAM),
        (dict(it=F32), E_PARAM), (dict(tt=F16), E_PARAM), (dict(k=0), E_PARAM),
        (dict(k=1025, idx_ld=2000, top_ld=2000), E_PARAM), (dict(idx_ld=7), E_PARAM),
        (dict(top_ld=7), E_PARAM), (dict(T=0.0), E_PARAM), (dict(T=-1.0), E_PARAM),
        (dict(T=NAN), E_PARAM), (dict(T=INF), E_PARAM), (dict(scale=NAN), E_PARAM),
        (dict(z=0), E_NULL), (dict(idx=0), E_NULL), (dict(top=0), E_NULL), (dict(z=A + 1), E_ALIGN),
        (dict(idx=A + MB + 4), E_ALIGN), (dict(top=A + 2 * MB + 1), E_ALIGN),
        (dict(rs=A + 3 * MB + 2), E_ALIGN)]
    lost = [(dict(loss=0), E_NULL), (dict(lse=0), E_NULL), (dict(loss=A + 5 * MB), E_OVERLAP),
            (dict(loss=A), E_OVERLAP), (dict(lse=A + 3 * MB + 12), E_OVERLAP)]
    slope = [(dict(dz=0), E_NULL), (dict(dz_ld=99), E_PARAM), (dict(dz=A + 6 * MB + 1), E_ALIGN),
             (dict(dz=A + 2), E_OVERLAP), (dict(dz=A, dz_ld=101), E_OVERLAP),
             (dict(dz=A + MB), E_OVERLAP), (dict(dz=A + 2 * MB), E_OVERLAP)]
    none = dict(rows=0, z=0, idx=0, top=0)
    refuses(lib.distill_loss, {**head, **tail, **out}, shared + lost + [(none, OK)])
    refuses(lib.distill_loss_grad, {**head, **tail, **out, **dz},
            shared + lost + slope + [(dict(none, dz=0), OK)])
    refuses(lib.distill_grad, {**head, "lse": A + 5 * MB, **tail, **dz},
            shared + slope + [(dict(lse=0), E_NULL), (dict(lse=A + 6 * MB), E_OVERLAP), (none, OK)])


def test_binding_refuses_host_tensors_distill():
    import torch

    z, i, t, r = torch.zeros(4, 9), torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2), torch.zeros(4)
    for call in (lambda: gcq.distill_loss(z, i, t), lambda: gcq.distill_grad(z, r, i, t),
                 lambda: gcq.distill_loss_grad(z, i, t)):
        with pytest.raises(ValueError):
            call()
