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
        (dict(kt=F32), E_PARAM), (dict(n=(1 << 30) + 1), E_PARAM), (dict(scale=NAN), E_PARAM),
        (dict(scale=INF), E_PARAM), (dict(ld=1 << 60), E_PARAM), (dict(table=0), E_NULL),
        (dict(tokens=0), E_NULL), (dict(out=0), E_NULL), (dict(table=A + 1), E_ALIGN),
        (dict(tokens=A + MB + 4), E_ALIGN), (dict(out=A + 2 * MB + 1), E_ALIGN),
        (dict(out=A + 1598), E_OVERLAP), (dict(out=A + MB + 78), E_OVERLAP),
        (dict(n=0, table=0, tokens=0, out=0), OK)])


def test_embed_sort(lib):
    good = dict(tokens=A, kt=I32, n=100, vocab=50, plan=A + MB)
    refuses(lib.embed_sort, good, [
        (dict(vocab=0), E_PARAM), (dict(vocab=1 << 31), E_PARAM), (dict(kt=BF16), E_PARAM),
        (dict(n=(1 << 30) + 1), E_PARAM), (dict(tokens=0), E_NULL), (dict(plan=0), E_NULL),
        (dict(tokens=A + 2), E_ALIGN), (dict(plan=A + MB + 2), E_ALIGN),
        (dict(plan=A + 396), E_OVERLAP), (dict(n=0, tokens=0, plan=0), OK)])
    assert lib.embed_plan_words(0) == 0 and lib.embed_plan_words((1 << 30) + 1) == 0
    assert lib.embed_plan_words(100) >= 200


def test_embed_grad(lib):
    good = dict(grad=A, gt=BF16, ld=8, plan=A + MB, n=100, vocab=50, dim=8, scale=1.0, add=0,
                out=A + 2 * MB, out_ld=8, work=A + 3 * MB)
    refuses(lib.embed_grad, good, [
        (dict(gt=I64), E_PARAM), (dict(ld=7), E_PARAM), (dict(vocab=0), E_PARAM),
        (dict(dim=0), E_PARAM), (dict(scale=NAN), E_PARAM), (dict(out_ld=3), E_PARAM),
        (dict(n=(1 << 30) + 1), E_PARAM), (dict(grad=0), E_NULL), (dict(plan=0), E_NULL),
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
    plan = gcq.EmbedPlan(torch.zeros(16, dtype=torch.int32), 4, 4)
    with pytest.raises(ValueError):
        gcq.embed_grad(t, plan)
    with pytest.raises(ValueError):
        gcq.embed_grad_rows(t, plan)
