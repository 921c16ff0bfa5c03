"""The language-model operators on tables and matrices whose elements lie past
2^32: a call on rows far apart, or at a large table's end, gives bit for bit
what it gives on the same rows side by side, and writes nothing else."""
import pytest

pytestmark = pytest.mark.gpu


def rows_apart(x, ld, fill=None):
    """x's rows, ld elements apart, past 2^32 elements in all."""
    import torch

    rows, cols = x.shape
    assert (rows - 1) * ld > 2 ** 32
    big = torch.empty((rows - 1) * ld + cols, dtype=x.dtype, device="cuda")
    view = big.as_strided((rows, cols), (ld, 1))
    view.copy_(x) if fill is None else view.fill_(fill)
    return view


def test_embedding_tables(gpu):
    import torch

    V, D, n = 2 ** 20 + 70, 4099, 700          # 4.3e9 elements
    gen = torch.Generator(device="cuda").manual_seed(1)
    tok = torch.randint(V - 64, V, (n,), device="cuda", generator=gen)
    tok[::3] = torch.randint(0, V, tok[::3].shape, device="cuda", generator=gen)
    tok[0], tok[1], tok[2] = V - 1, 0, -1
    ids, at = torch.unique(tok.clamp(min=0), return_inverse=True)
    at[2] = -1

    print("[gpu] lookup", V, D, n, flush=True)
    table = torch.empty(V, D, dtype=torch.bfloat16, device="cuda")
    small = torch.randn(len(ids), D, device="cuda", generator=gen).to(torch.bfloat16)
    table[ids] = small
    out = rows_apart(torch.zeros(n, D, dtype=torch.bfloat16, device="cuda"), 2 ** 23, fill=7.0)
    gpu.embed_lookup(table, tok, 0.5, out=out)
    want = gpu.embed_lookup(small, at, 0.5)
    assert torch.equal(out, want)
    del table, out

    print("[gpu] gradient", V, D, n, flush=True)
    g = rows_apart(torch.randn(n, D, device="cuda", generator=gen).to(torch.bfloat16), 2 ** 23)
    plan, few = gpu.embed_sort(tok, V), gpu.embed_sort(at, len(ids))
    near = g.contiguous()
    want = gpu.embed_grad(near, few, 0.5)
    table = torch.full((V, D), 3.0, device="cuda")
    gpu.embed_grad(g, plan, 0.5, out=table)
    assert torch.equal(table[ids], want)
    assert int((table != 0).any(1).sum()) == int((want != 0).any(1).sum())
    table.fill_(3.0)
    gpu.embed_grad(g, plan, 0.5, out=table, accumulate=True)
    base = torch.full_like(want, 3.0)
    assert torch.equal(table[ids], gpu.embed_grad(near, few, 0.5, out=base, accumulate=True))
    assert int((table != 3).any(1).sum()) == int((base != 3).any(1).sum())
    del table

    print("[gpu] row-sparse", V, D, n, flush=True)
    rows = rows_apart(torch.zeros(n, D, device="cuda"), 2 ** 23, fill=7.0)
    got, _, count = gpu.embed_grad_rows(g, plan, 0.5, rows=rows)
    u = int(count)
    names = tok[tok >= 0].unique()
    assert u == len(names) and torch.equal(got[:u].long(), names)
    assert torch.equal(rows[:u], gpu.embed_grad_rows(near, plan, 0.5)[1][:u])
    assert (rows[u:] == 7).all()


@pytest.mark.parametrize("dim", [1000, 40001])
def test_norm_rows(gpu, dim):
    import torch

    n, ld = 1100, 2 ** 22
    gen = torch.Generator(device="cuda").manual_seed(2)

    def some():
        return torch.randn(n, dim, device="cuda", generator=gen).to(torch.bfloat16)

    x, res, dy, w = some(), some(), some(), torch.rand(dim, device="cuda") + 0.5
    far = [rows_apart(t, ld) for t in (x, res, dy)]
    print("[gpu] norm", n, dim, flush=True)
    y, h, rstd = gpu.rms_norm(x, w, 1e-6, residual=res)
    fy, fh, frstd = gpu.rms_norm(far[0], w, 1e-6, residual=far[1],
                                 y=rows_apart(y, ld, fill=7.0), h=rows_apart(y, ld, fill=7.0))
    assert torch.equal(fy, y) and torch.equal(fh, h) and torch.equal(frstd, rstd)
    codes, scales, _, _ = gpu.rms_norm_q8(x, w, 1e-6, residual=res)
    bytes_ = rows_apart(torch.zeros(n, dim, dtype=torch.uint8, device="cuda"), ld)
    _, fscales, _, _ = gpu.rms_norm_q8(far[0], w, 1e-6, residual=far[1], codes=bytes_, h=fh)
    assert torch.equal(bytes_, codes.view(torch.uint8)) and torch.equal(fscales, scales)
    dx, dw = gpu.rms_norm_grad(dy, h, w, rstd, dh=x)
    fdx, fdw = gpu.rms_norm_grad(far[2], fh, w, rstd, dh=far[0], dx=fy)
    assert torch.equal(fdx, dx) and torch.equal(fdw, dw)


@pytest.mark.parametrize("vocab", [1000, 70001])
def test_distillation_rows(gpu, vocab):
    import torch

    n, k, ld = 1100, 9, 2 ** 22
    gen = torch.Generator(device="cuda").manual_seed(3)
    z = torch.randn(n, vocab, device="cuda", generator=gen).to(torch.bfloat16)
    idx = torch.randint(0, vocab, (n, k), device="cuda", generator=gen, dtype=torch.int32)
    top = torch.randn(n, k, device="cuda", generator=gen)
    far, fidx, ftop = rows_apart(z, ld), rows_apart(idx, ld), rows_apart(top, ld)
    print("[gpu] distill", n, vocab, flush=True)
    loss, lse = gpu.distill_loss(z, idx, top, 2.0)
    floss, flse = gpu.distill_loss(far, fidx, ftop, 2.0)
    assert torch.equal(floss, loss) and torch.equal(flse, lse)
    out = rows_apart(z, ld, fill=7.0)
    gpu.distill_grad(far, lse, fidx, ftop, 2.0, out=out)
    assert torch.equal(out, gpu.distill_grad(z, lse, idx, top, 2.0))
    want = gpu.distill_loss_grad(z, idx, top, 2.0)
    got = gpu.distill_loss_grad(far, fidx, ftop, 2.0, out=far)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
