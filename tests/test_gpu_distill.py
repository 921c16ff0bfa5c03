"""Distillation from a teacher's top logits against a plain 64-bit
implementation.

Tolerances, e = 2^-24, E half a step of the gradient's type.  Every q_v is an
exponential of an argument x of magnitude up to X: the argument is off by at
most 4 e X + 4 e (a difference, the factor's rounding, a product), so q_v by
that much relative, plus 4 e for the exponential itself, plus the sum's error:
at most 64 + V / 1024 additions in a chain.  With X <= 64 here:
R(V) = (4 * 64 + 72 + V / 1024) e."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

TYPES = ["float32", "float16", "bfloat16"]
HALF = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
TINY = {"float32": 2.0 ** -150, "float16": 2.0 ** -25, "bfloat16": 2.0 ** -134}
E = 2.0 ** -24
SHAPES = [(1, 1, 1), (2, 5, 3), (3, 64, 4), (5, 1000, 7), (4, 1025, 64), (3, 4099, 100),
          (2, 32768, 257), (3, 33333, 1024), (2, 70001, 16), (600, 130, 5)]


def dtype(name):
    import torch

    return getattr(torch, name)


def rel(vocab):
    return (4 * 64 + 72 + vocab / 1024) * E


def case(seed, rows, vocab, k, kind, index="int64", absent=0.1, extra=0, sigma=2.5):
    import torch

    rs = np.random.default_rng(seed)
    z = torch.from_numpy((rs.standard_normal((rows, vocab + extra)) * sigma).astype(np.float32))
    z = z.to(dtype(kind)).cuda()[:, :vocab]
    idx = rs.integers(0, vocab, (rows, k))              # the same index twice, too
    gone = rs.random((rows, k)) < absent
    idx = np.where(gone, rs.choice([-1, vocab, -2 ** 31, 2 ** 31 - 1], (rows, k)), idx)
    top = -np.cumsum(rs.random((rows, k)) * 0.5, 1) + 6.0
    sc = rs.random(rows).astype(np.float32) + 0.5
    sc[rs.random(rows) < 0.2] = 0.0
    sc[0] = 0.75
    return (z, torch.from_numpy(idx).to(dtype(index)).cuda(),
            torch.from_numpy(top.astype(np.float32)).to(dtype(kind)).cuda(), torch.from_numpy(sc).cuda())


def plain(z, idx, top, T, rs, scale):
    """(loss, lse, dz, p, size of the loss' terms) in 64 bits."""
    import torch

    V = z.shape[1]
    zt = z.double() / T
    lse = torch.logsumexp(zt, 1)
    s = (rs.double() if rs is not None else torch.ones(z.shape[0], device="cuda").double()) * scale
    idx = idx.long()
    real = (idx >= 0) & (idx < V)
    t = torch.where(real, top.double() / T, -math.inf)
    some = (t > -math.inf).any(1) & (s != 0)
    p = torch.where(some[:, None] & real, torch.softmax(t, 1), 0.0)
    at = torch.where(real, idx, 0)
    logp = torch.where(p > 0, torch.log(p.clamp(min=1e-300)), 0.0)
    logq = torch.where(p > 0, zt.gather(1, at) - lse[:, None], 0.0)
    loss = s * (p * (logp - logq)).sum(1)
    size = s.abs() * (p * (logp.abs() + logq.abs() + lse.abs()[:, None] + 1)).sum(1)
    P = torch.zeros_like(zt).scatter_add_(1, at, p)
    q = torch.softmax(zt, 1)
    f = torch.where(some, s / T, 0.0)[:, None]
    return (torch.where(some, loss, 0.0), torch.where(s != 0, lse, 0.0), f * (q - P),
            f.abs() * (q + P), size)


def check(got, want, V, kind):
    loss, lse, dz = got
    l0, e0, d0, size, lsize = want
    r = rel(V)
    if loss is not None:
        assert ((loss.double() - l0).abs() <= r * lsize).all(), ((loss.double() - l0).abs().max())
        assert ((lse.double() - e0).abs() <= r * (1 + e0.abs())).all()
    if dz is not None:
        off = (dz.double() - d0).abs()
        assert (off <= HALF[kind] * d0.abs() + r * size + TINY[kind]).all(), off.max()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("index", ["int32", "int64"])
@pytest.mark.parametrize("T", [1.0, 2.0, 0.7])
def test_against_plain(gpu, kind, index, T):
    import torch

    for n, (rows, V, k) in enumerate(SHAPES):
        print("[gpu] distill", kind, index, T, rows, V, k, flush=True)
        z, idx, top, rs = case(n, rows, V, k, kind, index, extra=n % 3)
        scale = T * T / rows
        row_scale = rs if n % 2 else None
        want = plain(z, idx, top, T, row_scale, scale)
        want = (*want[:3], want[3], want[4])
        wide = torch.full((rows, V + 3), 7.0, dtype=dtype(kind), device="cuda")
        loss, lse = gpu.distill_loss(z, idx, top, T, row_scale, scale)
        check((loss, lse, None), want, V, kind)
        dz = gpu.distill_grad(z, lse, idx, top, T, row_scale, scale, out=wide[:, :V])
        check((None, None, dz), want, V, kind)
        assert (wide[:, V:] == 7.0).all()
        both = gpu.distill_loss_grad(z, idx, top.float() if n % 2 else top, T, row_scale, scale)
        check(both, want, V, kind)
        z2 = z.clone()
        assert torch.equal(gpu.distill_loss_grad(z2, idx, top, T, row_scale, scale, out=z2)[2], both[2])
        z2 = z.clone()
        assert torch.equal(gpu.distill_grad(z2, lse, idx, top, T, row_scale, scale, out=z2), dz)


@pytest.mark.parametrize("kind", TYPES)
def test_many_rows(gpu, kind):
    """Logits past the size from which they are read non-temporally."""
    import torch

    rows, V = (420, 70001) if kind == "float32" else (800, 70001)
    z, idx, top, rs = case(11, rows, V, 33, kind, extra=2)
    want = plain(z, idx, top, 1.5, rs, 3.0)
    loss, lse = gpu.distill_loss(z, idx, top, 1.5, rs, 3.0)
    check((loss, lse, None), want, V, kind)
    check((None, None, gpu.distill_grad(z, lse, idx, top, 1.5, rs, 3.0)), want, V, kind)
    check(gpu.distill_loss_grad(z, idx, top, 1.5, rs, 3.0), want, V, kind)


@pytest.mark.parametrize("kind", TYPES)
def test_row_lengths(gpu, kind):
    """Rows around the lengths at which more or less of a row is kept between
    the two passes, and other numbers of entries beside it."""
    import torch

    size = torch.finfo(dtype(kind)).bits // 8
    for nbytes, k in ((8192, 1), (8192, 1024), (16384, 40), (18432, 1024), (32768, 5), (40000, 300),
                      (65536, 1024), (73728, 8), (98304, 64), (114688, 1024), (131072, 1),
                      (204800, 40), (212992, 1024)):
        for V in (nbytes // size - 1, nbytes // size, nbytes // size + 1):
            print("[gpu] distill", kind, V, k, flush=True)
            z, idx, top, rs = case(V, 3, V, k, kind, extra=V % 3)
            want = plain(z, idx, top, 1.5, rs, 2.0)
            wide = torch.full((3, V + 3), 7.0, dtype=dtype(kind), device="cuda")
            got = gpu.distill_loss_grad(z, idx, top, 1.5, rs, 2.0, out=wide[:, :V])
            check(got, want, V, kind)
            assert (wide[:, V:] == 7.0).all()
            assert torch.equal(gpu.distill_loss_grad(z, idx, top, 1.5, rs, 2.0, out=z)[2], got[2])


def test_rows_with_nothing(gpu):
    """No entry, entries of -inf alone, masked rows, logits of -inf or of the
    type's lowest value, and rows that hold NaN but are not read."""
    import torch

    V, k, inf = 300, 4, math.inf
    z = torch.randn(8, V, device="cuda")
    idx = torch.arange(k, device="cuda").repeat(8, 1) * 7
    top = torch.zeros(8, k, device="cuda")
    s = torch.ones(8, device="cuda")
    idx[0] = -1                                   # no entry
    top[1] = -inf                                 # entries without weight
    s[2], z[2], top[2] = 0.0, math.nan, math.nan  # masked: not read
    z[3] = -inf                                   # no logit
    z[4, 10:] = -inf                              # a masked vocabulary; 14 and 21 are out of it
    z[5, 100:] = torch.finfo(torch.float32).min
    z[6, 7] = -inf                                # an entry where the student has nothing ...
    top[6, 1] = -inf                              # ... and the teacher neither
    z[7, 299] = math.nan
    loss, lse = gpu.distill_loss(z, idx, top, 2.0, s)
    dz = gpu.distill_grad(z, lse, idx, top, 2.0, s)
    l2, e2, d2 = gpu.distill_loss_grad(z, idx, top, 2.0, s)
    for l, e, d in ((loss, lse, dz), (l2, e2, d2)):
        assert (l[:3] == 0).all() and (d[:3] == 0).all() and e[2] == 0
        assert l[3] == inf and e[3] == -inf and (d[3] == 0).all()
        assert l[4] == inf and (d[4, 30:] == 0).all() and torch.isfinite(d[4]).all()
        assert torch.isfinite(l[5]) and (d[5, 100:] == 0).all()
        assert torch.isfinite(l[6]) and d[6, 7] == 0
        assert torch.isnan(l[7]) and torch.isnan(d[7]).all()
    want = plain(z[5:7], idx[5:7], top[5:7], 2.0, s[5:7], 1.0)
    want[2][1, 7] = 0.0
    assert ((loss[5].double() - want[0][0]).abs() <= rel(V) * want[4][0])
    assert ((dz[5].double() - want[2][0]).abs() <= rel(V) * want[3][0] + TINY["float32"]).all()


def test_large_logits(gpu):
    """Logits far from zero: only differences count."""
    import torch

    z, idx, top, _ = case(3, 4, 5000, 8, "float32")
    l0, e0, d0 = gpu.distill_loss_grad(z, idx, top, 1.0)
    up = (z * 1024).round() / 1024                  # so that adding 4096 is exact
    l1, e1, d1 = gpu.distill_loss_grad(up, idx, top, 1.0)
    l2, e2, d2 = gpu.distill_loss_grad(up + 4096, idx, top, 1.0)
    assert torch.equal(d1, d2) and torch.equal(l1, l2)
    d3 = gpu.distill_grad(up + 4096, e2, idx, top, 1.0)
    # lse itself is rounded, by half of a step of 2^-11 at 4096: q moves by that much
    size = plain(up, idx, top, 1.0, None, 1.0)[3]
    assert ((d3 - d2).abs() <= (2.0 ** -12 + 2 * rel(5000)) * size).all()


def test_gradient_by_differences(gpu):
    import torch

    z, idx, top, rs = case(5, 3, 200, 6, "float32", absent=0.2)
    dz = gpu.distill_loss_grad(z, idx, top, 1.5, rs, 2.25)[2]
    v = torch.randn(z.shape, generator=torch.Generator().manual_seed(1)).cuda()
    h = 1e-4
    up = plain(z.double() + h * v.double(), idx, top, 1.5, rs, 2.25)[0].sum()
    down = plain(z.double() - h * v.double(), idx, top, 1.5, rs, 2.25)[0].sum()
    # h^2 times a third derivative of order 10, 64-bit noise 1e-12; 600 float32 terms
    assert abs(float((up - down) / (2 * h)) - float((dz.double() * v.double()).sum())) <= 1e-6 + 600 * 8 * E


def test_strided_and_empty(gpu):
    import torch

    z, idx, top, rs = case(7, 6, 777, 9, "float16", "int32")
    want = gpu.distill_loss_grad(z, idx, top, 1.0, rs)
    pad = torch.zeros(6, 20, dtype=torch.int32, device="cuda")
    pad[:, 3:12] = idx
    tpad = torch.zeros(6, 30, dtype=torch.float16, device="cuda")
    tpad[:, 5:14] = top
    got = gpu.distill_loss_grad(z, pad[:, 3:12], tpad[:, 5:14], 1.0, rs)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    e = gpu.distill_loss_grad(z[:0], idx[:0], top[:0])
    assert e[0].numel() == 0 and e[2].shape == (0, 777)


def test_graphs_and_streams(gpu):
    import torch

    cases = [case(20 + i, 70, 3001, 12, "bfloat16") for i in range(3)]

    def step(z, idx, top, rs):
        loss, lse = gpu.distill_loss(z, idx, top, 2.0, rs)
        return loss, lse, gpu.distill_grad(z, lse, idx, top, 2.0, rs), \
            *gpu.distill_loss_grad(z, idx, top, 2.0, rs)

    want = [step(*c) for c in cases]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(*cases[1])
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))
    graphs = []
    for _ in range(2):
        held = tuple(t.clone() for t in cases[0])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step(*held)
        graphs.append((graph, held, got))
    for i in (2, 1, 0, 2):
        for graph, held, got in graphs:
            for a, b in zip(held, cases[i]):
                a.copy_(b)
            graph.replay()
            step(*cases[(i + 1) % 3])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
