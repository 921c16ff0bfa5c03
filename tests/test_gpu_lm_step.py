"""The language-model operators together, as a training step of a small student
uses them, up to the compressed gradient: lookup, a residual block with its
norm (plain, and through 8 bits), the tied head, distillation, every gradient
back, and the embedding's gradient into the 2-bit quantizer and the row-sparse
exchange of several workers.

Compared with the same step in 64 bits by torch's own differentiation.  The
step chains five products of at most 512 terms: each is off by at most 512 *
2^-24 of its terms' magnitudes, which are at most sqrt(512) times the result's
norm for the random data here, so gradients agree within 5 * 512 * 2^-24 *
sqrt(512) < 4e-3 of their norm."""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

N, V, D, K, T, EPS = 200, 300, 64, 12, 2.0, 1e-5
SCALE = D ** 0.5


def batch(seed):
    import torch

    rs = np.random.default_rng(seed)
    tok = np.minimum((V ** rs.random(N)).astype(np.int64) - 1, V - 1)
    tok[rs.random(N) < 0.05] = -1
    idx = np.stack([rs.permutation(V)[:K] for _ in range(N)])
    idx[rs.random((N, K)) < 0.05] = -1
    top = 3.0 - np.cumsum(rs.random((N, K)) * 0.3, 1)
    keep = (tok >= 0).astype(np.float32)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    return dev(tok), dev(idx), dev(top.astype(np.float32)), dev(keep / keep.sum())


def weights():
    import torch

    rs = np.random.default_rng(9)
    return [torch.from_numpy(a.astype(np.float32)).cuda() for a in
            (rs.standard_normal((V, D)) * 0.1, rs.standard_normal((D, D)) / SCALE,
             1.0 + 0.1 * rs.standard_normal(D))]


def step(gpu, E, W, w, data, q8):
    """(loss, gradients of E (tied), W and w, gradient of x, the normed y)."""
    import torch

    tok, idx, top, rs = data
    x = gpu.embed_lookup(E, tok, SCALE)
    a = x @ W
    if q8:
        codes, scales, h, rstd = gpu.rms_norm_q8(a, w, EPS, group=32, residual=x)
        y = codes.float() * scales.repeat_interleave(32, 1)
    else:
        y, h, rstd = gpu.rms_norm(a, w, EPS, residual=x)
    z = y @ E.T.contiguous()
    loss, _, dz = gpu.distill_loss_grad(z, idx, top, T, rs, T * T, out=z)
    dE = dz.T.contiguous() @ y
    dh, dw = gpu.rms_norm_grad(dz @ E, h, w, rstd)
    dx = dh + dh @ W.T.contiguous()
    plan = gpu.embed_sort(tok, V)
    gpu.embed_grad(dx, plan, SCALE, out=dE, accumulate=True)
    return loss.sum(), dE, x.T.contiguous() @ dh, dw, dx, y


def reference(E, W, w, data, q8, y_used):
    """The same in 64 bits; with q8 the 8-bit values stand for y and its
    gradient passes straight on."""
    import torch

    tok, idx, top, rs = data
    E, W, w = (t.double().requires_grad_() for t in (E, W, w))
    ok = tok >= 0
    x = torch.where(ok[:, None], SCALE * E[torch.where(ok, tok, 0)], 0.0)
    h = x @ W + x
    y = h * (h.square().mean(1, keepdim=True) + EPS).rsqrt() * w
    if q8:
        y = y + (y_used.double() - y).detach()
    z = y @ E.T / T
    real = idx >= 0
    p = torch.softmax((top.double() / T).masked_fill(~real, -np.inf), 1)
    logq = torch.log_softmax(z, 1).gather(1, torch.where(real, idx, 0))
    logp = torch.where(real, torch.log(p.clamp(min=1e-300)), 0.0)
    loss = (rs.double() * T * T * (p * (logp - logq)).sum(1)).sum()
    loss.backward()
    return loss.detach(), E.grad, W.grad, w.grad


def off(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("q8", [False, True])
def test_step(gpu, q8):
    E, W, w = weights()
    data = batch(1)
    got = step(gpu, E, W, w, data, q8)
    want = reference(E, W, w, data, q8, got[5])
    for name, a, b in zip(("loss", "E", "W", "w"), got, want):
        assert off(a, b) < 4e-3, name


def test_steps_gradient_into_the_quantizer(gpu):
    """Two workers' gradients through the 2-bit quantizer and the reduce, as a
    data-parallel step sends them: words and residuals as the oracle has them."""
    import torch

    E, W, w = weights()
    t = 0.01
    words = []
    for seed in (1, 2):
        dE = step(gpu, E, W, w, batch(seed), False)[1]
        g = dE.reshape(-1)
        r = torch.zeros_like(g)
        words.append(gpu.gc2_quantize(g, r, t))
        r_host = np.zeros(g.numel(), np.float32)
        want = oracle.gc2_quantize(g.cpu().numpy(), r_host, t)
        assert np.array_equal(words[-1].cpu().numpy().view(np.uint32), want)
        assert np.array_equal(r.cpu().numpy().view(np.uint32), r_host.view(np.uint32))
        assert (want != 0).any()
    total = gpu.gc2_dequant_reduce(words, V * D, t)
    host = oracle.gc2_dequant_reduce([x.cpu().numpy().view(np.uint32) for x in words], V * D, t)
    assert np.array_equal(total.cpu().numpy().view(np.uint32), host.view(np.uint32))


def test_steps_gradient_row_sparse(gpu):
    """An untied table: three workers send (ids, rows); merged, they are the
    gradient of the three batches together.  A sum of up to 600 rows in two
    orders: 600 * 2^-23 of its magnitudes."""
    import torch

    E, W, w = weights()
    ids, rows, toks, dxs = [], [], [], []
    for seed in (1, 2, 3):
        data = batch(seed)
        dx = step(gpu, E, W, w, data, False)[4]
        plan = gpu.embed_sort(data[0], V)
        i, r, c = gpu.embed_grad_rows(dx, plan, SCALE)
        u = int(c)
        assert u == torch.unique(data[0][data[0] >= 0]).numel()
        ids.append(i[:u])
        rows.append(r[:u])
        toks.append(data[0])
        dxs.append(dx)
    merged = gpu.embed_grad(torch.cat(rows), gpu.embed_sort(torch.cat(ids), V))
    whole = gpu.embed_grad(torch.cat(dxs), gpu.embed_sort(torch.cat(toks), V), SCALE)
    mag = gpu.embed_grad(torch.cat(dxs).abs(), gpu.embed_sort(torch.cat(toks), V), SCALE)
    assert ((merged - whole).abs() <= 600 * 2.0 ** -23 * mag).all()


def test_two_devices_are_refused(gpu):
    """Tensors of another device than the call's others are refused before
    anything is launched (checked with a host tensor where there is one GPU)."""
    import torch

    E, W, w = weights()
    with pytest.raises(ValueError):
        gpu.embed_lookup(E, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        gpu.rms_norm(E, w.cpu(), EPS)
    with pytest.raises(ValueError):
        gpu.distill_loss(E, torch.zeros(V, 2, dtype=torch.int64), torch.zeros(V, 2, device="cuda"))
    with pytest.raises(TypeError):
        gpu.rms_norm(E.double(), w, EPS)
    with pytest.raises(TypeError):
        gpu.embed_lookup(E, torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError):
        gpu.rms_norm(E, w[:5], EPS)
    with pytest.raises(ValueError):
        gpu.rms_norm_q8(E, w, EPS, group=48)
    with pytest.raises(ValueError):
        gpu.embed_lookup(E.T, torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        gpu.embed_lookup(E[:1].expand(5, D), torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(gpu.GcqError):   # out over the table
        gpu.embed_lookup(E, torch.zeros(3, dtype=torch.int64, device="cuda"), out=E[:3])
    plan = gpu.embed_sort(torch.zeros(3, dtype=torch.int64, device="cuda"), V)
    with pytest.raises(ValueError):     # a gradient of another batch than the plan's
        gpu.embed_grad(E[:4], plan)
    with pytest.raises(ValueError):
        gpu.embed_grad(E[:3], plan, accumulate=True)
