"""The RMS norm, its 8-bit output and its gradient against plain 64-bit
implementations.

Tolerances, with e = 2^-24 (half a float32 step, relative) and E half a step
of the output's type.  A row's mean of squares of D terms, each rounded once
and summed with no cancellation, is off by at most (D / lanes + 12) e
relative, D / lanes <= 64 for registers and (D / 1024) above; its inverse
root by half of that plus 4 e.  K(D) = 64 + D / 1024 e covers them.  y adds three
roundings and its own."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

TYPES = ["float32", "float16", "bfloat16"]
HALF = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
E = 2.0 ** -24
EPS = 1e-5

SHAPES = [(1, 1), (3, 7), (5, 64), (4, 100), (2, 511), (7, 513), (3, 1025), (1, 2048), (2, 4100),
          (1030, 40), (1025, 1030), (2, 8192), (3, 8197), (2, 16384), (2, 16389), (2, 33001),
          (3, 2500), (1030, 200), (1100, 65)]


def dtype(name):
    import torch

    return getattr(torch, name)


def few(dim):
    return (64 + dim / 1024) * E


def make(rs, rows, dim, kind, sigma=1.0, extra=0):
    import torch

    a = torch.from_numpy((rs.standard_normal((rows, dim + extra)) * sigma).astype(np.float32))
    a = a.to(dtype(kind)).cuda()
    return a[:, :dim] if extra else a


def near(got, want, rel, what, least=0.0):
    """|got - want| <= rel * |want| + least, elementwise."""
    got, want = got.double(), want.double()
    bad = (got - want).abs() > rel * want.abs() + least
    assert not bad.any(), (what, bad.sum().item(), got[bad][:4], want[bad][:4])


def tiny(kind):
    """Half the step of a type's subnormal values."""
    return {"float32": 2.0 ** -150, "float16": 2.0 ** -25, "bfloat16": 2.0 ** -134}[kind]


def plain(x, w, eps, res=None):
    h = x.double() + (res.double() if res is not None else 0.0)
    rstd = (h.square().mean(1) + eps).rsqrt()
    return h, rstd, h * rstd[:, None] * w.double()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("w32", [False, True])
@pytest.mark.parametrize("with_res", [False, True])
def test_norm(gpu, kind, w32, with_res):
    import torch

    rs = np.random.default_rng(1)
    for rows, dim in SHAPES:
        print("[gpu] norm", kind, w32, with_res, rows, dim, flush=True)
        extra = 3 if rows % 2 else 0
        x = make(rs, rows, dim, kind, 2.0, extra)
        res = make(rs, rows, dim, kind, 5.0, extra) if with_res else None
        w = make(rs, 1, dim, "float32" if w32 else kind)[0]
        wide = torch.full((rows, dim + 2), 7.0, dtype=dtype(kind), device="cuda")
        y, h, rstd = gpu.rms_norm(x, w, EPS, residual=res, y=wide[:, :dim])
        hd, rd, yd = plain(x, w, EPS, res)
        near(rstd, rd, few(dim), "rstd")
        if with_res:
            near(h, hd, HALF[kind] + E, "h", tiny(kind))
        else:
            assert h is x
        # in float32 h itself is rounded: off by e of its value, as y then is
        near(y, yd, HALF[kind] + few(dim) + 4 * E, "y", tiny(kind))
        assert (wide[:, dim:] == 7.0).all()
        if with_res:   # the residual updated in place gives the same
            r2 = res.clone()
            y2, h2, rstd2 = gpu.rms_norm(x, w, EPS, residual=r2, h=r2)
            assert torch.equal(y2, y) and torch.equal(h2, h) and torch.equal(rstd2, rstd)


def e4m3_values():
    """Every finite e4m3 value by code: sign, 4 exponent bits (bias 7), 3
    fraction bits; 0x7f and 0xff are NaN."""
    out = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        out[c] = math.nan if c & 127 == 127 else (-v if c & 128 else v)
    return out


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("group", [0, 32, 64, 128])
def test_norm_q8(gpu, kind, group):
    import torch

    rs = np.random.default_rng(2)
    table = torch.from_numpy(e4m3_values()).cuda()
    for rows, dim in SHAPES:
        for with_res in (False, True):
            print("[gpu] q8", kind, group, rows, dim, with_res, flush=True)
            x = make(rs, rows, dim, kind, 2.0, rows % 3)
            x[rows // 2, dim // 3:] = 0.0                  # groups of zeros
            res = make(rs, rows, dim, kind) * (x != 0) if with_res else None
            w = make(rs, 1, dim, kind)[0]
            wide = torch.full((rows, dim + 5), 9, dtype=torch.uint8, device="cuda")
            codes, scales, h, rstd = gpu.rms_norm_q8(x, w, EPS, group=group, residual=res,
                                                     codes=wide[:, :dim])
            hd, rd, yd = plain(x, w, EPS, res)
            near(rstd, rd, few(dim), "rstd")
            g = group or dim
            at = torch.arange(dim, device="cuda") // g
            top = torch.zeros(rows, -(-dim // g), dtype=torch.float64, device="cuda")
            top.scatter_reduce_(1, at.expand(rows, dim), yd.abs(), "amax")
            rel = few(dim) + 6 * E
            near(scales, top / 448.0, rel, "scales")
            v = table[codes.long()]
            assert not torch.isnan(v).any()
            # the code is a nearest e4m3 value of y / scale, up to the error of
            # that quotient: within half a step of it, the step being 2^-3 of
            # the value's power of two and 2^-9 at least
            s = scales.double()[:, at]
            q = torch.where(s > 0, yd / s.clamp(min=1e-300), 0.0)
            _, ex = torch.frexp(q)
            step = torch.exp2((ex - 1).clamp(min=-6).double() - 3.0)
            off = (v - q).abs()
            assert (off <= step / 2 + 2 * rel * q.abs()).all(), (off - step / 2).max()
            assert (wide[:, dim:] == 9).all()
            c8, s8, _, _ = gpu.rms_norm_q8(x, w, EPS, group=group, residual=res)
            assert torch.equal(c8.view(torch.uint8), codes) and torch.equal(s8.view(-1), scales.view(-1))


def test_q8_every_code(gpu):
    """A row whose normed values are e4m3 values times a power of two (their
    largest 448): every code comes back exactly, ties go to even."""
    import torch

    vals = e4m3_values()
    vals = vals[np.isfinite(vals)]
    ties = np.array([17.0, 19.0, -17.0, 2.0 ** -10, 3 * 2.0 ** -10, 1.0625])   # between neighbours
    even = np.array([16.0, 20.0, -16.0, 0.0, 2.0 ** -8, 1.0])
    x = np.concatenate([vals, ties])
    x = np.concatenate([x, np.full(512 - x.size, 448.0)])
    # eps makes the row's mean a power of four: rstd is then a power of two
    ms = float(np.mean(x * x))
    up = 4.0 ** math.ceil(math.log(ms, 4))
    xt = torch.from_numpy(x.astype(np.float32)).cuda()[None]
    codes, scales, _, rstd = gpu.rms_norm_q8(xt, torch.ones(512, device="cuda"), up - ms, group=0)
    got = codes.double().cpu().numpy()[0]
    want = np.concatenate([vals, even, np.full(512 - vals.size - ties.size, 448.0)])
    if float(rstd) == up ** -0.5:      # the mean's rounding may miss the power
        assert np.array_equal(got, want)
    else:
        off = np.abs(got - x)
        assert (off <= np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -10) * 1.0001).all()


def test_q8_edges(gpu):
    """Zero rows, tiny rows, infinities and NaN."""
    import torch

    x = torch.zeros(4, 256, device="cuda")
    x[1] = 1e-38
    x[2, 3] = float("nan")
    x[3, 200] = float("inf")
    w = torch.ones(256, device="cuda")
    codes, scales, _, rstd = gpu.rms_norm_q8(x, w, 1.0, group=128)
    f = codes.float()
    assert (f[0] == 0).all() and (scales[0] == 0).all() and rstd[0] == 1.0
    # 1e-38 / 448 is below the least normal number: the scale stops there
    assert (scales[1] == 2.0 ** -126).all()
    assert (f[1].double() * scales[1, 0].double() - 1e-38).abs().max() <= 2.0 ** -4 * 1e-38
    assert torch.isnan(f[2]).all()
    assert torch.isnan(f[3, 200]) and (f[3, :128] == 0).all()
    w[5] = float("nan")                                   # one column
    f, s, _, _ = gpu.rms_norm_q8(torch.ones(1, 256, device="cuda"), w, 0.0, group=128)
    assert torch.isnan(f.float()[0, 5]) and int(torch.isnan(f.float()).sum()) == 1
    assert (f.float()[0, 6:] == 448.0).all()


def plain_grad(dy, h, w, rstd, dh):
    dy, h, w, r = dy.double(), h.double(), w.double(), rstd.double()[:, None]
    u = dy * w
    c = (u * h).mean(1, keepdim=True)
    dx = r * (u - h * r * r * c) + (dh.double() if dh is not None else 0.0)
    size = r * (u.abs() + (h * r * r).abs() * (u * h).abs().mean(1, keepdim=True))
    if dh is not None:
        size = size + dh.double().abs()
    return dx, size, (dy * h * r).sum(0), (dy * h * r).abs().sum(0)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("w32", [False, True])
@pytest.mark.parametrize("with_dh", [False, True])
def test_norm_grad(gpu, kind, w32, with_dh):
    import torch

    rs = np.random.default_rng(3)
    for rows, dim in SHAPES + [(2100, 33), (3000, 600)]:
        print("[gpu] grad", kind, w32, with_dh, rows, dim, flush=True)
        extra = rows % 2
        dy, h = make(rs, rows, dim, kind, 0.5, extra), make(rs, rows, dim, kind, 2.0)
        dh = make(rs, rows, dim, kind, 0.3, extra) if with_dh else None
        w = make(rs, 1, dim, "float32" if w32 else kind)[0]
        rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
        dxd, size, dwd, dwsize = plain_grad(dy, h, w, rstd, dh)
        wide = torch.full((rows, dim + 3), 7.0, dtype=dtype(kind), device="cuda")
        dx, dw = gpu.rms_norm_grad(dy, h, w, rstd, dh=dh, dx=wide[:, :dim])
        # every term of dx goes through the mean's sum (few) and six roundings
        off = (dx.double() - dxd).abs()
        assert (off <= HALF[kind] * dxd.abs() + (few(dim) + 8 * E) * size + tiny(kind)).all()
        # a column's sum: at most rows + 16 additions in a chain, two roundings a term
        assert ((dw.double() - dwd).abs() <= (rows + 20) * E * dwsize + 1e-44).all()
        assert (wide[:, dim:] == 7.0).all()
        base = torch.from_numpy(rs.standard_normal(dim).astype(np.float32)).cuda()
        dx2, dw2 = gpu.rms_norm_grad(dy, h, w, rstd, dh=dh, dweight=base.clone(), accumulate=True)
        assert torch.equal(dx2, dx) and torch.equal(dw2, base + dw)
        if with_dh:
            d3 = dh.clone()
            dx3, _ = gpu.rms_norm_grad(dy, h, w, rstd, dh=d3, dx=d3)
            assert torch.equal(dx3, dx)


# rows that share a wavefront, three vectors a lane (64 and 256 lanes), two of 512 lanes to 8 bits, and
# matrices past the sizes from
# which accesses are non-temporal
MANY = [(1100, 9000), (1030, 200), (20001, 100), (5000, 65), (1030, 700), (1025, 1400), (1025, 2500), (1025, 5000), (9000, 4100)]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("rows,dim", MANY)
def test_many_rows(gpu, kind, rows, dim):
    import torch

    print("[gpu] many rows", kind, rows, dim, flush=True)
    g = torch.Generator(device="cuda").manual_seed(rows + dim)
    x, res, dy = (torch.randn(rows, dim, generator=g, device="cuda").to(dtype(kind)) for _ in range(3))
    w = torch.randn(dim, generator=g, device="cuda")
    hd, rd, yd = plain(x, w, EPS, res)
    y, h, rstd = gpu.rms_norm(x, w, EPS, residual=res)
    near(rstd, rd, few(dim), "rstd")
    near(h, hd, HALF[kind] + E, "h", tiny(kind))
    near(y, yd, HALF[kind] + few(dim) + 4 * E, "y", tiny(kind))
    codes, scales, h8, rstd8 = gpu.rms_norm_q8(x, w, EPS, group=128, residual=res)
    assert torch.equal(h8, h)
    near(rstd8, rd, few(dim), "rstd to 8 bits")
    v = codes.float().double() * scales.double()[:, torch.arange(dim, device="cuda") // 128]
    # half a step of three fraction bits, or of the smallest code
    least = 2.0 ** -10 * scales.double()[:, torch.arange(dim, device="cuda") // 128]
    assert ((v - yd).abs() <= (2.0 ** -4 + 3 * few(dim)) * yd.abs() + least).all()
    dxd, size, dwd, dwsize = plain_grad(dy, h, w, rstd, res)
    dx, dw = gpu.rms_norm_grad(dy, h, w, rstd, dh=res)
    off = (dx.double() - dxd).abs()
    assert (off <= HALF[kind] * dxd.abs() + (few(dim) + 8 * E) * size + tiny(kind)).all()
    assert ((dw.double() - dwd).abs() <= (rows + 40) * E * dwsize + 1e-44).all()


def test_grad_is_the_norms(gpu):
    """Differences of the 64-bit norm along random directions."""
    import torch

    rs = np.random.default_rng(4)
    rows, dim, t = 6, 96, 1e-5
    x, w, g, vx = (make(rs, *s, "float32") for s in ((rows, dim), (1, dim), (rows, dim), (rows, dim)))
    vw = make(rs, 1, dim, "float32")
    _, _, rstd = gpu.rms_norm(x, w[0], EPS)
    dx, dw = gpu.rms_norm_grad(g, x, w[0], rstd)

    def f(s):
        _, _, y = plain(x.double() + s * vx.double(), w[0].double() + s * vw[0].double(), EPS)
        return float((y * g.double()).sum())

    diff = (f(t) - f(-t)) / (2 * t)
    mine = float((dx.double() * vx.double()).sum() + (dw.double() * vw[0].double()).sum())
    # the difference: t^2 times a third derivative of order 10^3, and 64-bit
    # noise of 2^-52 * 600 / t; the gradients: 600 terms of a few e each
    assert abs(diff - mine) <= 1e-6 + 600 * 100 * E


def test_rows_without_work(gpu):
    import torch

    w = torch.ones(8, device="cuda")
    e = torch.zeros(0, 8, device="cuda")
    y, h, rstd = gpu.rms_norm(e, w, EPS)
    assert y.shape == (0, 8) and rstd.numel() == 0
    assert gpu.rms_norm_q8(e, w, EPS, group=32)[1].shape == (0, 1)
    dx, dw = gpu.rms_norm_grad(e, e, w, rstd, dweight=torch.ones(8, device="cuda"))
    assert (dw == 0).all()
    _, dw = gpu.rms_norm_grad(e, e, w, rstd, dweight=torch.ones(8, device="cuda"), accumulate=True)
    assert (dw == 1).all()


def test_graphs_and_streams(gpu):
    """Two captured graphs, replayed with eager work between: the same bits."""
    import torch

    rs = np.random.default_rng(5)
    ins = [tuple(make(rs, 300, 520, "bfloat16") for _ in range(3)) for _ in range(3)]
    w = make(rs, 1, 520, "float32")[0]

    def step(x, r, g):
        c, s, h, rstd = gpu.rms_norm_q8(x, w, EPS, group=64, residual=r)
        return c.view(torch.uint8), s, h, *gpu.rms_norm_grad(g, h, w, rstd, dh=r)

    want = [step(*i) for i in ins]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(*ins[1])
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))
    graphs = []
    for _ in range(2):
        held = tuple(t.clone() for t in ins[0])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step(*held)
        graphs.append((graph, held, got))
    for i in (2, 1, 0, 2):
        for graph, held, got in graphs:
            for a, b in zip(held, ins[i]):
                a.copy_(b)
            graph.replay()
            step(*ins[(i + 1) % 3])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
