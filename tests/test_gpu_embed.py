"""Embedding lookup and its gradient against plain 64-bit implementations.

The lookup is one product rounded once, so it is compared exactly with the
float32 product rounded to the output's type.  A gradient's element is a sum
of c terms in float32: any order of c - 1 additions is off by at most
(c - 1) * 2^-24 * (sum of the terms' magnitudes) to first order, and the final
scale adds half a step; the tolerance takes c + 2 half steps."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

TYPES = ["float32", "float16", "bfloat16"]


def dtype(name):
    import torch

    return getattr(torch, name)


def tokens_of(rs, n, vocab, kind):
    if kind == "one":                 # every position the same token
        return np.full(n, vocab // 2, np.int64)
    if kind == "padding":             # nothing but padding
        return np.where(np.arange(n) % 2 == 0, -1, vocab).astype(np.int64)
    if kind == "distinct":
        return rs.permutation(max(n, vocab))[:n].astype(np.int64) % vocab
    t = np.minimum((vocab ** rs.random(n)).astype(np.int64) - 1, vocab - 1)   # frequent ones first
    t[rs.random(n) < 0.05] = -1
    t[rs.random(n) < 0.02] = vocab
    t[rs.random(n) < 0.01] = -2 ** 31
    return t


def grads(rs, n, dim, dt, extra=0):
    import torch

    g = torch.from_numpy(rs.standard_normal((n, dim + extra)).astype(np.float32)).to(dt).cuda()
    return g[:, :dim] if extra else g


def want_grad(g, tok, vocab, scale):
    """(gradient, magnitude of its terms, count) in 64 bits on the host."""
    a = g.double().cpu().numpy()
    d, m, c = np.zeros((vocab, a.shape[1])), np.zeros((vocab, a.shape[1])), np.zeros(vocab, int)
    ok = (tok >= 0) & (tok < vocab)
    np.add.at(d, tok[ok], a[ok])
    np.add.at(m, tok[ok], np.abs(a[ok]))
    np.add.at(c, tok[ok], 1)
    s = float(np.float32(scale))
    return d * s, m * abs(s), c


def close(got, want, mag, count):
    tol = (count[:, None] + 2) * 2.0 ** -24 * mag
    bad = np.abs(got - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("table_type", TYPES)
@pytest.mark.parametrize("out_type", TYPES)
@pytest.mark.parametrize("index", ["int32", "int64"])
def test_lookup(gpu, table_type, out_type, index):
    import torch

    rs = np.random.default_rng(1)
    for n, vocab, dim, extra in [(1, 1, 1, 0), (7, 33, 8, 0), (64, 100, 100, 0), (33, 1000, 1025, 0),
                                 (5, 77, 4096, 3), (300, 50, 65, 1)]:
        print("[gpu] lookup", table_type, out_type, index, n, vocab, dim, flush=True)
        tok = tokens_of(rs, n, vocab, "text")
        table = grads(rs, vocab, dim, dtype(table_type), extra)
        t = torch.from_numpy(tok).clamp(-2 ** 31, 2 ** 31 - 1).to(dtype(index)).cuda()
        wide = torch.full((n, dim + extra), 7.0, dtype=dtype(out_type), device="cuda")
        out = gpu.embed_lookup(table, t, 3.7, out=wide[:, :dim])
        ok = torch.from_numpy((tok >= 0) & (tok < vocab)).cuda()
        rows = table.float()[torch.where(ok, t.long(), 0)] * 3.7
        want = torch.where(ok[:, None], rows, 0.0).to(dtype(out_type))
        assert torch.equal(out, want)
        assert (wide[:, dim:] == 7.0).all()


def test_lookup_keeps_special_values(gpu):
    import torch

    table = torch.tensor([[float("inf"), float("nan"), -0.0, 1e-41]], device="cuda")
    out = gpu.embed_lookup(table, torch.zeros(2, dtype=torch.int64, device="cuda"))
    assert out[1, 0] == float("inf") and torch.isnan(out[1, 1])
    assert torch.equal(out[1, 2:].view(torch.int32), table[0, 2:].view(torch.int32))
    assert gpu.embed_lookup(table, torch.zeros(0, dtype=torch.int64, device="cuda")).shape == (0, 4)


@pytest.mark.parametrize("n,vocab", [(1, 1), (2, 2 ** 31 - 1), (65, 3), (4096, 600), (4097, 600),
                                     (8193, 50000), (16384, 131072), (16385, 131072),
                                     (5000, 40), (20000, 131073), (70001, 2 ** 20 + 1),
                                     (9000, 2 ** 31 - 1), (300000, 70000)])
@pytest.mark.parametrize("index", ["int32", "int64"])
def test_sort_is_stable(gpu, n, vocab, index):
    import torch

    print("[gpu] sort", n, vocab, index, flush=True)
    tok = tokens_of(np.random.default_rng(n), n, vocab, "text").clip(-2 ** 31, 2 ** 31 - 1)
    t = torch.from_numpy(tok).to(dtype(index)).cuda()
    plan = gpu.embed_sort(t, vocab)
    key = np.where((tok >= 0) & (tok < vocab), tok, vocab)
    order = np.argsort(key, kind="stable")
    w = plan.words.cpu().numpy()
    assert np.array_equal(w[:n], key[order])
    assert np.array_equal(w[n:2 * n], order)


@pytest.mark.parametrize("kind", ["text", "one", "padding", "distinct"])
@pytest.mark.parametrize("grad_type", TYPES)
def test_gradient(gpu, kind, grad_type):
    import torch

    rs = np.random.default_rng(2)
    for n, vocab, dim, extra in [(1, 5, 3, 0), (31, 40, 64, 0), (32, 40, 1, 0), (33, 9, 8, 5),
                                 (1000, 200, 129, 0), (5003, 300, 40, 0), (257, 31, 2049, 1)]:
        print("[gpu] gradient", kind, grad_type, n, vocab, dim, flush=True)
        tok = tokens_of(rs, n, vocab, kind)
        g = grads(rs, n, dim, dtype(grad_type), extra)
        bad = torch.from_numpy((tok < 0) | (tok >= vocab)).cuda()
        g[bad] = float("nan")                      # padding is not read
        plan = gpu.embed_sort(torch.from_numpy(tok).cuda(), vocab)
        want, mag, count = want_grad(torch.where(bad[:, None], 0.0, g), tok, vocab, -2.5)

        wide = torch.full((vocab, dim + extra), 7.0, device="cuda")
        out = gpu.embed_grad(g, plan, -2.5, out=wide[:, :dim])
        close(out.double().cpu().numpy(), want, mag, count)
        assert (out[torch.from_numpy(count == 0).cuda()] == 0).all()
        assert (wide[:, dim:] == 7.0).all()

        base = torch.from_numpy(rs.standard_normal((vocab, dim)).astype(np.float32)).cuda()
        acc = gpu.embed_grad(g, plan, -2.5, out=base.clone(), accumulate=True)
        old = base.double().cpu().numpy()
        close(acc.double().cpu().numpy(), old + want, mag + np.abs(old), count)
        assert torch.equal(acc[torch.from_numpy(count == 0).cuda()],
                           base[torch.from_numpy(count == 0).cuda()])

        most = min(n, vocab)
        ids = torch.full((most + 2,), -9, dtype=torch.int32, device="cuda")
        rows = torch.full((most + 2, dim), 7.0, device="cuda")
        ids, rows, cnt = gpu.embed_grad_rows(g, plan, -2.5, ids=ids, rows=rows)
        u = int(cnt)
        named = np.flatnonzero(count)
        assert u == named.size and np.array_equal(ids[:u].cpu().numpy(), named)
        assert torch.equal(rows[:u], out[torch.from_numpy(named).cuda()])
        assert (ids[u:] == -9).all() and (rows[u:] == 7.0).all()


@pytest.mark.parametrize("n,vocab,dim", [(40000, 3000, 1024), (70001, 20000, 1030)])
def test_gradient_of_many(gpu, n, vocab, dim):
    """Long runs and segments of thousands of positions; the reference sums in
    64 bits on the GPU."""
    import torch

    rs = np.random.default_rng(7)
    tok = tokens_of(rs, n, vocab, "text")
    g = grads(rs, n, dim, torch.bfloat16)
    ok = torch.from_numpy((tok >= 0) & (tok < vocab)).cuda()
    at = torch.where(ok, torch.from_numpy(tok).cuda(), 0)
    gd = torch.where(ok[:, None], g.double(), 0.0)
    want = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda").index_add_(0, at, gd)
    mag = torch.zeros_like(want).index_add_(0, at, gd.abs())
    count = torch.zeros(vocab, dtype=torch.float64, device="cuda").index_add_(0, at, ok.double())
    plan = gpu.embed_sort(torch.from_numpy(tok).cuda(), vocab)
    out = gpu.embed_grad(g, plan)
    assert ((out.double() - want).abs() <= (count[:, None] + 2) * 2.0 ** -24 * mag).all()
    ids, rows, cnt = gpu.embed_grad_rows(g, plan)
    named = torch.nonzero(count)[:, 0]
    assert int(cnt) == named.numel() and torch.equal(ids[:int(cnt)].long(), named)
    assert torch.equal(rows[:int(cnt)], out[named])
    base = torch.ones(vocab, dim, device="cuda")
    acc = gpu.embed_grad(g, plan, out=base.clone(), accumulate=True)
    assert torch.equal(acc, out + 1.0)


def test_gradient_of_nothing(gpu):
    import torch

    plan = gpu.embed_sort(torch.zeros(0, dtype=torch.int32, device="cuda"), 5)
    g = torch.zeros(0, 3, device="cuda")
    assert torch.equal(gpu.embed_grad(g, plan), torch.zeros(5, 3, device="cuda"))
    ids, rows, count = gpu.embed_grad_rows(g, plan)
    assert int(count) == 0 and ids.numel() == 0
    one = torch.ones(5, 3, device="cuda")
    assert torch.equal(gpu.embed_grad(g, plan, out=one.clone(), accumulate=True), one)


def test_gradient_is_the_lookups(gpu):
    """<out, g> differs by <d, step> when the table moves by step: the lookup
    is linear, so the difference is exact up to rounding."""
    import torch

    rs = np.random.default_rng(3)
    tok = torch.from_numpy(tokens_of(rs, 400, 50, "text")).cuda()
    table, step, g = (torch.from_numpy(rs.standard_normal(s).astype(np.float32)).cuda()
                      for s in ((50, 24), (50, 24), (400, 24)))
    d = gpu.embed_grad(g, gpu.embed_sort(tok, 50), 1.5)
    a = (gpu.embed_lookup(table, tok, 1.5).double() * g.double()).sum()
    b = (gpu.embed_lookup(table + step, tok, 1.5).double() * g.double()).sum()
    terms = 400 * 24   # each off by a few half steps of values below about 20
    assert abs(float(b - a) - float((d.double() * step.double()).sum())) < terms * 2.0 ** -24 * 60


def test_repeats_bit_for_bit_and_in_graphs(gpu):
    """The same bits every time, eagerly and replayed from two captured graphs
    with workspaces of their own, with eager work between the replays."""
    import torch

    rs = np.random.default_rng(4)
    n, vocab, dim = 6000, 500, 96
    batches = [(torch.from_numpy(tokens_of(rs, n, vocab, "text")).cuda(), grads(rs, n, dim, torch.bfloat16))
               for _ in range(3)]

    def step(tok, g):
        plan = gpu.embed_sort(tok, vocab)
        return gpu.embed_grad(g, plan, 2.0), gpu.embed_grad_rows(g, plan, 2.0,
                                                                 ids=torch.zeros(vocab, dtype=torch.int32, device="cuda"),
                                                                 rows=torch.zeros(vocab, dim, device="cuda"))

    want = [step(*b) for b in batches]
    again = step(*batches[0])
    assert torch.equal(again[0], want[0][0]) and torch.equal(again[1][1], want[0][1][1])
    graphs = []
    for _ in range(2):
        tok, g = batches[0][0].clone(), batches[0][1].clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(tok, g)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step(tok, g)
        graphs.append((graph, tok, g, got))
    for i in (1, 2, 0, 1):
        for graph, tok, g, got in graphs:
            tok.copy_(batches[i][0])
            g.copy_(batches[i][1])
            graph.replay()
            step(*batches[(i + 1) % 3])
            torch.cuda.synchronize()
            assert torch.equal(got[0], want[i][0])
            assert all(torch.equal(a, b) for a, b in zip(got[1], want[i][1]))


def test_on_another_stream(gpu):
    import torch

    rs = np.random.default_rng(5)
    tok = torch.from_numpy(tokens_of(rs, 5000, 300, "text")).cuda()
    g = grads(rs, 5000, 64, torch.float32)
    want = gpu.embed_grad(g, gpu.embed_sort(tok, 300))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = gpu.embed_grad(g, gpu.embed_sort(tok, 300))
    side.synchronize()
    assert torch.equal(got, want)


def test_workers_messages_merge_in_order(gpu):
    """Row-sparse messages of three workers, concatenated, merged by the same
    calls: the sum over workers in worker order."""
    import torch

    rs = np.random.default_rng(6)
    vocab, dim, n = 90, 33, 200
    total = torch.zeros(vocab, dim, device="cuda")
    mag = torch.zeros(vocab, dim, device="cuda")
    ids, rows = [], []
    for _ in range(3):
        tok = torch.from_numpy(tokens_of(rs, n, vocab, "text")).cuda()
        g = grads(rs, n, dim, torch.float32)
        plan = gpu.embed_sort(tok, vocab)
        i, r, c = gpu.embed_grad_rows(g, plan, ids=torch.full((vocab,), -1, dtype=torch.int32, device="cuda"))
        ids.append(i)
        rows.append(r)
        d = gpu.embed_grad(g, plan)
        total += d
        mag += d.abs()
    # a token has at most three rows: the plain sum in worker order, except
    # where the end of a run of sorted positions splits them.  Each side rounds
    # at most twice, by half a step of at most the magnitudes' sum.
    merged = gpu.embed_grad(torch.cat(rows), gpu.embed_sort(torch.cat(ids), vocab))
    assert ((merged - total).abs() <= 4 * 2.0 ** -24 * mag).all()
    assert (merged == total).float().mean() > 0.5
