"""The language-model operators beside torch's autograd: a tensor whose
gradient would be lost is refused, what a call writes has its version raised,
and the calls work as the two halves of a torch.autograd.Function."""
import pytest

import gradient_compression_distributed_amd as gcq


def test_lost_gradients_are_refused_on_the_host():
    """The first matrix's check comes before that of its device."""
    import torch

    x, w, i = torch.zeros(4, 4, requires_grad=True), torch.zeros(4), torch.zeros(4, dtype=torch.int64)
    t, k = torch.zeros(4, 2), torch.zeros(4, 2, dtype=torch.int64)
    plan = gcq.EmbedPlan(torch.zeros(16, dtype=torch.int32), 4, 4)
    calls = (lambda: gcq.embed_lookup(x, i), lambda: gcq.embed_grad(x, plan),
             lambda: gcq.embed_grad_rows(x, plan), lambda: gcq.rms_norm(x, w, 1e-6),
             lambda: gcq.rms_norm_q8(x, w, 1e-6), lambda: gcq.rms_norm_grad(x, x, w, w),
             lambda: gcq.distill_loss(x, k, t), lambda: gcq.distill_grad(x, w, k, t),
             lambda: gcq.distill_loss_grad(x, k, t))
    for call in calls:
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="GPU memory"):
            call()


def operands():
    """{call: (function of keyword tensors, the tensors, names of those written)}."""
    import torch

    def f(*shape):
        return torch.randn(*shape, device="cuda")

    n, v, d, k = 6, 10, 32, 3
    tok = torch.arange(n, device="cuda")
    plan = gcq.embed_sort(tok, v)
    idx = torch.arange(n * k, device="cuda").reshape(n, k) % v
    x, w, rstd, z, top = f(n, d), f(d), f(n).abs() + 0.5, f(n, v), f(n, k)
    work = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    return {
        "embed_lookup": (lambda **a: gcq.embed_lookup(tokens=tok, **a), dict(table=f(v, d), out=f(n, d)), {"out"}),
        "embed_grad": (lambda **a: gcq.embed_grad(plan=plan, work=work, **a), dict(grad=x, out=f(v, d)), {"out"}),
        "embed_grad_rows": (lambda **a: gcq.embed_grad_rows(
            plan=plan, ids=torch.zeros(n, dtype=torch.int32, device="cuda"), **a),
            dict(grad=x, rows=f(n, d)), {"rows"}),
        "rms_norm": (lambda **a: gcq.rms_norm(eps=1e-6, **a),
                     dict(x=x, weight=w, residual=f(n, d), y=f(n, d), h=f(n, d), rstd=f(n)), {"y", "h", "rstd"}),
        "rms_norm_q8": (lambda **a: gcq.rms_norm_q8(eps=1e-6, group=32, **a),
                        dict(x=x, weight=w, residual=f(n, d), scales=f(n, 1), h=f(n, d), rstd=f(n)),
                        {"scales", "h", "rstd"}),
        "rms_norm_grad": (gcq.rms_norm_grad, dict(dy=f(n, d), h=x, weight=w, rstd=rstd, dh=f(n, d), dx=f(n, d),
                                                  dweight=f(d)), {"dx", "dweight"}),
        "distill_loss": (lambda **a: gcq.distill_loss(index=idx, **a),
                         dict(logits=z, teacher=top, row_scale=f(n), loss=f(n), lse=f(n)), {"loss", "lse"}),
        "distill_grad": (lambda **a: gcq.distill_grad(index=idx, **a),
                         dict(logits=z, lse=f(n), teacher=top, row_scale=f(n), out=f(n, v)), {"out"}),
        "distill_loss_grad": (lambda **a: gcq.distill_loss_grad(index=idx, **a),
                              dict(logits=z, teacher=top, row_scale=f(n), loss=f(n), lse=f(n), out=f(n, v)),
                              {"loss", "lse", "out"}),
    }


@pytest.mark.gpu
def test_lost_gradients_are_refused(gpu):
    """Each tensor of each call; under no_grad the same call goes through."""
    import torch

    for name, (call, tensors, _) in operands().items():
        for which, t in tensors.items():
            print("[gpu] refuses a gradient", name, which, flush=True)
            asks = {**tensors, which: t.clone().requires_grad_()}
            with pytest.raises(ValueError, match=f"{which} requires a gradient"):
                call(**asks)
            with torch.no_grad():
                call(**asks)
            call(**{**tensors, which: torch.nn.Parameter(t.clone(), requires_grad=False)})


@pytest.mark.gpu
def test_what_is_written_has_a_new_version(gpu):
    import torch

    for name, (call, tensors, written) in operands().items():
        before = {k: t._version for k, t in tensors.items()}
        call(**tensors)
        moved = {k for k, t in tensors.items() if t._version > before[k]}
        assert moved == written, name
    tok = torch.arange(5, device="cuda")
    plan = gpu.embed_sort(tok, 9)
    v = plan.words._version
    gpu.embed_sort(tok, 9, plan)
    assert plan.words._version > v
    with torch.inference_mode():                  # tensors without a version
        a = torch.ones(3, 8, device="cuda")
        gpu.rms_norm(a, torch.ones(8, device="cuda"), 1e-6, residual=a.clone())


@pytest.mark.gpu
def test_overwriting_a_saved_tensor_is_noticed(gpu):
    """exp saves its result; the gradient is put in its place; its backward
    pass must not run on what is there now."""
    import torch

    for write in (lambda z, idx, top: gpu.distill_loss_grad(z, idx, top, out=z),
                  lambda z, idx, top: gpu.rms_norm(torch.ones_like(z), torch.ones(8, device="cuda"), 1e-6,
                                                   residual=z, h=z)):
        leaf = torch.zeros(3, 8, device="cuda", requires_grad=True)
        z = leaf.exp()
        write(z.detach(), torch.zeros(3, 2, dtype=torch.int64, device="cuda"), torch.zeros(3, 2, device="cuda"))
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            z.sum().backward()


@pytest.mark.gpu
def test_as_autograd_functions(gpu):
    """Lookup and norm as Functions inside a small graph, against torch's own
    differentiation in 64 bits.  Sums of at most 64 terms, each a chain of a
    few roundings: 200 * 2^-24 of the gradients' norms."""
    import torch

    class Lookup(torch.autograd.Function):
        @staticmethod
        def forward(ctx, table, tok):
            ctx.save_for_backward(tok)
            ctx.vocab = table.shape[0]
            return gpu.embed_lookup(table, tok, 2.0)

        @staticmethod
        def backward(ctx, g):
            tok, = ctx.saved_tensors
            return gpu.embed_grad(g.contiguous(), gpu.embed_sort(tok, ctx.vocab), 2.0), None

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            y, _, rstd = gpu.rms_norm(x, w, 1e-5)
            ctx.save_for_backward(x, w, rstd)
            return y

        @staticmethod
        def backward(ctx, g):
            x, w, rstd = ctx.saved_tensors
            return gpu.rms_norm_grad(g.contiguous(), x, w, rstd)

    gen = torch.Generator(device="cuda").manual_seed(1)
    table = torch.randn(20, 16, device="cuda", generator=gen, requires_grad=True)
    w = torch.rand(16, device="cuda", generator=gen).add_(0.5).requires_grad_()
    tok = torch.randint(0, 20, (64,), device="cuda", generator=gen)
    c = torch.randn(64, 16, device="cuda", generator=gen)
    (Norm.apply(Lookup.apply(table, tok), w) * c).sum().backward()
    t2, w2 = table.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    x = 2.0 * t2[tok]
    (x * (x.square().mean(1, keepdim=True) + 1e-5).rsqrt() * w2 * c.double()).sum().backward()
    for a, b in ((table.grad, t2.grad), (w.grad, w2.grad)):
        assert float((a.double() - b).norm() / b.norm()) < 200 * 2.0 ** -24
