"""Rows whose mask leaves nothing, written as the type's lowest value: the
student's softmax over equal logits is uniform, in loss and in the gradient
that comes with it, at temperatures where their quotient overflows as well.

Tolerances, E half a step of the type and e = 2^-24: every exponent is exactly
0, so q is 1 / V rounded twice; the entries' weights are off by a few e, and
the loss adds a logarithm and a few roundings of terms below 12: 100 e."""
import math

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("vocab", [1, 77, 4096, 50021, 131072])
@pytest.mark.parametrize("T", [0.5, 1.0, 2.0])
def test_rows_of_the_lowest_value(gpu, kind, vocab, T):
    import torch

    dt = getattr(torch, kind)
    z = torch.full((3, vocab), torch.finfo(dt).min, dtype=dt, device="cuda")
    k = min(4, vocab)
    idx = torch.arange(k, device="cuda").repeat(3, 1) * (vocab // k)
    top = torch.tensor([0.0, -0.5, -1.0, -2.0], device="cuda")[:k].repeat(3, 1)
    print("[gpu] lowest", kind, vocab, T, flush=True)
    loss, lse, dz = gpu.distill_loss_grad(z, idx, top, T)
    p = torch.softmax(top.double() / T, 1)
    want = (p * p.log()).sum(1) + math.log(vocab)
    assert ((loss.double() - want).abs() <= 100 * 2.0 ** -24).all()
    d = torch.full((3, vocab), 1.0 / vocab, dtype=torch.float64, device="cuda").scatter_add_(1, idx, -p) / T
    size = torch.full_like(d, 1.0 / vocab).scatter_add_(1, idx, p) / T
    half = torch.finfo(dt).eps / 2
    least = {"float32": 2.0 ** -150, "float16": 2.0 ** -25, "bfloat16": 2.0 ** -134}[kind]
    assert ((dz.double() - d).abs() <= half * d.abs() + 30 * 2.0 ** -24 * size + least).all()
    # the loss alone the same, and a weight of 0 leaves such rows out of all
    assert ((gpu.distill_loss(z, idx, top, T)[0].double() - want).abs() <= 100 * 2.0 ** -24).all()
    none = torch.zeros(3, device="cuda")
    l0, e0 = gpu.distill_loss(z, idx, top, T, none)
    assert (l0 == 0).all() and (e0 == 0).all()
    assert (gpu.distill_grad(z, e0, idx, top, T, none) == 0).all()
