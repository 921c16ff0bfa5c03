"""Temperatures at the ends of what distillation takes: refusals on the host
(fake device addresses that are never dereferenced), and the least temperature
that is not refused against 64-bit values."""
import numpy as np
import pytest

import gradient_compression_distributed_amd as gcq

OK, E_PARAM = 0, -3
A, MB = 0x7F0000000000, 1 << 24
F32, I32 = 0, 3


@pytest.mark.parametrize("form", ["distill_loss", "distill_grad", "distill_loss_grad"])
def test_refused_where_a_factor_overflows(form):
    """log2(e) / T or scale / T infinite; others pass (no rows: no launch)."""
    fn = getattr(gcq.load(), form)

    def call(T, scale=1.0, rows=4):
        args = [A, F32, rows, 100, 100]
        if form == "distill_grad":
            args += [A + 5 * MB]
        args += [A + MB, I32, 8, A + 2 * MB, F32, 8, 8, T, None, scale]
        if form != "distill_grad":
            args += [A + 4 * MB, A + 5 * MB]
        if form != "distill_loss":
            args += [A + 6 * MB, 100]
        return fn(*args, None)

    for T in (1e-45, 1e-40, 4.2e-39):
        assert call(T) == E_PARAM, T
    assert call(1e-30, 1e10) == E_PARAM and call(1e-30, -1e10) == E_PARAM
    for T, scale in ((4.3e-39, 1.0), (1e-30, 1e7), (3e38, 1.0), (3e38, -3e38), (1.0, 0.0)):
        assert call(T, scale, rows=0) == OK, (T, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", [60, 5000, 40000])
def test_least_temperature(gpu, vocab):
    """Logits and temperature of subnormal size: their quotients are ordinary,
    and so are loss, lse and T * gradient.  The tolerance is the other
    temperatures' (test_gpu_distill): differences of subnormal numbers are
    exact, and lse * T, rounded to a multiple of 2^-149, moves an exponent by
    2^-150 / T < 3 * 2^-24."""
    import torch

    from tests.test_gpu_distill import check, plain

    T = float(np.float32(4.5e-39))
    rs = np.random.default_rng(vocab)
    z = torch.from_numpy((rs.standard_normal((3, vocab)) * 2.5 * T).astype(np.float32)).cuda()
    idx = torch.from_numpy(rs.integers(0, vocab, (3, 9))).cuda()
    top = torch.from_numpy((rs.random((3, 9)) * 3 * T).astype(np.float32)).cuda()
    want = plain(z, idx, top, T, None, 1.0)
    print("[gpu] least temperature", vocab, flush=True)
    loss, lse = gpu.distill_loss(z, idx, top, T)
    check((loss, lse, None), want, vocab, "float32")
    check((None, None, gpu.distill_grad(z, lse, idx, top, T)), want, vocab, "float32")
    check(gpu.distill_loss_grad(z, idx, top, T), want, vocab, "float32")
    assert torch.isfinite(lse).all()
