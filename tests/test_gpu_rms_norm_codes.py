"""rms_norm_q8's codes one by one: every e4m3 value, every tie between two of
them and values right beside the ties, for scales whose reciprocals are
rounded, and scales at both ends of their range.

eps makes rstd a power of two whatever the row holds (the mean of squares is
lost when eps is added to it) and the weights are powers of two, or the scale
itself, so y is exact, its largest magnitude is 448 scales, the scale comes
out exactly and every expected code is known."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

# non-negative finite e4m3 values by code
CODES = [math.ldexp(c, -9) if c < 8 else math.ldexp(8 + c % 8, (c >> 3) - 10) for c in range(127)]


def pattern():
    """(values, their codes, whether each is a tie): 448, every code of either
    sign, and every tie, whose code is the even neighbour."""
    v, want, tie = [448.0], [126], [False]
    for c in range(127):
        v += [CODES[c], -CODES[c]]
        want += [c, c | 128]
        tie += [False, False]
        if c < 126:
            mid, even = (CODES[c] + CODES[c + 1]) / 2, c if c % 2 == 0 else c + 1
            v += [mid, -mid]
            want += [even, even | 128]
            tie += [True, True]
    return np.array(v), np.array(want, np.uint8), np.array(tie)


def laid_out(a, dim, group):
    """The pattern repeated over dim columns, a piece of it behind the leading
    448 in every group."""
    group = group or dim
    out, rest, at = np.empty(dim, a.dtype), a[1:], 0
    for g0 in range(0, dim, group):
        n = min(group, dim - g0) - 1
        out[g0] = a[0]
        out[g0 + 1:g0 + 1 + n] = rest[(at + np.arange(n)) % rest.size]
        at += n
    return out


def codes_of(gpu, x, w, eps, group):
    import torch

    codes, scales, _, rstd = gpu.rms_norm_q8(x, w, eps, group=group)
    return codes.view(torch.uint8).cpu().numpy(), scales.cpu().numpy(), rstd.cpu().numpy()


@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("dim", [250, 1000, 2048, 8192, 20000])
def test_every_code_and_tie(gpu, group, dim):
    """Rows of scales 3, 5, 7 ... times a power of two in float32; every split
    of a row over lanes.  The products need 5 + 11 bits."""
    import torch

    v, want, tie = (laid_out(a, dim, group) for a in pattern())
    s = np.arange(3, 2048, 2 if dim < 2048 else 30, dtype=np.float64)
    x = torch.from_numpy((v[None] * s[:, None] * 2.0 ** -40).astype(np.float32)).cuda()
    print("[gpu] codes", group, dim, len(s), flush=True)
    got, scales, rstd = codes_of(gpu, x, torch.ones(dim, device="cuda"), 1.0, group)
    assert (rstd == 1.0).all()                    # 1 + 2^-40 at most
    assert (scales == (s * 2.0 ** -40)[:, None]).all()
    # a step of float32 off a tie, its own neighbour is the nearest
    assert (got == want[None]).all(), int((got != want[None]).sum())
    for away in (np.inf, 0.0):
        off = x.cpu().numpy()
        off[:, tie] = np.nextafter(off[:, tie], np.float32(away) * np.sign(off[:, tie]))
        other, _, _ = codes_of(gpu, torch.from_numpy(off).cuda(), torch.ones(dim, device="cuda"), 1.0,
                               group)
        mags = np.abs(v[tie])
        up = np.searchsorted(CODES, mags)         # the larger neighbour's code
        near = (up if away else up - 1) | (want[tie] & 128)
        # the quotient is rounded to float32 first and may come back to the tie
        assert ((other[:, tie] == near[None]) | (other[:, tie] == want[tie][None])).all()
        assert (other[:, ~tie] == want[~tie][None]).all()


@pytest.mark.parametrize("kind", ["float16", "bfloat16"])
@pytest.mark.parametrize("group", [0, 64, 128])
@pytest.mark.parametrize("rows,dim", [(2, 250), (1100, 250), (2, 4096), (1030, 4096), (2, 20000)])
def test_every_code_and_tie_16_bit(gpu, kind, group, rows, dim):
    """x holds the codes' values, float32 weights the scale; rstd is 2^-30."""
    import torch

    v, want = (laid_out(a, dim, group) for a in pattern()[:2])
    x = torch.from_numpy(v.astype(np.float32)).to(getattr(torch, kind)).cuda()
    assert torch.equal(x.double().cpu(), torch.from_numpy(v))
    x = x.expand(rows, dim).contiguous()
    for s in (1.0, 3.0, 41.0, 113.0, 641.0, 2047.0):
        got, scales, rstd = codes_of(gpu, x, torch.full((dim,), s, device="cuda"), 2.0 ** 60, group)
        assert (rstd == 2.0 ** -30).all() and (scales == s * 2.0 ** -30).all()
        assert (got == want[None]).all(), (s, int((got != want[None]).sum()))


@pytest.mark.parametrize("group", [0, 32])
def test_scales_at_their_ends(gpu, group):
    """The least scale (2^-126), scales whose quotients pass through subnormal
    numbers, the largest, and an infinite one: finite values become 0, the
    infinity NaN."""
    import torch

    dim = 512
    v, want, _ = (laid_out(a, dim, group) for a in pattern())
    w = torch.ones(dim, device="cuda")
    for s in (2.0 ** -126, 3 * 2.0 ** -127, 129 * 2.0 ** -130, 2.0 ** 100, 3 * 2.0 ** 100):
        up = 2.0 ** 127 if s > 1 else 1.0         # x stays small beside eps, the weights bring y to its size
        x = torch.from_numpy((v * s / up).astype(np.float32)).cuda()[None]
        assert (x[0].double().cpu().numpy() == v * s / up).all()
        got, scales, rstd = codes_of(gpu, x, w * up, 1.0, group)
        assert rstd[0] == 1.0 and (scales == s).all()
        assert (got[0] == want).all()
    w[7] = math.inf
    got, scales, _ = codes_of(gpu, torch.ones(1, dim, device="cuda"), w, 0.0, group)
    g = group or dim
    assert scales[0, 0] == math.inf and got[0, 7] & 127 == 127
    assert (np.delete(got[0, :g], 7) == 0).all() and (got[0, g:] == 126).all()
