"""Workspace sizes of the language-model operators: one that is made for the
largest batch and the longest row serves every smaller call."""
import numpy as np
import pytest

import gradient_compression_distributed_amd as gcq

F32, F16, BF16 = range(3)


def never_falls(sizes, what):
    drop = np.flatnonzero(np.diff(np.array(sizes, dtype=np.int64)) < 0)
    assert drop.size == 0, (what, drop[:4])


# every size up to past the largest threshold, then far ones
STEPS = [*range(0, 20000), *range(20000, 300000, 997), 1 << 20, 1 << 22]


@pytest.mark.parametrize("fixed", [1, 8, 64, 255, 256, 257, 1000, 2048, 2049, 4096, 8192, 131072, 1 << 22])
def test_embed_sizes_never_fall(fixed):
    lib = gcq.load()
    never_falls([lib.embed_work_bytes(n, fixed) for n in [*STEPS, 1 << 24]], ("positions", fixed))
    never_falls([lib.embed_work_bytes(fixed, dim) for dim in STEPS], ("columns", fixed))


def test_plan_sizes_never_fall():
    lib = gcq.load()
    never_falls([lib.embed_plan_words(n) for n in [*STEPS, 1 << 24]], "positions")


@pytest.mark.parametrize("kind", [F32, F16, BF16])
@pytest.mark.parametrize("fixed", [1, 3, 16, 17, 255, 256, 257, 700, 1023, 1024, 1025, 4096, 65536, 1 << 22])
def test_norm_sizes_never_fall(kind, fixed):
    lib = gcq.load()
    never_falls([lib.rms_norm_work_bytes(rows, fixed, kind) for rows in [*STEPS, 1 << 24]], ("rows", fixed))
    never_falls([lib.rms_norm_work_bytes(fixed, dim, kind) for dim in STEPS], ("columns", fixed))


@pytest.mark.gpu
def test_one_workspace_serves_smaller_batches(gpu):
    """Batches of falling size through one workspace with a guard behind it:
    the results of a workspace of their own, and the guard untouched."""
    import torch

    vocab = 500
    for n0, dim0 in ((8192, 4096), (16384, 2048), (4100, 300), (40, 64)):
        need = gpu.embed_work_bytes(n0, dim0)
        room = torch.full((need + (32 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
        for n, dim in ((n0, dim0), (n0 - 32, dim0), (n0 - 1, dim0 - 1), (n0 // 2, dim0), (n0 // 2, dim0 // 2 + 1),
                       (33, dim0), (32, dim0), (min(n0, 9), 3), (1, dim0)):
            print("[gpu] one workspace", n0, dim0, n, dim, flush=True)
            gen = torch.Generator(device="cuda").manual_seed(n + dim)
            tok = torch.randint(0, vocab, (n,), device="cuda", generator=gen)
            g = torch.randn(n, dim, device="cuda", generator=gen).to(torch.bfloat16)
            plan = gpu.embed_sort(tok, vocab)
            got = gpu.embed_grad(g, plan, work=room[:need])
            assert torch.equal(got, gpu.embed_grad(g, plan))
            ids, rows, count = gpu.embed_grad_rows(g, plan, work=room[:need])
            assert torch.equal(rows[:int(count)], got[ids[:int(count)].long()])
            assert (room[need:] == 0x5A).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
def test_one_workspace_serves_shorter_rows(gpu, kind):
    import torch

    dtype = getattr(torch, kind)
    for rows0, dim0 in ((1500, 16400), (1500, 8192), (1300, 6000), (20, 1000)):
        need = gpu.rms_norm_work_bytes(rows0, dim0, dtype)
        room = torch.full((need + (32 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
        for rows, dim in ((rows0, dim0), (rows0, dim0 - 1), (rows0, dim0 // 2), (rows0, dim0 // 3), (rows0 - 1, dim0 // 8),
                          (rows0, 64), (rows0 // 2, dim0), (1, 1)):
            print("[gpu] one workspace", kind, rows0, dim0, rows, dim, flush=True)
            gen = torch.Generator(device="cuda").manual_seed(rows + dim)
            dy, h = (torch.randn(rows, dim, device="cuda", generator=gen).to(dtype) for _ in range(2))
            w, rstd = torch.ones(dim, device="cuda"), torch.ones(rows, device="cuda")
            dx, dw = gpu.rms_norm_grad(dy, h, w, rstd, work=room[:need])
            want = gpu.rms_norm_grad(dy, h, w, rstd)
            assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
            assert (room[need:] == 0x5A).all()
