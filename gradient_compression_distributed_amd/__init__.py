"""MI355X (gfx950) gradient-compression hot path: Python binding.

A thin ctypes layer over ``libgcq.so`` (the C ABI of ``include/gcq.h``).
Every step of the path runs in the library's HIP kernels; this module only
checks tensor metadata, passes raw device pointers and the current HIP
stream, and turns a negative status into ``GcqError``.  PyTorch supplies
device memory and streams.  There is no CPU fallback: if the library is
missing, ``load()`` raises.

Packed words (2-bit codes, QSGD nibbles) are held in ``torch.int32``
tensors as raw 32-bit patterns (view them as uint32 on the host).

No call records anything for autograd.  The language-model operators refuse
tensors that require a gradient while gradients are recorded (call them under
``torch.no_grad()``, in a ``torch.autograd.Function``, or with detached
tensors), and raise the version of what they write, as torch's own in-place
operations do.
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "GcqError", "load", "lib_path", "gc2_quantize", "gc2_quantize_buckets",
    "gc2_quantize_buckets_noalloc", "GC2_NOALLOC_MAX_BUCKETS",
    "gc2_dequant_reduce", "qsgd_quantize", "qsgd_dequant", "gc2_packed_words",
    "qsgd_num_buckets", "qsgd_nibble_words", "MAX_WORKERS", "set_tuning", "get_tuning", "BucketList",
    "cdsgd_update_quantize", "cdsgd_local_update", "cdsgd_compresses",
    "qsgd_quantize_maxnorm", "qsgd_dequant_average",
    "saps_mask", "saps_gather", "saps_merge", "saps_mask_words", "saps_num_tiles",
    "qsgd_elias_encode", "qsgd_elias_decode", "qsgd_elias_max_words",
    "probe_stream", "probe_reduce",
    "embed_lookup", "embed_sort", "EmbedPlan", "embed_grad", "embed_grad_rows",
    "embed_plan_words", "embed_work_bytes",
    "rms_norm", "rms_norm_q8", "rms_norm_grad", "rms_norm_work_bytes",
    "distill_loss", "distill_grad", "distill_loss_grad",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_NAME = "libgcq.so"
MAX_WORKERS = 64

_lib = None


class GcqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.gcq_status_string(status).decode() if _lib is not None else str(status)
        super().__init__(f"{where}: status {status} ({msg})")


class Tuning(ctypes.Structure):
    """Mirror of ``gcq_tuning`` (launch knobs; results never depend on them)."""
    _fields_ = [(f, ctypes.c_int) for f in (
        "gc2_unroll", "gc2_nt", "gc2_blocks_per_cu", "dq_nt_loads", "dq_nt_stores",
        "dq_lds_stores", "dq_blocks_per_cu", "dq_fp4_decode", "qsgd_nt", "qsgd_rcp",
        "qsgd_dequant_nt", "qsgd_blocks_per_cu", "qsgd_dequant_blocks_per_cu",
        "qsgd_buckets_per_wave", "dq_words_per_thread", "dq_resident_per_cu",
        "gc2_resident_per_cu", "cdsgd_resident_per_cu", "qsgd_avg_resident_per_cu")]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class Gc2Bucket(ctypes.Structure):
    _fields_ = [("g", ctypes.c_void_p), ("r", ctypes.c_void_p), ("out_words", ctypes.c_void_p),
                ("n", ctypes.c_size_t), ("t", ctypes.c_float)]


def lib_path() -> str:
    return os.path.join(_PKG, LIB_NAME)


def load():
    """Load libgcq.so from the package directory (raises if it is absent)."""
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run __graft_entry__.build() "
                           "(hipcc --offload-arch=gfx950) first")
    lib = ctypes.CDLL(path)
    vp, sz, u32, u64, f32, i32 = (ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint32,
                                  ctypes.c_uint64, ctypes.c_float, ctypes.c_int)
    lib.gc2_quantize.argtypes = [vp, vp, sz, f32, vp, vp]
    lib.gc2_quantize.restype = i32
    lib.gc2_quantize_buckets.argtypes = [ctypes.POINTER(Gc2Bucket), u32, vp]
    lib.gc2_quantize_buckets.restype = i32
    lib.gc2_quantize_buckets_noalloc.argtypes = [ctypes.POINTER(Gc2Bucket), u32, vp]
    lib.gc2_quantize_buckets_noalloc.restype = i32
    lib.gc2_dequant_reduce.argtypes = [ctypes.POINTER(vp), u32, sz, f32, vp, vp]
    lib.gc2_dequant_reduce.restype = i32
    lib.gcq_probe_reduce.argtypes = [ctypes.POINTER(vp), u32, sz, vp, vp]
    lib.gcq_probe_reduce.restype = i32
    lib.gcq_probe_stream.argtypes = [vp, vp, vp, vp, sz, vp]
    lib.gcq_probe_stream.restype = i32
    lib.qsgd_quantize.argtypes = [vp, sz, u32, u32, u64, vp, vp, vp]
    lib.qsgd_quantize.restype = i32
    lib.qsgd_dequant.argtypes = [vp, vp, sz, u32, u32, vp, vp]
    lib.qsgd_dequant.restype = i32
    lib.cdsgd_update_quantize.argtypes = [vp, vp, vp, sz, f32, f32, vp, vp]
    lib.cdsgd_update_quantize.restype = i32
    lib.qsgd_quantize_maxnorm.argtypes = [vp, sz, u32, u32, u64, vp, vp, vp]
    lib.qsgd_quantize_maxnorm.restype = i32
    lib.qsgd_dequant_average.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(vp), u32, sz, u32,
                                         u32, vp, vp]
    lib.qsgd_dequant_average.restype = i32
    lib.qsgd_elias_max_words.argtypes = [sz, u32]
    lib.qsgd_elias_max_words.restype = sz
    lib.qsgd_elias_encode.argtypes = [vp, vp, sz, u32, vp, vp, sz, vp]
    lib.qsgd_elias_encode.restype = i32
    lib.qsgd_elias_decode.argtypes = [vp, sz, vp, sz, u32, vp, vp, vp]
    lib.qsgd_elias_decode.restype = i32
    lib.saps_mask.argtypes = [sz, f32, u64, vp, vp, vp]
    lib.saps_mask.restype = i32
    lib.saps_gather.argtypes = [vp, sz, vp, vp, vp, sz, vp]
    lib.saps_gather.restype = i32
    lib.saps_merge.argtypes = [vp, sz, vp, vp, vp, sz, vp]
    lib.saps_merge.restype = i32
    lib.saps_mask_words.argtypes = [sz]
    lib.saps_mask_words.restype = sz
    lib.saps_num_tiles.argtypes = [sz]
    lib.saps_num_tiles.restype = sz
    lib.cdsgd_local_update.argtypes = [vp, vp, sz, f32, vp]
    lib.cdsgd_local_update.restype = i32
    lib.gc2_packed_words.argtypes = [sz]
    lib.gc2_packed_words.restype = sz
    lib.qsgd_num_buckets.argtypes = [sz, u32]
    lib.qsgd_num_buckets.restype = sz
    lib.qsgd_nibble_words.argtypes = [sz]
    lib.qsgd_nibble_words.restype = sz
    lib.gcq_status_string.argtypes = [i32]
    lib.gcq_status_string.restype = ctypes.c_char_p
    lib.gcq_get_tuning.argtypes = [ctypes.POINTER(Tuning)]
    lib.gcq_get_tuning.restype = i32
    lib.gcq_set_tuning.argtypes = [ctypes.POINTER(Tuning)]
    lib.gcq_set_tuning.restype = i32
    lib.embed_lookup.argtypes = [vp, i32, sz, sz, sz, vp, i32, sz, f32, vp, i32, sz, vp]
    lib.embed_lookup.restype = i32
    lib.embed_sort.argtypes = [vp, i32, sz, sz, vp, vp]
    lib.embed_sort.restype = i32
    lib.embed_grad.argtypes = [vp, i32, sz, vp, sz, sz, sz, f32, i32, vp, sz, vp, vp]
    lib.embed_grad.restype = i32
    lib.embed_grad_rows.argtypes = [vp, i32, sz, vp, sz, sz, sz, f32, vp, vp, sz, vp, vp, vp]
    lib.embed_grad_rows.restype = i32
    lib.embed_plan_words.argtypes = [sz]
    lib.embed_plan_words.restype = sz
    lib.embed_work_bytes.argtypes = [sz, sz]
    lib.embed_work_bytes.restype = sz
    lib.rms_norm.argtypes = [vp, i32, sz, sz, sz, vp, sz, vp, i32, f32, vp, sz, vp, sz, vp, vp]
    lib.rms_norm.restype = i32
    lib.rms_norm_q8.argtypes = [vp, i32, sz, sz, sz, vp, sz, vp, i32, f32, u32, vp, sz, vp, vp, sz,
                                vp, vp]
    lib.rms_norm_q8.restype = i32
    lib.rms_norm_grad.argtypes = [vp, i32, sz, sz, sz, vp, sz, vp, i32, vp, vp, sz, vp, sz, vp, i32,
                                  vp, vp]
    lib.rms_norm_grad.restype = i32
    lib.rms_norm_work_bytes.argtypes = [sz, sz, i32]
    lib.rms_norm_work_bytes.restype = sz
    lib.distill_loss.argtypes = [vp, i32, sz, sz, sz, vp, i32, sz, vp, i32, sz, u32, f32, vp, f32,
                                 vp, vp, vp]
    lib.distill_loss.restype = i32
    lib.distill_grad.argtypes = [vp, i32, sz, sz, sz, vp, vp, i32, sz, vp, i32, sz, u32, f32, vp,
                                 f32, vp, sz, vp]
    lib.distill_grad.restype = i32
    lib.distill_loss_grad.argtypes = [vp, i32, sz, sz, sz, vp, i32, sz, vp, i32, sz, u32, f32, vp,
                                      f32, vp, vp, vp, sz, vp]
    lib.distill_loss_grad.restype = i32
    _lib = lib
    return lib


# ---------------------------------------------------------------- helpers
def gc2_packed_words(n: int) -> int:
    return int(load().gc2_packed_words(n))


def qsgd_num_buckets(n: int, d: int) -> int:
    return int(load().qsgd_num_buckets(n, d))


def qsgd_nibble_words(n: int) -> int:
    return int(load().qsgd_nibble_words(n))


def _dev(x, dtype, name, min_numel=0):
    import torch

    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if x.device.type != "cuda":
        raise ValueError(f"{name} must live in GPU memory (got {x.device})")
    if x.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {x.dtype})")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if x.numel() < min_numel:
        raise ValueError(f"{name} holds {x.numel()} elements, needs {min_numel}")
    return x


def _ptr(x):
    return ctypes.c_void_p(x.data_ptr() if x is not None and x.numel() else 0)


def _stream(device=None):
    import torch

    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check(status: int, where: str):
    if status != 0:
        raise GcqError(status, where)


def get_tuning() -> dict:
    """Current launch knobs as a dict (see ``gcq_tuning`` in include/gcq.h)."""
    t = Tuning()
    _check(load().gcq_get_tuning(ctypes.byref(t)), "gcq_get_tuning")
    return t.as_dict()


def set_tuning(**knobs) -> dict:
    """Change some launch knobs (speed only; results are identical).
    Returns the previous settings, so ``set_tuning(**old)`` restores them."""
    t = Tuning()
    _check(load().gcq_get_tuning(ctypes.byref(t)), "gcq_get_tuning")
    old = t.as_dict()
    for k, v in knobs.items():
        if k not in old:
            raise KeyError(f"unknown tuning knob {k!r}")
        setattr(t, k, int(v))
    _check(load().gcq_set_tuning(ctypes.byref(t)), "gcq_set_tuning")
    return old


# -------------------------------------------------------------- the calls
def gc2_quantize(g, r, t: float, out=None):
    """One 2-bit quantize step: returns the packed words, updates ``r``."""
    import torch

    lib = load()
    _dev(g, torch.float32, "g")
    n = g.numel()
    _dev(r, torch.float32, "r", n)
    if out is None:
        out = torch.empty(gc2_packed_words(n), dtype=torch.int32, device=g.device)
    _dev(out, torch.int32, "out", gc2_packed_words(n))
    _check(lib.gc2_quantize(_ptr(g), _ptr(r), n, ctypes.c_float(t), _ptr(out),
                            _stream(g.device)), "gc2_quantize")
    return out


def cdsgd_compresses(count: int, k: int) -> bool:
    """CD-SGD's k-step switch (Algorithm 1, section 3.2.1): iteration
    ``count`` compresses its gradient unless ``count % k == 0``, when the
    full-precision gradient is pushed instead (host logic only)."""
    if k < 1:
        raise ValueError("k must be >= 1")
    return count % k != 0


def cdsgd_update_quantize(g, r, w, t: float, eta: float, out=None):
    """A compressing CD-SGD iteration on one buffer: ``w -= eta * g`` (local
    update) and one 2-bit quantize step of (g, r); returns the packed words."""
    import torch

    lib = load()
    _dev(g, torch.float32, "g")
    n = g.numel()
    _dev(r, torch.float32, "r", n)
    _dev(w, torch.float32, "w", n)
    if out is None:
        out = torch.empty(gc2_packed_words(n), dtype=torch.int32, device=g.device)
    _dev(out, torch.int32, "out", gc2_packed_words(n))
    _check(lib.cdsgd_update_quantize(_ptr(g), _ptr(r), _ptr(w), n, ctypes.c_float(t),
                                     ctypes.c_float(eta), _ptr(out), _stream(g.device)),
           "cdsgd_update_quantize")
    return out


def cdsgd_local_update(g, w, eta: float):
    """A correction iteration's local update: ``w -= eta * g``."""
    import torch

    lib = load()
    _dev(g, torch.float32, "g")
    _dev(w, torch.float32, "w", g.numel())
    _check(lib.cdsgd_local_update(_ptr(g), _ptr(w), g.numel(), ctypes.c_float(eta),
                                  _stream(g.device)), "cdsgd_local_update")


class BucketList:
    """A checked, reusable descriptor array for gc2_quantize_buckets.

    Holds references to the tensors so their memory outlives the list;
    building it once and reusing it every step keeps per-call host work to
    the library's own checks and one launch."""

    def __init__(self, buckets):
        import torch

        self.tensors = list(buckets)
        self.array = (Gc2Bucket * max(len(buckets), 1))()
        self.device = None
        for i, (g, r, out, t) in enumerate(buckets):
            _dev(g, torch.float32, f"buckets[{i}].g")
            n = g.numel()
            _dev(r, torch.float32, f"buckets[{i}].r", n)
            _dev(out, torch.int32, f"buckets[{i}].out", gc2_packed_words(n))
            self.array[i] = Gc2Bucket(g.data_ptr() if n else 0, r.data_ptr() if n else 0,
                                      out.data_ptr() if n else 0, n, t)
            self.device = self.device or g.device
        self.count = len(buckets)


def gc2_quantize_buckets(buckets):
    """Fused launch over ``[(g, r, out, t), ...]`` (or a ``BucketList``);
    each bucket is quantized exactly as gc2_quantize would."""
    lib = load()
    bl = buckets if isinstance(buckets, BucketList) else BucketList(buckets)
    _check(lib.gc2_quantize_buckets(bl.array, bl.count, _stream(bl.device)),
           "gc2_quantize_buckets")


def gc2_quantize_buckets_noalloc(buckets):
    """gc2_quantize_buckets through the entry point that allocates nothing
    (its descriptor table is a fixed device array of the library, at most
    GC2_NOALLOC_MAX_BUCKETS buckets; calls that may overlap on one device
    race on it)."""
    lib = load()
    bl = buckets if isinstance(buckets, BucketList) else BucketList(buckets)
    _check(lib.gc2_quantize_buckets_noalloc(bl.array, bl.count, _stream(bl.device)),
           "gc2_quantize_buckets_noalloc")


GC2_NOALLOC_MAX_BUCKETS = 4096


def gc2_dequant_reduce(words, n: int, t: float, acc=None):
    """acc = sum over workers 0..W-1 (in order) of the dequantized codes."""
    import torch

    lib = load()
    W = len(words)
    nw = gc2_packed_words(n)
    for i, w in enumerate(words):
        _dev(w, torch.int32, f"words[{i}]", nw)
    if acc is None:
        acc = torch.empty(n, dtype=torch.float32, device=words[0].device)
    _dev(acc, torch.float32, "acc", n)
    ptrs = (ctypes.c_void_p * max(W, 1))(*[w.data_ptr() for w in words])
    _check(lib.gc2_dequant_reduce(ptrs, W, n, ctypes.c_float(t), _ptr(acc),
                                  _stream(acc.device)), "gc2_dequant_reduce")
    return acc


def probe_stream(a, c, b=None, words=None):
    """Measurement probe with the 2-bit quantizer's access pattern and no
    arithmetic: c = a ^ b (bitwise; c = a without b), plus a packed-word
    stream when ``words`` is given.  n = a.numel() must be a multiple of 1024."""
    import torch

    lib = load()
    _dev(a, torch.float32, "a")
    n = a.numel()
    _dev(c, torch.float32, "c", n)
    if b is not None:
        _dev(b, torch.float32, "b", n)
    if words is not None:
        _dev(words, torch.int32, "words", n // 16)
    _check(lib.gcq_probe_stream(_ptr(a), _ptr(b) if b is not None else None, _ptr(c),
                                _ptr(words) if words is not None else None, n,
                                _stream(a.device)), "gcq_probe_stream")


def probe_reduce(words, n: int, acc):
    """Measurement probe: gc2_dequant_reduce's kernel with the decode replaced
    by an XOR (acc[16 i] = XOR of the workers' word i, other sums +0)."""
    import torch

    lib = load()
    W = len(words)
    nw = gc2_packed_words(n)
    for i, w in enumerate(words):
        _dev(w, torch.int32, f"words[{i}]", nw)
    _dev(acc, torch.float32, "acc", n)
    ptrs = (ctypes.c_void_p * max(W, 1))(*[w.data_ptr() for w in words])
    _check(lib.gcq_probe_reduce(ptrs, W, n, _ptr(acc), _stream(acc.device)), "gcq_probe_reduce")
    return acc


def qsgd_quantize(g, d: int, s: int, seed: int, norms=None, nibbles=None, maxnorm: bool = False):
    """Bucketed QSGD: returns (norms float32[ceil(n/d)], nibbles int32[ceil(n/8)]).
    With ``maxnorm`` the bucket scale is the largest magnitude (Knowl 8)."""
    import torch

    lib = load()
    _dev(g, torch.float32, "g")
    n = g.numel()
    nb, nw = qsgd_num_buckets(n, d), qsgd_nibble_words(n)
    if norms is None:
        norms = torch.empty(nb, dtype=torch.float32, device=g.device)
    if nibbles is None:
        nibbles = torch.empty(nw, dtype=torch.int32, device=g.device)
    _dev(norms, torch.float32, "norms", nb)
    _dev(nibbles, torch.int32, "nibbles", nw)
    fn = lib.qsgd_quantize_maxnorm if maxnorm else lib.qsgd_quantize
    _check(fn(_ptr(g), n, d, s, ctypes.c_uint64(seed & 0xFFFFFFFFFFFFFFFF),
              _ptr(norms), _ptr(nibbles), _stream(g.device)), "qsgd_quantize")
    return norms, nibbles


def qsgd_quantize_maxnorm(g, d: int, s: int, seed: int, scales=None, nibbles=None):
    """QSGD with max-norm bucket scales: returns (scales, nibbles)."""
    return qsgd_quantize(g, d, s, seed, norms=scales, nibbles=nibbles, maxnorm=True)


def qsgd_dequant_average(scales, nibbles, n: int, d: int, s: int, out=None):
    """Mean over K workers (order 0..K-1) of their decoded QSGD messages."""
    import torch

    lib = load()
    K = len(scales)
    if K != len(nibbles):
        raise ValueError("scales and nibbles differ in length")
    for i in range(K):
        _dev(scales[i], torch.float32, f"scales[{i}]", qsgd_num_buckets(n, d))
        _dev(nibbles[i], torch.int32, f"nibbles[{i}]", qsgd_nibble_words(n))
    if out is None:
        out = torch.empty(n, dtype=torch.float32, device=scales[0].device)
    _dev(out, torch.float32, "out", n)
    sp = (ctypes.c_void_p * max(K, 1))(*[x.data_ptr() for x in scales])
    npp = (ctypes.c_void_p * max(K, 1))(*[x.data_ptr() for x in nibbles])
    _check(lib.qsgd_dequant_average(sp, npp, K, n, d, s, _ptr(out), _stream(out.device)),
           "qsgd_dequant_average")
    return out


def qsgd_dequant(norms, nibbles, n: int, d: int, s: int, out=None):
    """out = +-(norm * level) / s per element."""
    import torch

    lib = load()
    _dev(norms, torch.float32, "norms", qsgd_num_buckets(n, d))
    _dev(nibbles, torch.int32, "nibbles", qsgd_nibble_words(n))
    if out is None:
        out = torch.empty(n, dtype=torch.float32, device=norms.device)
    _dev(out, torch.float32, "out", n)
    _check(lib.qsgd_dequant(_ptr(norms), _ptr(nibbles), n, d, s, _ptr(out),
                            _stream(out.device)), "qsgd_dequant")
    return out


# ------------------------------------------------------------------ SAPS
def saps_mask_words(n: int) -> int:
    return int(load().saps_mask_words(n))


def saps_num_tiles(n: int) -> int:
    return int(load().saps_num_tiles(n))


def saps_mask(n: int, c: float, seed: int, mask=None, offsets=None, device="cuda"):
    """Shared-seed Bernoulli(1/c) mask: returns (mask words int32, tile
    offsets int64 with the total kept count last)."""
    import torch

    lib = load()
    if mask is None:
        mask = torch.empty(saps_mask_words(n), dtype=torch.int32, device=device)
    if offsets is None:
        offsets = torch.empty(saps_num_tiles(n) + 1, dtype=torch.int64, device=device)
    _dev(mask, torch.int32, "mask", saps_mask_words(n))
    _dev(offsets, torch.int64, "offsets", saps_num_tiles(n) + 1)
    _check(lib.saps_mask(n, ctypes.c_float(c), ctypes.c_uint64(seed & 0xFFFFFFFFFFFFFFFF),
                         _ptr(mask), _ptr(offsets), _stream(offsets.device)), "saps_mask")
    return mask, offsets


def saps_count(offsets) -> int:
    """The total kept count (synchronizes with the device)."""
    return int(offsets[-1].item())


def saps_gather(x, mask, offsets, values=None):
    """The kept components of ``x`` in index order."""
    import torch

    lib = load()
    _dev(x, torch.float32, "x")
    _dev(mask, torch.int32, "mask", saps_mask_words(x.numel()))
    _dev(offsets, torch.int64, "offsets", saps_num_tiles(x.numel()) + 1)
    if values is None:
        values = torch.empty(saps_count(offsets), dtype=torch.float32, device=x.device)
    _dev(values, torch.float32, "values")
    _check(lib.saps_gather(_ptr(x), x.numel(), _ptr(mask), _ptr(offsets), _ptr(values),
                           values.numel(), _stream(x.device)), "saps_gather")
    return values


def saps_merge(x, mask, offsets, peer_values):
    """x[kept] = (x[kept] + peer_values) * 0.5, in place."""
    import torch

    lib = load()
    _dev(x, torch.float32, "x")
    _dev(mask, torch.int32, "mask", saps_mask_words(x.numel()))
    _dev(offsets, torch.int64, "offsets", saps_num_tiles(x.numel()) + 1)
    _dev(peer_values, torch.float32, "peer_values")
    _check(lib.saps_merge(_ptr(x), x.numel(), _ptr(mask), _ptr(offsets), _ptr(peer_values),
                          peer_values.numel(), _stream(x.device)), "saps_merge")


# ------------------------------------------------------- QSGD Elias coding
def qsgd_elias_max_words(n: int, d: int) -> int:
    return int(load().qsgd_elias_max_words(n, d))


def qsgd_elias_encode(norms, nibbles, n: int, d: int, offsets=None, out=None):
    """Elias-omega coded buckets: returns (bit offsets int64[nb + 1], words
    int32[capacity]); the coded length in bits is the last offset."""
    import torch

    lib = load()
    nb = qsgd_num_buckets(n, d)
    _dev(norms, torch.float32, "norms", nb)
    _dev(nibbles, torch.int32, "nibbles", qsgd_nibble_words(n))
    if offsets is None:
        offsets = torch.empty(nb + 1, dtype=torch.int64, device=norms.device)
    if out is None:
        out = torch.empty(max(qsgd_elias_max_words(n, d), 1), dtype=torch.int32,
                          device=norms.device)
    _dev(offsets, torch.int64, "offsets", nb + 1)
    _dev(out, torch.int32, "out")
    _check(lib.qsgd_elias_encode(_ptr(norms), _ptr(nibbles), n, d, _ptr(offsets), _ptr(out),
                                 out.numel(), _stream(out.device)), "qsgd_elias_encode")
    return offsets, out


def qsgd_elias_decode(words, offsets, n: int, d: int, norms=None, nibbles=None):
    """Returns (norms, nibbles) of Elias-coded buckets."""
    import torch

    lib = load()
    nb = qsgd_num_buckets(n, d)
    _dev(words, torch.int32, "words")
    _dev(offsets, torch.int64, "offsets", nb + 1)
    if norms is None:
        norms = torch.empty(nb, dtype=torch.float32, device=words.device)
    if nibbles is None:
        nibbles = torch.empty(qsgd_nibble_words(n), dtype=torch.int32, device=words.device)
    _dev(norms, torch.float32, "norms", nb)
    _dev(nibbles, torch.int32, "nibbles", qsgd_nibble_words(n))
    _check(lib.qsgd_elias_decode(_ptr(words), words.numel(), _ptr(offsets), n, d, _ptr(norms),
                                 _ptr(nibbles), _stream(words.device)), "qsgd_elias_decode")
    return norms, nibbles


# ------------------------------------------------- language-model operators
# Matrices are 2-D tensors whose rows are contiguous; rows may lie further
# apart than their length (a slice of columns).  A call runs on the device of
# its tensors, on that device's current stream, whatever device is current.
# Calls record nothing for autograd: where gradients are recorded, a tensor that
# requires one is refused (its gradient would be lost without a word), and the
# version of every tensor that a call writes is raised, so that a backward pass
# that saved it before says so.
# What a call needs of torch, looked up once (by _lm): the small calls take a
# few microseconds, and an import statement or a Stream object is a part of it.
_torch = _tensor = _type_codes = _raw_stream = _current_device = _wrote = None


def _lm():
    """The library, with the names above set."""
    global _torch, _tensor, _type_codes, _raw_stream, _current_device, _wrote
    if _torch is None:
        import torch

        load()
        _type_codes = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.int32: 3,
                       torch.int64: 4}
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
        _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        _wrote = getattr(torch._C, "_increment_version", torch.autograd.graph.increment_version)
        _torch, _tensor = torch, torch.Tensor
    return _lib if _lib is not None else load()


def _type_code(x, name, allowed=(0, 1, 2)):
    """The C ABI's enum gcq_type of a tensor's element type."""
    code = _type_codes.get(x.dtype, -1)
    if code not in allowed:
        raise TypeError(f"{name} has type {x.dtype}, which this call does not take")
    return code


def _on(x, name, device=None):
    """Refuses what is not a GPU tensor (on ``device``, an index, if given) and
    one whose gradient would be lost; returns the index of its device."""
    try:
        at = x.get_device()
        lost = x.requires_grad
    except AttributeError:
        raise TypeError(f"{name} must be a torch tensor") from None
    if lost and _torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, which this call does not record: call it "
                         "under torch.no_grad() or in a torch.autograd.Function, or detach it")
    if at < 0:
        raise ValueError(f"{name} must live in GPU memory (got {x.device})")
    if device is not None and at != device:
        raise ValueError(f"{name} is on device {at}, the call's other tensors on {device}")
    return at


def _row_distance(x, name, rows, cols):
    """The distance of a matrix's rows in elements."""
    ld, step = x.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    if rows <= 1:
        return cols
    if ld < cols:
        raise ValueError(f"{name}: rows overlap")
    return ld


def _first(x, name):
    """A call's first matrix: (index of the device, rows, columns, distance of
    the rows)."""
    dev = _on(x, name)
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be a matrix")
    rows, cols = shape
    return dev, rows, cols, _row_distance(x, name, rows, cols)


def _matrix(x, name, rows, cols, device, written=False):
    """Checks a matrix of rows x cols (at least ``rows`` rows if it is
    written); returns the distance of its rows in elements."""
    if type(x) is not _tensor or x.get_device() != device or x.requires_grad:
        _on(x, name, device)
    shape = x.shape
    if shape != (rows, cols) and (len(shape) != 2 or shape[1] != cols or not written or shape[0] < rows):
        raise ValueError(f"{name} has shape {tuple(shape)}, needs ({rows}, {cols})")
    return _row_distance(x, name, shape[0], cols)


def _vector(x, name, n, device, dtype=None, at_least=False):
    """Checks a contiguous tensor of n elements (or at least n, or any number
    for None); returns how many it holds."""
    if type(x) is not _tensor or x.get_device() != device or x.requires_grad:
        _on(x, name, device)
    if dtype is not None and x.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {x.dtype})")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    have = x.numel()
    if have != n and n is not None and (have < n or not at_least):
        raise ValueError(f"{name} holds {have} elements, needs {n}")
    return have


def _call(fn, where, device, *args):
    """fn(*args, stream) on a device's current stream, with that device
    current while it runs."""
    if _current_device() == device:
        status = fn(*args, _raw_stream(device))
    else:
        with _torch.cuda.device(device):
            status = fn(*args, _raw_stream(device))
    if status != 0:
        raise GcqError(status, where)


def embed_plan_words(n: int) -> int:
    return int(load().embed_plan_words(n))


def embed_work_bytes(n: int, dim: int) -> int:
    return int(load().embed_work_bytes(n, dim))


def embed_lookup(table, tokens, scale: float = 1.0, out=None):
    """out[i] = scale * table[tokens[i]], rounded once to out's type (the
    table's by default).  Tokens outside the table are padding: zero rows."""
    lib, torch = _lm(), _torch
    dev, vocab, dim, ld = _first(table, "table")
    n = _vector(tokens, "tokens", None, dev)
    if out is None:
        out = torch.empty((n, dim), dtype=table.dtype, device=table.device)
    out_ld = _matrix(out, "out", n, dim, dev)
    _call(lib.embed_lookup, "embed_lookup", dev, table.data_ptr(), _type_code(table, "table"),
          vocab, dim, ld, tokens.data_ptr(), _type_code(tokens, "tokens", (3, 4)), n, scale,
          out.data_ptr(), _type_code(out, "out"), out_ld)
    _wrote((out,))
    return out


class EmbedPlan:
    """Positions ordered by token (embed_sort): the plan's words and the
    sizes they belong to."""

    def __init__(self, words, n: int, vocab: int):
        self.words, self.n, self.vocab = words, n, vocab


def embed_sort(tokens, vocab: int, plan=None) -> EmbedPlan:
    """The plan of a batch's tokens for embed_grad and embed_grad_rows.  A
    plan of as many tokens is overwritten if given."""
    lib, torch = _lm(), _torch
    dev = _on(tokens, "tokens")
    n = _vector(tokens, "tokens", None, dev)
    if plan is None:
        plan = EmbedPlan(torch.empty(lib.embed_plan_words(n), dtype=torch.int32,
                                     device=tokens.device), n, vocab)
    elif plan.n != n:
        raise ValueError(f"the plan given is for {plan.n} tokens, not {n}")
    _vector(plan.words, "plan", lib.embed_plan_words(n), dev, torch.int32, at_least=True)
    _call(lib.embed_sort, "embed_sort", dev, tokens.data_ptr(),
          _type_code(tokens, "tokens", (3, 4)), n, vocab, plan.words.data_ptr())
    plan.vocab = vocab
    _wrote((plan.words,))
    return plan


def _embed_grad_args(lib, grad, plan, work):
    """The checks embed_grad and embed_grad_rows share; (device, row length,
    distance of the gradient's rows, workspace)."""
    torch = _torch
    dev, rows, dim, ld = _first(grad, "grad")
    if not isinstance(plan, EmbedPlan):
        raise TypeError("plan must be an EmbedPlan (embed_sort)")
    if rows != plan.n:
        raise ValueError(f"grad has {rows} rows, the plan {plan.n} tokens")
    _vector(plan.words, "plan", lib.embed_plan_words(plan.n), dev, torch.int32, at_least=True)
    need = lib.embed_work_bytes(plan.n, dim)
    if work is None:
        work = torch.empty(need, dtype=torch.uint8, device=grad.device)
    else:
        _vector(work, "work", need, dev, torch.uint8, at_least=True)
    return dev, dim, ld, work


def embed_grad(grad, plan: EmbedPlan, scale: float = 1.0, out=None, accumulate: bool = False,
               work=None):
    """The table's gradient, float32: out[v] = scale * (sum of grad[i] over
    the positions i of token v), zero where no token is; with ``accumulate``
    it is added to out instead."""
    lib, torch = _lm(), _torch
    dev, dim, ld, work = _embed_grad_args(lib, grad, plan, work)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = torch.empty((plan.vocab, dim), dtype=torch.float32, device=grad.device)
    out_ld = _matrix(out, "out", plan.vocab, dim, dev)
    _type_code(out, "out", (0,))
    _call(lib.embed_grad, "embed_grad", dev, grad.data_ptr(), _type_code(grad, "grad"), ld,
          plan.words.data_ptr(), plan.n, plan.vocab, dim, scale, accumulate, out.data_ptr(), out_ld,
          work.data_ptr())
    _wrote((out,))
    return out


def embed_grad_rows(grad, plan: EmbedPlan, scale: float = 1.0, ids=None, rows=None, count=None,
                    work=None):
    """The same gradient in row-sparse form: (ids int32, rows float32, count
    int32[1]).  The first ``count`` ids are the batch's different tokens in
    ascending order and the same rows their gradients; what is behind them is
    left as it was.  ids and rows hold at least min(n, vocab) entries."""
    lib, torch = _lm(), _torch
    dev, dim, ld, work = _embed_grad_args(lib, grad, plan, work)
    most = min(plan.n, plan.vocab)
    if ids is None:
        ids = torch.empty(most, dtype=torch.int32, device=grad.device)
    if rows is None:
        rows = torch.empty((most, dim), dtype=torch.float32, device=grad.device)
    if count is None:
        count = torch.empty(1, dtype=torch.int32, device=grad.device)
    _vector(ids, "ids", most, dev, torch.int32, at_least=True)
    _vector(count, "count", 1, dev, torch.int32)
    rows_ld = _matrix(rows, "rows", most, dim, dev, written=True)
    _type_code(rows, "rows", (0,))
    _call(lib.embed_grad_rows, "embed_grad_rows", dev, grad.data_ptr(), _type_code(grad, "grad"),
          ld, plan.words.data_ptr(), plan.n, plan.vocab, dim, scale, ids.data_ptr(),
          rows.data_ptr(), rows_ld, count.data_ptr(), work.data_ptr())
    _wrote((ids, rows, count))
    return ids, rows, count


def rms_norm_work_bytes(rows: int, dim: int, dtype) -> int:
    return int(_lm().rms_norm_work_bytes(rows, dim, _type_codes.get(dtype, -1)))


def _rms_args(x, weight, residual, h, rstd):
    """The checks rms_norm and rms_norm_q8 share; (device, rows, dim, type,
    arguments of x and the residual, arguments of the weight, h, its
    arguments, rstd)."""
    torch = _torch
    dev, rows, dim, ld = _first(x, "x")
    kind = _type_code(x, "x")
    res, res_ld, h_at, h_ld = None, 0, None, 0
    if residual is not None:
        res_ld = _matrix(residual, "residual", rows, dim, dev)
        _type_code(residual, "residual", (kind,))
        res = residual.data_ptr()
        if h is residual:
            h_at, h_ld = res, res_ld
        else:
            if h is None:
                h = torch.empty((rows, dim), dtype=x.dtype, device=x.device)
            h_ld = _matrix(h, "h", rows, dim, dev)
            _type_code(h, "h", (kind,))
            h_at = h.data_ptr()
    elif h is not None:
        raise ValueError("h is x itself without a residual")
    _vector(weight, "weight", dim, dev)
    if rstd is None:
        rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
    else:
        _vector(rstd, "rstd", rows, dev, torch.float32)
    return (dev, rows, dim, kind, (x.data_ptr(), kind, rows, dim, ld, res, res_ld, weight.data_ptr(),
                                   _type_code(weight, "weight", (kind, 0))),
            x if residual is None else h, (h_at, h_ld, rstd.data_ptr()), rstd)


def rms_norm(x, weight, eps: float, residual=None, y=None, h=None, rstd=None):
    """Root-mean-square norm of x (+ residual), times weight: returns (y, h,
    rstd).  h is the sum, rounded to x's type (x itself without a residual;
    it may be given as the residual, which is then updated), rstd what
    rms_norm_grad needs."""
    lib, torch = _lm(), _torch
    dev, rows, dim, kind, args, h, tail, rstd = _rms_args(x, weight, residual, h, rstd)
    if y is None:
        y = torch.empty((rows, dim), dtype=x.dtype, device=x.device)
    y_ld = _matrix(y, "y", rows, dim, dev)
    _type_code(y, "y", (kind,))
    _call(lib.rms_norm, "rms_norm", dev, *args, eps, y.data_ptr(), y_ld, *tail)
    _wrote((y, rstd) if residual is None else (y, rstd, h))
    return y, h, rstd


def rms_norm_q8(x, weight, eps: float, group: int = 128, residual=None, codes=None, scales=None,
                h=None, rstd=None):
    """rms_norm with y as e4m3 codes (torch.float8_e4m3fn) and a float32 scale
    per group of 32, 64 or 128 columns (group 0: per row): y is about code *
    scale.  Returns (codes, scales [rows, groups], h, rstd)."""
    lib, torch = _lm(), _torch
    dev, rows, dim, _, args, h, tail, rstd = _rms_args(x, weight, residual, h, rstd)
    if group not in (0, 32, 64, 128):
        raise ValueError(f"group must be 0, 32, 64 or 128 (got {group})")
    parts = -(-dim // group) if group else 1
    if codes is None:
        codes = torch.empty((rows, dim), dtype=torch.float8_e4m3fn, device=x.device)
    if scales is None:
        scales = torch.empty((rows, parts), dtype=torch.float32, device=x.device)
    codes_ld = _matrix(codes, "codes", rows, dim, dev)
    if codes.dtype not in (torch.float8_e4m3fn, torch.uint8):
        raise TypeError(f"codes must be float8_e4m3fn or uint8 (got {codes.dtype})")
    _vector(scales, "scales", rows * parts, dev, torch.float32)
    _call(lib.rms_norm_q8, "rms_norm_q8", dev, *args, eps, group, codes.data_ptr(), codes_ld,
          scales.data_ptr(), *tail)
    _wrote((codes, scales, rstd) if residual is None else (codes, scales, rstd, h))
    return codes, scales, h, rstd


def rms_norm_grad(dy, h, weight, rstd, dh=None, dx=None, dweight=None, accumulate: bool = False,
                  work=None):
    """Gradients of rms_norm for dy (and dh, the gradient that reaches h
    otherwise): returns (dx, dweight).  dx is the gradient of x and of the
    residual; it may be given as dh.  dweight is float32; with ``accumulate``
    it is added to."""
    lib, torch = _lm(), _torch
    dev, rows, dim, ld = _first(dy, "dy")
    kind = _type_code(dy, "dy")
    h_ld = _matrix(h, "h", rows, dim, dev)
    _type_code(h, "h", (kind,))
    _vector(weight, "weight", dim, dev)
    _vector(rstd, "rstd", rows, dev, torch.float32)
    dh_at, dh_ld = None, 0
    if dh is not None:
        _type_code(dh, "dh", (kind,))
        dh_at, dh_ld = dh.data_ptr(), _matrix(dh, "dh", rows, dim, dev)
    if dx is None:
        dx = torch.empty((rows, dim), dtype=dy.dtype, device=dy.device)
    dx_ld = _matrix(dx, "dx", rows, dim, dev)
    _type_code(dx, "dx", (kind,))
    if dweight is None:
        if accumulate:
            raise ValueError("accumulate needs dweight")
        dweight = torch.empty(dim, dtype=torch.float32, device=dy.device)
    _vector(dweight, "dweight", dim, dev, torch.float32)
    need = lib.rms_norm_work_bytes(rows, dim, kind)
    if work is None:
        work = torch.empty(need, dtype=torch.uint8, device=dy.device)
    else:
        _vector(work, "work", need, dev, torch.uint8, at_least=True)
    _call(lib.rms_norm_grad, "rms_norm_grad", dev, dy.data_ptr(), kind, rows, dim, ld, h.data_ptr(),
          h_ld, weight.data_ptr(), _type_code(weight, "weight", (kind, 0)), rstd.data_ptr(), dh_at,
          dh_ld, dx.data_ptr(), dx_ld, dweight.data_ptr(), accumulate, work.data_ptr())
    _wrote((dx, dweight))
    return dx, dweight


def _distill_args(logits, index, teacher, temperature, row_scale, scale):
    """The checks the three calls share; (device, rows, vocab, type, the
    logits' arguments, the arguments behind them)."""
    dev, rows, vocab, ld = _first(logits, "logits")
    kind = _type_code(logits, "logits")
    _on(index, "index", dev)
    k = index.shape[-1] if index.dim() else 0
    idx_ld = _matrix(index, "index", rows, k, dev)
    top_ld = _matrix(teacher, "teacher", rows, k, dev)
    if row_scale is not None:
        _vector(row_scale, "row_scale", rows, dev, _torch.float32)
    return (dev, rows, vocab, kind, (logits.data_ptr(), kind, rows, vocab, ld),
            (index.data_ptr(), _type_code(index, "index", (3, 4)), idx_ld, teacher.data_ptr(),
             _type_code(teacher, "teacher", (kind, 0)), top_ld, k, temperature,
             None if row_scale is None else row_scale.data_ptr(), scale))


def _row_floats(x, name, rows, dev, like):
    """A float32 vector of a value per row, new if none is given."""
    torch = _torch
    if x is None:
        return torch.empty(rows, dtype=torch.float32, device=like.device)
    _vector(x, name, rows, dev, torch.float32)
    return x


def _dlogits(out, logits, rows, vocab, kind, dev):
    torch = _torch
    if out is None:
        out = torch.empty((rows, vocab), dtype=logits.dtype, device=logits.device)
    _type_code(out, "out", (kind,))
    return out, _matrix(out, "out", rows, vocab, dev)


def distill_loss(logits, index, teacher, temperature: float = 1.0, row_scale=None,
                 scale: float = 1.0, loss=None, lse=None):
    """Distillation from a teacher's top logits: returns (loss, lse), float32
    per row.  ``index`` and ``teacher`` are [rows, k]: the teacher's entries
    and their logits (an index outside the vocabulary marks an absent one).
    loss = s * KL(softmax(teacher / T) || softmax(logits / T)), the student's
    softmax over the whole vocabulary, s = scale * row_scale; rows with s = 0
    are not read."""
    lib = _lm()
    dev, rows, _, _, head, tail = _distill_args(logits, index, teacher, temperature, row_scale, scale)
    loss = _row_floats(loss, "loss", rows, dev, logits)
    lse = _row_floats(lse, "lse", rows, dev, logits)
    _call(lib.distill_loss, "distill_loss", dev, *head, *tail, loss.data_ptr(), lse.data_ptr())
    _wrote((loss, lse))
    return loss, lse


def distill_grad(logits, lse, index, teacher, temperature: float = 1.0, row_scale=None,
                 scale: float = 1.0, out=None):
    """The gradient of sum(loss) in the logits, from distill_loss's lse;
    ``row_scale`` may carry the gradient from above.  out may be the logits."""
    lib, torch = _lm(), _torch
    dev, rows, vocab, kind, head, tail = _distill_args(logits, index, teacher, temperature, row_scale,
                                                       scale)
    _vector(lse, "lse", rows, dev, torch.float32)
    out, ld = _dlogits(out, logits, rows, vocab, kind, dev)
    _call(lib.distill_grad, "distill_grad", dev, *head, lse.data_ptr(), *tail, out.data_ptr(), ld)
    _wrote((out,))
    return out


def distill_loss_grad(logits, index, teacher, temperature: float = 1.0, row_scale=None,
                      scale: float = 1.0, loss=None, lse=None, out=None):
    """distill_loss and distill_grad in one launch: (loss, lse, dlogits).  out
    may be the logits, which it then replaces."""
    lib = _lm()
    dev, rows, vocab, kind, head, tail = _distill_args(logits, index, teacher, temperature, row_scale,
                                                       scale)
    loss = _row_floats(loss, "loss", rows, dev, logits)
    lse = _row_floats(lse, "lse", rows, dev, logits)
    out, ld = _dlogits(out, logits, rows, vocab, kind, dev)
    _call(lib.distill_loss_grad, "distill_loss_grad", dev, *head, *tail, loss.data_ptr(),
          lse.data_ptr(), out.data_ptr(), ld)
    _wrote((loss, lse, out))
    return loss, lse, out
