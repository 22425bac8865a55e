"""Binding of the paged-cache operators: block tables and slot maps
(hga_paged_plan), per-head norms with the position rotation and its gradient
(hga_qk_norm_rope, hga_qk_norm_rope_backward), and attention of one new token
over the pages (hga_paged_decode).

A serving step of a layer that attends over every cached token (or a window):

    plan = hga_paged_plan(cache.lens, new_tokens, cache.free_pages, cache.free_count,
                          cache.block_table, cache.page_size, n_slots,
                          lens_out=cache.lens, free_count_out=cache.free_count)
    q, _, _ = hga_qk_norm_rope(q, k, v, plan["pos"], rope, q_weight=wq, k_weight=wk,
                               k_pages=cache.k_pages, v_pages=cache.v_pages, slot=plan["slot"])
    out = hga_paged_decode(q, cache.k_pages, cache.v_pages, cache.block_table, cache.lens)

As in the rest of the package, these functions check their tensors, pass pointers
and raise HGAError on a refusal; they never synchronise.  With `stream`, tensors
that a call allocates are recorded on that stream.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional

import torch

from . import HGAError, _aligned_span, _check, _dtype_code, _F32, _need, _stream, load

# A small step's call is bound by its host side, so the checks below read each
# attribute of a tensor once and leave the wording of a refusal to _need.

_I32 = torch.int32
_P = ctypes.c_void_p
_LAYOUTS = {"half": 0, "interleaved": 1}
_SCALINGS = {"none": 0, "linear": 1, "yarn": 2}


class _PagedDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "Hq", "Hkv", "D", "dtype", "num_pages",
                                              "page_size", "max_pages")]


class _PlanIO(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("lens", "new_tokens", "release", "free_pages", "free_count",
                                  "block_table", "lens_out", "free_count_out", "cu_tokens",
                                  "granted", "slot", "pos")]


class _Rope(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("layout", "rotary_dim", "scaling", "original_len")]
                + [(n, ctypes.c_double) for n in ("theta", "factor", "beta_fast", "beta_slow",
                                                  "magnitude")])


class _QkIO(ctypes.Structure):
    _fields_ = ([(n, _P) for n in ("q", "k", "v")]
                + [(n, ctypes.c_int64) for n in ("q_stride", "k_stride", "v_stride")]
                + [("q_weight", _P), ("k_weight", _P), ("eps", ctypes.c_double)]
                + [(n, _P) for n in ("pos", "q_out", "k_out", "v_out", "slot", "k_pages",
                                     "v_pages")]
                + [("num_slots", ctypes.c_int64)])


class _QkGradIO(ctypes.Structure):
    _fields_ = ([("q", _P), ("k", _P), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                 ("q_weight", _P), ("k_weight", _P), ("eps", ctypes.c_double), ("pos", _P),
                 ("d_q", _P), ("d_k", _P), ("d_v", _P), ("grad_dtype", ctypes.c_int32),
                 ("dq", _P), ("dk", _P), ("dv", _P)]
                + [(n, ctypes.c_int64) for n in ("dq_stride", "dk_stride", "dv_stride")]
                + [("d_q_weight", _P), ("d_k_weight", _P)])


class _TokenDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "Hq", "Hkv", "D", "dtype")]


def declare(lib):
    """The argument types of the entry points, set when the library is loaded."""
    sz, i32 = ctypes.c_size_t, ctypes.c_int32
    lib.hga_paged_plan.argtypes = [_P, _P, i32, _P, sz, _P]
    lib.hga_qk_norm_rope.argtypes = [_P, _P, _P, _P]
    lib.hga_qk_norm_rope_backward.argtypes = [_P, _P, _P, _P, sz, _P]
    lib.hga_paged_decode.argtypes = [_P, _P, _P, _P, _P, _P, i32, i32, ctypes.c_double, _P, _P, _P,
                                     sz, _P]
    for f in ("hga_paged_plan", "hga_qk_norm_rope", "hga_qk_norm_rope_backward",
              "hga_paged_decode"):
        getattr(lib, f).restype = ctypes.c_int
    lib.hga_paged_plan_workspace.argtypes = [i32, i32]
    lib.hga_qk_norm_rope_backward_workspace.argtypes = [_P]
    lib.hga_paged_decode_workspace.argtypes = [_P]
    for f in ("hga_paged_plan_workspace", "hga_qk_norm_rope_backward_workspace",
              "hga_paged_decode_workspace"):
        getattr(lib, f).restype = sz


class HGARope(NamedTuple):
    """A position rotation (hga_rope in include/hga.h).  rotary_dim None: the
    whole head; 0: none.  layout "half" (pairs i, i + R/2) or "interleaved"
    (2i, 2i + 1).  scaling "none", "linear" or "yarn" (factor; for yarn also
    original_len, beta_fast, beta_slow).  magnitude 0: 1, for yarn
    0.1 ln(factor) + 1."""
    rotary_dim: Optional[int] = None
    theta: float = 1e6
    layout: str = "half"
    scaling: str = "none"
    factor: float = 1.0
    original_len: int = 0
    beta_fast: float = 32.0
    beta_slow: float = 1.0
    magnitude: float = 0.0

    def c(self, D: int) -> _Rope:
        if self.layout not in _LAYOUTS:
            raise HGAError(f"layout {self.layout!r}: one of {sorted(_LAYOUTS)}")
        if self.scaling not in _SCALINGS:
            raise HGAError(f"scaling {self.scaling!r}: one of {sorted(_SCALINGS)}")
        return _Rope(_LAYOUTS[self.layout], D if self.rotary_dim is None else self.rotary_dim,
                     _SCALINGS[self.scaling], self.original_len, self.theta, self.factor,
                     self.beta_fast, self.beta_slow, self.magnitude)


class PagedKVCache:
    """The buffers of a paged cache (caller-owned device memory): the page
    pools, the block table of up to B sequences of max_pages pages each, their
    lengths, and the stack of free pages."""

    def __init__(self, B: int, num_pages: int, page_size: int, max_pages: int, Hkv: int, D: int,
                 dtype, device="cuda"):
        z = dict(device=device)
        self.page_size = page_size
        self.k_pages = torch.zeros(num_pages, page_size, Hkv, D, dtype=dtype, **z)
        self.v_pages = torch.zeros(num_pages, page_size, Hkv, D, dtype=dtype, **z)
        self.block_table = torch.full((B, max_pages), -1, dtype=_I32, **z)
        self.lens = torch.zeros(B, dtype=_I32, **z)
        self.free_pages = torch.arange(num_pages - 1, -1, -1, dtype=_I32, **z)
        self.free_count = torch.full((1,), num_pages, dtype=_I32, **z)


@functools.lru_cache(maxsize=64)
def _rope(rope: HGARope, D: int) -> _Rope:
    return rope.c(D)


_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") \
    else lambda index: torch.cuda.current_stream(index).cuda_stream


def _launch(what, fn, dev, stream, *args):
    """fn(*args, stream) with the call's device current."""
    st = _raw_stream(dev.index) if stream is None else _stream(stream, dev)
    if torch.cuda.current_device() == dev.index:
        status = fn(*args, st)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, st)
    if status:
        _check(status, what)


def _new(shape, dtype, dev, stream):
    t = torch.empty(shape, dtype=dtype, device=dev)
    if stream is not None:
        t.record_stream(stream)       # freed by the caller before `stream` is done with it
    return t


def _work(nbytes, dev, workspace, stream):
    """(tensor kept for the call, aligned address, bytes from there)."""
    if workspace is None:
        workspace = _new(nbytes + 256, torch.uint8, dev, stream)
        base = (workspace.data_ptr() + 255) & -256
        return workspace, base, nbytes
    _need(workspace, "workspace", device=dev)
    return (workspace,) + _aligned_span(workspace.data_ptr(),
                                        workspace.numel() * workspace.element_size(), nbytes)


def _dense(t, name, shape, dtype, dev):
    """The address of a contiguous tensor of that shape, type and device."""
    if type(t) is not torch.Tensor or t.dtype is not dtype or t.shape != shape \
            or t.get_device() != dev.index or not t.is_contiguous():
        _need(t, name, shape, dtype, dev)
    return t.data_ptr()


def _ints(t, name, shape, dev):
    return _dense(t, name, shape, _I32, dev)


def _token_stride(t, name, lead, H, D, dtype, dev):
    """Elements between the tokens of [tokens, H, D] or [B, T, H, D]: rows of D
    adjacent, heads D apart, tokens evenly spaced (a view of a fused buffer)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise HGAError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev.index:
        raise HGAError(f"{name} is on {t.device}, the call's tensors are on {dev}")
    if t.dtype is not dtype:
        raise HGAError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != lead + (H, D):
        raise HGAError(f"{name} has shape {tuple(t.shape)}, expected {tuple(lead + (H, D))}")
    s = t.stride()
    if s[-1] != 1 or (H > 1 and s[-2] != D):
        raise HGAError(f"{name}: heads must be adjacent rows of {D} (strides {s})")
    if len(lead) == 2:
        B, T = lead
        if B > 1 and T > 1 and s[0] != T * s[1]:
            raise HGAError(f"{name}: tokens must be evenly spaced (strides {s})")
        step = s[1] if T > 1 else s[0] if B > 1 else H * D
    else:
        step = s[0] if lead[0] > 1 else H * D
    return step


def hga_paged_plan(lens, new_tokens, free_pages, free_count, block_table, page_size: int,
                   n_slots: int, *, release=None, lens_out=None, free_count_out=None,
                   cu_tokens=None, granted=None, slot=None, pos=None, workspace=None, stream=None):
    """Block table, slot map and positions of one step from the sequences'
    lengths (include/hga.h has the rules).  lens, new_tokens, release [B],
    free_pages [num_pages], free_count [1], block_table [B, max_pages], all
    int32.  New pages are written into block_table (and, with release, freed
    ones onto free_pages); lens_out and free_count_out may be lens and
    free_count.  Returns dict(lens, free_count, cu_tokens [B+1], granted [B],
    slot [n_slots], pos [n_slots])."""
    lib = load()
    _need(block_table, "block_table", dtype=_I32)
    if block_table.dim() != 2:
        raise HGAError("block_table must be [B, max_pages]")
    dev = block_table.device
    B, max_pages = block_table.shape
    _count(n_slots, "n_slots")
    _count(page_size, "page_size")
    _need(free_pages, "free_pages", dtype=_I32, device=dev)
    P = free_pages.numel()
    given = (lens_out, free_count_out, cu_tokens, granted, slot, pos)
    sizes = (B, 1, B + 1, B, n_slots, n_slots)
    if any(t is None for t in given):
        # one allocation for what the caller does not bring
        new = _new(sum(n for t, n in zip(given, sizes) if t is None), _I32, dev, stream)
        parts = iter(new.split([n for t, n in zip(given, sizes) if t is None]))
        lens_out, free_count_out, cu_tokens, granted, slot, pos = (
            next(parts) if t is None else t for t in given)
    ptr = [t.data_ptr() if g is None else _ints(t, name, (n,), dev) for t, g, n, name in zip(
        (lens_out, free_count_out, cu_tokens, granted, slot, pos), given, sizes,
        ("lens_out", "free_count_out", "cu_tokens", "granted", "slot", "pos"))]
    io = _PlanIO(_ints(lens, "lens", (B,), dev), _ints(new_tokens, "new_tokens", (B,), dev),
                 None if release is None else _ints(release, "release", (B,), dev),
                 free_pages.data_ptr(), _ints(free_count, "free_count", (1,), dev),
                 block_table.data_ptr(), *ptr)
    dims = _PagedDims(B, 0, 0, 0, 0, P, page_size, max_pages)
    ws, base, avail = _work(lib.hga_paged_plan_workspace(B, n_slots), dev, workspace, stream)
    _launch("hga_paged_plan", lib.hga_paged_plan, dev, stream, ctypes.byref(dims),
            ctypes.byref(io), n_slots, base, avail)
    return dict(lens=lens_out, free_count=free_count_out, cu_tokens=cu_tokens, granted=granted,
                slot=slot, pos=pos)


def _count(x, name):
    """A count that fits the C interface's int32 (ctypes would wrap a larger one)."""
    if not 0 <= x < 1 << 31:
        raise HGAError(f"{name} is {x}, expected 0 .. 2^31 - 1")
    return x


def _lead(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() not in (3, 4):
        raise HGAError(f"{name} must be [tokens, H, D] or [B, T, H, D]")
    return t.shape[:-2], t.shape[-2], t.shape[-1]


def _tokens(lead):
    return lead if len(lead) == 2 else (1, lead[0])


def hga_qk_norm_rope(q, k, v, pos, rope: HGARope, *, q_weight=None, k_weight=None,
                     eps: float = 1e-6, k_pages=None, v_pages=None, slot=None, q_out=None,
                     k_out=None, v_out=None, stream=None):
    """Per-head RMS norms of q and k (each where its weight [D] is given) and
    the rotation at pos, in one pass.  q [tokens, Hq, D] or [B, T, Hq, D], k and
    v with Hkv heads: dense, or views of a fused QKV buffer.  pos: int32 of the
    leading shape (None with rotary_dim 0).  With k_pages, v_pages
    [num_pages, page_size, Hkv, D] and slot (int32, leading shape; -1: not
    written), keys and values go to the pages, and to k_out and v_out only where
    these are given; without them, to new dense tensors.  v may be None.
    Returns (q_out, k_out, v_out)."""
    lib = load()
    lead, Hq, D = _lead(q, "q")
    _, Hkv, _ = _lead(k, "k")
    dev, dt = q.device, q.dtype
    code = _dtype_code(q)
    qs = _token_stride(q, "q", lead, Hq, D, dt, dev)
    ks = _token_stride(k, "k", lead, Hkv, D, dt, dev)
    vs = 0 if v is None else _token_stride(v, "v", lead, Hkv, D, dt, dev)
    paged = k_pages is not None or v_pages is not None
    if paged and (k_pages is None or (v_pages is None) != (v is None) or slot is None):
        raise HGAError("k_pages, v_pages (with v) and slot come together")
    if q_out is None:
        q_out = _new(lead + (Hq, D), dt, dev, stream)
    if not paged and k_out is None:
        k_out = _new(lead + (Hkv, D), dt, dev, stream)
    if not paged and v is not None and v_out is None:
        v_out = _new(lead + (Hkv, D), dt, dev, stream)
    if v is None and v_out is not None:
        raise HGAError("v_out without v")
    kv = lead + (Hkv, D)
    num_slots = 0
    if paged:
        if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
            raise HGAError("k_pages must be [num_pages, page_size, Hkv, D]")
        shape = k_pages.shape[:2] + (Hkv, D)
        num_slots = shape[0] * shape[1]
        _dense(k_pages, "k_pages", shape, dt, dev)
        if v_pages is not None:
            _dense(v_pages, "v_pages", shape, dt, dev)
    r = _rope(rope, D)
    if pos is None and r.rotary_dim:
        raise HGAError("pos is needed with a rotation")
    io = _QkIO(q.data_ptr(), k.data_ptr(), None if v is None else v.data_ptr(), qs, ks, vs,
               None if q_weight is None else _dense(q_weight, "q_weight", (D,), dt, dev),
               None if k_weight is None else _dense(k_weight, "k_weight", (D,), dt, dev), eps,
               None if pos is None else _ints(pos, "pos", lead, dev),
               _dense(q_out, "q_out", lead + (Hq, D), dt, dev),
               None if k_out is None else _dense(k_out, "k_out", kv, dt, dev),
               None if v_out is None else _dense(v_out, "v_out", kv, dt, dev),
               _ints(slot, "slot", lead, dev) if paged else None,
               k_pages.data_ptr() if paged else None,
               v_pages.data_ptr() if v_pages is not None else None, num_slots)
    dims = _TokenDims(*_tokens(lead), Hq, Hkv, D, code)
    _launch("hga_qk_norm_rope", lib.hga_qk_norm_rope, dev, stream, ctypes.byref(dims),
            ctypes.byref(r), ctypes.byref(io))
    return q_out, k_out, v_out


def hga_qk_norm_rope_backward(q, k, d_q, d_k, pos, rope: HGARope, *, q_weight=None, k_weight=None,
                              eps: float = 1e-6, d_v=None, dq=None, dk=None, dv=None,
                              workspace=None, stream=None):
    """Gradients of hga_qk_norm_rope.  q, k, pos, rope, weights and eps as in the
    forward; d_q, d_k (and d_v) the dense gradients of its dense outputs, fp32
    (as hga_attend_backward gives them) or in q's dtype.  dq, dk, dv may be
    views of one fused buffer.  Returns (dq, dk, dv, dq_weight, dk_weight): dq,
    dk, dv in q's dtype (dv None without d_v), the weights' gradients fp32 [D]
    (None without the weight)."""
    lib = load()
    lead, Hq, D = _lead(q, "q")
    _, Hkv, _ = _lead(k, "k")
    dev, dt = q.device, q.dtype
    code = _dtype_code(q)
    qs = _token_stride(q, "q", lead, Hq, D, dt, dev)
    ks = _token_stride(k, "k", lead, Hkv, D, dt, dev)
    if not isinstance(d_q, torch.Tensor) or d_q.dtype not in (torch.float32, dt):
        raise HGAError(f"d_q must be a float32 or {dt} tensor")
    gt = d_q.dtype
    if (d_v is None) and dv is not None:
        raise HGAError("dv without d_v")
    kv = lead + (Hkv, D)
    dq = _new(lead + (Hq, D), dt, dev, stream) if dq is None else dq
    dk = _new(kv, dt, dev, stream) if dk is None else dk
    dv = _new(kv, dt, dev, stream) if dv is None and d_v is not None else dv
    dqw = None if q_weight is None else _new(D, torch.float32, dev, stream)
    dkw = None if k_weight is None else _new(D, torch.float32, dev, stream)
    r = _rope(rope, D)
    if pos is None and r.rotary_dim:
        raise HGAError("pos is needed with a rotation")
    io = _QkGradIO(q.data_ptr(), k.data_ptr(), qs, ks,
                   None if q_weight is None else _dense(q_weight, "q_weight", (D,), dt, dev),
                   None if k_weight is None else _dense(k_weight, "k_weight", (D,), dt, dev), eps,
                   None if pos is None else _ints(pos, "pos", lead, dev),
                   _dense(d_q, "d_q", lead + (Hq, D), gt, dev), _dense(d_k, "d_k", kv, gt, dev),
                   None if d_v is None else _dense(d_v, "d_v", kv, gt, dev),
                   _F32 if gt is torch.float32 else code,
                   dq.data_ptr(), dk.data_ptr(), None if dv is None else dv.data_ptr(),
                   _token_stride(dq, "dq", lead, Hq, D, dt, dev),
                   _token_stride(dk, "dk", lead, Hkv, D, dt, dev),
                   0 if dv is None else _token_stride(dv, "dv", lead, Hkv, D, dt, dev),
                   None if dqw is None else dqw.data_ptr(), None if dkw is None else dkw.data_ptr())
    dims = _TokenDims(*_tokens(lead), Hq, Hkv, D, code)
    ws, base, avail = _work(lib.hga_qk_norm_rope_backward_workspace(ctypes.byref(dims)), dev,
                            workspace, stream)
    _launch("hga_qk_norm_rope_backward", lib.hga_qk_norm_rope_backward, dev, stream,
            ctypes.byref(dims), ctypes.byref(r), ctypes.byref(io), base, avail)
    return dq, dk, dv, dqw, dkw


def hga_paged_decode(q, k_pages, v_pages, block_table, lens, *, window: int = 0, sinks: int = 0,
                     scale: float = 0.0, out=None, want_lse: bool = False, lse=None,
                     workspace=None, stream=None):
    """Attention of one new token per sequence over its pages.  q [B, Hq, D]
    (rotated), k_pages and v_pages [num_pages, page_size, Hkv, D], block_table
    [B, max_pages] and lens [B] int32 (the new token's key and value already
    written, lens counting it).  window > 0: only the last `window` tokens and
    the first `sinks` are visible.  scale 0: 1/sqrt(D).  -> out [B, Hq, D] (and
    lse [B, Hq] fp32 when asked)."""
    lib = load()
    _need(q, "q")
    if q.dim() != 3:
        raise HGAError("q must be [B, Hq, D]")
    B, Hq, D = q.shape
    dev, dt = q.device, q.dtype
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
        raise HGAError("k_pages must be [num_pages, page_size, Hkv, D]")
    P, page, Hkv, _ = k_pages.shape
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise HGAError("block_table must be [B, max_pages]")
    max_pages = block_table.shape[1]
    if out is None:
        out = _new((B, Hq, D), dt, dev, stream)
    if lse is None and want_lse:
        lse = _new((B, Hq), torch.float32, dev, stream)
    dims = _PagedDims(B, Hq, Hkv, D, _dtype_code(q), P, page, max_pages)
    nbytes = lib.hga_paged_decode_workspace(ctypes.byref(dims))
    ws, base, avail = _work(nbytes, dev, workspace, stream)
    pages = (P, page, Hkv, D)
    _launch("hga_paged_decode", lib.hga_paged_decode, dev, stream, ctypes.byref(dims),
            q.data_ptr(), _dense(k_pages, "k_pages", pages, dt, dev),
            _dense(v_pages, "v_pages", pages, dt, dev),
            _ints(block_table, "block_table", (B, max_pages), dev), _ints(lens, "lens", (B,), dev),
            _count(window, "window"), _count(sinks, "sinks"), scale,
            _dense(out, "out", (B, Hq, D), dt, dev),
            None if lse is None else _dense(lse, "lse", (B, Hq), torch.float32, dev), base, avail)
    return (out, lse) if lse is not None else out
