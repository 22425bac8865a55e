"""The paged-cache operators: block tables and slot maps (hga_paged_plan),
per-head norms with the position rotation and its gradient (hga_qk_norm_rope,
hga_qk_norm_rope_backward), and attention of one new token over the pages
(hga_paged_decode).

A serving step of a layer that attends over every cached token (or a window), with
one new token in every row, so that row b of q is sequence b (the attention takes one
token a sequence: plan and norms lay out whole prompts, but attention of a prompt over
pages is not among these operators):

    plan = hga_paged_plan(cache.lens, new_tokens, cache.free_pages, cache.free_count,
                          cache.block_table, cache.page_size, n_slots,
                          lens_out=cache.lens, free_count_out=cache.free_count)
    q, _, _ = hga_qk_norm_rope(q, k, v, plan["pos"], rope, q_weight=wq, k_weight=wk,
                               k_pages=cache.k_pages, v_pages=cache.v_pages, slot=plan["slot"])
    out = hga_paged_decode(q, cache.k_pages, cache.v_pages, cache.block_table, cache.lens)

As in the rest of the package, these functions check their tensors, pass pointers
to the C ABI and raise HGAError on a refusal; they never synchronise.  The checks
and the marshalling are compiled (csrc/binding.cpp, module _paged).  With `stream`,
tensors that a call allocates belong to that stream, as if allocated under
torch.cuda.stream(stream).
"""
from __future__ import annotations

import importlib
import os
from typing import NamedTuple, Optional

import torch

from . import HGAError, load

_ext = None


def _module():
    """The compiled binding (raises if it has not been built)."""
    global _ext
    if _ext is None:
        load()                        # reports a missing library first
        if not os.path.exists(os.path.join(os.path.dirname(os.path.abspath(__file__)), "_paged.so")):
            raise HGAError("_paged.so is missing: build it with "
                           "hierarchical_kv_routing_b200._build.build()")
        ext = importlib.import_module("hierarchical_kv_routing_b200._paged")
        ext.set_errors(HGAError, torch.cuda.OutOfMemoryError)
        _ext = ext
    return _ext


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


class PagedKVCache:
    """The buffers of a paged cache (caller-owned device memory): the page
    pools, the block table of up to B sequences of max_pages pages each, their
    lengths, and the stack of free pages."""

    def __init__(self, B: int, num_pages: int, page_size: int, max_pages: int, Hkv: int, D: int,
                 dtype, device="cuda"):
        z = dict(device=device)
        i = dict(dtype=torch.int32, **z)
        self.page_size = page_size
        self.k_pages = torch.zeros(num_pages, page_size, Hkv, D, dtype=dtype, **z)
        self.v_pages = torch.zeros(num_pages, page_size, Hkv, D, dtype=dtype, **z)
        self.block_table = torch.full((B, max_pages), -1, **i)
        self.lens = torch.zeros(B, **i)
        self.free_pages = torch.arange(num_pages - 1, -1, -1, **i)
        self.free_count = torch.full((1,), num_pages, **i)


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
    return (_ext or _module()).plan(lens, new_tokens, free_pages, free_count, block_table, page_size,
                                    n_slots, release, lens_out, free_count_out, cu_tokens, granted,
                                    slot, pos, workspace, stream)


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
    return (_ext or _module()).qk(q, k, v, pos, rope, q_weight, k_weight, eps, k_pages, v_pages, slot,
                                  q_out, k_out, v_out, stream)


def hga_qk_norm_rope_backward(q, k, d_q, d_k, pos, rope: HGARope, *, q_weight=None, k_weight=None,
                              eps: float = 1e-6, d_v=None, dq=None, dk=None, dv=None,
                              workspace=None, stream=None):
    """Gradients of hga_qk_norm_rope.  q, k, pos, rope, weights and eps as in the
    forward; d_q, d_k (and d_v) the dense gradients of its dense outputs, fp32
    (as hga_attend_backward gives them) or in q's dtype.  dq, dk, dv may be
    views of one fused buffer.  Returns (dq, dk, dv, dq_weight, dk_weight): dq,
    dk, dv in q's dtype (dv None without d_v), the weights' gradients fp32 [D]
    (None without the weight)."""
    return (_ext or _module()).qk_backward(q, k, d_q, d_k, pos, rope, q_weight, k_weight, eps, d_v, dq,
                                           dk, dv, workspace, stream)


def hga_paged_decode(q, k_pages, v_pages, block_table, lens, *, window: int = 0, sinks: int = 0,
                     scale: float = 0.0, out=None, want_lse: bool = False, lse=None,
                     workspace=None, stream=None):
    """Attention of one new token per sequence over its pages.  q [B, Hq, D]
    (rotated), k_pages and v_pages [num_pages, page_size, Hkv, D], block_table
    [B, max_pages] and lens [B] int32 (the new token's key and value already
    written, lens counting it).  window > 0: only the last `window` tokens and
    the first `sinks` are visible.  scale 0: 1/sqrt(D).  -> out [B, Hq, D] (and
    lse [B, Hq] fp32 when asked)."""
    return (_ext or _module()).decode(q, k_pages, v_pages, block_table, lens, window, sinks, scale, out,
                                      want_lse, lse, workspace, stream)
