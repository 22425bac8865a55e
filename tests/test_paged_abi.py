"""The paged-cache operators' argument checks: refused on the host, before
anything is launched (the fake pointers below are never dereferenced, and no call
here is valid enough to launch), and the reference's own pins."""
import ctypes

import numpy as np
import pytest
import torch

import hierarchical_kv_routing_b200 as hga
from hierarchical_kv_routing_b200 import _build
from tests import paged_reference as ref

A = 1 << 24
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 6
P, I32, I64, F64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double


def struct(name, *fields):
    """A structure of include/hga.h: (type, "names ...") in order."""
    return type(name, (ctypes.Structure,), {"_fields_": [(n, t) for t, ns in fields for n in ns.split()]})


PagedDims = struct("hga_paged_dims", (I32, "B Hq Hkv D dtype num_pages page_size max_pages"))
PlanIO = struct("hga_paged_plan_io", (P, "lens new_tokens release free_pages free_count block_table "
                                         "lens_out free_count_out cu_tokens granted slot pos"))
Rope = struct("hga_rope", (I32, "layout rotary_dim scaling original_len"),
              (F64, "theta factor beta_fast beta_slow magnitude"))
QkIO = struct("hga_qk_io", (P, "q k v"), (I64, "q_stride k_stride v_stride"), (P, "q_weight k_weight"),
              (F64, "eps"), (P, "pos q_out k_out v_out slot k_pages v_pages"), (I64, "num_slots"))
GradIO = struct("hga_qk_grad_io", (P, "q k"), (I64, "q_stride k_stride"), (P, "q_weight k_weight"),
                (F64, "eps"), (P, "pos d_q d_k d_v"), (I32, "grad_dtype"), (P, "dq dk dv"),
                (I64, "dq_stride dk_stride dv_stride"), (P, "d_q_weight d_k_weight"))


def rope(**kw):
    d = dict(layout=0, rotary_dim=64, scaling=0, original_len=0, theta=1e6, factor=1.0, beta_fast=32.0,
             beta_slow=1.0, magnitude=0.0)
    d.update(kw)
    return Rope(**d)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    hga.load()
    lib = ctypes.CDLL(hga.lib_path())             # argument types of this module's own
    sz = ctypes.c_size_t
    lib.hga_paged_plan.argtypes = [P, P, I32, P, sz, P]
    lib.hga_qk_norm_rope.argtypes = [P, P, P, P]
    lib.hga_qk_norm_rope_backward.argtypes = [P, P, P, P, sz, P]
    lib.hga_paged_decode.argtypes = [P, P, P, P, P, P, I32, I32, F64, P, P, P, sz, P]
    lib.hga_paged_plan_workspace.argtypes = [I32, I32]
    for f in ("plan", "decode"):
        getattr(lib, f"hga_paged_{f}_workspace").restype = sz
    lib.hga_qk_norm_rope_backward_workspace.restype = sz
    return lib


def pdims(**kw):
    d = dict(B=4, Hq=8, Hkv=2, D=64, dtype=1, num_pages=100, page_size=16, max_pages=10)
    d.update(kw)
    return PagedDims(**d)


BAD_PAGES = [(dict(B=0), INVALID), (dict(num_pages=0), INVALID), (dict(page_size=0), INVALID),
             (dict(page_size=-16), INVALID), (dict(max_pages=0), INVALID), (dict(page_size=24), UNSUPPORTED),
             (dict(B=65536), UNSUPPORTED), (dict(num_pages=1 << 27), UNSUPPORTED),
             (dict(max_pages=1 << 27), UNSUPPORTED), (dict(B=60000, max_pages=60000), UNSUPPORTED)]
BAD_HEADS = [(dict(Hq=0), INVALID), (dict(Hkv=3), INVALID), (dict(D=96), UNSUPPORTED),
             (dict(dtype=2), INVALID), (dict(Hq=1 << 17, Hkv=1), UNSUPPORTED)]


def plan_io(**kw):
    d = {n: A for n, _ in PlanIO._fields_}
    d.update(kw)
    return PlanIO(**d)


def call_plan(lib, d, io, n=8, ws=A, nbytes=1 << 20):
    return lib.hga_paged_plan(ctypes.byref(d), ctypes.byref(io), n, ws, nbytes, None)


@pytest.mark.parametrize("bad,code", BAD_PAGES)
def test_plan_dims(lib, bad, code):
    assert call_plan(lib, pdims(**bad), plan_io()) == code


def test_plan_pointers_and_workspace(lib):
    for f in ("lens", "new_tokens", "free_pages", "free_count", "block_table", "lens_out",
              "free_count_out", "cu_tokens", "granted", "slot", "pos"):
        assert call_plan(lib, pdims(), plan_io(**{f: None})) == INVALID, f
    for f, _ in PlanIO._fields_:
        assert call_plan(lib, pdims(), plan_io(**{f: A + 2})) == INVALID, f
    assert call_plan(lib, pdims(), plan_io(), n=-1) == INVALID
    assert lib.hga_paged_plan(None, None, 0, None, 0, None) == INVALID
    need = lib.hga_paged_plan_workspace(4, 8)
    assert need >= 16
    assert call_plan(lib, pdims(), plan_io(), nbytes=need - 1) == WORKSPACE
    assert call_plan(lib, pdims(), plan_io(), ws=None) == WORKSPACE
    assert call_plan(lib, pdims(), plan_io(), ws=A + 16) == WORKSPACE
    assert lib.hga_paged_plan_workspace(0, 8) == 0 and lib.hga_paged_plan_workspace(4, -1) == 0


def decode_call(lib, d, **kw):
    a = dict(q=A, k=A, v=A, table=A, lens=A, window=0, sinks=0, scale=0.0, out=A, lse=None, ws=A,
             nbytes=1 << 28)
    a.update(kw)
    return lib.hga_paged_decode(ctypes.byref(d), a["q"], a["k"], a["v"], a["table"], a["lens"],
                                a["window"], a["sinks"], a["scale"], a["out"], a["lse"], a["ws"],
                                a["nbytes"], None)


@pytest.mark.parametrize("bad,code", BAD_PAGES + BAD_HEADS)
def test_decode_dims(lib, bad, code):
    assert decode_call(lib, pdims(**bad)) == code
    assert lib.hga_paged_decode_workspace(ctypes.byref(pdims(**bad))) == 0


def test_decode_pointers_values_and_workspace(lib):
    for f in ("q", "k", "v", "table", "lens", "out"):
        assert decode_call(lib, pdims(), **{f: None}) == INVALID
    for f in ("q", "k", "v", "out"):
        assert decode_call(lib, pdims(), **{f: A + 8}) == INVALID
    for f in ("table", "lens", "lse"):
        assert decode_call(lib, pdims(), **{f: A + 2}) == INVALID
    for kw in (dict(window=-1), dict(sinks=-1), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf"))):
        assert decode_call(lib, pdims(), **kw) == INVALID
    # more units of work than 32 bits count
    assert decode_call(lib, pdims(B=1024, max_pages=1 << 20, page_size=1024)) == UNSUPPORTED
    need = lib.hga_paged_decode_workspace(ctypes.byref(pdims()))
    assert need > 0
    assert decode_call(lib, pdims(), nbytes=need - 1) == WORKSPACE
    assert decode_call(lib, pdims(), ws=None) == WORKSPACE
    assert decode_call(lib, pdims(), ws=A + 128) == WORKSPACE


def tdims(**kw):
    d = dict(B=1, T=7, Hq=4, Hkv=2, D=64, dtype=1)
    d.update(kw)
    return hga._Dims(**d)


def qk_io(**kw):
    d = dict(q=A, k=A, v=A, q_stride=512, k_stride=512, v_stride=512, q_weight=A, k_weight=A, eps=1e-6,
             pos=A, q_out=A, k_out=A, v_out=A)
    d.update(kw)
    return QkIO(**d)


def grad_io(**kw):
    d = {n: A for n in ("q", "k", "q_weight", "k_weight", "pos", "d_q", "d_k", "d_v", "dq", "dk", "dv",
                        "d_q_weight", "d_k_weight")}
    d.update({n: 512 for n in ("q_stride", "k_stride", "dq_stride", "dk_stride", "dv_stride")})
    d.update(eps=1e-6, grad_dtype=1)
    d.update(kw)
    return GradIO(**d)


def call_qk(lib, d, io, r=None):
    r = r or rope()
    return lib.hga_qk_norm_rope(ctypes.byref(d), ctypes.byref(r), ctypes.byref(io), None)


def call_grad(lib, d, io, r=None, ws=A, nbytes=1 << 24):
    r = r or rope()
    return lib.hga_qk_norm_rope_backward(ctypes.byref(d), ctypes.byref(r), ctypes.byref(io), ws, nbytes,
                                         None)


@pytest.mark.parametrize("bad,code", BAD_HEADS + [(dict(B=0), INVALID), (dict(T=-1), INVALID),
                                                  (dict(B=1 << 16, T=1 << 16), UNSUPPORTED)])
def test_qk_dims(lib, bad, code):
    assert call_qk(lib, tdims(**bad), qk_io()) == code
    assert call_grad(lib, tdims(**bad), grad_io()) == code
    assert lib.hga_qk_norm_rope_backward_workspace(ctypes.byref(tdims(**bad))) == 0


@pytest.mark.parametrize("bad,code", [
    (dict(rotary_dim=80), INVALID), (dict(rotary_dim=-16), INVALID), (dict(rotary_dim=24), UNSUPPORTED),
    (dict(theta=1.0), INVALID), (dict(theta=float("nan")), INVALID), (dict(theta=float("inf")), INVALID),
    (dict(scaling=1, factor=0.5), INVALID), (dict(scaling=1, factor=float("inf")), INVALID),
    (dict(scaling=2, factor=2.0), INVALID),
    (dict(scaling=2, factor=2.0, original_len=64, beta_slow=0.0), INVALID),
    (dict(scaling=2, factor=2.0, original_len=64, beta_slow=33.0), INVALID),
    (dict(magnitude=-1.0), INVALID), (dict(magnitude=float("nan")), INVALID),
    (dict(layout=2), INVALID), (dict(layout=-1), INVALID), (dict(scaling=3), INVALID)])
def test_rope_values(lib, bad, code):
    # a good rotation first: the constants kept of it are not used for the bad one
    assert call_qk(lib, tdims(), qk_io(q=None), rope(rotary_dim=32)) == INVALID
    assert call_qk(lib, tdims(), qk_io(q=None), rope(**bad)) == code
    assert call_grad(lib, tdims(), grad_io(d_q=None), rope(**bad)) == code


def test_values_beyond_fp32(lib):
    """What the kernels take in fp32 and would be infinite there."""
    assert call_qk(lib, tdims(T=0), qk_io(), rope(magnitude=1e38)) == 0
    assert call_qk(lib, tdims(T=0), qk_io(), rope(magnitude=1e39)) == INVALID
    assert call_grad(lib, tdims(), grad_io(d_q=None), rope(magnitude=1e39)) == INVALID
    assert call_qk(lib, tdims(), qk_io(eps=1e39)) == INVALID
    assert call_grad(lib, tdims(), grad_io(eps=1e39)) == INVALID
    for scale in (1e39, 3e38):              # times log2(e), as the kernel has it
        assert decode_call(lib, pdims(), scale=scale) == INVALID


def test_qk_pointers_and_strides(lib):
    for f in ("q", "k", "v", "pos"):
        assert call_qk(lib, tdims(), qk_io(**{f: None})) == INVALID, f
    for f in ("q", "k", "v", "q_out", "k_out", "v_out", "q_weight", "k_weight"):
        assert call_qk(lib, tdims(), qk_io(**{f: A + 8})) == INVALID, f
    for f, v in (("q_stride", 255), ("q_stride", 260), ("k_stride", 127), ("v_stride", 0),
                 ("v_stride", 1 << 50), ("q_stride", -512)):
        assert call_qk(lib, tdims(), qk_io(**{f: v})) == INVALID, f
    for eps in (-1e-6, float("nan"), float("inf")):
        assert call_qk(lib, tdims(), qk_io(eps=eps)) == INVALID
        assert call_grad(lib, tdims(), grad_io(eps=eps)) == INVALID
    for kw in (dict(k_pages=A), dict(k_pages=A, slot=A), dict(k_pages=A, slot=A + 2, num_slots=8),
               dict(v_pages=A, num_slots=8), dict(k_pages=A + 4, slot=A, num_slots=8)):
        assert call_qk(lib, tdims(), qk_io(**kw)) == INVALID
    assert call_qk(lib, tdims(), qk_io(k_pages=A, slot=A, num_slots=1 << 31)) == UNSUPPORTED


def test_qk_grad_pointers_and_workspace(lib):
    for f in ("q", "k", "pos", "d_q", "d_k", "dq", "dk", "d_v", "dv", "q_weight", "d_q_weight",
              "k_weight", "d_k_weight"):
        assert call_grad(lib, tdims(), grad_io(**{f: None})) == INVALID, f
    for f in ("q", "k", "d_q", "d_k", "d_v", "dq", "dk", "dv", "q_weight", "k_weight"):
        assert call_grad(lib, tdims(), grad_io(**{f: A + 8})) == INVALID, f
    for f in ("d_q_weight", "d_k_weight", "pos"):
        assert call_grad(lib, tdims(), grad_io(**{f: A + 2})) == INVALID, f
    for f in ("q_stride", "k_stride", "dq_stride", "dk_stride", "dv_stride"):
        assert call_grad(lib, tdims(), grad_io(**{f: 4})) == INVALID, f
    assert call_grad(lib, tdims(dtype=0), grad_io(grad_dtype=1)) == INVALID
    assert call_grad(lib, tdims(), grad_io(grad_dtype=2)) == INVALID
    need = lib.hga_qk_norm_rope_backward_workspace(ctypes.byref(tdims()))
    assert need > 0
    assert call_grad(lib, tdims(), grad_io(), nbytes=need - 1) == WORKSPACE
    assert call_grad(lib, tdims(), grad_io(), ws=None) == WORKSPACE
    assert call_grad(lib, tdims(), grad_io(), ws=A + 64) == WORKSPACE


def test_binding_refuses_cpu_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(2, 2, 64)
    with pytest.raises(hga.HGAError):
        hga.hga_paged_plan(i, i, i, i[:1], torch.zeros(2, 3, dtype=torch.int32), 16, 4)
    with pytest.raises(hga.HGAError):
        hga.hga_qk_norm_rope(x, x, x, i, hga.HGARope())
    with pytest.raises(hga.HGAError):
        hga.hga_qk_norm_rope_backward(x, x, x, x, i, hga.HGARope())
    with pytest.raises(hga.HGAError):
        hga.hga_paged_decode(x, x[None], x[None], torch.zeros(2, 3, dtype=torch.int32), i)


def test_reference_plan_pins():
    """By hand: two rows, pages of 4, a stack of three."""
    r = ref.plan([3, 4], [2, 1], [7, 8, 9], 3, [[0, -1, -1], [1, -1, -1]], 4, 4)
    assert r["cu_tokens"] == [0, 2, 3] and r["granted"] == [2, 1] and r["lens"] == [5, 5]
    assert r["table"] == [[0, 9, -1], [1, 8, -1]] and r["free_count"] == [1]
    assert r["slot"] == [3, 36, 32, -1] and r["pos"] == [3, 4, 4, 0]
    r = ref.plan([4, 4, 1], [1, 1, 1], [9, 0, 0], 1, [[0, -1], [1, -1], [2, -1]], 4, 3)
    assert r["granted"] == [1, 0, 1] and r["slot"] == [36, -1, 9]      # the page goes to the first
    r = ref.plan([5, 1], [0, 9], [3, 0, 0, 0, 0], 1, [[0, 1, -1], [2, -1, -1]], 4, 9, [1, 0])
    assert r["free"][:3] == [3, 0, 1] and r["lens"] == [0, 10] and r["table"][1] == [2, 1, 0]


def test_reference_rotation_pins():
    """Complex rotation for both layouts; the transpose undoes it; attention over a
    window that covers everything is attention over everything."""
    rng = np.random.default_rng(0)
    x, pos = rng.normal(size=(5, 2, 64)), np.arange(5) * 7
    for layout in ("half", "interleaved"):
        for R in (0, 16, 48, 64):
            w = ref.rates(R, 1e4)
            y = ref.rotate(x, pos, R, layout, w, 1.0)
            a, b = ref.members(R, layout)
            z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos[:, None, None] * w)
            assert np.allclose(y[..., a], z.real) and np.allclose(y[..., b], z.imag)
            assert np.array_equal(y[..., R:], x[..., R:])
            assert np.allclose(ref.rotate(y, pos, R, layout, w, 1.0, back=True), x)
    w = ref.rates(64, 1e4, "yarn", 4.0, 4096)
    base = ref.rates(64, 1e4)
    assert np.allclose(w[0], base[0]) and np.allclose(w[-1], base[-1] / 4)
    assert (np.diff(w / base) <= 1e-12).all()
    assert ref.visible(9, 3, 2) == [0, 1, 6, 7, 8] and ref.visible(3, 9, 2) == [0, 1, 2]
    assert ref.visible(4, 0, 2) == [0, 1, 2, 3]


def test_qk_grad_of_no_tokens_checks_the_weights(lib):
    """Without tokens the kernel still runs (it writes the weights' zero gradients) and
    reads the weights in 16-byte words."""
    for f in ("q_weight", "k_weight"):
        for off in (2, 8):
            assert call_grad(lib, tdims(T=0), grad_io(**{f: A + off})) == INVALID, f
    for f in ("d_q_weight", "d_k_weight"):
        assert call_grad(lib, tdims(T=0), grad_io(**{f: A + 2})) == INVALID, f


def test_values_below_fp32(lib):
    """What fp32 holds as 0 or with fewer bits (below 2^-126): an eps of 0 would make a
    row of zeros NaN, a magnitude of 0 its rotated part 0.  0 itself and 2^-126 are taken."""
    for bad in (1e-50, 5e-324, 1e-45, 2.0 ** -127):
        assert call_qk(lib, tdims(T=0), qk_io(), rope(magnitude=bad)) == INVALID
        assert call_grad(lib, tdims(), grad_io(d_q=None), rope(magnitude=bad)) == INVALID
        assert call_qk(lib, tdims(), qk_io(eps=bad)) == INVALID
        assert call_grad(lib, tdims(), grad_io(eps=bad)) == INVALID
        assert decode_call(lib, pdims(), scale=bad) == INVALID
    for good in (0.0, 2.0 ** -126):
        assert call_qk(lib, tdims(T=0), qk_io(), rope(magnitude=good)) == 0
        assert call_grad(lib, tdims(), grad_io(eps=good, d_q_weight=A + 2)) == INVALID
        assert decode_call(lib, pdims(), scale=good, ws=None) == WORKSPACE
        assert call_grad(lib, tdims(), grad_io(eps=good), ws=None) == WORKSPACE


def test_yarn_ramp_that_would_run_backwards(lib):
    """lo and hi by the header's formula: where hi < lo, pairs that turn often would be
    slowed and the others not.  hi = lo and a first or last pair on the ramp are taken."""
    def ends(theta, L, fast, slow, R=64):
        d = lambda t: R * np.log(L / (2 * np.pi * t)) / (2 * np.log(theta))
        return max(0.0, np.floor(d(fast))), min(R - 1.0, np.ceil(d(slow)))
    seen = set()
    for theta, L, fast, slow in [(1e6, 3, 32.0, 1.0), (1e6, 6, 32.0, 1.0), (1e6, 7, 32.0, 1.0),
                                 (10.0, 1 << 20, 32.0, 1.0), (10.0, 1 << 14, 32.0, 1.0), (1e4, 4096, 32.0, 1.0),
                                 (1e4, 4096, 1e9, 1e9), (1e4, 100, 16.0, 15.0), (1e4, 4096, 4.0, 4.0)]:
        lo, hi = ends(theta, L, fast, slow)
        r = rope(scaling=2, factor=4.0, theta=theta, original_len=L, beta_fast=fast, beta_slow=slow)
        want = INVALID if hi < lo else 0
        assert call_qk(lib, tdims(T=0), qk_io(), r) == want, (theta, L, lo, hi)
        seen.add(want)
    assert seen == {0, INVALID}
