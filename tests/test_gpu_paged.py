"""The paged-cache operators on the GPU against their definitions in 64 bits:
block tables and slot maps, norms with rotation and their gradient, attention of
one new token over pages, and a run of them together."""
import math

import numpy as np
import pytest
import torch

from tests import paged_reference as ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def hga(gpu_lib):
    return gpu_lib


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().double().cpu().numpy()


# ------------------------------------------------------------------ plan --

def plan_state(rng, B, page, M, spare, full=False):
    """Lengths within the rows, shuffled pages, `spare` free ones."""
    lens = rng.integers(0, M * page + 1, B)
    if full:
        lens[:] = M * page
    held = -(-lens // page)
    P = int(held.sum()) + spare
    ids = rng.permutation(P)
    table, at = np.full((B, M), -1), 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = np.full(max(P, 1), -7)
    free[:P - at] = ids[at:]
    return lens, table, free, P - at


def check_plan(hga, lens, new, table, free, count, page, n_slots, release=None, in_place=False):
    want = ref.plan(lens.tolist(), new.tolist(), free.tolist(), count, table.tolist(), page, n_slots,
                    None if release is None else release.tolist())
    tl, tt, tf, tc = i32(lens), i32(table), i32(free), i32([count])
    kw = dict(lens_out=tl, free_count_out=tc) if in_place else {}
    r = hga.hga_paged_plan(tl, i32(new), tf, tc, tt, page, n_slots,
                           release=None if release is None else i32(release), **kw)
    got = {k: v.tolist() for k, v in r.items()}
    got.update(table=tt.tolist(), free=tf.tolist())
    for k in want:
        assert got[k] == want[k], k
    if not in_place:
        assert tl.tolist() == lens.tolist() and tc.tolist() == [count]
    return want


@pytest.mark.parametrize("B,page,M,top,pad", [
    (1, 16, 1, 1, 0), (1, 1, 7, 3, 2), (3, 16, 4, 5, 0), (33, 8, 9, 2, 5), (256, 16, 30, 1, 0),
    (1023, 4, 6, 3, 1), (1024, 4, 6, 3, 0), (1025, 32, 5, 3, 64), (2500, 2, 6, 9, 3)])
def test_plan_steps(hga, B, page, M, top, pad):
    rng = np.random.default_rng(B + page)
    for spare in (0, B // 3 + 1, 4 * B):
        lens, table, free, count = plan_state(rng, B, page, M, spare)
        new = rng.integers(0, top + 1, B)
        n = int(new.sum())
        check_plan(hga, lens, new, table, free, count, page, n + pad)
        check_plan(hga, lens, new, table, free, count, page, n + pad, in_place=True,
                   release=(rng.random(B) < 0.3).astype(int))
    assert hga.hga_device_status() == 0


@pytest.mark.parametrize("n", [2047, 2048, 2049, 8192, 70001])
def test_plan_prompts_in_both_fills(hga, n):
    """Prompts whose tokens the scanning CTA fills itself, and beyond."""
    rng = np.random.default_rng(n)
    new = rng.multinomial(n, np.ones(7) / 7)
    new[3] += new[2]
    new[2] = 0
    lens, page, M = np.array([0, 5, 16, 31, 0, 1, 64]), 16, 3000
    table, free, count = np.full((7, M), -1), rng.permutation(9000), 9000 - 20
    free[count:] = -1
    at = count
    for b in range(7):
        for j in range(-(-lens[b] // page)):
            table[b, j] = 8980 + b
    free = np.array([x for x in free if x < 8970 and x >= 0] + [0] * 100)
    count = len(free) - 100
    check_plan(hga, lens, new, table, free, count, page, n + 3)
    check_plan(hga, lens, new, table, free, 200, page, n + 3)      # most have to wait
    assert at and hga.hga_device_status() == 0


def test_plan_row_full_and_map_full(hga):
    """A row without room and tokens beyond the map are refused, the others served."""
    rng = np.random.default_rng(3)
    lens, table, free, count = plan_state(rng, 5, 4, 3, 20)
    lens[:] = [12, 11, 0, 12, 3]
    table = np.arange(15).reshape(5, 3)
    free, count = np.arange(15, 55), 25               # pages 15 .. 39 of a pool of 40
    new = np.array([1, 1, 4, 0, 9])
    w = check_plan(hga, lens, new, table, free, count, 4, 15)
    assert w["granted"] == [0, 1, 4, 0, 9]
    w = check_plan(hga, lens, new, table, free, count, 4, 14)      # the last one's end lies beyond
    assert w["granted"] == [0, 1, 4, 0, 0]
    w = check_plan(hga, lens, new, table, free, count, 4, 0)
    assert w["granted"] == [0, 0, 0, 0, 0]
    assert hga.hga_device_status() == 0


def test_plan_bad_values_are_reported(hga):
    """Bad counts and page ids are left out and reported; the other rows are served."""
    for lens, new, table, free, count in [
            ([-3, 2], [1, 1], [[0, 1], [2, 3]], [4, 5], 2),
            ([9, 2], [1, 1], [[0, 1], [2, 3]], [4, 5], 2),
            ([3, 2], [-1, 1], [[0, 1], [2, 3]], [4, 5], 2),
            ([3, 2], [0, 1], [[0, 1], [2, 3]], [4, 5], 77)]:
        r = hga.hga_paged_plan(i32(lens), i32(new), i32(free + [9] * 14), i32([count]), i32(table), 4, 2)
        assert r["granted"].tolist()[1] == 1
        assert 2 * 4 + 2 in r["slot"].tolist()
        assert hga.hga_device_status() == 5 and hga.hga_device_status() == 0
    t = i32([[0, -1], [99, 3]])
    r = hga.hga_paged_plan(i32([4, 2]), i32([1, 1]), i32([-5] * 8), i32([8]), t, 4, 2)
    assert r["slot"].tolist() == [-1, -1] and t.tolist() == [[0, -1], [99, 3]]
    assert hga.hga_device_status() == 5
    # a release of bad and of too many pages: what fits is given back
    free = i32([5, 6, 0, 0])
    r = hga.hga_paged_plan(i32([8, 8, 8]), i32([0, 0, 0]), free, i32([2]), i32([[0, 44], [-1, 1], [2, 3]]),
                           4, 0, release=i32([1, 1, 1]))
    assert free.tolist() == [5, 6, 0, 1] and r["free_count"].tolist() == [4]
    assert r["lens"].tolist() == [0, 0, 0]
    assert hga.hga_device_status() == 5 and hga.hga_device_status() == 0


@pytest.mark.parametrize("bad", [0, 1, 40])
def test_plan_releases_long_rows(hga, bad):
    """More pages given back than one sweep of the scanning CTA, some ids bad: the good
    ones lie on the stack in order."""
    rng = np.random.default_rng(bad)
    B, page, M = 9, 2, 4000
    lens = rng.integers(page * M * 3 // 4, page * M, B)
    held = -(-lens // page)
    P = int(held.sum()) + 50
    ids = rng.permutation(P)
    table, at = np.full((B, M), -1), 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = np.full(P, -7)
    free[:50] = ids[at:]
    release = np.ones(B, int)
    release[4] = 0
    if not bad:
        check_plan(hga, lens, rng.integers(0, 9, B), table, free, 50, page, 100, release)
        assert hga.hga_device_status() == 0
        return
    for _ in range(bad):
        table[rng.integers(0, B), rng.integers(0, M * 3 // 4)] = rng.choice([-1, P, 2 ** 31 - 1, -2 ** 31])
    want = free[:50].tolist()
    for b in range(B):
        if release[b]:
            want += [x for x in table[b, :held[b]].tolist() if 0 <= x < P]
    tf = i32(free)
    r = hga.hga_paged_plan(i32(lens), i32([0] * B), tf, i32([50]), i32(table), page, 0, release=i32(release))
    assert r["free_count"].tolist() == [len(want)] and tf[:len(want)].tolist() == want
    bads = sum(not 0 <= x < P for b in range(B) if release[b] for x in table[b, :held[b]])
    assert hga.hga_device_status() == (5 if bads else 0)


def test_plan_releases_a_row_of_the_largest_size(hga):
    """One row of 2^31 - 1 pages of one token, all given back: the last sweep over its
    entries ends beyond 31 bits."""
    n = 2 ** 31 - 1
    table = torch.arange(n, dtype=torch.int32, device="cuda")
    free = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    r = hga.hga_paged_plan(i32([n]), i32([0]), free, i32([0]), table.view(1, n), 1, 1, release=i32([1]))
    assert r["free_count"].tolist() == [n] and r["lens"].tolist() == [0]
    assert torch.equal(free, table)
    assert hga.hga_device_status() == 0


# ------------------------------------------------------------- rotation --

ROPES = [
    dict(rotary_dim=None, theta=1e4), dict(rotary_dim=0), dict(rotary_dim=16, theta=5e5),
    dict(rotary_dim=48, layout="interleaved", theta=1e6),
    dict(rotary_dim=None, layout="interleaved", scaling="linear", factor=4.0),
    dict(rotary_dim=64, scaling="yarn", factor=4.0, original_len=4096, theta=1e6),
    dict(rotary_dim=32, layout="interleaved", scaling="yarn", factor=7.5, original_len=512,
         beta_fast=24.0, beta_slow=2.0, theta=1e4, magnitude=1.25),
]


def rope_ref(r, D):
    R = D if r.get("rotary_dim") is None else r["rotary_dim"]
    scal = {k: r[k] for k in ("scaling", "factor", "original_len", "beta_fast", "beta_slow") if k in r}
    w = ref.rates(R, r.get("theta", 1e6), **scal)
    m = ref.magnitude(r.get("scaling", "none"), r.get("factor", 1.0), r.get("magnitude", 0.0))
    return R, r.get("layout", "half"), w, m


def qkv(seed, N, Hq, Hkv, D, dtype, pad=0):
    """A fused buffer (with `pad` more columns) and its views."""
    g = torch.Generator().manual_seed(seed)
    W = (Hq + 2 * Hkv) * D + pad
    x = (torch.randn(N, W, generator=g) * torch.exp(torch.randn(W, generator=g))).to(DT[dtype]).cuda()
    return (x, x[:, :Hq * D].view(N, Hq, D), x[:, Hq * D:(Hq + Hkv) * D].view(N, Hkv, D),
            x[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].view(N, Hkv, D))


def weights(seed, D, dtype):
    g = torch.Generator().manual_seed(seed)
    return [(1 + 0.3 * torch.randn(D, generator=g)).to(DT[dtype]).cuda() for _ in range(2)]


SHAPES = [("bf16", 5, 4, 2, 128), ("bf16", 37, 3, 1, 64), ("f32", 5, 2, 1, 64), ("f32", 33, 5, 5, 128),
          ("bf16", 1, 32, 4, 128), ("bf16", 2600, 8, 8, 64), ("f32", 1, 1, 1, 128)]


@pytest.mark.parametrize("r", ROPES, ids=lambda r: "-".join(str(v) for v in r.values()))
@pytest.mark.parametrize("dtype,N,Hq,Hkv,D", SHAPES)
def test_qk_norm_rope(hga, dtype, N, Hq, Hkv, D, r):
    _, q, k, v = qkv(N, N, Hq, Hkv, D, dtype, pad=16)
    qw, kw = weights(N + 1, D, dtype)
    rng = np.random.default_rng(N)
    pos = rng.integers(0, 1 << 20, N)
    pos[0] = 0
    R, layout, w, m = rope_ref(r, D)
    for a, b in ((qw, kw), (None, kw), (qw, None)):
        qo, ko, vo = hga.hga_qk_norm_rope(q, k, v, i32(pos), hga.HGARope(**r), q_weight=a, k_weight=b,
                                          eps=1e-5)
        for x, y, wt in ((q, qo, a), (k, ko, b)):
            want, bound = ref.norm_rope(f64(x), None if wt is None else f64(wt), pos, R, layout, w, m,
                                        1e-5, dtype)
            assert ref.worst(f64(y), want, bound) <= 1
        assert torch.equal(vo, v)
    # the leading shape [B, T] of a strided buffer
    if N % 2 == 0:
        x4 = [t.unflatten(0, (2, N // 2)) for t in (q, k, v)]
        q4, k4, _ = hga.hga_qk_norm_rope(*x4, i32(pos.reshape(2, -1)), hga.HGARope(**r), q_weight=qw,
                                         k_weight=None, eps=1e-5)
        assert torch.equal(q4.flatten(0, 1), qo) and torch.equal(k4.flatten(0, 1), ko)


def test_qk_positions_far_and_negative(hga):
    """Angles do not lose positions: far, negative, and the ends of 32 bits."""
    pos = np.array([0, 1, 977, 65536, 10 ** 6, -1, -12345, 1 << 24, 2 ** 31 - 1, -2 ** 31])
    _, q, k, v = qkv(4, 10, 2, 1, 64, "f32")
    qo, _, _ = hga.hga_qk_norm_rope(q, k, None, i32(pos), hga.HGARope(theta=1e4))
    # the rates, rounded to 64 bits, turn by at most 2^31 2^-53 more or less: 2.4e-7
    want, bound = ref.norm_rope(f64(q), None, pos, 64, "half", ref.rates(64, 1e4), 1.0, 0, "f32")
    assert ref.worst(f64(qo), want, bound + 2.4e-7 * np.abs(f64(q)).max(-1, keepdims=True)) <= 1


@pytest.mark.parametrize("dtype,N,Hkv,D,page", [("bf16", 9, 4, 128, 4), ("f32", 130, 1, 64, 16),
                                                 ("bf16", 1, 8, 64, 1)])
def test_qk_into_pages(hga, dtype, N, Hkv, D, page):
    """Rows go to their slots and nowhere else; -1 writes nothing, a bad slot is
    reported; dense keys are written beside the pages where they are asked for."""
    _, q, k, v = qkv(N, N, Hkv * 2, Hkv, D, dtype)
    qw, kw = weights(1, D, dtype)
    P = -(-N // page) + 2
    rng = np.random.default_rng(N)
    slot = rng.permutation(P * page)[:N]
    if N > 8:
        slot[[2, N - 1]] = -1
    rope = hga.HGARope(theta=1e4)
    dense = hga.hga_qk_norm_rope(q, k, v, i32(np.arange(N)), rope, q_weight=qw, k_weight=kw)
    kp = torch.full((P, page, Hkv, D), float("nan"), dtype=DT[dtype], device="cuda")
    vp = kp.clone()
    k2 = torch.empty_like(dense[1])
    qo, ko, vo = hga.hga_qk_norm_rope(q, k, v, i32(np.arange(N)), rope, q_weight=qw, k_weight=kw,
                                      k_pages=kp, v_pages=vp, slot=i32(slot), k_out=k2)
    assert torch.equal(qo, dense[0]) and torch.equal(ko, dense[1]) and vo is None
    for pages, rows in ((kp, dense[1]), (vp, dense[2])):
        want = torch.full((P * page, Hkv, D), float("nan"), dtype=DT[dtype], device="cuda")
        for t in range(N):
            if slot[t] >= 0:
                want[slot[t]] = rows[t]
        assert torch.equal(pages.view(-1, Hkv, D).nan_to_num(7.0), want.nan_to_num(7.0))
    assert hga.hga_device_status() == 0
    for bad in (P * page, -2, 2 ** 31 - 1):
        s2 = i32(slot)
        s2[0] = bad
        kq = kp.clone()
        hga.hga_qk_norm_rope(q, k, v, i32(np.arange(N)), rope, q_weight=qw, k_weight=kw, k_pages=kq,
                             v_pages=vp, slot=s2)
        assert hga.hga_device_status() == 5
        assert torch.equal(kq.nan_to_num(7.0), kp.nan_to_num(7.0))


def test_qk_empty_and_zero_rows(hga):
    """No tokens; and a row of zeros, which the norm leaves at zero."""
    rope = hga.HGARope()
    e = torch.empty(0, 2, 64, device="cuda")
    qo, ko, vo = hga.hga_qk_norm_rope(e, e, e, i32([]), rope)
    assert qo.shape == e.shape
    w = torch.ones(64, device="cuda")
    _, _, _, dqw, dkw = hga.hga_qk_norm_rope_backward(e, e, e, e, i32([]), rope, q_weight=w, k_weight=w)
    assert not dqw.any() and not dkw.any()
    z = torch.zeros(3, 2, 64, device="cuda")
    qo, _, _ = hga.hga_qk_norm_rope(z, z, z, i32([1, 2, 3]), rope, q_weight=w, k_weight=w)
    assert not qo.any()
    dq, _, _, dqw, _ = hga.hga_qk_norm_rope_backward(z, z, z + 1, z + 1, i32([0, 0, 0]), rope,
                                                     q_weight=w, k_weight=w, eps=1e-6)
    assert torch.allclose(dq, torch.full_like(dq, 1e3), rtol=1e-6) and not dqw.any()


@pytest.mark.parametrize("r", ROPES, ids=lambda r: "-".join(str(v) for v in r.values()))
@pytest.mark.parametrize("dtype,N,Hq,Hkv,D", SHAPES)
def test_qk_backward(hga, dtype, N, Hq, Hkv, D, r):
    """Against the formula: into a fused buffer's views (its other columns left as
    they were), with gradients of either type, with and without weights."""
    x, q, k, v = qkv(N + 5, N, Hq, Hkv, D, dtype, pad=16)
    qw, kw = weights(N + 6, D, dtype)
    rng = np.random.default_rng(N)
    pos = rng.integers(0, 1 << 20, N)
    R, layout, w, m = rope_ref(r, D)
    g = torch.Generator().manual_seed(N)
    for gt in ({"f32"} | {dtype}):
        d = [torch.randn(N, h, D, generator=g).to(DT[gt]).cuda() for h in (Hq, Hkv, Hkv)]
        for a, b in ((qw, kw), (None, kw), (None, None)):
            buf = torch.full_like(x, 123.0)
            o = [buf[:, :Hq * D].view(N, Hq, D), buf[:, Hq * D:(Hq + Hkv) * D].view(N, Hkv, D),
                 buf[:, (Hq + Hkv) * D:-16].view(N, Hkv, D)]
            kw2 = dict(q_weight=a, k_weight=b, eps=1e-5, d_v=d[2])
            dq, dk, dv, da, db = hga.hga_qk_norm_rope_backward(
                q, k, d[0], d[1], i32(pos), hga.HGARope(**r), dq=o[0], dk=o[1], dv=o[2], **kw2)
            assert (buf[:, -16:] == 123.0).all()
            for xi, di, wt, got, gotw in ((q, d[0], a, dq, da), (k, d[1], b, dk, db)):
                (want, bound), dw = ref.norm_rope_grad(f64(xi), f64(di), None if wt is None else f64(wt),
                                                       pos, R, layout, w, m, 1e-5, dtype)
                assert ref.worst(f64(got), want, bound) <= 1
                assert (gotw is None) == (dw is None)
                if dw is not None:
                    assert ref.worst(f64(gotw), *dw) <= 1
            assert torch.equal(dv, d[2].to(DT[dtype]))
            again = hga.hga_qk_norm_rope_backward(q, k, d[0], d[1], i32(pos), hga.HGARope(**r), **kw2)
            assert all(s is None and t is None or torch.equal(s, t)
                       for s, t in zip(again, (dq, dk, dv, da, db)))


@pytest.mark.parametrize("size", [1e16, 1e-16])
@pytest.mark.parametrize("dtype,N,Hq,Hkv,D", [("f32", 5, 3, 1, 64), ("bf16", 5, 4, 2, 128)])
def test_qk_rows_far_from_one(hga, dtype, N, Hq, Hkv, D, size):
    """Rows whose squares fit fp32 while the cube of their inverse norm does not."""
    _, q, k, v = qkv(N, N, Hq, Hkv, D, dtype)
    q, k = q * size, k * size
    qw, kw = weights(N + 1, D, dtype)
    pos = np.arange(N) * 37
    R, layout, w, m = rope_ref({}, D)
    rope = hga.HGARope()
    g = torch.Generator().manual_seed(N)
    d = [torch.randn(N, h, D, generator=g).cuda() for h in (Hq, Hkv)]
    y = hga.hga_qk_norm_rope(q, k, v, i32(pos), rope, q_weight=qw, k_weight=kw, eps=0.0)
    r = hga.hga_qk_norm_rope_backward(q, k, d[0], d[1], i32(pos), rope, q_weight=qw, k_weight=kw, eps=0.0)
    for x, dy, wt, gy, gx, gw in ((q, d[0], qw, y[0], r[0], r[3]), (k, d[1], kw, y[1], r[1], r[4])):
        assert ref.worst(f64(gy), *ref.norm_rope(f64(x), f64(wt), pos, R, layout, w, m, 0.0, dtype)) <= 1
        dx, dw = ref.norm_rope_grad(f64(x), f64(dy), f64(wt), pos, R, layout, w, m, 0.0, dtype)
        assert ref.worst(f64(gx), *dx) <= 1 and ref.worst(f64(gw), *dw) <= 1


def test_qk_backward_against_differences():
    """The formula the kernels are held to is the derivative: central differences
    of the 64-bit forward in a random direction."""
    rng = np.random.default_rng(0)
    for r in ROPES:
        R, layout, w, m = rope_ref(r, 64)
        x, dy, wt = rng.normal(size=(3, 2, 64)), rng.normal(size=(3, 2, 64)), rng.normal(size=64)
        pos = np.array([0, 17, 901])

        def loss(x, wt):
            return (ref.norm_rope(x, wt, pos, R, layout, w, m, 1e-5, "f32")[0] * dy).sum()
        (dx, _), (dw, _) = ref.norm_rope_grad(x, dy, wt, pos, R, layout, w, m, 1e-5, "f32")
        ex, ew, h = rng.normal(size=x.shape), rng.normal(size=64), 1e-5
        assert abs((loss(x + h * ex, wt) - loss(x - h * ex, wt)) / (2 * h) - (dx * ex).sum()) < 1e-6
        assert abs((loss(x, wt + h * ew) - loss(x, wt - h * ew)) / (2 * h) - (dw * ew).sum()) < 1e-6


# --------------------------------------------------------------- decode --

def pages_for(seed, lens, Hkv, D, dtype, page, M=None, junk=float("nan")):
    """Pools of NaN (or junk) with the sequences' rows written in, on shuffled pages."""
    g = torch.Generator().manual_seed(seed)
    held = [-(-n // page) for n in lens]
    M = M or max(held + [1])
    P = sum(held) + 3
    ids = torch.randperm(P, generator=g)
    kp = torch.full((P, page, Hkv, D), junk, dtype=DT[dtype])
    vp = kp.clone()
    table, at = torch.full((len(lens), M), -1, dtype=torch.int32), 0
    for b, n in enumerate(lens):
        rows = [torch.randn(held[b] * page, Hkv, D, generator=g).to(DT[dtype]) for _ in range(2)]
        for x, pool in zip(rows, (kp, vp)):
            x[n:] = junk
            pool[ids[at:at + held[b]]] = x.view(held[b], page, Hkv, D)
        table[b, :held[b]] = ids[at:at + held[b]].to(torch.int32)
        at += held[b]
    return kp.cuda(), vp.cuda(), table.cuda()


def queries(seed, B, Hq, D, dtype, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (size * torch.randn(B, Hq, D, generator=g)).to(DT[dtype]).cuda()


def check_decode(hga, q, kp, vp, table, lens, dtype, window=0, sinks=0, scale=0.0, skip=(), **kw):
    out, lse = hga.hga_paged_decode(q, kp, vp, table, i32(lens), window=window, sinks=sinks,
                                    scale=scale, want_lse=True, **kw)
    want = ref.decode(f64(q), f64(kp), f64(vp), table.cpu().numpy(), lens, window, sinks, dtype,
                      scale or None, skip)
    assert ref.worst(f64(out), want[0], want[2]) <= 1
    assert ref.worst(f64(lse), want[1], want[3]) <= 1
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (4, 4, 128), (8, 8, 64), (32, 4, 128), (6, 2, 64),
                                      (5, 1, 128), (9, 1, 64), (16, 1, 128), (20, 1, 64), (34, 2, 128),
                                      (40, 4, 64), (7, 7, 128), (50, 2, 64), (64, 2, 64), (33, 1, 64)])
@pytest.mark.parametrize("page", [16, 64])
def test_decode_heads_and_lengths(hga, dtype, Hq, Hkv, D, page):
    """Lengths of nothing, one token, and both sides of pages, tiles and units."""
    for lens in ([0], [1], [0, 1, 15, 16, 17, 31, 32, 33], [127, 64, 0, 128, 129, 257, 65, 63],
                 [700, 3, 1300]):
        kp, vp, table = pages_for(len(lens), lens, Hkv, D, dtype, page)
        q = queries(7, len(lens), Hq, D, dtype)
        out, _ = check_decode(hga, q, kp, vp, table, lens, dtype)
        again, _ = hga.hga_paged_decode(q, kp, vp, table, i32(lens), want_lse=True)
        assert torch.equal(out, again)
    assert hga.hga_device_status() == 0


@pytest.mark.parametrize("dtype,Hq,Hkv,D", [("bf16", 8, 4, 64), ("f32", 2, 1, 128), ("bf16", 12, 2, 128)])
@pytest.mark.parametrize("page", [1, 2, 8, 128, 1024])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (37, 5), (100, 64), (64, 300),
                                          (5000, 3), (0, 9)])
def test_decode_window_and_sinks(hga, dtype, Hq, Hkv, D, page, window, sinks):
    lens = [0, 1, 2, 5, 37, 100, 141, 401, 900]
    kp, vp, table = pages_for(window + page, lens, Hkv, D, dtype, page)
    q = queries(sinks, len(lens), Hq, D, dtype)
    check_decode(hga, q, kp, vp, table, lens, dtype, window, sinks)
    assert hga.hga_device_status() == 0


def test_decode_window_reads_no_page_outside(hga):
    """Table entries of pages that hold no visible token may be anything."""
    lens, page = [513, 300, 40], 16
    kp, vp, table = pages_for(1, lens, 2, 64, "bf16", page)
    q = queries(1, 3, 4, 64, "bf16")
    out, _ = check_decode(hga, q, kp, vp, table, lens, "bf16", window=64, sinks=20)
    t2 = table.clone()
    for b, n in enumerate(lens):
        for j in range(table.shape[1]):
            if not any(t // page == j for t in ref.visible(n, 64, 20)):
                t2[b, j] = 1 << 30
    assert torch.equal(hga.hga_paged_decode(q, kp, vp, t2, i32(lens), window=64, sinks=20), out)
    assert hga.hga_device_status() == 0


@pytest.mark.parametrize("dtype,Hq,Hkv,D,lens", [
    ("bf16", 8, 1, 128, [20000]), ("bf16", 4, 4, 64, [9000, 1, 0, 4000]), ("f32", 3, 1, 64, [6000, 5000]),
    ("bf16", 16, 2, 64, [30, 12000, 64, 640] * 3), ("f32", 16, 8, 128, [33] * 100 + [2000])])
def test_decode_split_rows_are_joined(hga, dtype, Hq, Hkv, D, lens):
    """Rows longer than one CTA's share, next to short and empty ones."""
    kp, vp, table = pages_for(3, lens, Hkv, D, dtype, 32)
    q = queries(3, len(lens), Hq, D, dtype)
    a, la = check_decode(hga, q, kp, vp, table, lens, dtype)
    b, lb = hga.hga_paged_decode(q, kp, vp, table, i32(lens), want_lse=True)
    assert torch.equal(a, b) and torch.equal(la, lb)
    # a wider table changes the launch, not what is attended
    wide = torch.full((len(lens), 4 * table.shape[1]), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    check_decode(hga, q, kp, vp, wide, lens, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_more_rows_than_ctas(hga, dtype):
    """More items than CTAs (joins are then found by CTA), with empty rows among them."""
    rng = np.random.default_rng(2)
    lens = rng.integers(0, 150, 700).tolist()
    lens[5], lens[699], lens[0] = 2500, 0, 0
    kp, vp, table = pages_for(9, lens, 1, 64, dtype, 16)
    q = queries(9, 700, 2, 64, dtype)
    check_decode(hga, q, kp, vp, table, lens, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_large_scores(hga, dtype):
    """Scores of hundreds, both signs: the running maximum has to carry the sums,
    and rising and falling orders of it both occur."""
    lens = [300, 333]
    kp, vp, table = pages_for(5, lens, 2, 64, dtype, 16)
    ramp = torch.linspace(-20, 20, 16, device="cuda").view(1, 16, 1, 1).to(kp.dtype)
    q = queries(5, 2, 4, 64, dtype, size=8.0)
    check_decode(hga, q, kp * ramp, vp, table, lens, dtype)
    check_decode(hga, q, kp * ramp.flip(1), vp, table, lens, dtype, scale=0.5)
    check_decode(hga, q, kp * ramp, vp, table, lens, dtype, window=50, sinks=9)


def test_decode_nan_and_infinity_at_attended_keys(hga):
    """What is attended counts: a NaN key reaches its heads' rows and no others."""
    lens = [1, 200, 90]
    kp, vp, table = pages_for(5, lens, 2, 64, "bf16", 16, junk=float("inf"))
    q = queries(5, 3, 4, 64, "bf16")
    clean, _ = check_decode(hga, q, kp, vp, table, lens, "bf16")
    kp[table[0, 0], 0, 1] = float("nan")
    vp[table[1, 3], 2, 0, 7] = float("nan")
    out, lse = hga.hga_paged_decode(q, kp, vp, table, i32(lens), want_lse=True)
    assert out[0, 2:].isnan().all() and lse[0, 2:].isnan().all()
    assert torch.equal(out[0, :2], clean[0, :2]) and torch.equal(out[2], clean[2])
    assert out[1, :2, 7].isnan().all() and not out[1, 2:].isnan().any()


def test_decode_bad_pages_and_lengths_are_reported(hga):
    """Keys of a bad page are left out, a bad length counts as none; others are served."""
    lens, page = [100, 64, 40], 16
    kp, vp, table = pages_for(6, lens, 2, 64, "bf16", page)
    q = queries(6, 3, 4, 64, "bf16")
    clean, _ = check_decode(hga, q, kp, vp, table, lens, "bf16")
    for bad in (-1, kp.shape[0], 2 ** 31 - 1, -2 ** 31):
        t2 = table.clone()
        t2[0, 2] = bad
        t2[1, :] = bad
        check_decode(hga, q, kp, vp, t2, lens, "bf16", skip=(bad,))
        assert hga.hga_device_status() == 5 and hga.hga_device_status() == 0
    for bad in (-1, table.shape[1] * page + 1, 2 ** 31 - 1, -2 ** 31):
        out, lse = hga.hga_paged_decode(q, kp, vp, table, i32([bad, 64, 40]), want_lse=True)
        assert not out[0].any() and (lse[0] == -math.inf).all() and torch.equal(out[1:], clean[1:])
        assert hga.hga_device_status() == 5 and hga.hga_device_status() == 0


def test_decode_page_written_twice_and_shared(hga):
    """Two sequences may share pages (a common prefix), one row may hold a page twice."""
    kp, vp, table = pages_for(8, [64, 64], 2, 64, "bf16", 16)
    table[1, :3] = table[0, :3]
    table[0, 1] = table[0, 0]
    check_decode(hga, queries(8, 2, 4, 64, "bf16"), kp, vp, table, [64, 60], "bf16")


def test_decode_offsets_beyond_32_bits(hga):
    """Pools of more than 2^32 bytes: rows at their far end are found."""
    page, Hkv, D = 64, 8, 128
    P = (1 << 32) // (page * Hkv * D * 2) + 40
    kp = torch.zeros(P, page, Hkv, D, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    lens, rows = [130, 64], [P - 1, P - 3, 0, P - 2]
    g = torch.Generator(device="cuda").manual_seed(1)
    for r in rows:
        kp[r].normal_(generator=g)
        vp[r].normal_(generator=g)
    table = i32([[P - 1, 0, P - 3], [P - 2, -1, -1]])
    q = queries(2, 2, 16, D, "bf16")
    out, lse = hga.hga_paged_decode(q, kp, vp, table, i32(lens), want_lse=True)
    small = {p: i for i, p in enumerate(rows)}
    t2 = np.array([[small[P - 1], small[0], small[P - 3]], [small[P - 2], 0, 0]])
    want = ref.decode(f64(q), f64(kp[rows]), f64(vp[rows]), t2, lens, 0, 0, "bf16")
    assert ref.worst(f64(out), want[0], want[2]) <= 1 and ref.worst(f64(lse), want[1], want[3]) <= 1
    # and written: the last slot of the pool
    _, q1, k1, v1 = qkv(3, 1, 8, 8, D, "bf16")
    hga.hga_qk_norm_rope(q1, k1, v1, i32([5]), hga.HGARope(), k_pages=kp, v_pages=vp,
                         slot=i32([P * page - 1]))
    assert torch.equal(vp[P - 1, page - 1], v1[0])


# -------------------------------------------- streams, graphs, workspaces --

def test_decode_workspace_needs_no_value_and_is_shared_in_order(hga):
    """Calls of different shapes on one workspace of anything; a second stream."""
    sizes = [([300, 20], 8, 2, 64), ([5000], 8, 1, 128), ([40] * 90, 4, 4, 64)]
    ws = torch.full((1 << 26,), 0xFF, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    for rep in range(2):
        for lens, Hq, Hkv, D in sizes:
            kp, vp, table = pages_for(4, lens, Hkv, D, "bf16", 16)
            q = queries(4, len(lens), Hq, D, "bf16")
            check_decode(hga, q, kp, vp, table, lens, "bf16", workspace=ws)
            torch.cuda.synchronize()
            check_decode(hga, q, kp, vp, table, lens, "bf16", stream=side) if rep == 0 else None
            torch.cuda.synchronize()


def test_two_decodes_at_once(hga):
    """Two streams, each with its own workspace, at the same time."""
    jobs = []
    for i in range(2):
        lens = [4000 + 100 * i, 17, 2500]
        kp, vp, table = pages_for(20 + i, lens, 4, 128, "bf16", 16)
        jobs.append((queries(i, 3, 32, 128, "bf16"), kp, vp, table, i32(lens), torch.cuda.Stream()))
    alone = [hga.hga_paged_decode(*j[:5]) for j in jobs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [hga.hga_paged_decode(*j[:5], stream=j[5]) for j in jobs]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone, got))


def test_captured_step_follows_the_lengths(hga):
    """plan, norms and rotation, attention in one CUDA graph: replays follow the
    lengths on the device, row by row as eager steps do; two graphs share a workspace."""
    torch.manual_seed(0)
    B, page, Hq, Hkv, D, n = 5, 4, 8, 2, 64, 8
    rope = hga.HGARope(theta=1e4)
    wq, wk = weights(0, D, "bf16")

    def cache():
        c = hga.PagedKVCache(B, 40, page, 12, Hkv, D, torch.bfloat16)
        return c, torch.zeros(B, dtype=torch.int32, device="cuda"), \
            torch.zeros(n, (Hq + 2 * Hkv), D, dtype=torch.bfloat16, device="cuda"), \
            torch.zeros(B, dtype=torch.int32, device="cuda")

    def step(c, new, x, rel, ws):
        p = hga.hga_paged_plan(c.lens, new, c.free_pages, c.free_count, c.block_table, page, n,
                               release=rel, lens_out=c.lens, free_count_out=c.free_count)
        q, _, _ = hga.hga_qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], p["pos"], rope,
                                       q_weight=wq, k_weight=wk, k_pages=c.k_pages,
                                       v_pages=c.v_pages, slot=p["slot"])
        last = (p["cu_tokens"][1:] - 1).clamp(min=0).long()
        return hga.hga_paged_decode(q[last], c.k_pages, c.v_pages, c.block_table, c.lens,
                                    workspace=ws), p

    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    eager, graphed = cache(), cache()
    step(*cache(), ws)                                    # loads the kernels
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(*graphed, ws)
        graphs.append((g, out))
    rng = np.random.default_rng(0)
    for i in range(30):
        new = i32(rng.multinomial(rng.integers(0, n + 1), np.ones(B) / B))
        x = torch.randn(n, Hq + 2 * Hkv, D).to(torch.bfloat16).cuda()
        rel = i32(rng.random(B) < 0.1)
        for _, a, b, c in (eager, graphed):
            a.copy_(new), b.copy_(x), c.copy_(rel)
        want, p = step(*eager, ws)
        g, (got, pg) = graphs[i % 2]
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(want, got)
        for k in p:
            assert torch.equal(p[k], pg[k]), k
        for a, b in zip(vars(eager[0]).values(), vars(graphed[0]).values()):
            assert not isinstance(a, torch.Tensor) or torch.equal(a, b)
    assert hga.hga_device_status() == 0


def test_allocations_of_another_stream_do_not_wait_for_this_one(hga):
    """With `stream`, a call's new tensors come from that stream's memory: a block that
    the current stream has freed but still writes to is not handed out."""
    _, q, k, v = qkv(1, 1024, 8, 2, 64, "bf16")
    pos = i32(np.arange(1024))
    want = hga.hga_qk_norm_rope(q, k, v, pos, hga.HGARope())
    kp, vp, table = pages_for(1, [200] * 64, 2, 64, "bf16", 16)
    qd, lens = queries(1, 64, 64, 64, "bf16"), i32([200] * 64)
    dec = hga.hga_paged_decode(qd, kp, vp, table, lens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for op, ref_out in ((lambda: hga.hga_qk_norm_rope(q, k, v, pos, hga.HGARope(), stream=side), want),
                        (lambda: (hga.hga_paged_decode(qd, kp, vp, table, lens, stream=side),), (dec,))):
        late = [torch.empty_like(t) for t in ref_out]
        torch.cuda._sleep(200_000_000)
        for t in late:
            t.fill_(7.0)
        del late, t
        got = op()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref_out))


def test_results_are_ordinary_tensors(hga):
    """What comes back can be changed in place and differentiated through."""
    _, q, k, v = qkv(1, 6, 4, 2, 64, "f32")
    o = list(hga.hga_qk_norm_rope(q, k, v, i32(np.arange(6)), hga.HGARope()))
    p = hga.hga_paged_plan(i32([1, 2]), i32([1, 1]), i32([2, 3]), i32([2]), i32([[0, 0], [1, 0]]), 4, 4)
    before = {n: t.clone() for n, t in p.items()}
    p["slot"].add_(5)
    assert all(torch.equal(p[n], before[n] + (5 if n == "slot" else 0)) for n in p)
    for t in o:
        assert not t.is_inference() and not t.requires_grad
        t.mul_(2.0).requires_grad_()
    sum((t * t).sum() for t in o).backward()
    assert all(torch.equal(t.grad, 2 * t) for t in o)


def test_binding_refusals(hga):
    """Tensors of the wrong kind are refused with a message before anything runs."""
    rope = hga.HGARope()
    x, q, k, v = qkv(1, 6, 4, 2, 64, "bf16")
    pos = i32(np.arange(6))
    kp, vp, table = pages_for(1, [20, 3], 2, 64, "bf16", 16)
    qd, lens = queries(1, 2, 4, 64, "bf16"), i32([20, 3])
    d = [torch.zeros(6, h, 64, device="cuda") for h in (4, 2, 2)]
    slot = i32(np.arange(6))
    cases = [
        lambda: hga.hga_qk_norm_rope(q.cpu(), k, v, pos, rope),
        lambda: hga.hga_qk_norm_rope(q.half(), k.half(), v.half(), pos, rope),
        lambda: hga.hga_qk_norm_rope(q, k.float(), v, pos, rope),
        lambda: hga.hga_qk_norm_rope(q, k[:5], v, pos, rope),
        lambda: hga.hga_qk_norm_rope(q[..., :32], k[..., :32], None, pos, hga.HGARope(0)),
        lambda: hga.hga_qk_norm_rope(q[:, ::2], k, v, pos, rope),
        lambda: hga.hga_qk_norm_rope(q[:1].expand(6, 4, 64), k, v, pos, rope),
        lambda: hga.hga_qk_norm_rope(q.transpose(-1, -2), k, v, pos, rope),
        lambda: hga.hga_qk_norm_rope(q, k, v, pos.long(), rope),
        lambda: hga.hga_qk_norm_rope(q, k, v, pos[:5], rope),
        lambda: hga.hga_qk_norm_rope(q, k, v, None, rope),
        lambda: hga.hga_qk_norm_rope(q, k, v, pos, rope, q_weight=torch.ones(64, device="cuda")),
        lambda: hga.hga_qk_norm_rope(q, k, v, pos, rope, k_pages=kp, slot=slot),
        lambda: hga.hga_qk_norm_rope(q, k, v, pos, rope, k_pages=kp, v_pages=vp),
        lambda: hga.hga_qk_norm_rope(q, k, v, pos, rope, k_pages=kp, v_pages=vp.float(), slot=slot),
        lambda: hga.hga_qk_norm_rope(q, k, None, pos, rope, v_out=d[1]),
        lambda: hga.hga_qk_norm_rope(q, k, v, pos, rope, q_out=d[0]),
        lambda: hga.hga_qk_norm_rope(q, k, v, pos, rope, eps=-1.0),
        lambda: hga.hga_qk_norm_rope(q, k, v, pos, rope._replace(layout="neox")),
        lambda: hga.hga_qk_norm_rope(q, k, v, pos, rope._replace(scaling="ntk")),
        lambda: hga.hga_qk_norm_rope(q, k, v, pos, rope._replace(rotary_dim=24)),
        lambda: hga.hga_qk_norm_rope(q, k, v, pos, "half"),
        lambda: hga.hga_qk_norm_rope(q.unflatten(0, (2, 3)), k, v, pos, rope),
        lambda: hga.hga_qk_norm_rope(x[:, 4:260].unflatten(-1, (4, 64)), k, v, pos, rope),  # 8 bytes off
        lambda: hga.hga_qk_norm_rope_backward(q, k, d[0].half(), d[1].half(), pos, rope),
        lambda: hga.hga_qk_norm_rope_backward(q, k, d[0], d[1].bfloat16(), pos, rope),
        lambda: hga.hga_qk_norm_rope_backward(q, k, d[0], d[1], pos, rope, dv=d[2]),
        lambda: hga.hga_qk_norm_rope_backward(q, k, d[0], d[1], pos, rope, dq=d[0]),
        lambda: hga.hga_qk_norm_rope_backward(q, k, d[0], d[1], pos, rope,
                                              workspace=torch.empty(8, device="cuda"),
                                              q_weight=torch.ones(64, device="cuda").bfloat16()),
        lambda: hga.hga_paged_decode(qd.float(), kp, vp, table, lens),
        lambda: hga.hga_paged_decode(qd[:, ::2], kp, vp, table, lens),
        lambda: hga.hga_paged_decode(qd, kp, vp[:1], table, lens),
        lambda: hga.hga_paged_decode(qd, kp.transpose(1, 2), vp.transpose(1, 2), table, lens),
        lambda: hga.hga_paged_decode(qd, kp, vp, table.t(), lens),
        lambda: hga.hga_paged_decode(qd, kp, vp, table, lens.long()),
        lambda: hga.hga_paged_decode(qd, kp, vp, table, lens[:1]),
        lambda: hga.hga_paged_decode(qd[:, :3], kp, vp, table, lens),
        lambda: hga.hga_paged_decode(qd, kp, vp, table, lens, window=-1),
        lambda: hga.hga_paged_decode(qd, kp, vp, table, lens, window=1 << 31),
        lambda: hga.hga_paged_decode(qd, kp, vp, table, lens, window=5, sinks=-2),
        lambda: hga.hga_paged_decode(qd, kp, vp, table, lens, scale=-1.0),
        lambda: hga.hga_paged_decode(qd, kp, vp, table, lens, out=qd.float()),
        lambda: hga.hga_paged_decode(qd, kp, vp, table, lens, workspace=torch.empty(64, device="cuda")),
        lambda: hga.hga_paged_decode(qd[:0], kp, vp, table[:0], lens[:0]),
        lambda: hga.hga_paged_plan(lens, lens, slot, i32([0]), table, 3, 4),
        lambda: hga.hga_paged_plan(lens, lens, slot, i32([0]), table, 16, -1),
        lambda: hga.hga_paged_plan(lens, lens.long(), slot, i32([0]), table, 16, 4),
        lambda: hga.hga_paged_plan(lens[:1], lens, slot, i32([0]), table, 16, 4),
        lambda: hga.hga_paged_plan(lens, lens, slot, i32([0]), table, 16, 4, slot=slot),
        lambda: hga.hga_paged_plan(lens, lens, slot, i32([0, 0]), table, 16, 4),
        lambda: hga.hga_paged_plan(lens, lens, slot, i32([0]), table[0], 16, 4),
    ]
    before = x.clone()
    for i, call in enumerate(cases):
        with pytest.raises(hga.HGAError):
            call()
            pytest.fail(f"case {i} was not refused")
    torch.cuda.synchronize()
    assert torch.equal(before, x) and hga.hga_device_status() == 0


def test_captured_gradient_follows_its_inputs(hga):
    """The gradient in two CUDA graphs on one workspace: replays follow the inputs, in a
    batched [B, T] layout with an odd head count."""
    N, Hq, Hkv, D = 22, 5, 1, 64
    rope = hga.HGARope(rotary_dim=32, layout="interleaved", theta=1e4)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    w = weights(3, D, "bf16")
    x, q, k, v = qkv(1, N, Hq, Hkv, D, "bf16")
    d = [torch.randn(2, N // 2, h, D, device="cuda") for h in (Hq, Hkv, Hkv)]
    pos = i32(np.arange(N).reshape(2, -1))

    def call(ws=None):
        return hga.hga_qk_norm_rope_backward(q.unflatten(0, (2, -1)), k.unflatten(0, (2, -1)), d[0], d[1],
                                             pos, rope, q_weight=w[0], k_weight=w[1], d_v=d[2],
                                             workspace=ws)
    call(ws)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call(ws)
        graphs.append((g, out))
    for i in range(4):
        x.copy_(qkv(50 + i, N, Hq, Hkv, D, "bf16")[0])
        d[0].normal_(), pos.add_(i)
        want = call()
        g, got = graphs[i % 2]
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_first_calls_in_a_capture(hga):
    """A process whose first call of every operator is captured: the graph replays."""
    import os
    import subprocess
    import sys
    code = """
import torch, hierarchical_kv_routing_b200 as hga
z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)
i = lambda *s: z(*s, dtype=torch.int32)
c = hga.PagedKVCache(2, 8, 4, 4, 2, 64, torch.bfloat16)
new, x, w = i(2) + 1, torch.randn(2, 8, 64, device="cuda").bfloat16(), z(64).bfloat16() + 1
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    p = hga.hga_paged_plan(c.lens, new, c.free_pages, c.free_count, c.block_table, 4, 2,
                           lens_out=c.lens, free_count_out=c.free_count)
    q, _, _ = hga.hga_qk_norm_rope(x[:, :4], x[:, 4:6], x[:, 6:], p["pos"], hga.HGARope(), q_weight=w,
                                   k_weight=w, k_pages=c.k_pages, v_pages=c.v_pages, slot=p["slot"])
    out = hga.hga_paged_decode(q, c.k_pages, c.v_pages, c.block_table, c.lens)
    grads = hga.hga_qk_norm_rope_backward(x[:, :4], x[:, 4:6], q, q[:, :2].contiguous(), p["pos"],
                                          hga.HGARope(), q_weight=w, k_weight=w)
g.replay()
torch.cuda.synchronize()
assert c.lens.tolist() == [1, 1] and torch.equal(out[:, :2], x[:, 6:7].expand(2, 2, 64))
assert all(t is None or t.isfinite().all() for t in grads) and hga.hga_device_status() == 0
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


# ------------------------------------------------------ a run of them all --

@pytest.mark.parametrize("dtype,layout", [("bf16", "half"), ("f32", "interleaved")])
def test_serving_run_against_dense_attention(hga, dtype, layout):
    """Prompts of several lengths, then steps of one token, rows released and taken
    again: every step's attention equals dense attention over what was written."""
    B, page, Hq, Hkv, D, window, sinks = 4, 8, 6, 2, 64, 24, 3
    c = hga.PagedKVCache(B, 30, page, 12, Hkv, D, DT[dtype])
    rope = hga.HGARope(theta=1e4, layout=layout, rotary_dim=32)
    wq, wk = weights(2, D, dtype)
    rng = np.random.default_rng(1)
    kept = {b: ([], []) for b in range(B)}
    plans = [([17, 0, 40, 8], None)] + [([1, 0, 1, 1], None)] * 3 + [([1, 30, 20, 1], [0, 0, 1, 0])] \
        + [([1, 1, 1, 1], None)] * 10
    for i, (new, rel) in enumerate(plans):
        N = sum(new)
        _, q, k, v = qkv(100 + i, N, Hq, Hkv, D, dtype)
        p = hga.hga_paged_plan(c.lens, i32(new), c.free_pages, c.free_count, c.block_table, page, N,
                               release=None if rel is None else i32(rel), lens_out=c.lens,
                               free_count_out=c.free_count)
        assert p["granted"].tolist() == new
        # the dense outputs of a second call are what the pages must hold
        qo, _, _ = hga.hga_qk_norm_rope(q, k, v, p["pos"], rope, q_weight=wq, k_weight=wk,
                                        k_pages=c.k_pages, v_pages=c.v_pages, slot=p["slot"])
        _, ko, vo = hga.hga_qk_norm_rope(q, k, v, p["pos"], rope, q_weight=wq, k_weight=wk)
        at = 0
        for b in range(B):
            if rel is not None and rel[b]:
                kept[b] = ([], [])
            for t in range(at, at + new[b]):
                kept[b][0].append(f64(ko[t]))
                kept[b][1].append(f64(vo[t]))
            at += new[b]
        ends = torch.tensor(np.maximum(np.cumsum(new) - 1, 0), device="cuda")
        ql = qo[ends].contiguous()
        lens = [len(kept[b][0]) for b in range(B)]
        assert c.lens.tolist() == lens
        for w, s in ((0, 0), (window, sinks)):
            out, lse = hga.hga_paged_decode(ql, c.k_pages, c.v_pages, c.block_table, c.lens, window=w,
                                            sinks=s, want_lse=True)
            top = max(max(lens), 1)
            kk, vv = np.zeros((B, top, Hkv, D)), np.zeros((B, top, Hkv, D))
            for b in range(B):
                if lens[b]:
                    kk[b, :lens[b]], vv[b, :lens[b]] = np.stack(kept[b][0]), np.stack(kept[b][1])
            want = ref.decode(f64(ql), kk, vv, np.arange(B)[:, None], lens, w, s, dtype)
            assert ref.worst(f64(out), want[0], want[2]) <= 1
            assert ref.worst(f64(lse), want[1], want[3]) <= 1
    assert rng is not None and hga.hga_device_status() == 0


def test_training_run_through_routed_attention(hga):
    """Fused QKV -> norms (no rotation) -> routed attention with every group opened
    -> its backward -> the norms' backward: the gradients of the fused buffer and of
    the weights equal automatic differentiation of dense attention in 64 bits."""
    N, Hq, Hkv, D, theta = 192, 4, 2, 64, 1e4
    prm = hga.HGAParams(F=1, L=1, K_c=8, K_g=32, g_s=16, rope_theta=theta)
    x, q, k, v = qkv(11, N, Hq, Hkv, D, "f32")
    wq, wk = weights(12, D, "f32")
    pos = i32(np.arange(N))[None]
    none = hga.HGARope(rotary_dim=0)
    qn, kn, vn = hga.hga_qk_norm_rope(q[None], k[None], v[None], None, none, q_weight=wq, k_weight=wk)
    k_rot, s_c, s_g = hga.hga_build_summaries(kn, pos, prm)
    _, sel = hga.hga_route(qn, pos, s_c, s_g, prm)
    out, lse = hga.hga_attend(qn, pos, k_rot, vn, sel, prm, want_lse=True)
    d_out = torch.randn(out.shape, generator=torch.Generator().manual_seed(1)).cuda()
    dqn, dkn, dvn = hga.hga_attend_backward(qn, pos, k_rot, vn, sel, lse, d_out, prm)
    dx = torch.empty_like(x)
    views = [dx[None, :, a * D:b * D].unflatten(-1, (-1, D)) for a, b in
             ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv))]
    _, _, _, dwq, dwk = hga.hga_qk_norm_rope_backward(
        q[None], k[None], dqn, dkn, None, none, q_weight=wq, k_weight=wk, d_v=dvn, dq=views[0],
        dk=views[1], dv=views[2])

    X, W1, W2 = (t.double().cpu().requires_grad_() for t in (x, wq, wk))
    h = X.view(N, -1, D)
    ang = torch.arange(N).double()[:, None] * theta ** (-2 * torch.arange(D // 2).double() / D)

    def turned(y, w):
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w
        z = torch.complex(y[..., :D // 2], y[..., D // 2:]) * torch.polar(torch.ones_like(ang), ang)[:, None]
        return torch.cat([z.real, z.imag], -1)
    Q, K = turned(h[:, :Hq], W1), turned(h[:, Hq:Hq + Hkv], W2)
    K, V = (t.repeat_interleave(Hq // Hkv, 1) for t in (K, h[:, Hq + Hkv:]))
    s = torch.einsum("ihd,jhd->hij", Q, K) / math.sqrt(D)
    s = s.masked_fill(torch.triu(torch.ones(N, N, dtype=torch.bool), 1), -math.inf)
    O = torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), V)
    (O * d_out[0].double().cpu()).sum().backward()
    # fp32 throughout: the attention backward is held to 1e-5 of its terms' magnitude
    # (and normwise), the norms add 64 F; normwise, with cancellation, 2e-5
    for got, want in ((dx, X.grad), (dwq, W1.grad), (dwk, W2.grad)):
        e = got.double().cpu() - want
        assert float(e.norm() / want.norm()) <= 2e-5
    O = O.detach()
    assert float((out[0].double().cpu() - O).abs().max()) <= 1e-5 * float(O.abs().max())
