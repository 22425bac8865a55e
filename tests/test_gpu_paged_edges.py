"""The paged-cache operators on the GPU at the edges of what they accept, against
their definitions in 64 bits."""
import numpy as np
import pytest
import torch

from tests import paged_reference as ref
from tests.test_gpu_paged import f64, i32, pages_for, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hga(gpu_lib):
    return gpu_lib


# --------------------------------------------------------------- decode --

@pytest.mark.parametrize("Hq,Hkv,D", [(4, 4, 128), (32, 4, 128), (16, 1, 128), (20, 1, 128), (8, 8, 64),
                                      (3, 1, 64), (16, 1, 64), (24, 1, 64), (64, 2, 64)])
def test_decode_weights_keep_16_bits(hga, Hq, Hkv, D):
    """The softmax weights' product with bf16 values, entry by entry where the sum is
    small against its terms.

    A weight is taken as the sum of two bf16: the first at most 2^-7 of it short, the
    second the rest, rounded by at most half a step: 2^-7 2^-8 = 2^-15 of the weight.
    Everything else of the bound is the definition's for fp32, and one rounding of
    the output; a single bf16 weight may be 2^-8 off."""
    lens = [48, 33, 7, 64, 1, 30, 17, 52]
    kp, vp, table = pages_for(Hq, lens, Hkv, D, "bf16", 16)
    q = queries(Hq + 1, len(lens), Hq, D, "bf16")
    out, lse = hga.hga_paged_decode(q, kp, vp, table, i32(lens), want_lse=True)
    want, wlse, bound, blse = ref.decode(f64(q), f64(kp), f64(vp), table.cpu().numpy(), lens, 0, 0, "f32")
    mag = ref.decode(f64(q), f64(kp), np.abs(f64(vp)), table.cpu().numpy(), lens, 0, 0, "f32")[0]
    bound = bound + 2.0 ** -15 * mag + ref.STEP["bf16"] * np.abs(want)
    assert ref.worst(f64(out), want, bound) <= 1
    assert ref.worst(f64(lse), wlse, blse) <= 1


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 128), (16, 1, 128), (6, 2, 64), (24, 1, 64)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_decode_infinite_values_stay_infinite(hga, Hq, Hkv, D, sign):
    """A value of infinity under a positive weight gives infinity, whatever bits the
    weight has: weights of 1 (a row's first maximum), of a power of two, and others."""
    for lens in ([1], [2], [40], [16, 200]):
        kp, vp, table = pages_for(D, lens, Hkv, D, "bf16", 16, junk=0.0)
        q = queries(5, len(lens), Hq, D, "bf16", size=0.5)
        if lens == [2]:
            q.zero_()                                  # both weights 1
        n = lens[-1] - 1
        vp[table[-1, n // 16], n % 16, :, 3] = sign * float("inf")
        out = hga.hga_paged_decode(q, kp, vp, table, i32(lens))
        assert (out[-1, :, 3] == sign * float("inf")).all()
        rest = torch.cat([out[-1, :, :3], out[-1, :, 4:]], -1)
        assert torch.isfinite(rest).all() and torch.isfinite(out[:-1]).all()


@pytest.mark.parametrize("dtype,D,off", [("bf16", 64, 0), ("bf16", 128, 5), ("f32", 128, 0), ("f32", 64, 17)])
def test_decode_rows_of_the_largest_size(hga, dtype, D, off):
    """A row within a unit of 2^31 keys (pages are shared, so it takes little memory):
    all of it, and with a window at its far end.

    The keys of the last two pages score 40, all others 0, so that these m keys make the
    result: the n others together weigh n e^-40 < 2^-26 of one of them.  lse = 40 +
    log(m + (n - m) e^-40): the score, its scale and the sum are a few roundings of
    fp32 at 43 and below, less than 2^-18 40 = 1.5e-4 together, where one key more or
    less of m <= 32 is 0.03.  The m scores are equal, so the values' mean is good to
    2^-19 and the output's rounding."""
    page, M = 16, (1 << 27) - 1
    n = M * page - off
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    kp = torch.zeros(3, page, 1, D, dtype=dt, device="cuda")
    vp = torch.ones(3, page, 1, D, dtype=dt, device="cuda")
    kp[1:] = 8.0
    vp[1], vp[2] = 3.0, 5.0
    table = torch.zeros(1, M, dtype=torch.int32, device="cuda")
    table[0, M - 2], table[0, M - 1] = 1, 2
    q = torch.full((1, 1, D), 0.5, dtype=dt, device="cuda")
    lens = i32([n])
    s = 40.0
    scale = s / (4.0 * D)                         # q.k of the last pages is 4 D
    in1, in2 = page - max(0, off - page), page - min(off, page)
    m = in1 + in2
    want_lse = s + np.log(m + (n - m) * np.exp(-s))
    want = (3.0 * in1 + 5.0 * in2) / m
    out, lse = hga.hga_paged_decode(q, kp, vp, table, lens, scale=scale, want_lse=True)
    assert abs(float(lse) - want_lse) <= 2 ** -18 * s
    assert (out.double() - want).abs().max() <= (2 ** -19 + ref.STEP[dtype]) * want
    out, lse = hga.hga_paged_decode(q, kp, vp, table, lens, scale=scale, want_lse=True, window=100, sinks=7)
    assert abs(float(lse) - (s + np.log(m + (107 - m) * np.exp(-s)))) <= 2 ** -18 * s
    assert (out.double() - want).abs().max() <= (2 ** -19 + ref.STEP[dtype]) * want
    assert hga.hga_device_status() == 0


# ---------------------------------------------------- norms and rotation --

def test_qk_backward_of_no_tokens(hga):
    """Zero gradients of the weights; weights that are not on 16 bytes are refused, as
    with tokens."""
    x = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(72, dtype=torch.bfloat16, device="cuda")
    call = lambda wt: hga.hga_qk_norm_rope_backward(x, x[:, :2], x, x[:, :2], i32([]), hga.HGARope(),
                                                    q_weight=wt, k_weight=w[8:])
    for at in (1, 4):
        with pytest.raises(hga.HGAError):
            call(w[at:at + 64])
    dq, dk, _, dqw, dkw = call(w[:64])
    assert dq.shape == x.shape and not dqw.any() and not dkw.any()
    assert hga.hga_device_status() == 0


def same_bits(a, b):
    """Equal, signs of zero included; NaN where the other is."""
    nan = a.isnan() & b.isnan()
    return bool((((a == b) & (a.signbit() == b.signbit())) | nan).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,R", [(64, 0), (64, 16), (64, 48), (128, 0), (128, 32), (128, 112)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_qk_unrotated_dimensions_pass_through(hga, dtype, D, R, layout):
    """Without a norm the dimensions from rotary_dim on come out as they went in,
    infinity, NaN and -0 included, and reach no other; with one, an infinite value makes
    its row's mean square infinite: 0 everywhere (x times 0) but NaN at itself.  The
    gradient likewise passes what comes in."""
    g = torch.Generator().manual_seed(D + R)
    x = torch.randn(9, 3, D, generator=g).to(dtype).cuda()
    odd = x.clone()
    odd[0, 0, R], odd[1, 1, D - 1], odd[2, 2, R + 5] = float("inf"), -float("inf"), float("nan")
    odd[3, :, R:] = -0.0
    odd[4, 0, R + 2:D] = float("inf")
    pos = i32(np.arange(9) * 1000 + 1)
    rope = hga.HGARope(rotary_dim=R, layout=layout)
    run = lambda t, **kw: hga.hga_qk_norm_rope(t, t, t, pos, rope, **kw)
    clean, got = run(x), run(odd)
    for a, b, v in zip(got[:2], clean[:2], (odd, odd)):
        assert same_bits(a[..., R:], v[..., R:])
        assert same_bits(a[..., :R], b[..., :R])
    back = lambda d: hga.hga_qk_norm_rope_backward(x, x, d, d, pos, rope)[:2]
    for a, b in zip(back(odd), back(x)):
        assert same_bits(a[..., R:], odd[..., R:])
        assert same_bits(a[..., :R], b[..., :R])
    w = torch.ones(D, dtype=dtype, device="cuda")
    for a in run(odd, q_weight=w, k_weight=w)[:2]:
        assert same_bits(a[5:], run(x, q_weight=w, k_weight=w)[0][5:])
        for t, h in ((0, 0), (1, 1), (4, 0)):
            inf = odd[t, h].isinf()
            assert a[t, h][inf].isnan().all() and (a[t, h][~inf] == 0).all()


# ---------------------------------------------------------------- status --

def test_device_status_of_several_operators(hga):
    """One status for every kernel's word: kept until it is cleared, cleared as a whole."""
    def bad_plan():
        hga.hga_paged_plan(i32([-1]), i32([1]), i32([0] * 4), i32([4]), i32([[0]]), 4, 1)

    def bad_slot():
        x = torch.zeros(1, 1, 64, device="cuda")
        kp = torch.zeros(1, 4, 1, 64, device="cuda")
        hga.hga_qk_norm_rope(x, x, x, i32([0]), hga.HGARope(), k_pages=kp, v_pages=kp.clone(), slot=i32([4]))

    def bad_length():
        kp, vp, table = pages_for(1, [4], 1, 64, "f32", 4)
        hga.hga_paged_decode(queries(1, 1, 1, 64, "f32"), kp, vp, table, i32([99]))
    assert hga.hga_device_status() == 0
    for calls in ((bad_plan,), (bad_slot,), (bad_length,), (bad_plan, bad_slot, bad_length)):
        for f in calls:
            f()
        assert hga.hga_device_status(clear=False) == 5
        assert hga.hga_device_status(clear=False) == 5
        assert hga.hga_device_status() == 5 and hga.hga_device_status() == 0
    other = torch.cuda.Stream()
    bad_slot()
    torch.cuda.synchronize()
    assert hga.hga_device_status(stream=other) == 5 and hga.hga_device_status() == 0
    for _ in range(1100):                          # more calls than there are places for a result
        assert hga.hga_device_status(clear=False) == 0


def test_device_status_takes_one_read(hga):
    """A launch and a copy, not a copy for every kernel file's word: against the read of
    one value, which is a copy (measured 2 times; with a copy a word 8)."""
    import time
    x = torch.zeros(1, device="cuda")

    def median(f):
        t = []
        for _ in range(300):
            t0 = time.perf_counter()
            f()
            t.append(time.perf_counter() - t0)
        return sorted(t)[150]
    median(hga.hga_device_status)
    assert min(median(hga.hga_device_status) / median(x.item) for _ in range(3)) < 4


def test_an_argument_without_a_truth_value_raises_its_own_error(hga):
    kp, vp, table = pages_for(1, [4], 1, 64, "bf16", 4)
    with pytest.raises(RuntimeError, match="ambiguous"):
        hga.hga_paged_decode(queries(1, 1, 1, 64, "bf16"), kp, vp, table, i32([4]), want_lse=torch.zeros(2))


def test_weights_that_the_call_before_writes(hga):
    """The gradient of a weight as the next call's weight: the call starts while the one
    before is still running, and reads the weight after it."""
    g = torch.Generator().manual_seed(3)
    x, d = (torch.randn(5000, 3, 64, generator=g).cuda() for _ in range(2))
    w, pos, rope = torch.ones(64, device="cuda"), i32(np.arange(5000)), hga.HGARope()
    out = torch.empty(5000, 3, 64, device="cuda")
    for i in range(20):
        y = x * (i + 1) if i % 2 else x - i
        torch.cuda.synchronize()
        _, _, _, dqw, _ = hga.hga_qk_norm_rope_backward(y, y, d, d, pos, rope, q_weight=w, k_weight=w)
        hga.hga_qk_norm_rope(y, y, None, pos, rope, q_weight=dqw, k_weight=dqw, q_out=out)
        first = out.clone()
        torch.cuda.synchronize()
        hga.hga_qk_norm_rope(y, y, None, pos, rope, q_weight=dqw, k_weight=dqw, q_out=out)
        assert torch.equal(first, out)
