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
