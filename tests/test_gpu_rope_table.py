"""Rotary tables to the last bit of fp32."""
import pytest
import torch

import attn_fwd_04_b200 as fa
import serving_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,R,kw", [
    (1, 2, {}), (1000, 128, {}), (131072, 64, {}), (1 << 21, 16, {}),
    (131072, 128, dict(base=500000.0, scaling="yarn", factor=4.0, original=32768, low=1.0,
                       high=32.0, mscale=1.1386)),
    (40001, 96, dict(base=500000.0, scaling="turns", factor=8.0, original=8192)),
    (70000, 32, dict(base=1e6, scaling="ntk", factor=2.5)),
    (5000, 256, dict(scaling="linear", factor=3.0, mscale=0.1))])
def test_every_entry(n, R, kw):
    """An entry is rounded once to fp32 (half a step: 2^-24 of it).  Before that, in
    fp64: a frequency, base^(-2i/R), is good to some 2^-47 of itself (an exponent of up
    to 24 rounded twice, an exponential, a division), and so is its angle; a run of 16
    positions adds 16 times three roundings and the error of the step's sine and cosine,
    below 2^-46."""
    kw = dict(kw)
    mscale = kw.pop("mscale", 1.0)
    cos, sin = fa.fa_rope_table(n, R, kw.get("base", 10000.0), kw.get("scaling", "none"),
                                kw.get("factor", 1.0), kw.get("original", 0), kw.get("low", 1.0),
                                kw.get("high", 4.0), mscale)
    assert fa.fa_get_device_error() == fa.FA_OK
    ang = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * \
        ref.frequencies(R, **kw).cuda()
    for got, want in ((cos, ang.cos() * mscale), (sin, ang.sin() * mscale)):
        tol = 2.0 ** -24 * want.abs() + mscale * 2.0 ** -45 * (1 + ang)
        assert ((got.double() - want).abs() <= tol).all()
