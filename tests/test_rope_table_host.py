"""Refusals of rotary tables beyond those of single arguments, without a GPU."""
import pytest

import attn_fwd_04_b200 as fa
from attn_fwd_04_b200 import build as fa_build

A = 1 << 20  # never dereferenced


@pytest.mark.parametrize("kind", [1, 3, 4])
def test_angles_out_of_range(kind):
    """Frequencies divided by next to nothing, and their products with a position."""
    fa_build.build()
    for factor, n in ((1e-320, 64), (1e-306, 1 << 30)):
        assert fa.lib().fa_rope_table(A, A, n, 64, 1e4, kind, factor, 64, 1.0, 4.0, 1.0,
                                      None) == fa.FA_ERR_SHAPE


@pytest.mark.parametrize("R,base,factor", [(4, 1e200, 1e200), (4, 1e10, 1e-200),
                                           (64, 1e300, 1e300), (128, 5e5, 1e308)])
def test_a_scaled_base_out_of_range(R, base, factor):
    """base * factor^(R/(R-2)) overflows, or vanishes: its powers would be NaN."""
    fa_build.build()
    new = float(base)
    try:
        new *= factor ** (R / (R - 2))
    except OverflowError:
        new = float("inf")
    assert new == float("inf") or new == 0.0
    assert fa.lib().fa_rope_table(A, A, 64, R, base, 2, factor, 0, 0.0, 0.0, 1.0,
                                  None) == fa.FA_ERR_SHAPE
