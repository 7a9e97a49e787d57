"""Values at the edges of the types through the token preparation and the attention behind a prefix.

Tolerances are those of the tests whose inputs and checks are used here.
"""

import pytest

from test_qk_rope import Inputs

import scaled_dot_product_vt_gb300 as vt


@pytest.fixture(scope="module", autouse=True)
def _built():
    vt.build()
    vt.load()


# ---------------------------------------------------------------- token preparation

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("exponent", [-60, -47, 50, 58])
def test_rows_of_any_size_whose_squares_stay_in_range(dtype, exponent):
    """Rows of 2^exponent with eps = 0: mean(x^2) is a normal number, and so are both directions' results, while the
    third power of 1 / rms is not."""
    x = Inputs(dtype, 2, 3, 1, 20, 64, 48, 2, True, True, seed=13)
    for t, a in ((x.q, x.q64), (x.k, x.k64)):
        t.mul_(2.0 ** exponent)  # (exact)
        a *= 2.0 ** exponent
    x.eps = 0.0
    x.check_forward(*vt.qk_rope(x.q, x.k, x.freqs, x.pos, **x.form()))
    x.check_backward(*vt.qk_rope_bwd(x.gq, x.gk, x.freqs, x.pos, q=x.q, k=x.k, **x.form()))
