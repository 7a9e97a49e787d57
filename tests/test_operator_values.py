"""Values at the edges of the types through the token preparation and the attention behind a prefix.

Tolerances are those of the tests whose inputs and checks are used here.
"""

import numpy as np
import pytest

from test_attn_prefix import Problem
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


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D,R", [("bf16", 96, 64), ("bf16", 72, 48), ("bf16", 33, 14), ("bf16", 201, 150),
                                       ("f32", 128, 64), ("f32", 36, 10)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_columns_that_are_not_rotated_are_copied(dtype, D, R, interleaved, value):
    """Without the norm, y_j = x_j for j >= R: an infinity or NaN in one of them stays there, in both directions."""
    x = Inputs(dtype, 1, 3, 1, 9, D, R, 1, False, interleaved, seed=14)
    clean = vt.qk_rope(x.q, x.k, x.freqs, x.pos, **x.form())[0].clone()
    clean_b = vt.qk_rope_bwd(x.gq, x.gk, x.freqs, x.pos, **x.form())[0].clone()
    for at in (R, D - 1, (R + D) // 2):
        for t in (x.q, x.gq):
            t[:, 1, 4, at] = value
        clean[:, 1, 4, at] = clean_b[:, 1, 4, at] = value
    got = vt.qk_rope(x.q, x.k, x.freqs, x.pos, **x.form())[0]
    got_b = vt.qk_rope_bwd(x.gq, x.gk, x.freqs, x.pos, **x.form())[0]
    for a, b in ((got, clean), (got_b, clean_b)):
        assert x.torch.equal(a.isnan(), b.isnan()) and x.torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))
    assert x.torch.equal(got[..., R:].nan_to_num(7.0), x.q[..., R:].nan_to_num(7.0))


@pytest.mark.gpu
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_a_frequency_that_is_no_number_reaches_its_pair(value):
    x = Inputs("f32", 1, 2, 1, 7, 32, 32, 1, False, False, seed=15)
    want = vt.qk_rope(x.q, x.k, x.freqs, x.pos, **x.form())[0].clone()
    x.freqs[3] = value
    got = vt.qk_rope(x.q, x.k, x.freqs, x.pos, **x.form())[0]
    pair = [3, 19]
    assert got[..., pair].isnan().all()
    got[..., pair] = want[..., pair]
    assert x.torch.equal(got, want)


# ---------------------------------------------------------------- attention behind a prefix

# streamed once; the prefix in a launch of its own, streamed and on tiles; rows of one sequence on tiles
FORMS = [("f32", 3, 1, 50), ("f32", 40, 1, 1500), ("f32", 2, 40, 100), ("bf16", 3, 1, 50), ("bf16", 90, 1, 1100),
         ("bf16", 2, 70, 300)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,B,S_q,S_p", FORMS)
@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
def test_an_infinite_value_fills_its_column_alone(dtype, B, S_q, S_p, value):
    p = Problem(dtype, B, 4, 2, S_q, S_p, 80, 64, 64, lens=[80] * B, seed=16)
    before = p.run()[0].clone()
    p.vp[:, 7, 11] = value            # every query sees the prefix
    p.vc[0, :, 80 - S_q, 30] = value  # and this row of its own cache
    o, lse = p.run()
    assert (o[..., 11] == value).all() and (o[0, ..., 30] == value).all()
    o[..., 11] = before[..., 11]
    o[0, ..., 30] = before[0, ..., 30]
    p.check(o, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,B,S_q,S_p", FORMS)
def test_a_key_whose_score_is_minus_infinity_has_no_weight(dtype, B, S_q, S_p):
    p = Problem(dtype, B, 4, 2, S_q, S_p, 80, 64, 64, lens=[80] * B, seed=17)
    p.q[..., 5] = 0.75  # (exact in both types)
    p.q64[..., 5] = 0.75
    p.kp[:, 9, 5] = -float("inf")
    p.kc[:, :, 0, 5] = -float("inf")
    got = p.run()
    # the same rows as if those two keys were not there
    p.kp64, p.vp64 = np.delete(p.kp64, 9, axis=2), np.delete(p.vp64, 9, axis=2)
    p.kc64, p.vc64 = p.kc64[:, :, 1:], p.vc64[:, :, 1:]
    B, H, H_kv, S_q, S_p, S_c, D_qk, D_v = p.dims
    p.dims = (B, H, H_kv, S_q, S_p - 1, S_c - 1, D_qk, D_v)
    p.lens = p.lens - 1
    p.check(*got)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,B,S_q,S_p", FORMS)
@pytest.mark.parametrize("scale", [0.0, 1e-39])
def test_a_scale_of_nothing_weighs_every_key_alike(dtype, B, S_q, S_p, scale):
    """Scores of about 1e36 (64 products of less than 2^125, in fp32's range) times 0, or times 1e-39."""
    p = Problem(dtype, B, 4, 2, S_q, S_p, 80, 64, 64, lens=[80] * B, seed=18, scale=scale)
    big = 2.0 ** 59  # (exact)
    for t, a in ((p.q, p.q64), (p.kp, p.kp64), (p.kc, p.kc64)):
        t.mul_(big)
        a *= big
    p.check(*p.run())
