"""Attention over packed sequences at the ends of what its contract takes: a side without rows, many short sequences, first
rows that are out of order, gradients that nothing may reach.  Tolerances are those of test_attn_packed.py."""

import numpy as np
import pytest

from test_attn_packed import Problem

import scaled_dot_product_vt_gb300 as vt

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    vt.build()
    vt.load()


def test_contiguity_of_an_empty_tensor():
    """torch gives [2, 0] the strides (1, 1): nothing lies apart there."""
    torch = pytest.importorskip("torch")
    for shape in ((2, 0), (0, 5), (1, 0), (3, 1), (3, 5), (2, 0, 4), (2, 3, 4)):
        x = torch.empty(shape)
        assert vt._contiguous(x.shape, x.stride())
        vt._check_lse("lse", (x.shape, x.stride(), x.dtype, 0), 0, shape)
    for x in (torch.empty(3, 5)[:, :4], torch.empty(5, 3).T, torch.empty(2, 3, 4).transpose(0, 1), torch.empty(3, 1).expand(3, 2)):
        assert not vt._contiguous(x.shape, x.stride())
        with pytest.raises(ValueError):
            vt._check_lse("lse", (x.shape, x.stride(), x.dtype, 0), 0, tuple(x.shape))


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_side_has_no_rows(dtype):
    """Keys without a query have gradients of 0, queries without a key O = 0, a log-sum-exp of -inf and a gradient of 0."""
    p = Problem(dtype, 4, 2, 64, 40, [(30, 30), (200, 200)], seed=1, behind=0)
    torch = p.torch
    res, none = p.results(), torch.zeros_like(p.cu_q)
    q, do, o, lse = (x[:, :0] for x in (p.q, p.do, *res))
    dq, dk, dv = vt.attn_bwd_packed(do, q, p.k, p.v, o, lse, none, p.cu_k, dlse=lse, **p.form)
    assert dq.shape == q.shape and (dk == 0).all() and (dv == 0).all()
    for out in (None, o.clone()):
        o2, lse2 = vt.attn_fwd_packed(q, p.k, p.v, none, p.cu_k, out=out, lse=lse if out is not None else None, return_lse=True,
                                      **p.form)
        assert o2.shape == (4, 0, 40) and lse2.shape == (4, 0)
    k, v = p.k[:, :0], p.v[:, :0]
    o, lse = vt.attn_fwd_packed(p.q, k, v, p.cu_q, none, return_lse=True, **p.form)
    assert (o == 0).all() and (lse == -torch.inf).all()
    dq, dk, dv = vt.attn_bwd_packed(p.do, p.q, k, v, o, lse, p.cu_q, none, dlse=p.dlse, **p.form)
    assert (dq == 0).all() and dk.shape == k.shape and dv.shape == v.shape
    assert vt.vt_last_device_status() == 0


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("which", ["both", "queries", "keys"])
def test_arrays_that_decrease_are_reported_wherever_they_do(dtype, which):
    """Also by a sequence that no block belongs to, and in the array of the other side; rows of no sequence stay."""
    p = Problem(dtype, 2, 1, 64, 64, [(1000, 1000)] + [(0, 0)] * 60, seed=15, before=2)
    torch = p.torch
    res = p.results()
    for at, row in ((2, 10), (2, 990), (30, 400), (33, 3), (59, 999)):
        cu = p.cu[0].copy()
        cu[at] = 2 + row  # behind a sequence that ends before it starts, the next one shares rows with the first
        for x, side in ((p.cu_q, "queries"), (p.cu_k, "keys")):
            x.copy_(torch.tensor(cu if which in ("both", side) else p.cu[0]))
        (out, lse), gr = p.outputs()
        p.forward(out=out, lse=lse)
        assert vt.vt_last_device_status() == 6 and vt.vt_last_device_status() == 0, (at, row)
        p.backward(*res, dq=gr[0], dk=gr[1], dv=gr[2])
        assert vt.vt_last_device_status() == 6 and vt.vt_last_device_status() == 0, (at, row)
        for x, side in zip((out, lse, *gr), (0, 0, 0, 1, 1)):
            p.untouched(x, side)
        if which != "queries":  # no query at all: dK and dV are 0, and the keys' array is looked at
            empty = [x[:, :0] for x in (p.do, p.q, *res)]
            cu_q = torch.zeros_like(p.cu_q)
            _, dk, dv = vt.attn_bwd_packed(empty[0], empty[1], p.k, p.v, empty[2], empty[3], cu_q, p.cu_k, **p.form)
            assert vt.vt_last_device_status() == 6 and (dk[:, 2:12] == 0).all() and (dv[:, 2:12] == 0).all()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_short_sequences(dtype):
    """More than 32 * 32 of them, so that a slot is found in three rounds."""
    rng = np.random.default_rng(16)
    Problem(dtype, 1, 1, 16, 16, [(int(n), int(n)) for n in rng.integers(0, 3, 1100)], seed=16).check()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,mask,window", [([(300, 100), (70, 70), (5, 1)], "causal", 0),
                                                 ([(200, 200), (40, 40)], "window_complement", 60)])
def test_queries_without_a_key_add_nothing_whatever_their_dlse(dtype, lengths, mask, window):
    """A log-sum-exp of -inf often has a gradient that is NaN (exp of inf - inf)."""
    p = Problem(dtype, 4, 2, 64, 64, lengths, mask, window, seed=17, behind=0)
    torch = p.torch
    o, lse = p.results()
    none = lse == -torch.inf
    assert none.any()
    want = [x.clone() for x in p.backward(o, lse, dlse=torch.where(none, 0.0, p.dlse))]
    p.check_backward(*want, dlse=torch.where(none, 0.0, p.dlse))
    for bad in (float("nan"), float("inf")):
        got = p.backward(o, lse, dlse=torch.where(none, bad, p.dlse))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert (want[0][none] == 0).all()
