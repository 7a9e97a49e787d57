"""The debug library's index checks over the operators' launches: it finds nothing, and its results are the release library's."""

import pytest

from test_attn_packed import Problem as Packed
from test_attn_prefix import Problem as Prefix
from test_attn_tree import Tree

import scaled_dot_product_vt_gb300 as vt

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    vt.build()
    vt.load()


def same(monkeypatch, run):
    """run() under either library."""
    import torch
    want = [x.clone() for x in run()]
    assert vt.vt_last_device_status() == 0
    dbg = vt.load_debug()
    with monkeypatch.context() as m:
        m.setattr(vt, "load", lambda *a: dbg)
        got = [x.clone() for x in run()]
        assert vt.vt_last_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(got) == len(want)


PACKED = [
    # dtype, H, H_kv, D_qk, D_v, lengths, mask, window
    ("bf16", 8, 2, 128, 128, [(300, 300), (7, 7), (129, 200)], "causal", 0),                    # dK and dV by query heads
    ("bf16", 8, 8, 128, 128, [(1500, 1500), (900, 900), (256, 256)] * 2, "causal", 0),          # more blocks than SMs
    ("bf16", 16, 8, 128, 72, [(1300, 1300), (700, 1000), (30, 900)], "window", 200),
    ("bf16", 4, 1, 96, 128, [(500, 100), (0, 9), (7, 0)], "none", 0),
    ("f32", 8, 2, 128, 128, [(300, 300), (7, 7)], "causal", 0),
    ("f32", 8, 8, 72, 128, [(700, 700), (400, 600)] * 3, "window_complement", 50),
]


@gpu
@pytest.mark.parametrize("case", PACKED, ids=lambda c: "-".join(map(str, c[:5])) + f"-{c[6]}")
def test_packed(monkeypatch, case):
    dtype, H, H_kv, D_qk, D_v, lengths, mask, window = case
    p = Packed(dtype, H, H_kv, D_qk, D_v, lengths, mask, window, seed=1, behind=0)
    res = p.results()
    same(monkeypatch, lambda: (*p.forward(), *p.backward(*res, dlse=p.dlse)))


TREES = [
    # dtype, B, H, H_kv, nodes, S_p, S_c, D_qk, D_v
    ("bf16", 4, 8, 2, 8, 333, 100, 128, 128),      # streamed
    ("bf16", 40, 4, 2, 5, 1000, 37, 128, 128),     # the prefix in a launch of its own
    ("bf16", 16, 16, 8, 64, 0, 4000, 128, 128),    # tiles of a sequence's rows, the keys in shares
    ("bf16", 32, 16, 4, 25, 8192, 700, 128, 128),  # the prefix in a launch of its own, longest sequences first
    ("bf16", 40, 8, 2, 33, 300, 100, 64, 64),      # one launch
    ("bf16", 1, 32, 8, 64, 1024, 0, 128, 128),     # no cache
    ("f32", 5, 8, 2, 13, 1000, 90, 72, 72),
]


@gpu
@pytest.mark.parametrize("case", TREES, ids=lambda c: "-".join(map(str, c)))
def test_trees(monkeypatch, case):
    t = Tree(*case, seed=2)
    same(monkeypatch, t.run)
    same(monkeypatch, lambda: Prefix.run(t))
