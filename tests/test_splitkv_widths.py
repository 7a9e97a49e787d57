"""Split-KV shares for value widths that are no multiple of 4: every partial row starts on its own 32 bytes."""

import math

import numpy as np
import pytest

import oracle
import synth
from gpu_util import check, to_host64

import scaled_dot_product_vt_gb300 as vt


def test_workspace_rows_are_rounded_up():
    vt.build()
    up = lambda x: (x + 255) // 256 * 256
    rows = 2 * 3 * 5
    for D_v, ld in ((1, 8), (7, 8), (8, 8), (33, 40), (128, 128)):
        assert vt.vt_attn_splitkv_workspace_size(2, 3, 5, D_v, 4) == up(4 * rows * ld * 4) + 3 * up(4 * rows * 4)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D_qk,D_v", [(33, 33), (64, 18), (128, 127), (20, 5), (96, 71)])
def test_odd_value_widths(dtype, D_qk, D_v):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    vt.load()
    B, H, S_q, S_k, n = 1, 3, 131, 1500, 3
    q, k, v = synth.make_qkv(B, H, S_q, S_k, D_qk, D_v, dtype, seed=71)
    scale = float(np.float32(1.0 / math.sqrt(D_qk)))

    def put(a):  # rows padded to 16 bytes
        t = torch.from_numpy(a.view(np.int16).copy()).view(torch.bfloat16) if a.dtype == np.uint16 else torch.from_numpy(a)
        step = 16 // t.element_size()
        room = torch.zeros((*t.shape[:3], t.shape[3] + -t.shape[3] % step), dtype=t.dtype, device="cuda")
        room[..., :t.shape[3]] = t.cuda()
        return room[..., :t.shape[3]]

    out = put(np.zeros((B, H, S_q, D_v), dtype=v.dtype))
    vt.attn_fwd_splitkv(put(q), put(k), put(v), scale=scale, causal=True, n_split=n, out=out)
    assert vt.vt_last_device_status() == 0
    check(to_host64(out), oracle.attn_fwd(q, k, v, scale, True), dtype, f"D={D_qk}/{D_v} {n} shares")
