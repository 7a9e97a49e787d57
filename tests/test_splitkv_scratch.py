"""Scratch of the split-KV calls: a call asks for packed partial rows of D_v floats wherever packed rows take its
stores, so that buffers of that size and problems that just fit the fixed 32 MiB array are served."""

import math

import numpy as np
import pytest

import oracle
import synth
from gpu_util import check, to_host64

import scaled_dot_product_vt_gb300 as vt

A = 1 << 32  # fake, aligned, distinct "device" addresses: never dereferenced on the host's paths
CUDA, UNSUPPORTED, INVALID = 4, 2, 1  # a call that passes every check ends at the missing device


@pytest.fixture(scope="module", autouse=True)
def _built():
    vt.build()
    vt.load()


def packed_bytes(rows, D_v, n):
    up = lambda x: (x + 255) // 256 * 256
    return up(4 * rows * D_v * n) + 3 * up(4 * rows * n)


# widths whose packed rows take the shares' stores: multiples of 4 (16-byte stores), and the widths too narrow for one
WIDTHS = [(t, d) for t in (vt.VT_BF16, vt.VT_F32) for d in (4, 12, 20, 36, 60, 100, 8, 128)] + [
    (vt.VT_BF16, 1), (vt.VT_BF16, 7), (vt.VT_BF16, 15), (vt.VT_F32, 1), (vt.VT_F32, 3)]


def no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: a valid call would launch on these fake addresses")


def problem(dtype, D_v, S_q):
    row = lambda d: (d + 7) // 8 * 8
    st = lambda s, d: (s * row(d), s * row(d), row(d))
    return (A, st(S_q, 16), 2 * A, st(4096, 16), 3 * A, st(4096, D_v), 4 * A, st(S_q, D_v), 1, 1, S_q, 4096, 16, D_v,
            0.25, False, dtype)


@pytest.mark.parametrize("dtype,D_v", WIDTHS)
def test_the_fixed_array_takes_what_fits_it_packed(dtype, D_v):
    no_gpu()
    n = 4
    most = (32 << 20) // (4 * n * (D_v + 3))
    while packed_bytes(most, D_v, n) > 32 << 20:
        most -= 1
    while packed_bytes(most + 1, D_v, n) <= 32 << 20:
        most += 1
    assert vt.vt_attn_fwd_splitkv_noalloc(*problem(dtype, D_v, most), n, None) == CUDA
    assert vt.vt_attn_fwd_splitkv_noalloc(*problem(dtype, D_v, most + 1), n, None) == UNSUPPORTED


@pytest.mark.parametrize("dtype,D_v", WIDTHS)
def test_a_packed_workspace_is_taken(dtype, D_v):
    no_gpu()
    S_q, n = 1000, 5
    need = packed_bytes(S_q, D_v, n)
    assert vt.vt_attn_fwd_splitkv(*problem(dtype, D_v, S_q), n, 5 * A, need, None) == CUDA
    assert vt.vt_attn_fwd_splitkv(*problem(dtype, D_v, S_q), n, 5 * A, need - 1, None) == INVALID
    # what the function reports always serves
    assert need <= vt.vt_attn_splitkv_workspace_size(1, 1, S_q, D_v, n)


@pytest.mark.parametrize("D_v", [4, 12, 20, 36, 100, 104])
def test_multiples_of_four_report_packed_rows(D_v):
    assert vt.vt_attn_splitkv_workspace_size(2, 3, 5, D_v, 4) == packed_bytes(30, D_v, 4)


@pytest.mark.parametrize("dtype,D_v", [(vt.VT_BF16, 17), (vt.VT_BF16, 33), (vt.VT_F32, 5), (vt.VT_F32, 33)])
def test_other_widths_need_their_rounded_rows(dtype, D_v):
    no_gpu()
    need = packed_bytes(100, (D_v + 7) // 8 * 8, 3)
    assert vt.vt_attn_fwd_splitkv(*problem(dtype, D_v, 100), 3, 5 * A, need, None) == CUDA
    assert vt.vt_attn_fwd_splitkv(*problem(dtype, D_v, 100), 3, 5 * A, need - 1, None) == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D_v", [("bf16", 4), ("bf16", 7), ("bf16", 12), ("bf16", 20), ("bf16", 36), ("bf16", 100),
                                       ("bf16", 128), ("f32", 3), ("f32", 4), ("f32", 20), ("f32", 100)])
def test_packed_workspaces_on_the_gpu(dtype, D_v):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B, H, S_q, S_k, D_qk, n = 1, 3, 131, 1500, 64, 3
    q, k, v = synth.make_qkv(B, H, S_q, S_k, D_qk, D_v, dtype, seed=72)
    scale = float(np.float32(1.0 / math.sqrt(D_qk)))

    def put(a):  # rows padded to 16 bytes
        t = torch.from_numpy(a.view(np.int16).copy()).view(torch.bfloat16) if a.dtype == np.uint16 else torch.from_numpy(a)
        step = 16 // t.element_size()
        room = torch.zeros((*t.shape[:3], t.shape[3] + -t.shape[3] % step), dtype=t.dtype, device="cuda")
        room[..., :t.shape[3]] = t.cuda()
        return room[..., :t.shape[3]]

    need = packed_bytes(B * H * S_q, D_v, n)
    room = torch.full((need + 1024,), 7, dtype=torch.uint8, device="cuda")
    out = put(np.zeros((B, H, S_q, D_v), dtype=v.dtype))
    vt.attn_fwd_splitkv(put(q), put(k), put(v), scale=scale, causal=True, n_split=n, out=out, workspace=room[512:512 + need])
    assert vt.vt_last_device_status() == 0
    check(to_host64(out), oracle.attn_fwd(q, k, v, scale, True), dtype, f"D_v={D_v} {n} shares")
    assert (room[:512] == 7).all() and (room[512 + need:] == 7).all()
