"""Calls of the token preparation and of the attention behind a prefix that their documentation allows and that are easily
got wrong: raw stream handles, tensors that lie beside each other in one projection or cache, checked calls, and every
combination of launches with guard bytes around what it writes."""

import os
import subprocess
import sys

import numpy as np
import pytest

from test_attn_prefix import Problem
from test_qk_rope import A, Inputs, pack

import scaled_dot_product_vt_gb300 as vt


@pytest.fixture(scope="module", autouse=True)
def _built():
    vt.build()
    vt.load()


# ---------------------------------------------------------------- raw stream handles

@pytest.mark.gpu
def test_the_raw_handle_of_the_default_stream():
    """stream=0 (torch.cuda.default_stream().cuda_stream) is the default stream, whichever one is current."""
    x = Inputs("bf16", 1, 2, 1, 20, 64, 64, seed=21)
    torch = x.torch
    seen = lambda: torch.cuda.current_stream().cuda_stream
    side = torch.cuda.Stream()
    for current in (torch.cuda.default_stream(), side):
        with torch.cuda.stream(current):
            assert vt._elsewhere(seen, x.q, torch.cuda.default_stream().cuda_stream, (), {}) == 0
            assert vt._elsewhere(seen, x.q, side.cuda_stream, (), {}) == side.cuda_stream
            assert vt._elsewhere(seen, x.q, side, (), {}) == side.cuda_stream
    torch.cuda.synchronize()
    # the call reads what the stream wrote before it
    old = vt.qk_rope(x.q, x.k, x.freqs, x.pos, **x.form())
    torch.cuda._sleep(1 << 23)  # a few milliseconds
    x.pos.zero_()
    got = vt.qk_rope(x.q, x.k, x.freqs, x.pos, stream=0, **x.form())
    torch.cuda.synchronize()
    want = vt.qk_rope(x.q, x.k, x.freqs, x.pos, **x.form())
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and not torch.equal(got[0], old[0])


# ---------------------------------------------------------------- tensors beside each other (no GPU)

def no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: a valid call would launch on these fake addresses")


LAUNCH, REFUSED = 4, 1  # a call that passes every check ends at the missing device
APPEND = dict(lens=9 * A, cap=8, ko=7 << 28, kos=(256, 128, 16), vo=9 << 28, vos=(512, 256, 32))


@pytest.mark.parametrize("kw,code", [
    # one projection [B, S, H D + H_kv D + H_kv D_v] with D_v = 24: Q in place while K and V go to their caches
    (dict(APPEND, H_kv=2, D_v=24, q=A, qo=A, k=A + 64, v=A + 128, qs=(448, 16, 112), qos=(448, 16, 112),
          ks=(448, 16, 112), vs=(448, 24, 112)), LAUNCH),
    # ... V's first 8 columns are Q's last ones
    (dict(APPEND, H_kv=2, D_v=24, q=A, qo=A, k=A + 96, v=A + 48, qs=(448, 16, 112), qos=(448, 16, 112),
          ks=(448, 16, 112), vs=(448, 24, 112)), REFUSED),
    # ... V's last head reaches into the next token's Q
    (dict(APPEND, H_kv=2, D_v=24, q=A, qo=A, k=A + 64, v=A + 144, qs=(448, 16, 112), qos=(448, 16, 112),
          ks=(448, 16, 112), vs=(448, 24, 112)), REFUSED),
    # a gate of 8 columns between Q and K, both in place
    (dict(q=A, qo=A, k=A + 80, ko=A + 80, qs=(256, 16, 64), qos=(256, 16, 64), ks=(256, 16, 64), kos=(256, 16, 64)),
     LAUNCH),
    # every head's Q, K and V beside each other: [B, S, H, 3, D]
    (dict(H_kv=2, q=A, qo=A, k=A + 32, ko=A + 32, qs=(384, 48, 96), qos=(384, 48, 96), ks=(384, 48, 96),
          kos=(384, 48, 96)), LAUNCH),
    # ... K 8 columns too early
    (dict(H_kv=2, q=A, qo=A, k=A + 16, ko=A + 16, qs=(384, 48, 96), qos=(384, 48, 96), ks=(384, 48, 96),
          kos=(384, 48, 96)), REFUSED),
    # K and V rows beside each other in one cache [B, H_kv, cap, D + D_v]
    (dict(APPEND, H_kv=2, D_v=24, v=10 * A, vs=(192, 96, 24), ks=(128, 64, 16), ko=1 << 32, vo=(1 << 32) + 32,
          kos=(640, 320, 40), vos=(640, 320, 40)), LAUNCH),
    # K's rows and V's of a head one after the other: [B, H_kv, cap D + cap D_v]
    (dict(APPEND, H_kv=2, D_v=24, v=10 * A, vs=(192, 96, 24), ks=(128, 64, 16), ko=1 << 32, vo=(1 << 32) + 256,
          kos=(640, 320, 16), vos=(640, 320, 24)), LAUNCH),
    # ... with room for 7 rows of K
    (dict(APPEND, H_kv=2, D_v=24, v=10 * A, vs=(192, 96, 24), ks=(128, 64, 16), ko=1 << 32, vo=(1 << 32) + 224,
          kos=(640, 320, 16), vos=(640, 320, 24)), REFUSED),
])
def test_tensors_beside_each_other(kw, code):
    no_gpu()
    assert vt.vt_qk_rope_fwd(pack(**kw), None) == code


def test_overlap_is_found_exactly():
    """Random layouts of Q and K outputs in one buffer: a call is refused when two elements meet, and only then."""
    no_gpu()
    rng = np.random.default_rng(22)
    counts = [0, 0]
    for _ in range(3000):
        B, S, H, H_kv = (int(n) for n in rng.integers(1, 4, 4))
        tensors = []
        for heads in (H, H_kv):
            order = rng.permutation(3)
            n, st, reach = (B, heads, S), [0, 0, 0], 16
            for i in order:  # strides that nest, with gaps
                st[i] = reach + 8 * int(rng.integers(0, 6)) if n[i] > 1 else 8 * int(rng.integers(0, 9))
                reach = st[i] * (n[i] - 1) + reach if n[i] > 1 else reach
            tensors.append((n, st))
        if rng.random() < 0.5:  # heads and sequences of one projection
            tensors[1] = (tensors[1][0], [tensors[0][1][0], tensors[1][1][1], tensors[0][1][2]])
        at = 8 * int(rng.integers(-12, 40))
        cells = []
        for (n, st), first in zip(tensors, (0, at)):
            b, h, s = np.ogrid[:n[0], :n[1], :n[2]]
            cells.append((first + b * st[0] + h * st[1] + s * st[2]).reshape(-1, 1) + np.arange(16))
        nested, reach = True, 16  # the rule for an output's own strides
        for st, n in sorted((st, n) for n, st in zip(*tensors[1]) if n > 1):
            nested, reach = nested and st >= reach, reach + st * (n - 1)
        code = vt.vt_qk_rope_fwd(pack(B=B, S=S, H=H, H_kv=H_kv, q=1 << 32, k=2 << 32, qo=3 << 32, ko=(3 << 32) + 2 * at,
                                      qs=(512, 128, 16), ks=(512, 128, 16), qos=tensors[0][1], kos=tensors[1][1]), None)
        meet = len(np.intersect1d(*cells)) > 0
        if nested:  # (else it is refused whatever lies beside it)
            assert code == (REFUSED if meet else LAUNCH), (B, S, H, H_kv, tensors, at)
            counts[meet] += 1
        else:
            assert code == REFUSED
    assert min(counts) > 300


@pytest.mark.gpu
def test_a_projection_with_values_of_another_width():
    """Q rotated where it is, K and V appended, all from one [B, S, H D + H_kv D + H_kv D_v] projection."""
    B, S, H, H_kv, D, D_v, cap = 3, 5, 4, 2, 64, 40, 9
    x = Inputs("bf16", B, H, H_kv, S, D, D, seed=25)
    torch = x.torch
    room = torch.full((B, S, H * D + H_kv * (D + D_v)), 7.0, dtype=x.t, device="cuda")
    q, k, v = (t.unflatten(-1, (-1, d)).transpose(1, 2) for t, d in
               zip(room.split([H * D, H_kv * D, H_kv * D_v], -1), (D, D, D_v)))
    v64 = x.rng.standard_normal(v.shape)
    for t, a in ((q, x.q), (k, x.k), (v, torch.from_numpy(v64))):
        t.copy_(a)
    kept = [k.clone(), v.clone()]
    caches = [torch.full((B, H_kv, cap, d), 3.0, dtype=x.t, device="cuda") for d in (D, D_v)]
    lens = torch.tensor([S, cap, S + 1], dtype=torch.int32, device="cuda")
    got, _ = vt.qk_rope(q, k, x.freqs, x.pos, q_out=q, k_out=caches[0], v=v, v_out=caches[1], kv_len=lens, **x.form())
    assert got is q and torch.equal(k, kept[0]) and torch.equal(v, kept[1])
    rows = torch.stack([caches[0][b, :, n - S:n] for b, n in enumerate(lens.tolist())])
    x.check_forward(q, rows)
    for b, n in enumerate(lens.tolist()):
        assert torch.equal(caches[1][b, :, n - S:n], v[b])
        caches[0][b, :, n - S:n] = caches[1][b, :, n - S:n] = 3.0
    assert (caches[0] == 3).all() and (caches[1] == 3).all()
    assert vt.vt_last_device_status() == 0


# ---------------------------------------------------------------- checked calls

CHECKED = """
import torch, scaled_dot_product_vt_gb300 as vt
x = torch.randn(4, 32, 4096, 128, device="cuda", dtype=torch.bfloat16)
f, p = torch.ones(64, device="cuda"), torch.zeros(4, 4096, dtype=torch.int32, device="cuda")
vt.qk_rope_bwd(x, None, f, p, q=x, eps=1e-6)
torch.cuda.synchronize()
stream = torch.cuda.current_stream()
for call in (lambda: vt.qk_rope(x, None, f, p, eps=1e-6), lambda: vt.qk_rope_bwd(x, None, f, p, q=x, eps=1e-6),
             lambda: vt.attn_fwd_prefix(x, x[0], x[0], None, None)):
    call()
    assert stream.query()
    print("done")
"""


@pytest.mark.gpu
def test_checked_calls_wait_for_their_kernels():
    """VT_CHECK: every call reads its stream's status itself, so it returns after its kernels ended."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CHECKED], cwd=root, env=dict(os.environ, VT_CHECK="1"), capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["done"] * 3, r.stdout + r.stderr


# ---------------------------------------------------------------- every combination of launches

# dtype, B, H, H_kv, S_q, S_p, S_c, D_qk, D_v; shares of the prefix, and of the caches (1: a cluster writes O, or its one
# share, itself) on a device of 152 SMs
PLANS = [
    (("bf16", 2, 4, 2, 1, 20000, 9000, 96, 33), 9, 2),     # both launches stream, and a third adds their shares
    (("f32", 4, 4, 1, 1, 20000, 9000, 33, 7), 32, 4),
    (("bf16", 16, 2, 2, 1, 4096, 50, 128, 128), 2, 1),     # the prefix streamed for all rows
    (("bf16", 5, 6, 2, 1, 20000, 60, 72, 40), 9, 1),
    (("f32", 40, 8, 2, 1, 1500, 40, 128, 128), 4, 1),
    (("bf16", 33, 8, 1, 2, 1500, 9, 80, 128), 11, 1),      # on tiles: three query tiles of rows, the last one short
    (("bf16", 70, 4, 2, 1, 1000, 37, 64, 33), 7, 1),
    (("bf16", 40, 8, 2, 1, 8192, 200, 128, 72), 31, 1),
    (("bf16", 1, 4, 1, 2, 0, 20000, 128, 128), 0, 4),      # no prefix: the caches in shares
    (("bf16", 5, 8, 4, 2, 333, 70, 64, 40), 0, 1),         # one launch
    (("bf16", 3, 8, 2, 100, 129, 300, 128, 72), 0, 0),     # rows of a sequence on tiles
]


def shares_of(case):
    dtype, B, H, H_kv, S_q, S_p, S_c, D_qk, D_v = case
    need = vt.vt_attn_prefix_workspace_size(B, H, H_kv, S_q, S_p, S_c, D_qk, D_v, vt.VT_BF16 if dtype == "bf16" else vt.VT_F32)
    return need, need // (B * H * S_q * ((D_v + 7) // 8 * 8 + 3) * 4)


@pytest.mark.parametrize("case,prefix,cache", PLANS, ids=lambda c: "-".join(map(str, c)) if isinstance(c, tuple) else None)
def test_plans_are_the_ones_named(case, prefix, cache):
    import torch
    if torch.cuda.is_available() and torch.cuda.get_device_properties(0).multi_processor_count != 152:
        pytest.skip("a device of another size")
    _, shares = shares_of(case)
    assert shares in ((prefix, prefix + cache) if prefix and cache == 1 else (prefix + cache if prefix or cache > 1 else 0,))
    again = case[1] * case[3] * -(-case[4] * (case[2] // case[3]) // 16) * case[5] * (case[7] + case[8]) * (
        2 if case[0] == "bf16" else 4)
    assert prefix == 0 or again > ((16 if case[0] == "bf16" else 2) << 20)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens_first", [False, True])
@pytest.mark.parametrize("case,prefix,cache", PLANS, ids=lambda c: "-".join(map(str, c)) if isinstance(c, tuple) else None)
def test_every_combination_of_launches(case, prefix, cache, tokens_first):
    p = Problem(*case, seed=23, tokens_first=tokens_first)
    torch = p.torch
    _, B, H, _, S_q, _, _, _, D_v = case
    need, _ = shares_of(case)
    row = (D_v + 7) // 8 * 8 + 16  # 8 columns before and behind
    room = torch.full((B, S_q + 1, H, row), 7.0, dtype=p.t, device="cuda")
    out = room[:, :S_q, :, 8:8 + D_v].transpose(1, 2)
    lse_room = torch.full((B * H * S_q + 2,), 7.0, device="cuda")
    ws = torch.full((need + 1024,), 7, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        o, lse = p.run(out=out, lse=lse_room[1:-1].view(B, H, S_q), workspace=ws[512:512 + need] if need else None)
        assert o is out
        p.check(o, lse)
        out.fill_(7.0)
        assert (room == 7).all() and lse_room[0] == 7 and lse_room[-1] == 7
        assert (ws[:512] == 7).all() and (ws[512 + need:] == 7).all()
    assert vt.vt_last_device_status() == 0
