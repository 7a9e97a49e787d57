"""vt_qk_rope_fwd and vt_qk_rope_bwd: refusals (host only) and results against the 64-bit forms of rope_ref.

Tolerances.  A value is rounded once to its type: half a step, finfo(t).eps / 2 relative to it.  Before that, fp32
work: a rotated value is two products and a sum (3 roundings of the pair's size), its cosine and sine carry the
angle's rounding (pi * 2^-25) and theirs (2 steps), and the norm multiplies in a mean whose relative error is at most
half of the (2 * 4 * 4 + 5) additions on a value's path, a reciprocal root (2 steps) and two products: below 40
roundings of 2^-24 in all, 64 allowed.  The backward does this twice (the mean of w u z, then the difference): 128.
A weight gradient's value passes at most 400 additions (heads and tokens of a thread, 256 rows of a block, 19 + 32
partials).  Angles in fp64 carry |angle| 2^-51.
"""

import numpy as np
import pytest

import rope_ref as ref

import scaled_dot_product_vt_gb300 as vt

U32 = 2.0 ** -24
A = 1 << 24  # fake, aligned, distinct "device" addresses: never dereferenced on the refusal paths


# ---------------------------------------------------------------- refusals (no GPU)

def pack(**kw):
    """A valid two-head call, with fields replaced."""
    f = dict(size=vt._QK_ROPE_BYTES, B=2, H=2, H_kv=1, S=4, D=16, R=16, dtype=vt.VT_BF16, inter=0, norm=1, axes=1,
             eps=1e-6, reserved=0, q=A, k=2 * A, qs=(128, 64, 16), ks=(64, 64, 16), qw=3 * A, kw=4 * A, freqs=5 * A,
             pos=6 * A, ps=(8, 4, 1), qo=7 * A, ko=8 * A, qos=(128, 64, 16), kos=(64, 64, 16), lens=0, cap=0, D_v=0,
             v=0, vo=0, vs=(0, 0, 0), vos=(0, 0, 0), axis=bytes(128))
    f.update(kw)
    return vt._QK_ROPE_PTRS.pack(f["size"], f["q"], f["k"], f["qw"], f["kw"], f["freqs"], f["pos"], f["qo"], f["ko"],
                                 f["lens"], f["v"], f["vo"]) + vt._QK_ROPE_REST.pack(
        f["B"], f["H"], f["H_kv"], f["S"], f["D"], f["R"], f["cap"], f["D_v"], f["dtype"], f["inter"], f["norm"],
        f["axes"], f["eps"], f["reserved"], *f["qs"], *f["ks"], *f["qos"], *f["kos"], *f["vs"], *f["vos"], *f["ps"],
        f["axis"])


def bwd(**kw):
    ws, ws_bytes = kw.pop("ws", 16 * A), kw.pop("ws_bytes", 1 << 23)
    gq, gk, dqw, dkw = kw.pop("gq", 10 * A), kw.pop("gk", 11 * A), kw.pop("dqw", 12 * A), kw.pop("dkw", 13 * A)
    return vt.vt_qk_rope_bwd(pack(**kw), gq, (128, 64, 16), gk, (64, 64, 16), dqw, dkw, ws, ws_bytes, None)


@pytest.fixture(scope="module", autouse=True)
def _built():
    vt.build()
    vt.load()


CACHE = dict(lens=9 * A, cap=8, kos=(128, 128, 16), D_v=16, v=10 * A, vo=11 * A, vs=(64, 64, 16), vos=(128, 128, 16))
BOTH = [
    (dict(size=8), 1), (dict(reserved=1), 1), (dict(dtype=2), 1), (dict(B=-1), 1), (dict(H_kv=-1), 1), (dict(D=0), 1),
    (dict(R=0), 1), (dict(R=5), 1), (dict(R=18), 1), (dict(axes=0), 1), (dict(axes=5), 2),
    (dict(eps=float("nan")), 1), (dict(eps=-1.0), 1), (dict(axis=bytes(7) + b"\1" + bytes(120)), 1),
    (dict(D=258, R=16, qs=(2112, 1056, 264), ks=(1056, 1056, 264)), 2), (dict(S=(1 << 30) + 1), 2), (dict(B=1 << 31), 2),
    (dict(freqs=0), 1), (dict(freqs=5 * A + 2), 3), (dict(pos=0), 1), (dict(pos=6 * A + 1), 3), (dict(ps=(8, -4, 1)), 1),
    (dict(q=0), 1), (dict(q=A + 8), 3), (dict(qs=(128, 64, 12)), 3), (dict(qs=(128, 0, 16)), 1),
    (dict(qs=(1 << 40, 64, 16)), 2), (dict(qo=0), 1), (dict(qo=7 * A + 2), 3), (dict(kw=4 * A + 8), 3),
    (dict(qos=(128, 16, 16)), 1),                  # heads of the output share rows
    (dict(qo=2 * A), 1),                           # dq / q_out over k
    (dict(qo=A + 32), 1), (dict(qo=A, qos=(128, 16, 32)), 1),  # over q, but not the same tensor
    (dict(qo=3 * A), 1), (dict(ko=5 * A), 1), (dict(qo=8 * A), 1),
]


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(k=0), 1), (dict(CACHE, cap=-1), 1), (dict(CACHE, D_v=0), 1), (dict(CACHE, D_v=264, vs=(1056, 1056, 264)), 2),
    (dict(CACHE, vo=0), 1), (dict(CACHE, lens=9 * A + 2), 3), (dict(CACHE, ko=2 * A), 1), (dict(CACHE, vo=10 * A), 1),
    (dict(CACHE, vo=8 * A), 1), (dict(CACHE, kos=(64, 64, 16)), 1),  # cap rows do not fit between two sequences
])
def test_forward_refusals(kw, code):
    assert vt.vt_qk_rope_fwd(pack(**kw), None) == code


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(CACHE), 1), (dict(gq=None), 1), (dict(gk=11 * A + 4), 3), (dict(ws=None), 1), (dict(ws_bytes=1024), 1),
    (dict(ws=16 * A + 128), 3), (dict(ws=10 * A), 1), (dict(dqw=12 * A + 2), 3), (dict(dqw=13 * A), 1),
    (dict(dqw=16 * A), 1), (dict(qo=11 * A), 1),
])
def test_backward_refusals(kw, code):
    assert bwd(**kw) == code


def test_empty_problems_and_workspace_size():
    for kw in (dict(B=0), dict(S=0), dict(H=0, H_kv=0)):
        assert vt.vt_qk_rope_fwd(pack(q=0, qo=0, k=0, ko=0, **kw), None) == 0
    assert vt.load().vt_qk_rope_fwd(None, None) == 1
    assert vt.vt_qk_rope_bwd_workspace_size(0) == 0 == vt.vt_qk_rope_bwd_workspace_size(257)
    assert vt.vt_qk_rope_bwd_workspace_size(128) >= 2 * 128 * 4


def test_valid_calls_reach_the_launch():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: a valid call would launch on these fake addresses")
    assert vt.vt_qk_rope_fwd(pack(), None) == 4
    assert vt.vt_qk_rope_fwd(pack(qo=A, ko=2 * A), None) == 4           # in place
    assert vt.vt_qk_rope_fwd(pack(**CACHE), None) == 4
    # Q and K as heads of one projection, in place: their spans interleave, their rows do not
    fused = dict(qs=(256, 16, 64), qos=(256, 16, 64), ks=(256, 16, 64), kos=(256, 16, 64))
    assert vt.vt_qk_rope_fwd(pack(q=A, qo=A, k=A + 64, ko=A + 64, **fused), None) == 4
    assert vt.vt_qk_rope_fwd(pack(q=A, qo=A, k=A + 32, ko=A + 32, **fused), None) == 1   # K's head is Q's second
    assert vt.vt_qk_rope_fwd(pack(q=A, qo=A, k=A + 48, ko=A + 48, **fused), None) == 1   # between two heads
    assert vt.vt_qk_rope_fwd(pack(q=A, qo=A, k=A + 128, ko=A + 128, **fused), None) == 1  # the next token's row
    assert vt.vt_qk_rope_fwd(pack(**dict(CACHE, qo=A)), None) == 4
    assert vt.vt_qk_rope_fwd(pack(H_kv=0, k=0, ko=0), None) == 4
    assert vt.vt_qk_rope_fwd(pack(ps=(0, 0, 0)), None) == 4
    # the stride of an index with one value is not looked at
    assert vt.vt_qk_rope_fwd(pack(H_kv=1, ks=(64, 7, 16)), None) == 4
    assert bwd() == 4
    assert bwd(qo=10 * A, ko=11 * A) == 4                                # dq over dq_out
    assert bwd(qo=A) == 4                                                # dq over q
    assert bwd(dqw=None, dkw=None, ws=None, ws_bytes=0) == 4
    assert bwd(norm=0, q=0, k=0, ws=None, ws_bytes=0) == 4


def test_wrapper_refusals():
    import torch
    q = torch.zeros(1, 1, 2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        vt.qk_rope(q, None, torch.zeros(4), torch.zeros(1, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="pair_axis"):
        vt._pair_axis_bytes(None, 4, 2)
    with pytest.raises(ValueError, match="pair_axis"):
        vt._pair_axis_bytes((0, 1, 2, 0), 4, 2)


# ---------------------------------------------------------------- results (GPU)

def gpu(f):
    return pytest.mark.gpu(f)


class Inputs:
    """Random inputs on both sides: tensors on the GPU, and the same values in 64 bits."""

    def __init__(self, dtype, B, H, H_kv, S, D, R, axes=1, norm=True, interleaved=False, seed=0, far=0, tokens_first=False,
                 weights=True):
        import torch
        if not torch.cuda.is_available():
            pytest.skip("no CUDA device")
        self.torch = torch
        self.t = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.half_step = torch.finfo(self.t).eps / 2
        self.shape = (B, H, H_kv, S, D, R)
        rng = np.random.default_rng(seed)
        self.rng, self.interleaved, self.eps = rng, interleaved, (1e-5 if norm else None)
        self.tokens_first = tokens_first
        self.q, self.q64 = self.tensor(B, H, S, D)
        self.k, self.k64 = self.tensor(B, H_kv, S, D) if H_kv else (None, None)
        self.gq, self.gq64 = self.tensor(B, H, S, D)
        self.gk, self.gk64 = self.tensor(B, H_kv, S, D) if H_kv else (None, None)
        self.qw = self.kw = self.qw64 = self.kw64 = None
        if norm and weights:
            self.qw, self.qw64 = self.vector(D)
            self.kw, self.kw64 = self.vector(D)
        freqs = (10000.0 ** (-np.arange(R // 2) / max(R // 2, 1))).astype(np.float32)
        pos = rng.integers(0, 4000, (axes, B, S)) + far
        self.pair_axis = tuple(int(a) for a in rng.integers(0, axes, R // 2)) if axes > 1 else None
        self.freqs = torch.from_numpy(freqs).cuda()
        self.pos = torch.from_numpy(pos.astype(np.int32)).cuda()
        self.cos, self.sin = ref.cos_sin(pos, freqs, self.pair_axis or (0,) * (R // 2))
        self.angle_err = float(np.abs(pos).max()) * 2.0 ** -51

    def give(self, a):
        t = self.torch.from_numpy(a.astype(np.float32)).to(self.t)
        return t.cuda(), t.to(self.torch.float64).numpy()

    def vector(self, D):
        return self.give(1 + 0.2 * self.rng.standard_normal(D))

    def tensor(self, B, H, S, D):
        """[B,H,S,D] with rows padded to 16 bytes (and tokens before heads in memory, if asked)."""
        t, a = self.give(self.rng.standard_normal((B, H, S, D)))
        pad = -D % (16 // t.element_size()) + 16 // t.element_size()
        shape = (B, S, H, D + pad) if self.tokens_first else (B, H, S, D + pad)
        room = self.torch.full(shape, float("nan"), dtype=self.t, device="cuda")
        view = (room.transpose(1, 2) if self.tokens_first else room)[..., :D]
        view.copy_(t)
        return view, a

    def form(self):
        return dict(pair_axis=self.pair_axis, interleaved=self.interleaved, eps=self.eps, q_weight=self.qw,
                    k_weight=self.kw)

    def close(self, got, want, size, steps, what, once=True):
        got = got.to(self.torch.float64).cpu().numpy()
        tol = (self.half_step if once else U32) * np.abs(want) + (steps * U32 + self.angle_err) * size + 1e-38
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0].tolist()}: "
                               f"{got[bad][0]} for {want[bad][0]}, allowed {tol[bad][0]:.3e}")

    def check_forward(self, q_out, k_out):
        for got, x, w, n in ((q_out, self.q64, self.qw64, "q"), (k_out, self.k64, self.kw64, "k")):
            if x is None:
                assert got is None
                continue
            want, size = ref.forward(x, w, self.eps, self.cos, self.sin, self.interleaved)
            self.close(got, want, size, 64, n)

    def check_backward(self, dq, dk, dqw, dkw):
        for got, gw, g, x, w, n in ((dq, dqw, self.gq64, self.q64, self.qw64, "q"),
                                    (dk, dkw, self.gk64, self.k64, self.kw64, "k")):
            if x is None:
                assert got is None and gw is None
                continue
            want, size, want_w, size_w = ref.backward(g, x, w, self.eps, self.cos, self.sin, self.interleaved)
            self.close(got, want, size, 128, "d" + n)
            if want_w is None:
                assert gw is None
            else:
                self.close(gw, want_w, size_w, 400 + 128, f"d{n}_weight", once=False)


SHAPES = [
    # dtype, B, H, H_kv, S, D, R, axes, norm, interleaved
    ("bf16", 2, 4, 2, 33, 128, 128, 1, True, False),
    ("bf16", 1, 3, 1, 65, 128, 64, 2, True, True),
    ("bf16", 2, 5, 5, 7, 72, 72, 3, True, False),      # runs of 4 elements
    ("bf16", 1, 2, 1, 9, 96, 64, 4, False, True),
    ("bf16", 3, 1, 1, 1, 20, 10, 1, True, False),      # single elements
    ("bf16", 1, 2, 2, 5, 33, 14, 2, True, False),      # an odd width
    ("bf16", 1, 2, 1, 4, 201, 198, 1, True, True),     # an odd width over several chunks a thread
    ("bf16", 1, 40, 0, 3, 256, 256, 1, True, False),   # no K
    ("bf16", 1, 1, 1, 700, 16, 2, 1, False, False),
    ("f32", 2, 4, 2, 33, 128, 128, 1, True, False),
    ("f32", 1, 2, 2, 17, 72, 72, 3, False, True),
    ("f32", 1, 3, 3, 21, 20, 20, 1, True, False),
    ("f32", 1, 2, 1, 6, 255, 254, 2, True, False),
    ("f32", 1, 2, 1, 6, 256, 128, 2, True, True),
    ("f32", 4, 9, 3, 130, 64, 64, 1, True, False),
]


@gpu
@pytest.mark.parametrize("tokens_first", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_both_directions(shape, tokens_first):
    x = Inputs(*shape, seed=3, tokens_first=tokens_first)
    x.check_forward(*vt.qk_rope(x.q, x.k, x.freqs, x.pos, **x.form()))
    x.check_backward(*vt.qk_rope_bwd(x.gq, x.gk, x.freqs, x.pos, q=x.q, k=x.k, **x.form()))
    assert vt.vt_last_device_status() == 0


@gpu
@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 5000, -(1 << 31)])
def test_far_positions_keep_their_phase(far):
    x = Inputs("f32", 1, 2, 1, 40, 64, 64, seed=5, far=far)
    x.check_forward(*vt.qk_rope(x.q, x.k, x.freqs, x.pos, **x.form()))


@gpu
def test_norm_without_weights_and_rows_of_zeros():
    x = Inputs("f32", 1, 2, 1, 12, 64, 64, seed=6, weights=False)
    x.q[0, 1, 3] = 0
    x.q64[0, 1, 3] = 0
    x.check_forward(*vt.qk_rope(x.q, x.k, x.freqs, x.pos, **x.form()))
    x.check_backward(*vt.qk_rope_bwd(x.gq, x.gk, x.freqs, x.pos, q=x.q, k=x.k, **x.form()))


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place_and_padding_untouched(dtype):
    x = Inputs(dtype, 2, 4, 2, 19, 72, 48, 2, True, False, seed=7)
    pad = x.q._base[..., 72:]
    q, k = vt.qk_rope(x.q, x.k, x.freqs, x.pos, q_out=x.q, k_out=x.k, **x.form())
    assert q is x.q and k is x.k
    x.check_forward(q, k)
    assert x.torch.isnan(pad).all()
    x = Inputs(dtype, 2, 4, 2, 19, 72, 48, 2, True, False, seed=7)
    got = vt.qk_rope_bwd(x.gq, x.gk, x.freqs, x.pos, q=x.q, k=x.k, dq=x.gq, dk=x.k, **x.form())
    x.check_backward(*got)


@gpu
@pytest.mark.parametrize("dtype,S,D,D_v", [("bf16", 1, 128, 128), ("bf16", 3, 72, 40), ("f32", 4, 20, 33)])
def test_append_writes_its_rows_and_no_others(dtype, S, D, D_v):
    B, H, H_kv, cap = 5, 4, 2, 11
    x = Inputs(dtype, B, H, H_kv, S, D, D, seed=8)
    torch = x.torch
    kc, kc64 = x.tensor(B, H_kv, cap, D)
    vc, vc64 = x.tensor(B, H_kv, cap, D_v)
    v, v64 = x.tensor(B, H_kv, S, D_v)
    lens = np.array([S, cap, 0, cap + 1, S + 2])  # full, to the end, all padding, one past the end, inside
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    before = [t.clone() for t in (kc, vc)]
    q_out, k_out = vt.qk_rope(x.q, x.k, x.freqs, x.pos, k_out=kc, v=v, v_out=vc, kv_len=kv_len, **x.form())
    assert k_out is kc
    assert vt.vt_last_device_status() == 6  # the row at cap
    assert vt.vt_last_device_status() == 0
    want_q, size_q = ref.forward(x.q64, x.qw64, x.eps, x.cos, x.sin, False)
    want_k, size_k = ref.forward(x.k64, x.kw64, x.eps, x.cos, x.sin, False)
    x.close(q_out, want_q, size_q, 64, "q")
    size = np.zeros(kc64.shape)
    for b in range(B):
        for s in range(S):
            row = lens[b] - S + s
            if 0 <= row < cap:
                kc64[b, :, row], size[b, :, row], vc64[b, :, row] = want_k[b, :, s], size_k[b, :, s], v64[b, :, s]
                before[0][b, :, row], before[1][b, :, row] = kc[b, :, row], vc[b, :, row]
    x.close(kc, kc64, size, 64, "cache")
    assert torch.equal(kc, before[0]) and torch.equal(vc, before[1])
    assert np.array_equal(vc.to(torch.float64).cpu().numpy(), vc64)


@gpu
def test_given_outputs_shared_positions_and_keys_alone():
    x = Inputs("bf16", 3, 6, 2, 37, 64, 64, seed=12)
    torch = x.torch
    x.pos[:] = x.pos[:, :1]
    x.cos, x.sin = x.cos[:1].repeat(3, 0), x.sin[:1].repeat(3, 0)
    one = x.pos[0, 0].expand(3, -1)  # one row of positions for the batch: stride 0
    room = torch.full((3, 37, 8, 80), 7.0, dtype=x.t, device="cuda")
    q_out, k_out = room[:, :, :6, 8:72].transpose(1, 2), room[:, :, 6:, 8:72].transpose(1, 2)
    got = vt.qk_rope(x.q, x.k, x.freqs, one, q_out=q_out, k_out=k_out, **x.form())
    assert got[0] is q_out and got[1] is k_out
    x.check_forward(*got)
    assert (room[..., :8] == 7).all() and (room[..., 72:] == 7).all()
    # Q and K of one projection, rotated where they are
    room = torch.full((3, 37, 10, 64), 7.0, dtype=x.t, device="cuda")
    q, k = room[:, :, :6].transpose(1, 2), room[:, :, 6:8].transpose(1, 2)
    q.copy_(x.q)
    k.copy_(x.k)
    x.check_forward(*vt.qk_rope(q, k, x.freqs, one, q_out=q, k_out=k, **x.form()))
    assert (room[:, :, 8:] == 7).all()
    # an append of keys without values
    cache = torch.zeros(3, 2, 50, 64, dtype=x.t, device="cuda")
    lens = torch.full((3,), 40, dtype=torch.int32, device="cuda")
    vt.qk_rope(x.q, x.k, x.freqs, one, k_out=cache, kv_len=lens, **x.form())
    assert torch.equal(cache[:, :, 3:40], k_out) and not cache[:, :, 40:].any() and not cache[:, :, :3].any()


@gpu
def test_gradients_against_differences():
    # L(x + h d) - L(x - h d) over 2 h, both from the GPU forward, beside the same quotient in 64 bits
    x = Inputs("f32", 1, 2, 1, 9, 64, 48, 2, True, True, seed=9)
    torch = x.torch
    d = x.rng.standard_normal(x.q64.shape).astype(np.float32)
    h = 2.0 ** -6
    dq, _, dqw, _ = vt.qk_rope_bwd(x.gq, x.gk, x.freqs, x.pos, q=x.q, k=x.k, **x.form())

    def loss(sign):
        moved = (x.q.cpu().numpy() + np.float32(sign * h) * d).astype(np.float32)
        y, _ = vt.qk_rope(torch.from_numpy(moved).cuda(), x.k, x.freqs, x.pos, **x.form())
        want, size = ref.forward(moved.astype(np.float64), x.qw64, x.eps, x.cos, x.sin, True)
        return ((y.double().cpu().numpy() * x.gq64).sum(), (want * x.gq64).sum(),
                ((U32 * np.abs(want) + 64 * U32 * size) * np.abs(x.gq64)).sum())

    (hi, hi64, e1), (lo, lo64, e2) = loss(1), loss(-1)
    slope = float((dq.double().cpu().numpy() * d).sum())
    want, size, _, _ = ref.backward(x.gq64, x.q64, x.qw64, x.eps, x.cos, x.sin, True)
    slope64 = (want * d).sum()
    curve = abs((hi64 - lo64) / (2 * h) - slope64)  # what the quotient itself leaves, in 64 bits
    tol = (e1 + e2) / (2 * h) + curve + ((U32 * np.abs(want) + 128 * U32 * size) * np.abs(d)).sum()
    assert abs((hi - lo) / (2 * h) - slope) <= tol
    assert curve < 0.05 * abs(slope64)  # the quotient says something


@gpu
def test_weight_gradients_do_not_change_between_calls():
    x = Inputs("bf16", 2, 6, 2, 1500, 64, 64, seed=10)
    runs = [vt.qk_rope_bwd(x.gq, x.gk, x.freqs, x.pos, q=x.q, k=x.k, **x.form()) for _ in range(3)]
    for r in runs[1:]:
        assert all(x.torch.equal(a, b) for a, b in zip(runs[0], r))
    x.check_backward(*runs[0])


@gpu
def test_no_tokens_give_zero_weight_gradients():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    z = torch.empty(2, 4, 0, 64, device="cuda")
    k = torch.empty(2, 1, 0, 64, device="cuda")
    f, p = torch.ones(32, device="cuda"), torch.empty(2, 0, dtype=torch.int32, device="cuda")
    dq, dk, dqw, dkw = vt.qk_rope_bwd(z, k, f, p, q=z, k=k, eps=1e-6)
    assert dq.shape == z.shape and not dqw.any() and not dkw.any()
    assert vt.qk_rope(z, k, f, p, eps=1e-6)[0].shape == z.shape


@gpu
def test_another_stream_and_a_replayed_graph():
    x = Inputs("bf16", 2, 4, 2, 50, 128, 128, seed=11)
    torch = x.torch
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = vt.qk_rope(x.q, x.k, x.freqs, x.pos, **x.form())
    want_b = vt.qk_rope_bwd(x.gq, x.gk, x.freqs, x.pos, q=x.q, k=x.k, **x.form())
    got = vt.qk_rope(x.q, x.k, x.freqs, x.pos, stream=side, **x.form())
    assert vt.vt_last_device_status(side) == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = vt.qk_rope(x.q, x.k, x.freqs, x.pos, **x.form())
        got_b = vt.qk_rope_bwd(x.gq, x.gk, x.freqs, x.pos, q=x.q, k=x.k, **x.form())
    for t in (*got, *got_b):
        t.fill_(float("nan"))
    x.pos.add_(0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*got, *got_b), (*want, *want_b)))
