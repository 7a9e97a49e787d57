"""vt_attn_fwd_prefix: refusals (host only) and results against a plain 64-bit form.

Tolerances.  With |s| the row's largest sum of |scale q k| over its keys, a score is off by at most a few fp32
steps of |s| (D products accumulated in fp32: bounded by D 2^-24 |s|, taken as 2^-17 |s| for D <= 128); the fp32 form also
loses 2^-20 of every factor (two TF32 parts each, cut).  An error d of the scores changes every weight by a factor
1 +- 2 d, so O moves by at most 2 d times the spread of V, and LSE by d.  ex2, lg2 and the sums add 2^-20 of the sum.
bf16: P is rounded to bf16, half a step (2^-8... finfo.eps / 2) of each weight, for an error of at most
eps / 2 * sum w |v|, and O is rounded once.
"""

import numpy as np
import pytest

import rope_ref

import scaled_dot_product_vt_gb300 as vt

A = 1 << 24  # fake, aligned, distinct "device" addresses: never dereferenced on the refusal paths


# ---------------------------------------------------------------- refusals (no GPU)

def pack(**kw):
    f = dict(size=vt._ATTN_PREFIX_BYTES, B=2, H=4, H_kv=2, S_q=3, S_p=40, S_c=24, D_qk=16, D_v=8, dtype=vt.VT_BF16,
             scale=0.25, q=A, qs=(192, 48, 16), kp=2 * A, vp=3 * A, kps=(640, 16), vps=(320, 8), kc=4 * A, vc=5 * A,
             kcs=(768, 384, 16), vcs=(384, 192, 8), lens=6 * A, o=7 * A, os=(96, 24, 8), lse=8 * A, ws=9 * A,
             wsb=1 << 23)
    f.update(kw)
    return vt._ATTN_PREFIX_PTRS.pack(f["size"], f["q"], f["kp"], f["vp"], f["kc"], f["vc"], f["lens"], f["o"], f["lse"],
                                     f["ws"], f["wsb"]) + vt._ATTN_PREFIX_REST.pack(
        f["B"], f["H"], f["H_kv"], f["S_q"], f["S_p"], f["S_c"], f["D_qk"], f["D_v"], f["dtype"], f["scale"], *f["qs"],
        *f["kps"], *f["vps"], *f["kcs"], *f["vcs"], *f["os"])


@pytest.fixture(scope="module", autouse=True)
def _built():
    vt.build()
    vt.load()


# long enough a prefix that its partial results need the workspace
LONG = dict(B=64, H=8, H_kv=1, S_q=1, S_p=1 << 16, qs=(128, 16, 16), kps=(1 << 20, 16), vps=(1 << 19, 8),
            kcs=(384, 384, 16), vcs=(192, 192, 8), os=(64, 8, 8), wsb=1 << 30)


@pytest.mark.parametrize("kw,code", [
    (dict(size=8), 1), (dict(dtype=5), 1), (dict(B=-1), 1), (dict(S_p=-1), 1), (dict(S_c=-1), 1), (dict(D_qk=0), 1),
    (dict(D_v=0), 1), (dict(H_kv=0), 1), (dict(H_kv=3), 1), (dict(scale=float("nan")), 1),
    (dict(D_qk=129), 2), (dict(D_v=136), 2), (dict(S_p=(1 << 30) + 1), 2), (dict(S_p=1 << 29, S_c=(1 << 29) + 1), 2),
    (dict(B=1 << 20, H=1 << 10, S_q=2), 2),
    (dict(q=0), 1), (dict(kp=0), 1), (dict(vc=0), 1), (dict(o=0), 1), (dict(q=A + 8), 3), (dict(vp=3 * A + 2), 3),
    (dict(kps=(640, 20)), 3), (dict(kcs=(768, -384, 16)), 1), (dict(vcs=(1 << 40, 192, 8)), 2),
    (dict(lens=6 * A + 2), 3), (dict(lse=8 * A + 2), 1), (dict(os=(96, 8, 8)), 1),
    (dict(o=A), 1), (dict(o=2 * A + 64), 1), (dict(o=5 * A), 1), (dict(lse=7 * A), 1), (dict(lse=6 * A), 1),
    (dict(LONG, ws=0), 1), (dict(LONG, wsb=256), 1), (dict(LONG, ws=9 * A + 16), 3), (dict(LONG, ws=8 * A), 1),
    (dict(LONG, ws=4 * A), 1),
])
def test_refusals(kw, code):
    assert vt.vt_attn_fwd_prefix(pack(**kw), None) == code


def test_empty_problems_and_workspace_size():
    for kw in (dict(B=0), dict(S_q=0), dict(H=0)):
        assert vt.vt_attn_fwd_prefix(pack(q=0, o=0, **kw), None) == 0
    assert vt.load().vt_attn_fwd_prefix(None, None) == 1
    assert vt.vt_attn_prefix_workspace_size(0, 4, 2, 1, 100, 100, 64, 64, vt.VT_BF16) == 0
    assert vt.vt_attn_prefix_workspace_size(4, 4, 3, 1, 100, 100, 64, 64, vt.VT_BF16) == 0
    assert vt.vt_attn_prefix_workspace_size(64, 8, 1, 1, 1 << 16, 24, 16, 8, vt.VT_BF16) >= 64 * 8 * 11 * 4


def test_valid_calls_reach_the_launch():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: a valid call would launch on these fake addresses")
    assert vt.vt_attn_fwd_prefix(pack(), None) == 4
    assert vt.vt_attn_fwd_prefix(pack(**LONG), None) == 4
    assert vt.vt_attn_fwd_prefix(pack(S_p=0, kp=0, vp=0, kps=(0, 0)), None) == 4
    assert vt.vt_attn_fwd_prefix(pack(S_c=0, kc=0, vc=0, lens=0, lse=0), None) == 4
    assert vt.vt_attn_fwd_prefix(pack(S_p=0, S_c=0, kp=0, vp=0, kc=0, vc=0), None) == 4  # no key at all: O = 0


# ---------------------------------------------------------------- results (GPU)

def gpu(f):
    return pytest.mark.gpu(f)


class Problem:
    def __init__(self, dtype, B, H, H_kv, S_q, S_p, S_c, D_qk, D_v, lens=None, seed=0, scale=None, tokens_first=False,
                 beyond=float("nan"), spread=1.0):
        import torch
        if not torch.cuda.is_available():
            pytest.skip("no CUDA device")
        self.torch, self.t = torch, torch.bfloat16 if dtype == "bf16" else torch.float32
        self.rng, self.tokens_first = np.random.default_rng(seed), tokens_first
        self.dims = (B, H, H_kv, S_q, S_p, S_c, D_qk, D_v)
        self.scale = D_qk ** -0.5 if scale is None else scale
        self.q, self.q64 = self.tensor(B, H, S_q, D_qk, spread)
        kp, self.kp64 = self.tensor(1, H_kv, S_p, D_qk)
        vp, self.vp64 = self.tensor(1, H_kv, S_p, D_v)
        self.kp, self.vp = (kp[0], vp[0]) if S_p else (None, None)
        self.kc, self.kc64 = self.tensor(B, H_kv, S_c, D_qk)
        self.vc, self.vc64 = self.tensor(B, H_kv, S_c, D_v)
        self.lens = np.asarray(self.rng.integers(0, S_c + 1, B) if lens is None else lens)
        self.kv_len = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        for b, n in enumerate(self.lens):  # what lies behind a sequence has no influence
            self.kc[b, :, max(n, 0):] = beyond
            self.vc[b, :, max(n, 0):] = beyond

    def tensor(self, B, H, S, D, spread=1.0):
        t = self.torch.from_numpy((spread * self.rng.standard_normal((B, H, S, D))).astype(np.float32)).to(self.t)
        pad = -D % (16 // t.element_size()) + 16 // t.element_size()
        shape = (B, S, H, D + pad) if self.tokens_first else (B, H, S, D + pad)
        room = self.torch.full(shape, float("nan"), dtype=self.t, device="cuda")
        view = (room.transpose(1, 2) if self.tokens_first else room)[..., :D]
        view.copy_(t)
        return view, t.to(self.torch.float64).numpy()

    def run(self, **kw):
        return vt.attn_fwd_prefix(self.q, self.kp, self.vp, self.kc, self.vc, self.kv_len, scale=self.scale,
                                  return_lse=True, **kw)

    def check(self, o, lse):
        B, H, H_kv, S_q, S_p, S_c, D_qk, D_v = self.dims
        eps = self.torch.finfo(self.t).eps / 2
        bf = self.t == self.torch.bfloat16
        o, lse = (x.to(self.torch.float64).cpu().numpy() for x in (o, lse))
        for b in range(B):
            n = min(max(int(self.lens[b]), 0), S_c)
            for h in range(H):
                hk = h // (H // H_kv)
                k = np.concatenate([self.kp64[0, hk], self.kc64[b, hk, :n]])
                v = np.concatenate([self.vp64[0, hk], self.vc64[b, hk, :n]])
                for s in range(S_q):
                    seen = S_p + max(0, n - S_q + s + 1)
                    at = f"b={b} h={h} s={s} ({seen} keys)"
                    if seen == 0:
                        assert not o[b, h, s].any() and lse[b, h, s] == -np.inf, at
                        continue
                    x = self.scale * (k[:seen] @ self.q64[b, h, s])
                    size = (abs(self.scale) * (np.abs(k[:seen]) @ np.abs(self.q64[b, h, s]))).max()
                    d = size * (2.0 ** -17 + (0.0 if bf else 2.0 ** -19))
                    top = x.max()
                    w = np.exp(x - top)
                    want_lse = top + np.log(w.sum())
                    w /= w.sum()
                    want = w @ v[:seen]
                    mass = w @ np.abs(v[:seen])
                    tol = (2 * d + 2.0 ** -18) * mass + eps * np.abs(want) + (2 * eps * mass if bf else 0.0)
                    err = np.abs(o[b, h, s] - want)
                    assert (err <= tol).all(), f"{at}: O off by {err.max():.3e}, allowed {tol[err.argmax()]:.3e}"
                    tol = d + 2.0 ** -19 * (1 + abs(want_lse))
                    assert abs(lse[b, h, s] - want_lse) <= tol, f"{at}: LSE {lse[b, h, s]} for {want_lse}, +- {tol:.3e}"


CASES = [
    # dtype, B, H, H_kv, S_q, S_p, S_c, D_qk, D_v
    ("bf16", 1, 1, 1, 1, 1, 1, 8, 8),
    ("bf16", 4, 8, 2, 1, 333, 100, 128, 128),     # the prefix again for every sequence
    ("bf16", 70, 4, 2, 1, 1000, 37, 128, 128),    # the prefix once, shares of it
    ("bf16", 19, 6, 2, 1, 2051, 50, 72, 40),      # groups of 3, odd widths
    ("bf16", 9, 8, 1, 3, 515, 64, 96, 64),
    ("bf16", 5, 4, 4, 1, 700, 513, 64, 128),
    ("bf16", 3, 6, 2, 17, 900, 120, 128, 64),     # rows of a sequence over several tiles
    ("bf16", 2, 2, 1, 130, 400, 260, 64, 64),
    ("bf16", 6, 4, 2, 1, 0, 3000, 128, 128),      # no prefix
    ("bf16", 6, 4, 2, 2, 640, 0, 128, 128),       # no cache
    ("bf16", 2, 3, 1, 2, 0, 9, 33, 20),
    ("bf16", 33, 8, 1, 2, 1025, 9, 80, 128),      # three query tiles of gathered rows, the last one short
    ("bf16", 160, 64, 8, 4, 300, 5, 64, 64),      # more blocks of gathered rows than SMs
    ("bf16", 80, 64, 8, 8, 300, 8, 128, 128),
    ("bf16", 3, 8, 2, 100, 129, 300, 128, 128),   # chunks: the rows of a sequence fill tiles of their own
    ("bf16", 2, 4, 1, 70, 0, 200, 96, 64),
    ("bf16", 5, 8, 1, 33, 1000, 0, 128, 72),
    ("bf16", 40, 6, 2, 90, 70, 91, 40, 128),      # more of them than SMs
    ("bf16", 70, 4, 2, 1, 1000, 37, 64, 33),      # an odd value width in the shares
    ("bf16", 1, 4, 1, 2, 0, 20000, 128, 128),     # one sequence: its keys in shares
    ("bf16", 2, 4, 2, 1, 9000, 9000, 96, 33),     # the same behind a prefix of its own launch
    ("f32", 1, 2, 1, 1, 5000, 3000, 64, 64),
    ("f32", 1, 1, 1, 1, 1, 1, 4, 4),
    ("f32", 8, 8, 2, 1, 1000, 333, 72, 72),
    ("f32", 40, 8, 2, 1, 1500, 40, 128, 128),
    ("f32", 3, 4, 1, 5, 300, 77, 20, 36),
    ("f32", 2, 2, 2, 40, 100, 90, 64, 128),
    ("f32", 4, 4, 1, 1, 0, 1200, 33, 7),
]


@gpu
@pytest.mark.parametrize("tokens_first", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_against_the_definition(case, tokens_first):
    p = Problem(*case, seed=1, tokens_first=tokens_first)
    p.check(*p.run())
    assert vt.vt_last_device_status() == 0


@gpu
@pytest.mark.parametrize("dtype,S_q,D_v", [("bf16", 3, 64), ("f32", 3, 64), ("bf16", 70, 64), ("bf16", 70, 128)])
@pytest.mark.parametrize("S_p", [0, 5, 600])
def test_lengths_at_their_ends(dtype, S_q, D_v, S_p):
    # empty, one token, fewer than the queries, a block of keys and its neighbours, full
    lens = [0, 1, 2, 3, 15, 16, 17, 63, 64, 65, 69, 70, 71, 127, 128, 129]
    p = Problem(dtype, len(lens), 4, 2, S_q, S_p, 129, 64, D_v, lens=lens, seed=2)
    p.check(*p.run())
    p.lens[:] = 129
    o, lse = vt.attn_fwd_prefix(p.q, p.kp, p.vp, p.kc.nan_to_num(0.0), p.vc.nan_to_num(0.0), None, scale=p.scale,
                                return_lse=True)
    for a, t in ((p.kc64, p.kc), (p.vc64, p.vc)):
        a[:] = t.nan_to_num(0.0).double().cpu().numpy()
    p.check(o, lse)


@gpu
@pytest.mark.parametrize("S_q", [1, 64])
def test_lengths_outside_the_cache_are_reported(S_q):
    p = Problem("bf16", 3, 4, 2, S_q, 50, 20, 64, 64, lens=[-5, 20, 20], seed=3)
    p.kv_len[2] = 1 << 20
    p.check(*p.run())
    assert vt.vt_last_device_status() == 6
    assert vt.vt_last_device_status() == 0


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, -0.5, 3.0])
def test_scales_and_peaked_rows(dtype, scale):
    # streamed, and (bf16) on tiles of gathered rows
    for B, S_q, D in ((20, 1, 64), (90, 1, 64), (90, 1, 128), (2, 50, 64), (2, 50, 128)):
        p = Problem(dtype, B, 4, 1, S_q, 1100, 60, D, D, seed=4, scale=scale, spread=2.0)
        p.check(*p.run())


@gpu
@pytest.mark.parametrize("B,S_q,S_p", [(3, 1, 100), (90, 1, 1100), (2, 70, 300)])
def test_nan_stays_in_its_row(B, S_q, S_p):
    p = Problem("bf16", B, 4, 2, S_q, S_p, 80, 64, 64, lens=[80] * B, seed=11)
    want = [t.clone() for t in p.run()]
    p.q[1, 2, S_q - 1, 5] = float("nan")
    o, lse = p.run()
    assert p.torch.isnan(o[1, 2, S_q - 1]).all() and p.torch.isnan(lse[1, 2, S_q - 1])
    o[1, 2, S_q - 1], lse[1, 2, S_q - 1] = want[0][1, 2, S_q - 1], want[1][1, 2, S_q - 1]
    assert p.torch.equal(o, want[0]) and p.torch.equal(lse, want[1])


@gpu
def test_a_row_dominated_by_one_key_returns_its_value():
    p = Problem("bf16", 3, 2, 1, 1, 400, 30, 64, 64, lens=[30, 7, 1], seed=5)
    for b, n in enumerate(p.lens):
        for h in range(2):
            p.q[b, h, 0] = p.kc[b, 0, n - 1] * 8
    o, _ = p.run()
    for b, n in enumerate(p.lens):
        assert p.torch.equal(o[b, :, 0], p.vc[b, :, n - 1].expand(2, -1))


@gpu
def test_writes_nothing_else():
    p = Problem("bf16", 5, 6, 2, 2, 900, 40, 72, 40, seed=6)
    torch = p.torch
    room = torch.full((5, 3, 6, 64), 7.0, dtype=p.t, device="cuda")
    out = room[:, :2].transpose(1, 2)[..., 8:48]
    lse_room = torch.full((5 * 6 * 2 + 2,), 7.0, device="cuda")
    lse = lse_room[1:-1].view(5, 6, 2)
    need = vt.vt_attn_prefix_workspace_size(5, 6, 2, 2, 900, 40, 72, 40, vt.VT_BF16)
    ws = torch.full((need + 512,), 7, dtype=torch.uint8, device="cuda")
    p.check(*p.run(out=out, lse=lse, workspace=ws[:need] if need else None))
    out.fill_(7.0)
    assert (room == 7.0).all() and lse_room[0] == 7.0 and lse_room[-1] == 7.0 and (ws[need:] == 7).all()


@gpu
def test_runs_give_the_same_bits_on_any_stream_and_from_a_graph():
    p = Problem("bf16", 70, 8, 2, 1, 3000, 200, 128, 128, seed=7)
    torch = p.torch
    first = p.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = p.run(stream=side)
    assert vt.vt_last_device_status(side) == 0
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = p.run()
    for seed in (7, 8):  # the captured call with new inputs and lengths
        fresh = Problem("bf16", *p.dims, seed=seed, beyond=0.5)
        for name in ("q", "kp", "vp", "kc", "vc", "kv_len"):
            getattr(p, name).copy_(getattr(fresh, name))
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        want = fresh.run()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
def test_calls_at_once_on_two_streams():
    # each with a workspace of its own: the launches of both are in flight together, and in each of three the last
    # reads what the first two left
    ps = [Problem("bf16", 70, 8, 2, 1, 3000, 200, 128, 128, seed=s) for s in (20, 21)]
    torch = ps[0].torch
    want = [p.run() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    got = [[p.run(stream=s) for p, s in zip(ps, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for pair in got:
        for w, g in zip(want, pair):
            assert all(torch.equal(a, b) for a, b in zip(w, g))
    assert all(vt.vt_last_device_status(s) == 0 for s in streams)


@gpu
def test_long_caches_pass_32_bit_offsets():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    # two sequences 2^31 elements apart, rows 2^15 elements apart: offsets reach past 2^32 bytes and 2^31 elements
    B, S_c, D, row = 2, 70000, 64, 1 << 15
    room = torch.empty((1 << 31) + S_c * row + D, dtype=torch.bfloat16, device="cuda")
    kc = torch.as_strided(room, (B, 1, S_c, D), (1 << 31, 1 << 31, row, 1))
    vc = torch.as_strided(room, (B, 1, S_c, D), (1 << 31, 1 << 31, row, 1), D)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v, q = (torch.randn(n, generator=g, device="cuda").bfloat16() for n in
               ((B, 1, S_c, D), (B, 1, S_c, D), (B, 4, 1, D)))
    # (the second sequence's rows fall between the first one's: they share no row's 128 elements)
    kc[0].copy_(k[0]); vc[0].copy_(v[0])
    keep = 1 << 14
    kc2 = torch.as_strided(room, (1, S_c, D), (1 << 31, row, 1), (1 << 31) + keep)
    vc2 = torch.as_strided(room, (1, S_c, D), (1 << 31, row, 1), (1 << 31) + keep + D)
    kc2.copy_(k[1]); vc2.copy_(v[1])
    kc = torch.as_strided(room, (B, 1, S_c, D), ((1 << 31) + keep, 1 << 31, row, 1))
    vc = torch.as_strided(room, (B, 1, S_c, D), ((1 << 31) + keep, 1 << 31, row, 1), D)
    lens = torch.tensor([S_c, S_c - 1], dtype=torch.int32, device="cuda")
    got = vt.attn_fwd_prefix(q, None, None, kc, vc, lens, return_lse=True)
    want = vt.attn_fwd_prefix(q, None, None, k, v, lens, return_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x = torch.einsum("bhd,bkd->bhk", q[:, :, 0].double(), k[:, 0].double()) / 8
    x[1, :, S_c - 1:] = -float("inf")
    assert (got[1][:, :, 0].double() - torch.logsumexp(x, -1)).abs().max() < 1e-4


@gpu
@pytest.mark.parametrize("dtype,S", [("bf16", 1), ("bf16", 4), ("f32", 2)])
def test_steps_of_a_batch_behind_a_prefix(dtype, S):
    """Three steps as a server makes them: prepare the new tokens, append them, attend; the second is captured and
    replayed.  Every step's O is the one the definition gives on the caches it left."""
    B, H, H_kv, S_p, S_c, D = 6, 8, 2, 700, 40, 64
    p = Problem(dtype, B, H, H_kv, S, S_p, S_c, D, D, lens=[0, 1, 3, 9, 20, 28], seed=9, beyond=0.0)
    torch, rng = p.torch, p.rng
    freqs = torch.from_numpy((10000.0 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32)).cuda()
    w, w64 = p.tensor(1, 1, 2, D)
    qw, kw = w[0, 0, 0].contiguous(), w[0, 0, 1].contiguous()
    q, k, v = (p.tensor(B, n, S, D)[0] for n in (H, H_kv, H_kv))
    pos = torch.zeros((B, S), dtype=torch.int32, device="cuda")
    arange = torch.arange(S, device="cuda", dtype=torch.int32)

    def step():
        return vt.attn_prefix_step(q, k, v, freqs, pos, p.kp, p.vp, p.kc, p.vc, p.kv_len, eps=1e-6, q_weight=qw,
                                   k_weight=kw, scale=p.scale, return_lse=True)

    graph = None
    for n in range(3):
        fresh = [p.tensor(B, c, S, D) for c in (H, H_kv, H_kv)]
        for dst, (src, _) in zip((q, k, v), fresh):
            dst.copy_(src)
        p.kv_len += S
        p.lens = p.lens + S
        pos.copy_(S_p + p.kv_len[:, None] - S + arange)
        old = [p.kc.clone(), p.vc.clone()]
        if n == 1:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = step()
        if graph is not None:
            graph.replay()
        else:
            out = step()
        torch.cuda.synchronize()
        assert vt.vt_last_device_status() == 0
        # the rows appended, and no others
        cos, sin = rope_ref.cos_sin(pos.cpu().numpy()[None], freqs.cpu().numpy(), (0,) * (D // 2))
        want_k, size = rope_ref.forward(fresh[1][1], w64[0, 0, 1], 1e-6, cos, sin, False)
        for b in range(B):
            rows = slice(int(p.lens[b]) - S, int(p.lens[b]))
            err = np.abs(p.kc[b, :, rows].double().cpu().numpy() - want_k[b])
            assert (err <= torch.finfo(p.t).eps / 2 * np.abs(want_k[b]) + 64 * 2.0 ** -24 * size[b]).all()
            assert torch.equal(p.vc[b, :, rows], v[b])
            old[0][b, :, rows], old[1][b, :, rows] = p.kc[b, :, rows], p.vc[b, :, rows]
        assert torch.equal(old[0], p.kc) and torch.equal(old[1], p.vc)
        # attention, on the rotated queries as the first operator rounds them
        q_rot, _ = vt.qk_rope(q, None, freqs, pos, eps=1e-6, q_weight=qw)
        p.q64 = q_rot.double().cpu().numpy()
        p.kc64, p.vc64 = p.kc.double().cpu().numpy(), p.vc.double().cpu().numpy()
        p.check(*out)


# ---------------------------------------------------------------- sizes at the contract's limits (no GPU)

def test_plan_of_the_largest_sizes():
    """2^26 sequences of one row over 2^28 shared keys: the prefix read once per sequence would be 2^64 bytes, so it is
    read once for all of them, with partial results in the workspace."""
    assert vt.vt_attn_prefix_workspace_size(1 << 26, 1, 1, 1, 1 << 28, 16, 128, 128, vt.VT_F32) > 0


# ---------------------------------------------------------------- scalar arguments that change in place (no GPU)

def test_scalar_arguments_are_read_in_every_call(monkeypatch):
    """A scale or eps held in a tensor is taken at its value of the call, not at that of an earlier call with it."""
    import torch
    lib, seen = vt.load(), []

    class Recorder:
        def __getattr__(self, name):
            return getattr(lib, name)

        def vt_attn_fwd_prefix(self, args, stream):
            seen.append(vt._ATTN_PREFIX_REST.unpack(args[vt._ATTN_PREFIX_PTRS.size:])[9])
            return 0

        def vt_qk_rope_fwd(self, args, stream):
            seen.append(vt._QK_ROPE_REST.unpack(args[vt._QK_ROPE_PTRS.size:])[12])
            return 0

        def vt_qk_rope_bwd(self, args, *rest):
            seen.append(vt._QK_ROPE_REST.unpack(args[vt._QK_ROPE_PTRS.size:])[12])
            return 0

    monkeypatch.setattr(vt, "load", Recorder)
    monkeypatch.setattr(vt, "_here", lambda t: True)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    q, kc = torch.zeros(1, 2, 1, 16), torch.zeros(1, 2, 8, 16)
    freqs, pos = torch.ones(8), torch.zeros(1, 1, dtype=torch.int32)
    ws = torch.zeros(2 * 608 * 16 * 4, dtype=torch.uint8)
    number = torch.tensor(0.25)
    calls = (lambda: vt.attn_fwd_prefix(q, None, None, kc, kc, scale=number),
             lambda: vt.qk_rope(q, None, freqs, pos, eps=number),
             lambda: vt.qk_rope_bwd(q, None, freqs, pos, q=q, eps=number, workspace=ws))
    for call in calls:
        for value in (0.25, 0.5):
            number.fill_(value)
            call()
    assert seen == [0.25, 0.5] * 3


def test_pair_axis_takes_whole_numbers_only():
    import torch
    with pytest.raises(TypeError):
        vt._pair_axis_bytes((torch.tensor(0), torch.tensor(1)), 2, 2)
    assert vt._pair_axis_bytes((0, np.int64(1)), 2, 2)[:2] == b"\0\1"


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """A stream belongs to a device: work on tensors of another one would silently run elsewhere."""
    import types

    import torch

    class Stream:
        device = torch.device("cuda", 1)

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    on_0 = types.SimpleNamespace(is_cuda=True, device=torch.device("cuda", 0))
    with pytest.raises(ValueError, match="device"):
        vt._elsewhere(lambda: None, on_0, Stream(), (), {})
