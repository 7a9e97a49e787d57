"""vt_attn_fwd_packed and vt_attn_bwd_packed: refusals (host only) and results against a plain 64-bit form.

Tolerances.  With h = eps / 2 of the type (half a rounding step) and acc(n) = (n + 32) 2^-23 for a sum of n products in fp32
(2^-23 each: the tensor core cuts what it adds), f = 2^-19 for fp32 (two TF32 parts per factor lose 2^-20 of each) and 0 for
bf16 (products of bf16 are exact in fp32):
  a score s is off by d = (acc(D) + f) max_j sum |scale q k|, the log-sum-exp by d + 2^-19 (1 + |LSE|), and a weight
  P = exp(s - LSE) by r = 2 (2 d + 2^-19 (1 + |LSE|)) + 2^-20 of itself (e^x - 1 <= 2 x there);
  O:      (2 d + acc(n) + f) sum P |v| + h |O|, and 2 h sum P |v| more in bf16 (P is rounded);
  dV:     sum P |g| (r + acc(n) + f + [bf16] h) + h |dV|;
  delta = sum g o: o is rounded (h) and the sum is acc(D) off;  dP: (acc(D) + f) sum |g v|;
  dS:     P (dP's + delta's) + r |dS| + [bf16] h |dS|;
  dQ, dK: sum of dS's |scale k| (or |scale q|), (acc(n) + f) sum |dS scale k|, and h of the result.
"""

import math

import numpy as np
import pytest

import scaled_dot_product_vt_gb300 as vt

gpu = pytest.mark.gpu
A = 1 << 28  # fake, aligned, distinct "device" addresses: never dereferenced on the refusal paths


@pytest.fixture(scope="module", autouse=True)
def _built():
    vt.build()
    vt.load()


# ---------------------------------------------------------------- refusals (no GPU)

def pack(**kw):
    f = dict(size=vt._ATTN_PACKED_BYTES, q=A, k=2 * A, v=3 * A, cu_q=4 * A, cu_k=5 * A, o=6 * A, lse=7 * A, N=3, H=4, H_kv=2,
             T_q=40, T_k=50, D_qk=16, D_v=8, window=0, dtype=vt.VT_BF16, scale=0.25, mask=1, reserved=0, qs=(16, 64),
             ks=(16, 32), vs=(8, 16), os=(8, 32))
    f.update({k: v for k, v in kw.items() if k in f})
    return vt._ATTN_PACKED_PTRS.pack(f["size"], f["q"], f["k"], f["v"], f["cu_q"], f["cu_k"], f["o"], f["lse"]) + \
        vt._ATTN_PACKED_REST.pack(f["N"], f["H"], f["H_kv"], f["T_q"], f["T_k"], f["D_qk"], f["D_v"], f["window"], f["dtype"],
                                  f["scale"], f["mask"], f["reserved"], *f["qs"], *f["ks"], *f["vs"], *f["os"])


def grads(**kw):
    f = dict(gsize=vt._PACKED_GRADS_BYTES, do=8 * A, dlse=9 * A, dq=10 * A, dk=11 * A, dv=12 * A, ws=13 * A, wsb=1 << 20,
             dos=(8, 32), dqs=(16, 64), dks=(16, 32), dvs=(8, 16))
    f.update({k: v for k, v in kw.items() if k in f})
    return vt._PACKED_GRADS_PTRS.pack(f["gsize"], f["do"], f["dlse"], f["dq"], f["dk"], f["dv"], f["ws"], f["wsb"]) + \
        vt._PACKED_GRADS_REST.pack(*f["dos"], *f["dqs"], *f["dks"], *f["dvs"])


def forward(**kw):
    return vt.vt_attn_fwd_packed(pack(**kw), None)


def backward(**kw):
    return vt.vt_attn_bwd_packed(pack(**kw), grads(**kw), None)


BAD = [
    (dict(size=8), 1), (dict(reserved=1), 1), (dict(dtype=2), 1), (dict(N=-1), 1), (dict(H=-4), 1), (dict(T_q=-1), 1),
    (dict(T_k=-1), 1), (dict(D_qk=0), 1), (dict(D_v=0), 1), (dict(H_kv=0), 1), (dict(H_kv=3), 1),
    (dict(scale=float("inf")), 1), (dict(mask=4), 1), (dict(mask=-1), 1), (dict(mask=2), 1), (dict(mask=3, window=0), 1),
    (dict(mask=2, window=(1 << 40) + 1), 2), (dict(D_qk=129), 2), (dict(D_v=136), 2), (dict(T_q=(1 << 30) + 1), 2),
    (dict(T_k=(1 << 30) + 1), 2), (dict(N=(1 << 30) + 1), 2), (dict(N=1 << 30), 2), (dict(H=1 << 20, T_q=1 << 20), 2),
    (dict(q=0), 1), (dict(k=0), 1), (dict(v=0), 1), (dict(cu_q=0), 1), (dict(cu_k=0), 1), (dict(o=0), 1),
    (dict(q=A + 8), 3), (dict(v=3 * A + 2), 3), (dict(cu_q=4 * A + 2), 3), (dict(lse=7 * A + 2), 3), (dict(qs=(20, 64)), 3),
    (dict(ks=(16, -32)), 1), (dict(vs=(1 << 40, 16)), 2),
]


@pytest.mark.parametrize("kw,code", BAD)
def test_refusals(kw, code):
    assert forward(**kw) == code and backward(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(os=(8, 24)), 1),                                   # O's rows meet
    (dict(o=A), 1), (dict(o=3 * A + 16), 1), (dict(o=4 * A), 1), (dict(lse=2 * A), 1), (dict(lse=6 * A), 1),
])
def test_forward_outputs_that_meet(kw, code):
    assert forward(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(gsize=8), 1), (dict(lse=0), 1), (dict(do=0), 1), (dict(dq=0), 1), (dict(dk=0), 1), (dict(dv=0), 1),
    (dict(do=8 * A + 4), 3), (dict(dlse=9 * A + 1), 3), (dict(dqs=(16, 20)), 3), (dict(dks=(0, 32)), 1),
    (dict(dqs=(16, 48)), 1), (dict(dq=A), 1), (dict(dk=10 * A), 1), (dict(dv=11 * A), 1), (dict(dq=8 * A), 1),
    (dict(dk=6 * A), 1), (dict(dv=7 * A), 1), (dict(ws=0), 1), (dict(ws=13 * A + 16), 3), (dict(wsb=1024), 1),
    (dict(ws=12 * A), 1), (dict(ws=A), 1),
])
def test_backward_refusals(kw, code):
    assert backward(**kw) == code


def test_empty_problems():
    for kw in (dict(N=0), dict(H=0), dict(T_q=0, T_k=0)):
        none = dict(q=0, k=0, v=0, cu_q=0, cu_k=0, o=0, lse=0, do=0, dq=0, dk=0, dv=0, ws=0, wsb=0)
        assert forward(**kw, **none) == 0 and backward(**kw, **none) == 0
    assert forward(T_q=0, q=0, o=0) == 0
    assert vt.load().vt_attn_fwd_packed(None, None) == 1 and vt.load().vt_attn_bwd_packed(pack(), None, None) == 1
    size = vt.vt_attn_bwd_packed_workspace_size
    assert size(0, 4, 2, 9, 9, 16, 16, 1) == 0 and size(2, 4, 3, 9, 9, 16, 16, 1) == 0 and size(2, 4, 2, 9, 9, 130, 16, 1) == 0
    assert size(2, 4, 2, 300, 300, 16, 16, 1) >= 4 * 300 * 8


def test_valid_calls_reach_the_launch():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: a valid call would launch on these fake addresses")
    cases = (dict(), dict(dtype=vt.VT_F32, qs=(16, 64)), dict(mask=2, window=5), dict(lse=7 * A, dlse=0), dict(cu_k=4 * A),
             dict(T_k=0, k=0, v=0, dk=0, dv=0), dict(dq=10 * A, dk=10 * A + 128, dv=10 * A + 192, dqs=(16, 112),
                                                     dks=(16, 112), dvs=(8, 112)))  # one projection's gradient
    for kw in cases:
        assert backward(**kw) == 4, kw
        assert forward(**kw) == 4, kw
    assert forward(lse=0) == 4
    assert backward(T_q=0, q=0, o=0, lse=0, do=0, dq=0) == 4


# ---------------------------------------------------------------- results

class Problem:
    """Sequences of (queries, keys) rows behind `before` rows of none and ahead of `behind` more; everything outside the
    sequences is NaN, and rows are padded with NaN."""

    def __init__(self, dtype, H, H_kv, D_qk, D_v, lengths, mask="causal", window=0, seed=0, scale=None, spread=1.0, before=0,
                 behind=3, tokens_first=True):
        import torch
        if not torch.cuda.is_available():
            pytest.skip("no CUDA device")
        self.torch, self.t = torch, dict(bf16=torch.bfloat16, f32=torch.float32)[dtype]
        self.H, self.H_kv, self.D_qk, self.D_v, self.lengths = H, H_kv, D_qk, D_v, lengths
        self.form = dict(mask=mask, window=window, scale=float(np.float32(scale if scale is not None else D_qk ** -0.5)))
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.tokens_first, self.before, self.behind = tokens_first, before, behind
        self.cu = [np.cumsum([before] + [n[i] for n in lengths]) for i in (0, 1)]
        self.cu_q, self.cu_k = (torch.tensor(c, dtype=torch.int32, device="cuda") for c in self.cu)
        self.q, self.do = (self.rows(H, 0, D, spread) for D in (D_qk, D_v))
        self.k, self.v = (self.rows(H_kv, 1, D, spread) for D in (D_qk, D_v))
        self.dlse = torch.randn((H, self.cu[0][-1] + behind), generator=self.g, device="cuda")

    def room(self, H, T, D, fill):
        torch = self.torch
        pad = -D % (16 // self.t.itemsize) + 16 // self.t.itemsize
        x = torch.full((T, H, D + pad) if self.tokens_first else (H, T, D + pad), fill, dtype=self.t, device="cuda")
        return (x.transpose(0, 1) if self.tokens_first else x)[..., :D]

    def rows(self, H, side, D, spread=1.0):
        a, e = self.cu[side][0], self.cu[side][-1]
        x = self.room(H, int(e) + self.behind, D, float("nan"))
        x[:, a:e] = self.torch.randn((H, e - a, D), generator=self.g, device="cuda").mul(spread).to(self.t)
        return x

    def seen(self, n, m):
        """[n, m]: the keys that every query sees."""
        torch, mask, w = self.torch, self.form["mask"], self.form["window"]
        at = torch.arange(n, device="cuda")[:, None] + (m - n)
        key = torch.arange(m, device="cuda")[None]
        return {"none": key >= 0, "causal": key <= at, "window": (key <= at) & (key > at - w),
                "window_complement": key <= at - w}[mask].expand(n, m)

    def parts(self):
        d = self.torch.float64
        for i, (n, m) in enumerate(self.lengths):
            r, c = slice(self.cu[0][i], self.cu[0][i] + n), slice(self.cu[1][i], self.cu[1][i] + m)
            for h in range(self.H):
                hk = h // (self.H // self.H_kv)
                q, k, v, g = self.q[h, r].to(d), self.k[hk, c].to(d), self.v[hk, c].to(d), self.do[h, r].to(d)
                yield h, hk, r, c, q, k, v, g, self.seen(n, m)

    def weights(self, q, k, seen):
        torch, scale = self.torch, self.form["scale"]
        x = (scale * (q @ k.T)).masked_fill(~seen, -math.inf)
        lse = torch.logsumexp(x, -1) if k.shape[0] else torch.full((q.shape[0],), -math.inf, device="cuda").double()
        p = torch.where(seen, torch.exp(x - lse.clamp(min=-1e300)[:, None]), 0.0)
        size = (abs(scale) * (q.abs() @ k.abs().T)).masked_fill(~seen, 0.0)
        return p, lse, size.amax(-1) if k.shape[0] else torch.zeros_like(lse)

    def constants(self):
        bf = self.t == self.torch.bfloat16
        return self.torch.finfo(self.t).eps / 2, bf, 0.0 if bf else 2.0 ** -19, lambda n: (n + 32) * 2.0 ** -23

    def close(self, name, got, want, tol, at):
        err = (got.double() - want).abs()
        bad = ~(err <= tol)
        assert not bad.any(), f"{name} {at}: off by {err[bad].max():.3e} where {tol[bad].max():.3e} is allowed, got {got[bad][:4]}"

    def forward(self, **kw):
        return vt.attn_fwd_packed(self.q, self.k, self.v, self.cu_q, self.cu_k, return_lse=True, **self.form, **kw)

    def outputs(self, fill=7.0):
        """Results' rooms with `fill` in every place: (out, lse), (dq, dk, dv)."""
        torch = self.torch
        T_q, T_k = self.q.shape[1], self.k.shape[1]
        return ((self.room(self.H, T_q, self.D_v, fill), torch.full((self.H, T_q), fill, device="cuda")),
                (self.room(self.H, T_q, self.D_qk, fill), self.room(self.H_kv, T_k, self.D_qk, fill),
                 self.room(self.H_kv, T_k, self.D_v, fill)))

    def untouched(self, x, side, fill=7.0):
        a, e = self.cu[side][0], self.cu[side][-1]
        assert (x[:, :a] == fill).all() and (x[:, e:] == fill).all()
        if x.dim() == 3:  # and the columns behind the rows' last
            room = x._base
            assert (room[..., x.shape[2]:] == fill).all()

    def check_forward(self, o, lse):
        h2, bf, f, acc = self.constants()
        for h, hk, r, c, q, k, v, _, seen in self.parts():
            p, want_lse, size = self.weights(q, k, seen)
            n = seen.sum(-1)
            none = n == 0
            assert (o[h, r][none] == 0).all() and (lse[h, r][none] == -math.inf).all()
            d = (acc(self.D_qk) + f) * size
            want, mass = p @ v, p @ v.abs()
            tol = (2 * d + acc(n) + f + (2 * h2 if bf else 0.0))[:, None] * mass + h2 * want.abs() + 1e-30
            self.close("O", o[h, r], want, tol, (h, r))
            some = ~none
            self.close("LSE", lse[h, r][some], want_lse[some], (d + 2.0 ** -19 * (1 + want_lse.abs()))[some], (h, r))

    def results(self):
        """The forward's results as a user has them, from the definition: O rounded once, LSE in fp32."""
        torch = self.torch
        o, lse = self.room(self.H, self.q.shape[1], self.D_v, float("nan")), torch.full((self.H, self.q.shape[1]), math.nan,
                                                                                          device="cuda")
        for h, hk, r, c, q, k, v, _, seen in self.parts():
            p, want_lse, _ = self.weights(q, k, seen)
            o[h, r] = (p @ v).to(self.t)
            lse[h, r] = want_lse.float()
        return o, lse

    def backward(self, o, lse, dlse=None, **kw):
        return vt.attn_bwd_packed(self.do, self.q, self.k, self.v, o, lse, self.cu_q, self.cu_k, dlse=dlse, **self.form, **kw)

    def check_backward(self, dq, dk, dv, dlse=None):
        torch = self.torch
        h2, bf, f, acc = self.constants()
        scale = self.form["scale"]
        T_k = self.k.shape[1]
        sums = {x: torch.zeros((self.H_kv, T_k, D), dtype=torch.float64, device="cuda")
                for x, D in (("dk", self.D_qk), ("dk_tol", self.D_qk), ("dv", self.D_v), ("dv_tol", self.D_v))}
        for h, hk, r, c, q, k, v, g, seen in self.parts():
            p, lse, size = self.weights(q, k, seen)
            n = seen.sum(-1)
            lse = torch.where(n > 0, lse, 0.0)
            d = (acc(self.D_qk) + f) * size
            rel = (2 * (2 * d + 2.0 ** -19 * (1 + lse.abs())) + 2.0 ** -20)[:, None]
            o = p @ v
            gv, delta = g @ v.T, (g * o).sum(-1, keepdim=True)
            if dlse is not None:
                delta = delta - dlse[h, r].double()[:, None]
            ds = p * (gv - delta)
            dp_off = (acc(self.D_v) + f) * (g.abs() @ v.abs().T)
            delta_off = (g.abs() * o.abs()).sum(-1, keepdim=True) * (h2 + acc(self.D_v) + f) + delta.abs() * 2.0 ** -23
            ds_off = p * (dp_off + delta_off) * (1 + rel) + rel * ds.abs() + (h2 * ds.abs() if bf else 0.0)
            want = scale * (ds @ k)
            tol = abs(scale) * (ds_off @ k.abs() + (acc(k.shape[0]) + f) * (ds.abs() @ k.abs())) + h2 * want.abs() + 1e-30
            self.close("dQ", dq[h, r], want, tol, (h, r))
            many = acc(q.shape[0] * self.H // self.H_kv) + f
            sums["dk"][hk, c] += scale * (ds.T @ q)
            sums["dk_tol"][hk, c] += abs(scale) * (ds_off.T @ q.abs() + many * (ds.abs().T @ q.abs()))
            sums["dv"][hk, c] += p.T @ g
            sums["dv_tol"][hk, c] += (p * (rel + (h2 if bf else 0.0) + many)).T @ g.abs()
        a, e = self.cu[1][0], self.cu[1][-1]
        for name, got in (("dk", dk), ("dv", dv)):
            want = sums[name][:, a:e]
            self.close(name, got[:, a:e], want, sums[name + "_tol"][:, a:e] + h2 * want.abs() + 1e-30, "")

    def check(self, dlse=False):
        (out, lse), gr = self.outputs()
        o, l = self.forward(out=out, lse=lse)
        assert o.data_ptr() == out.data_ptr() and l.data_ptr() == lse.data_ptr()
        self.check_forward(o, l)
        self.untouched(o, 0)
        self.untouched(l, 0)
        dlse = self.dlse if dlse else None
        got = self.backward(*self.results(), dlse=dlse, dq=gr[0], dk=gr[1], dv=gr[2])
        self.check_backward(*got, dlse=dlse)
        for x, side in zip(got, (0, 1, 1)):
            self.untouched(x, side)
        assert vt.vt_last_device_status() == 0


CASES = [
    # dtype, H, H_kv, D_qk, D_v, lengths, mask, window
    ("bf16", 1, 1, 8, 8, [(1, 1)], "causal", 0),
    ("bf16", 4, 2, 128, 128, [(5, 5), (0, 0), (300, 300), (1, 1), (128, 128), (129, 129)], "causal", 0),
    ("bf16", 3, 1, 64, 64, [(127, 127), (256, 256), (257, 257), (64, 64)], "causal", 0),
    ("bf16", 6, 2, 72, 40, [(33, 500), (1, 700), (260, 300), (0, 9), (7, 0)], "causal", 0),       # chunks; one side empty
    ("bf16", 2, 2, 96, 64, [(300, 100), (10, 3), (50, 49)], "causal", 0),                          # first rows see nothing
    ("bf16", 4, 1, 128, 64, [(200, 333), (130, 130)], "none", 0),
    ("bf16", 2, 1, 64, 128, [(400, 400), (90, 600)], "window", 100),
    ("bf16", 2, 1, 128, 128, [(300, 300), (40, 40)], "window", 1),
    ("bf16", 2, 2, 128, 128, [(300, 400), (64, 64)], "window_complement", 70),
    ("bf16", 16, 2, 33, 20, [(70, 70)] * 9, "causal", 0),
    ("bf16", 2, 2, 16, 112, [(513, 513)], "none", 0),
    ("bf16", 40, 8, 64, 64, [(140, 140), (3, 3), (256, 256), (300, 300)], "causal", 0),             # more units than SMs
    ("bf16", 1, 1, 128, 128, [(1, 1)] * 300, "causal", 0),
    ("f32", 1, 1, 4, 4, [(1, 1)], "causal", 0),
    ("f32", 4, 2, 128, 128, [(5, 5), (0, 0), (200, 200), (1, 1), (64, 64), (65, 65)], "causal", 0),
    ("f32", 6, 2, 72, 40, [(33, 300), (1, 400), (160, 170), (0, 9), (7, 0)], "causal", 0),
    ("f32", 2, 1, 64, 96, [(150, 60), (90, 90)], "causal", 0),
    ("f32", 4, 1, 20, 36, [(100, 133), (60, 60)], "none", 0),
    ("f32", 2, 1, 96, 64, [(200, 200), (50, 150)], "window", 17),
    ("f32", 2, 2, 33, 7, [(100, 120), (64, 64)], "window_complement", 30),
    ("f32", 2, 1, 64, 64, [(80, 80)], "window", 1),
]


@gpu
@pytest.mark.parametrize("tokens_first", [True, False])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:5])) + f"-{len(c[5])}-{c[6]}")
def test_against_the_definition(case, tokens_first):
    dtype, H, H_kv, D_qk, D_v, lengths, mask, window = case
    Problem(dtype, H, H_kv, D_qk, D_v, lengths, mask, window, seed=1, before=0 if tokens_first else 5, behind=3,
            tokens_first=tokens_first).check(dlse=tokens_first)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, -0.5, 2.0])
def test_scales_and_peaked_rows(dtype, scale):
    Problem(dtype, 4, 2, 64, 64, [(150, 150), (30, 200)], seed=2, scale=scale, spread=1.5).check(dlse=True)
    Problem(dtype, 2, 1, 128, 128, [(150, 150)], "none", seed=3, scale=scale, spread=1.5).check()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_stays_in_its_sequence(dtype):
    p = Problem(dtype, 4, 2, 64, 128, [(100, 100), (77, 90), (140, 140), (5, 5)], seed=4)
    fwd = [x.clone() for x in p.forward()]
    res = p.results()
    bwd = [x.clone() for x in p.backward(*res)]
    n = slice(p.cu[0][1], p.cu[0][2]), slice(p.cu[1][1], p.cu[1][2])
    for x, s in ((p.q, n[0]), (p.k, n[1]), (p.v, n[1]), (p.do, n[0]), (res[0], n[0]), (res[1], n[0])):
        x[:, s] = float("nan")
    for got, want, side in zip((*p.forward(), *p.backward(*res)), (*fwd, *bwd), (0, 0, 0, 1, 1)):
        a, e = p.cu[side][0], p.cu[side][-1]
        assert p.torch.isnan(got[:, n[side]]).all()
        got[:, n[side]] = want[:, n[side]]
        assert p.torch.equal(got[:, a:e], want[:, a:e])


@gpu
def test_a_nan_query_spares_the_other_rows():
    p = Problem("bf16", 2, 1, 64, 64, [(200, 200)], seed=5)
    want = [x.clone() for x in p.forward()]
    p.q[1, 70, 3] = float("nan")
    o, lse = p.forward()
    assert p.torch.isnan(o[1, 70]).all() and p.torch.isnan(lse[1, 70])
    o[1, 70], lse[1, 70] = want[0][1, 70], want[1][1, 70]
    assert p.torch.equal(o[:, :200], want[0][:, :200]) and p.torch.equal(lse[:, :200], want[1][:, :200])


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_queries_of_one_key_have_no_gradient(dtype):
    """P is 1 whatever the score: dS is 0, and dLSE alone reaches it."""
    for lengths, mask, window in (([(50, 50)], "window", 1), ([(40, 1), (1, 1)], "none", 0), ([(1, 1)] * 5, "causal", 0)):
        p = Problem(dtype, 2, 1, 64, 64, lengths, mask, window, seed=6, behind=0)
        dq, dk, _ = p.backward(*p.results())
        assert (dq == 0).all() and (dk == 0).all()
        p.check(dlse=True)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_first_rows_that_are_not_in_order_are_reported(dtype):
    """Rows outside [0, T] count as the nearest inside, a sequence that ends before it starts as empty (the one behind it
    then starts at row 10, and shares rows 10 to 30 with the first)."""
    p = Problem(dtype, 2, 1, 64, 64, [(30, 30), (40, 40), (50, 50)], seed=7, behind=0)
    good = [x.clone() for x in p.forward()]
    grad = [x.clone() for x in p.backward(*p.results())]
    res = p.results()
    for cu, kept in (([-9, 30, 70, 120], slice(0, 120)), ([0, 30, 70, 1 << 20], slice(0, 120)),
                     ([0, 30, 10, 120], slice(0, 10))):
        p.cu_q.copy_(p.torch.tensor(cu))
        p.cu_k.copy_(p.torch.tensor(cu))
        got = p.forward()
        assert vt.vt_last_device_status() == 6 and vt.vt_last_device_status() == 0
        bwd = p.backward(*res)
        assert vt.vt_last_device_status() == 6 and vt.vt_last_device_status() == 0
        for a, b in zip((*got, *bwd), (*good, *grad)):
            assert p.torch.equal(a[:, kept], b[:, kept])


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_projection_and_its_gradient(dtype):
    """Q, K and V beside each other in one tensor, their gradients in another; cu_k left out."""
    import torch
    p = Problem(dtype, 6, 2, 64, 64, [(130, 130), (20, 20), (75, 75)], seed=8, behind=0)
    T = p.q.shape[1]
    qkv, dqkv = (torch.empty((T, 10, 64), dtype=p.t, device="cuda").transpose(0, 1) for _ in range(2))
    qkv[:6], qkv[6:8], qkv[8:] = p.q, p.k, p.v
    p.q, p.k, p.v = qkv[:6], qkv[6:8], qkv[8:]
    p.check_forward(*vt.attn_fwd_packed(p.q, p.k, p.v, p.cu_q, return_lse=True, **p.form))
    vt.attn_bwd_packed(p.do, p.q, p.k, p.v, *p.results(), p.cu_q, dq=dqkv[:6], dk=dqkv[6:8], dv=dqkv[8:], **p.form)
    p.check_backward(dqkv[:6], dqkv[6:8], dqkv[8:])


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_same_bits_on_any_stream_from_a_graph_and_with_a_workspace(dtype):
    p = Problem(dtype, 8, 2, 128, 128, [(300, 300), (7, 7), (450, 450), (129, 129)], seed=9, behind=0)
    torch = p.torch
    res = p.results()
    need = vt.vt_attn_bwd_packed_workspace_size(4, 8, 2, p.q.shape[1], p.k.shape[1], 128, 128, 1 if dtype == "bf16" else 0)
    room = torch.full((need + 512,), 7, dtype=torch.uint8, device="cuda")
    first = [x.clone() for x in (*p.forward(), *p.backward(*res, workspace=room[:need]))]
    assert (room[need:] == 7).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = (*p.forward(stream=side), *p.backward(*res, stream=side))
    assert vt.vt_last_device_status(side) == 0
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = (*p.forward(), *p.backward(*res))
    for lengths in ([(300, 300), (7, 7), (450, 450), (129, 129)], [(0, 0), (800, 800), (1, 1), (85, 85)]):
        fresh = Problem(dtype, 8, 2, 128, 128, lengths, seed=10, behind=0)  # new inputs and lengths
        fres = fresh.results()
        for name in ("q", "k", "v", "do", "cu_q", "cu_k"):
            getattr(p, name).copy_(getattr(fresh, name))
        for a, b in zip(res, fres):
            a.copy_(b)
        for x in got:
            x.fill_(float("nan"))
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (*fresh.forward(), *fresh.backward(*fres))))


@gpu
def test_calls_at_once_on_two_streams():
    ps = [Problem(d, 8, 2, 128, 64, [(300, 300), (700, 700), (33, 33)], seed=11, behind=0) for d in ("bf16", "f32")]
    torch = ps[0].torch
    res = [p.results() for p in ps]
    want = [(*p.forward(), *p.backward(*r)) for p, r in zip(ps, res)]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    got = [[(*p.forward(stream=s), *p.backward(*r, stream=s)) for p, r, s in zip(ps, res, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    for pair in got:
        for w, g in zip(want, pair):
            assert all(torch.equal(a, b) for a, b in zip(w, g))
    assert all(vt.vt_last_device_status(s) == 0 for s in streams)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_pass_32_bits(dtype):
    """Rows 2^15 elements (and more) apart: offsets pass 2^31 elements and 2^32 bytes.  Every tensor has columns of its own."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    T, D, row = 70000, 64, 1 << 15
    t = dict(bf16=torch.bfloat16, f32=torch.float32)[dtype]
    room = torch.empty((T, row), dtype=t, device="cuda")
    at = lambda i: torch.as_strided(room, (1, T, D), (row, row, 1), 64 * i)
    g = torch.Generator(device="cuda").manual_seed(1)
    small = [torch.randn((1, T, D), generator=g, device="cuda").to(t) for _ in range(4)]
    wide = [at(i) for i in range(4)]
    for a, b in zip(wide, small):
        a.copy_(b)
    cu = torch.tensor([0, 10, 69000, T], dtype=torch.int32, device="cuda")
    form = dict(mask="window", window=300, scale=0.125)
    results = []
    for (q, k, v, do), out in ((small, [None] * 4), (wide, [at(4 + i) for i in range(4)])):
        o, lse = vt.attn_fwd_packed(q, k, v, cu, return_lse=True, out=out[0], **form)
        results.append((o, lse, *vt.attn_bwd_packed(do, q, k, v, o, lse, cu, dq=out[1], dk=out[2], dv=out[3], **form)))
    assert all(torch.equal(a, b) for a, b in zip(*results))
    assert vt.vt_last_device_status() == 0


@gpu
def test_gradients_against_differences():
    """d/dt of sum(O g) + sum(LSE dl) along a direction, from the 64-bit definition: central differences with a step of 2^-10
    are off by 2^-20 / 6 of the third derivative, the fp32 gradients by 2^-17 of their terms: 1e-4 of the terms' sizes."""
    p = Problem("f32", 4, 2, 32, 32, [(20, 20), (9, 30), (40, 17)], seed=12, behind=0)
    torch = p.torch
    dl = torch.where(torch.isfinite(p.results()[1]), p.dlse, 0.0)
    grads_ = p.backward(*p.results(), dlse=dl)
    base = [x.clone() for x in (p.q, p.k, p.v)]
    way = [torch.randn(x.shape, generator=p.g, device="cuda") for x in base]

    def loss(step):
        total = 0.0
        for x, b, w in zip((p.q, p.k, p.v), base, way):
            x.copy_(b + step * w)
        for h, hk, r, c, q, k, v, g, seen in p.parts():
            # (the perturbed inputs in 64 bits, not their roundings)
            q, k, v = (b.double()[i, s] + step * w.double()[i, s] for b, w, i, s in
                       ((base[0], way[0], h, r), (base[1], way[1], hk, c), (base[2], way[2], hk, c)))
            pr, lse, _ = p.weights(q, k, seen)
            some = seen.any(-1)
            total += float((g * (pr @ v)).sum()) + float((lse[some] * dl[h, r].double()[some]).sum())
        return total

    got = sum(float((a.double() * w.double()).sum()) for a, w in zip(grads_, way))
    want = (loss(2.0 ** -10) - loss(-2.0 ** -10)) * 2.0 ** 9
    assert abs(got - want) <= 1e-4 * sum(float((a.double() * w.double()).abs().sum()) for a, w in zip(grads_, way))


@gpu
def test_the_debug_library_finds_nothing():
    """Its index checks pass, and its results are the release library's."""
    import torch
    dbg = vt.load_debug()
    for dtype, mask, window in (("bf16", "causal", 0), ("bf16", "window", 50), ("f32", "causal", 0)):
        p = Problem(dtype, 4, 2, 64, 64, [(200, 300), (1, 1), (0, 4), (140, 90), (300, 300)], mask, window, seed=14, behind=0)
        o, lse = p.forward()
        got = p.backward(o, lse)
        o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
        new = [torch.empty_like(x) for x in got]
        code = vt.VT_BF16 if dtype == "bf16" else vt.VT_F32
        st = lambda x: (x.stride(0), x.stride(1))
        dims = (len(p.lengths), 4, 2, p.q.shape[1], p.k.shape[1], 64, 64)
        args = pack(q=p.q.data_ptr(), k=p.k.data_ptr(), v=p.v.data_ptr(), cu_q=p.cu_q.data_ptr(), cu_k=p.cu_k.data_ptr(),
                    o=o2.data_ptr(), lse=lse2.data_ptr(), N=dims[0], H=4, H_kv=2, T_q=dims[3], T_k=dims[4], D_qk=64, D_v=64,
                    window=window, dtype=code, scale=p.form["scale"], mask=vt.MASKS[mask], qs=st(p.q), ks=st(p.k), vs=st(p.v),
                    os=st(o2))
        ws = torch.empty(vt.vt_attn_bwd_packed_workspace_size(*dims, code), dtype=torch.uint8, device="cuda")
        g = grads(do=p.do.data_ptr(), dlse=0, dq=new[0].data_ptr(), dk=new[1].data_ptr(), dv=new[2].data_ptr(), ws=ws.data_ptr(),
                  wsb=ws.numel(), dos=st(p.do), dqs=st(new[0]), dks=st(new[1]), dvs=st(new[2]))
        stream = torch.cuda.current_stream().cuda_stream
        assert dbg.vt_attn_fwd_packed(args, stream) == 0 and dbg.vt_attn_bwd_packed(args, g, stream) == 0
        assert dbg.vt_last_device_status(stream) == 0
        assert all(torch.equal(a, b) for a, b in zip((o, lse, *got), (o2, lse2, *new)))


@gpu
def test_wrappers_refuse():
    p = Problem("bf16", 4, 2, 64, 64, [(20, 20)], seed=13)
    torch = p.torch
    o, lse = p.results()
    bad = [
        (ValueError, dict(q=p.q[0])), (ValueError, dict(k=p.k[:, :-1])), (TypeError, dict(v=p.v.float())),
        (TypeError, dict(cu_q=p.cu_q.long())), (ValueError, dict(cu_k=p.cu_k[:1])), (ValueError, dict(cu_q=p.cu_q[:0])),
        (ValueError, dict(q=p.q.transpose(1, 2))), (ValueError, dict(cu_q=p.cu_q.cpu())), (TypeError, dict(q=p.q.half())),
    ]
    for error, kw in bad:
        a = dict(dict(q=p.q, k=p.k, v=p.v, cu_q=p.cu_q, cu_k=p.cu_k), **kw)
        with pytest.raises(error):
            vt.attn_fwd_packed(**a)
        with pytest.raises(error):
            vt.attn_bwd_packed(p.do, a["q"], a["k"], a["v"], o, lse, a["cu_q"], a["cu_k"])
    with pytest.raises(ValueError):
        vt.attn_fwd_packed(p.q, p.k, p.v, p.cu_q, p.cu_k, mask="diagonal")
    for kw in (dict(mask="window"), dict(mask="window", window=-3)):
        with pytest.raises(vt.VtError):
            vt.attn_fwd_packed(p.q, p.k, p.v, p.cu_q, p.cu_k, **kw)
    with pytest.raises(ValueError):
        vt.attn_fwd_packed(p.q, p.k, p.v, p.cu_q, p.cu_k, lse=lse[:, :-1])
    for kw in (dict(do=p.do[..., :-1]), dict(o=o[:1]), dict(lse=lse.double()), dict(lse=None)):
        a = dict(dict(do=p.do, o=o, lse=lse), **kw)
        with pytest.raises((ValueError, TypeError)):
            vt.attn_bwd_packed(a["do"], p.q, p.k, p.v, a["o"], a["lse"], p.cu_q, p.cu_k)
    with pytest.raises((ValueError, TypeError)):
        vt.attn_bwd_packed(p.do, p.q, p.k, p.v, o, lse, p.cu_q, p.cu_k, dlse=lse.bfloat16())
    with pytest.raises(vt.VtError):  # outputs on inputs
        vt.attn_bwd_packed(p.do, p.q, p.k, p.v, o, lse, p.cu_q, p.cu_k, dq=p.q)
    with pytest.raises(vt.VtError):
        vt.attn_fwd_packed(p.q, p.k, p.v, p.cu_q, p.cu_k, out=p.q)
