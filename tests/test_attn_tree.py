"""vt_attn_fwd_tree: refusals (host only) and results against a plain 64-bit form, with the tolerances of
test_attn_prefix.py; and the operators of a training and of a serving step run together."""

import math

import numpy as np
import pytest

import test_attn_prefix as prefix
from test_attn_packed import Problem as Packed

import scaled_dot_product_vt_gb300 as vt

gpu = pytest.mark.gpu
A = prefix.A


@pytest.fixture(scope="module", autouse=True)
def _built():
    vt.build()
    vt.load()


# ---------------------------------------------------------------- refusals (no GPU)

@pytest.mark.parametrize("kw,parents,code", [
    (dict(), 0, 1), (dict(), 11 * A + 2, 3), (dict(), 7 * A, 1), (dict(), 8 * A, 1), (dict(S_q=65), 11 * A, 2),
    (dict(size=8), 11 * A, 1), (dict(H_kv=3), 11 * A, 1), (dict(q=0), 11 * A, 1),
])
def test_refusals(kw, parents, code):
    assert vt.vt_attn_fwd_tree(prefix.pack(**kw), parents, None) == code


def test_empty_problems():
    for kw in (dict(B=0), dict(S_q=0), dict(H=0)):
        assert vt.vt_attn_fwd_tree(prefix.pack(q=0, o=0, **kw), None, None) == 0
    assert vt.load().vt_attn_fwd_tree(None, 11 * A, None) == 1


def test_valid_calls_reach_the_launch():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: a valid call would launch on these fake addresses")
    assert vt.vt_attn_fwd_tree(prefix.pack(), 11 * A, None) == 4
    assert vt.vt_attn_fwd_tree(prefix.pack(S_c=0, kc=0, vc=0, lens=0), 11 * A, None) == 4


# ---------------------------------------------------------------- results

def random_parents(rng, B, n, kind):
    if kind == "chain":
        return np.tile(np.arange(n) - 1, (B, 1))
    if kind == "roots":
        return np.full((B, n), -1)
    if kind == "star":
        return np.tile(np.minimum(np.arange(n) - 1, 0), (B, 1))
    return np.array([[int(rng.integers(-1, s)) if s else -1 for s in range(n)] for _ in range(B)])


class Tree(prefix.Problem):
    def __init__(self, *a, kind="random", **kw):
        super().__init__(*a, **kw)
        B, S_q = self.dims[0], self.dims[3]
        self.parents = random_parents(self.rng, B, S_q, kind)
        self.par = self.torch.tensor(self.parents, dtype=self.torch.int32, device="cuda")

    def run(self, **kw):
        return vt.attn_fwd_tree(self.q, self.kp, self.vp, self.kc, self.vc, self.par, self.kv_len, scale=self.scale,
                                return_lse=True, **kw)

    def check(self, o, lse):
        """As Problem.check, one node at a time: its keys are put where a query of its own would see them."""
        B, H, H_kv, S_q, S_p, S_c, D_qk, D_v = self.dims
        eps = self.torch.finfo(self.t).eps / 2
        bf = self.t == self.torch.bfloat16
        o, lse = (x.to(self.torch.float64).cpu().numpy() for x in (o, lse))
        for b in range(B):
            n = min(max(int(self.lens[b]), 0), S_c)
            for s in range(S_q):
                keys = list(range(max(0, n - S_q)))
                at, own = s, []
                while at >= 0:
                    own.append(n - S_q + at)
                    up = int(self.parents[b, at])
                    at = up if -1 <= up < at else -1
                keys += sorted(j for j in own if j >= 0)
                for h in range(H):
                    hk = h // (H // H_kv)
                    k = np.concatenate([self.kp64[0, hk], self.kc64[b, hk, keys]])
                    v = np.concatenate([self.vp64[0, hk], self.vc64[b, hk, keys]])
                    where = f"b={b} node={s} h={h} ({len(k)} keys)"
                    if len(k) == 0:
                        assert not o[b, h, s].any() and lse[b, h, s] == -np.inf, where
                        continue
                    x = self.scale * (k @ self.q64[b, h, s])
                    size = (abs(self.scale) * (np.abs(k) @ np.abs(self.q64[b, h, s]))).max()
                    d = size * (2.0 ** -17 + (0.0 if bf else 2.0 ** -19))
                    w = np.exp(x - x.max())
                    want_lse = x.max() + np.log(w.sum())
                    w /= w.sum()
                    want, mass = w @ v, w @ np.abs(v)
                    tol = (2 * d + 2.0 ** -18) * mass + eps * np.abs(want) + (2 * eps * mass if bf else 0.0)
                    err = np.abs(o[b, h, s] - want)
                    assert (err <= tol).all(), f"{where}: O off by {err.max():.3e}, allowed {tol[err.argmax()]:.3e}"
                    assert abs(lse[b, h, s] - want_lse) <= d + 2.0 ** -19 * (1 + abs(want_lse)), where


CASES = [
    # dtype, B, H, H_kv, nodes, S_p, S_c, D_qk, D_v
    ("bf16", 1, 1, 1, 1, 1, 1, 8, 8),
    ("bf16", 4, 8, 2, 8, 333, 100, 128, 128),      # streamed with the prefix
    ("bf16", 40, 4, 2, 5, 1000, 37, 128, 128),     # the prefix in a launch of its own
    ("bf16", 9, 6, 2, 13, 515, 64, 96, 40),        # groups of 3
    ("bf16", 3, 6, 2, 40, 300, 120, 72, 128),      # tiles of a sequence's rows
    ("bf16", 2, 8, 1, 64, 129, 300, 128, 128),     # four blocks of rows
    ("bf16", 5, 4, 4, 33, 0, 700, 64, 64),
    ("bf16", 3, 8, 2, 64, 0, 200, 64, 128),
    ("bf16", 1, 4, 1, 3, 0, 9000, 128, 64),        # one sequence: its keys in shares
    ("bf16", 2, 8, 1, 25, 0, 5000, 128, 128),      # few sequences of many rows and keys
    ("bf16", 30, 16, 4, 25, 2000, 300, 128, 64),   # many of them behind a prefix
    ("bf16", 3, 4, 2, 7, 200, 0, 64, 64),          # no cache: the prefix alone
    ("f32", 2, 2, 1, 3, 50, 30, 4, 4),
    ("f32", 5, 8, 2, 13, 400, 90, 72, 72),
    ("f32", 2, 4, 4, 64, 0, 200, 128, 128),
    ("f32", 2, 2, 1, 5, 0, 3000, 33, 20),
]


@gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_against_the_definition(case):
    t = Tree(*case, seed=1)
    t.check(*t.run())
    assert vt.vt_last_device_status() == 0


@gpu
@pytest.mark.parametrize("kind", ["chain", "roots", "star"])
@pytest.mark.parametrize("dtype,nodes", [("bf16", 3), ("bf16", 33), ("bf16", 64), ("f32", 9)])
def test_shapes_of_trees(dtype, nodes, kind):
    t = Tree(dtype, 3, 4, 2, nodes, 70, 150, 64, 64, kind=kind, seed=2)
    o, lse = t.run()
    t.check(o, lse)
    if kind == "chain":  # the call of the tokens in a row
        prefix.Problem.check(t, o, lse)


@gpu
@pytest.mark.parametrize("dtype,nodes,D_v", [("bf16", 5, 64), ("bf16", 40, 64), ("bf16", 40, 128), ("f32", 5, 64)])
@pytest.mark.parametrize("S_p", [0, 600])
def test_lengths_at_their_ends(dtype, nodes, D_v, S_p):
    # empty, shorter than the tree, the tree alone, trees that cross blocks of 16 and 128 keys
    lens = [0, 1, nodes - 1, nodes, nodes + 1, 16, 17, 31, 64, 127, 128, 129, 130, 150, 165, 200]
    t = Tree(dtype, len(lens), 4, 2, nodes, S_p, 200, 64, D_v, lens=lens, seed=3)
    t.check(*t.run())
    assert vt.vt_last_device_status() == 0


@gpu
@pytest.mark.parametrize("nodes", [4, 40])
def test_parents_that_are_no_earlier_node_are_reported(nodes):
    t = Tree("bf16", 3, 4, 2, nodes, 50, 90, 64, 64, lens=[90, 70, 50], seed=4)
    t.par[0, 1], t.par[1, 2], t.par[2, 3] = 1, -7, 1 << 30
    t.parents[0, 1], t.parents[1, 2], t.parents[2, 3] = -1, -1, -1
    t.check(*t.run())
    assert vt.vt_last_device_status() == 6
    assert vt.vt_last_device_status() == 0


NO_CACHE = [
    # dtype, B, H, H_kv, nodes, S_p, S_c, D_qk, D_v
    ("bf16", 1, 32, 8, 64, 1024, 0, 128, 128),     # 256 rows a key/value head, the prefix in shares
    ("bf16", 1, 8, 2, 40, 640, 0, 128, 128),
    ("bf16", 3, 6, 2, 40, 2000, 0, 72, 40),
    ("bf16", 40, 8, 2, 33, 300, 0, 64, 64),        # many sequences, one launch
    ("bf16", 2, 8, 1, 9, 1, 0, 64, 128),
    ("bf16", 20, 8, 2, 4, 3000, 0, 128, 64),       # streamed rows, the prefix on its own
    ("bf16", 1, 4, 1, 3, 4000, 0, 64, 64),         # streamed with the prefix, in shares
    ("f32", 2, 8, 2, 33, 700, 0, 64, 64),
    ("f32", 1, 2, 1, 5, 60, 0, 33, 20),
]


def test_a_tree_without_a_cache_has_its_own_plan():
    """Shares of the prefix (and so partial results) where a sequence's rows fill tiles: the kernel that reads the parents."""
    size = vt.vt_attn_tree_workspace_size
    assert size(1, 32, 8, 64, 1024, 0, 128, 128, vt.VT_BF16) > 0 == vt.vt_attn_prefix_workspace_size(
        1, 32, 8, 64, 1024, 0, 128, 128, vt.VT_BF16)


@gpu
@pytest.mark.parametrize("case", NO_CACHE, ids=lambda c: "-".join(map(str, c)))
def test_without_a_cache_the_nodes_see_the_prefix_alone(case):
    """And parents that are no earlier node are reported all the same."""
    t = Tree(*case, seed=9)
    B, nodes = t.dims[0], t.dims[3]
    for kv_len in (t.kv_len, None):  # (not read)
        t.kv_len = kv_len
        t.check(*t.run())
        assert vt.vt_last_device_status() == 0
    t.par[B - 1, nodes - 1] = nodes
    t.check(*t.run())
    assert vt.vt_last_device_status() == 6 and vt.vt_last_device_status() == 0


@gpu
@pytest.mark.parametrize("dtype,S_q", [("bf16", 1), ("bf16", 3), ("bf16", 20), ("f32", 3)])
def test_no_key_at_all(dtype, S_q):
    """O = 0 and a log-sum-exp of -inf, for tokens in a row and for trees."""
    t = Tree(dtype, 3, 8, 2, S_q, 0, 0, 64, 40, seed=10)
    for run in (t.run, lambda **kw: prefix.Problem.run(t, **kw)):
        out = t.torch.full((3, 8, S_q, 40), 7.0, dtype=t.t, device="cuda")
        o, lse = run(out=out)
        assert (o == 0).all() and (lse == -math.inf).all()
    assert vt.vt_last_device_status() == 0


@gpu
@pytest.mark.parametrize("B,nodes", [(70, 4), (20, 30)])
def test_writes_nothing_else_and_gives_the_same_bits(B, nodes):
    t = Tree("bf16", B, 8, 2, nodes, 1500, 200, 128, 72, seed=5)
    torch = t.torch
    first = t.run()
    room = torch.full((B, nodes + 1, 8, 96), 7.0, dtype=t.t, device="cuda")
    out = room[:, :nodes].transpose(1, 2)[..., 8:80]
    need = vt.vt_attn_tree_workspace_size(B, 8, 2, nodes, 1500, 200, 128, 72, vt.VT_BF16)
    ws = torch.full((need + 512,), 7, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = t.run(out=out, workspace=ws[:need] if need else None, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again)) and (ws[need:] == 7).all()
    out.fill_(7.0)
    assert (room == 7.0).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = t.run()
    fresh = Tree("bf16", B, 8, 2, nodes, 1500, 200, 128, 72, seed=6, beyond=0.5)
    for name in ("q", "kp", "vp", "kc", "vc", "kv_len", "par"):
        getattr(t, name).copy_(getattr(fresh, name))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, fresh.run()))


@gpu
def test_wrapper_refuses():
    t = Tree("bf16", 2, 4, 2, 5, 20, 30, 64, 64, seed=7)
    args = lambda par: (t.q, t.kp, t.vp, t.kc, t.vc, par, t.kv_len)
    for par in (None, t.par[:1], t.par.long(), t.par.cpu(), t.par.T.contiguous().T, t.par[:, :4]):
        with pytest.raises(ValueError):
            vt.attn_fwd_tree(*args(par))
    big = Tree("bf16", 1, 1, 1, 64, 0, 80, 64, 64, seed=8)
    q = big.q.repeat(1, 1, 2, 1)
    with pytest.raises(vt.VtError):
        vt.attn_fwd_tree(q, None, None, big.kc, big.vc, big.par.repeat(1, 2).contiguous(), big.kv_len)


# ---------------------------------------------------------------- steps

def turned(torch, x, pos, freqs, eps):
    """Norm and rotation of rows x [..., T, D] in 64 bits."""
    n = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    a = pos.double()[:, None] * freqs.double()
    lo, hi = n.chunk(2, -1)
    return torch.cat([lo * a.cos() - hi * a.sin(), lo * a.sin() + hi * a.cos()], -1)


@gpu
def test_a_training_step_of_packed_texts():
    """Norm and rotation, attention, its gradients, those of the norm, all on packed texts: fp32, against autograd in 64 bits.
    Five operators of relative errors below 2^-17 (the sums of a gradient row among them): 1e-4 of the largest gradient."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lengths, H, H_kv, D = [70, 1, 130, 33], 4, 2, 64
    T = sum(lengths)
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v, do = (torch.randn((T, h, D), generator=g, device="cuda").transpose(0, 1) for h in (H, H_kv, H_kv, H))
    pos = torch.cat([torch.arange(n, device="cuda") for n in lengths]).int()
    freqs = 10000.0 ** (-torch.arange(D // 2, device="cuda") / (D // 2))
    cu = torch.tensor(np.cumsum([0] + lengths), dtype=torch.int32, device="cuda")
    form = dict(freqs=freqs, positions=pos[None], eps=1e-6)
    qr, kr = vt.qk_rope(q[None], k[None], **form)
    o, lse = vt.attn_fwd_packed(qr[0], kr[0], v, cu, return_lse=True)
    dqr, dkr, dv = vt.attn_bwd_packed(do, qr[0], kr[0], v, o, lse, cu)
    dq, dk, _, _ = vt.qk_rope_bwd(dqr[None], dkr[None], q=q[None], k=k[None], **form)
    leaves = [x.double().requires_grad_() for x in (q, k, v)]
    a, b = (turned(torch, x, pos, freqs, 1e-6) for x in leaves[:2])
    outs = []
    for i in range(len(lengths)):
        s = slice(cu[i], cu[i + 1])
        x = torch.einsum("hqd,hkd->hqk", a[:, s], b[:, s].repeat_interleave(2, 0)) * D ** -0.5
        x = x.masked_fill(torch.ones(x.shape[1:], dtype=torch.bool, device="cuda").triu(1), -math.inf)
        outs.append(torch.softmax(x, -1) @ leaves[2][:, s].repeat_interleave(2, 0))
    want_o = torch.cat(outs, 1)
    want = torch.autograd.grad(want_o, leaves, do.double())
    assert (o - want_o).abs().max() <= 1e-4
    for got, w in zip((dq[0], dk[0], dv), want):
        assert (got - w).abs().max() <= 1e-4 * w.abs().max()
    assert vt.vt_last_device_status() == 0


@gpu
@pytest.mark.parametrize("dtype,tol", [("bf16", 3e-2), ("f32", 1e-4)])
def test_a_serving_step_of_drafted_trees(dtype, tol):
    """Prompts attended packed and laid into caches, then a tree of drafted tokens for each: appended, and attended.  bf16:
    O of unit values is off by its rounding, P's and those of the rotated keys (2^-9 of scores up to about 4): 3e-2."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    t = dict(bf16=torch.bfloat16, f32=torch.float32)[dtype]
    lengths, nodes, H, H_kv, D, cap = [5, 90, 40], 6, 4, 2, 64, 128
    B, T = len(lengths), sum(lengths)
    g = torch.Generator(device="cuda").manual_seed(2)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(t)
    freqs = 10000.0 ** (-torch.arange(D // 2, device="cuda") / (D // 2))
    cu = torch.tensor(np.cumsum([0] + lengths), dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(n, device="cuda") for n in lengths]).int()
    q, k, v = (rand(T, h, D).transpose(0, 1) for h in (H, H_kv, H_kv))
    qr, kr = vt.qk_rope(q[None], k[None], freqs, pos[None], eps=1e-6)
    o = vt.attn_fwd_packed(qr[0], kr[0], v, cu)
    k_cache, v_cache = torch.full((2, B, H_kv, cap, D), float("nan"), dtype=t, device="cuda")
    for b, n in enumerate(lengths):
        k_cache[b, :, :n], v_cache[b, :, :n] = kr[0][:, cu[b]:cu[b + 1]], v[:, cu[b]:cu[b + 1]]
    parents = torch.tensor([[-1, 0, 0, 1, 1, 2], [-1, 0, 1, 2, 3, 4], [-1, -1, 0, 1, 2, 0]], dtype=torch.int32, device="cuda")
    depth = torch.tensor([[0, 1, 1, 2, 2, 2], [0, 1, 2, 3, 4, 5], [0, 0, 1, 1, 2, 1]], device="cuda")
    nq, nk, nv = (rand(B, nodes, h, D).transpose(1, 2) for h in (H, H_kv, H_kv))
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda") + nodes
    npos = (torch.tensor(lengths, device="cuda")[:, None] + depth).int()
    nqr, _ = vt.qk_rope(nq, nk, freqs, npos, eps=1e-6, k_out=k_cache, kv_len=lens, v=nv, v_out=v_cache)
    tree = vt.attn_fwd_tree(nqr, None, None, k_cache, v_cache, parents, lens)
    assert vt.vt_last_device_status() == 0
    for b, n in enumerate(lengths):
        s = slice(cu[b], cu[b + 1])
        a, c = (turned(torch, x[:, s].double(), pos[s], freqs, 1e-6) for x in (q, k))
        na, nc = (turned(torch, x[b].double(), npos[b], freqs, 1e-6) for x in (nq, nk))
        for h in range(H):
            x = (a[h] @ c[h // 2].T * D ** -0.5).masked_fill(torch.ones((n, n), dtype=torch.bool, device="cuda").triu(1), -math.inf)
            assert (o[h, s] - torch.softmax(x, -1) @ v[h // 2, s].double()).abs().max() <= tol
            for node in range(nodes):
                path, at = [], node
                while at >= 0:
                    path.append(at)
                    at = int(parents[b, at])
                keys, vals = (torch.cat([y, z[path]]) for y, z in ((c[h // 2], nc[h // 2]),
                                                                   (v[h // 2, s].double(), nv[b, h // 2].double())))
                want = torch.softmax(keys @ na[h, node] * D ** -0.5, -1) @ vals
                assert (tree[b, h, node] - want).abs().max() <= tol
