"""Workloads of the token-preparation and shared-prefix operators: what a pass takes, its plain form in
elementary torch operations, and its value from the definition in 64 bits.

``rope``      per-head norm of the queries and keys and their rotation by one or more position axes,
              optionally appending the keys and values to a cache
``rope_bwd``  its gradients
``attn``      attention of a batch of sequences over a prefix that all share and over each one's own cache
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one new token for each of 16 sequences: normalised, rotated, appended to the cache (latency)
        dict(name="rope_step_bf16", op="rope", dtype="bf16", B=16, H=16, H_kv=4, S=1, D=128, R=128, axes=1, norm=True,
             interleaved=False, cap=256),
        # the prompts of four sequences, grouped heads
        dict(name="rope_prefill_bf16", op="rope", dtype="bf16", B=4, H=32, H_kv=8, S=2048, D=128, R=128, axes=1,
             norm=True, interleaved=False, cap=0),
        # patches of a video on a (time, height, width) grid, head width 72, rotation alone
        dict(name="rope_video_f32", op="rope", dtype="f32", B=2, H=16, H_kv=16, S=1000, D=72, R=72, axes=3, norm=False,
             interleaved=True, cap=0),
        # training on the prompts above
        dict(name="rope_bwd_bf16", op="rope_bwd", dtype="bf16", B=4, H=32, H_kv=8, S=2048, D=128, R=128, axes=1,
             norm=True, interleaved=False, cap=0),
        # training on images and text, two thirds of each head rotated, an odd length
        dict(name="rope_bwd_video_f32", op="rope_bwd", dtype="f32", B=1, H=8, H_kv=8, S=333, D=96, R=64, axes=3,
             norm=True, interleaved=True, cap=0),
        # four sequences just begun after a short prompt (latency)
        dict(name="attn_few_bf16", op="attn", dtype="bf16", B=4, H=16, H_kv=4, S_q=1, D_qk=128, D_v=128, S_p=333,
             cap=256, lo=1, hi=37),
        # serving: 64 sequences behind one long system prompt
        dict(name="attn_batch_bf16", op="attn", dtype="bf16", B=64, H=32, H_kv=8, S_q=1, D_qk=128, D_v=128, S_p=8192,
             cap=1024, lo=1, hi=1024),
        # long sequences of their own behind a shorter prompt: bound by the cache's bytes
        dict(name="attn_long_cache_bf16", op="attn", dtype="bf16", B=16, H=32, H_kv=8, S_q=1, D_qk=128, D_v=128,
             S_p=2048, cap=8192, lo=1, hi=8192),
        # no grouped heads, D_qk 96 and D_v 64, odd lengths
        dict(name="attn_ragged_bf16", op="attn", dtype="bf16", B=37, H=32, H_kv=32, S_q=1, D_qk=96, D_v=64, S_p=8191,
             cap=333, lo=0, hi=333),
        # four drafted tokens to be checked for each of 32 sequences, behind a long document
        dict(name="attn_draft_bf16", op="attn", dtype="bf16", B=32, H=16, H_kv=4, S_q=4, D_qk=128, D_v=128, S_p=32768,
             cap=512, lo=4, hi=512),
        # chunks of 256 prompt tokens behind the system prompt
        dict(name="attn_chunk_bf16", op="attn", dtype="bf16", B=8, H=32, H_kv=8, S_q=256, D_qk=128, D_v=128, S_p=8192,
             cap=1024, lo=256, hi=1024),
        # single precision, width 72
        dict(name="attn_f32", op="attn", dtype="f32", B=8, H=8, H_kv=2, S_q=1, D_qk=72, D_v=72, S_p=1000, cap=333,
             lo=1, hi=333),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = max(listed(), key=lambda c: work(c)["flops"])
    widest = max(listed(), key=lambda c: work(c)["bytes"])
    while True:
        op = rng.choice(["rope", "rope_bwd", "attn", "attn"])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        H_kv = rng.choice([1, 2, 4, 8])
        H = H_kv * rng.choice([1, 2, 3, 4, 8])
        D = rng.choice([64, 72, 96, 128])
        if op == "attn":
            cap = _between(rng, 1, 8192)
            S_q = min(rng.choice([1, 1, 1, 2, 3, 4, _between(rng, 5, 256)]), cap)
            c = dict(op=op, dtype=dtype, B=_between(rng, 1, 128), H=H, H_kv=H_kv, S_q=S_q, D_qk=D,
                     D_v=rng.choice([D, 64, 128]), S_p=_between(rng, 1, 32768), cap=cap, lo=S_q, hi=cap)
            if dtype == "f32" and work(c)["flops"] > 2e10:  # single precision: checks and small models
                continue
        else:
            append = op == "rope" and rng.random() < 0.4
            S = rng.choice([1, 1, 2, 4]) if append else _between(rng, 1, 4096)
            c = dict(op=op, dtype=dtype, B=_between(rng, 1, 64) if append else rng.choice([1, 2, 3, 4]), H=H, H_kv=H_kv,
                     S=S, D=D, R=rng.choice([D, D, D // 2, 64]), axes=rng.choice([1, 2, 3]), norm=rng.random() < 0.7,
                     interleaved=rng.random() < 0.4, cap=rng.choice([64, 100, 256]) if append else 0)
        w = work(c)
        if w["flops"] <= work(most)["flops"] and w["bytes"] <= work(widest)["bytes"]:
            return c


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "attn":
        keys = (c["lo"] + c["hi"]) / 2
        rows = c["B"] * c["H"] * c["S_q"]
        kv = c["H_kv"] * (c["S_p"] + c["B"] * keys) * (c["D_qk"] + c["D_v"])
        return {"bytes": e * (kv + rows * (c["D_qk"] + c["D_v"])) + 4 * rows,
                "flops": 2.0 * rows * (c["S_p"] + keys) * (c["D_qk"] + c["D_v"])}
    tokens = c["B"] * c["S"]
    x = tokens * (c["H"] + c["H_kv"]) * c["D"]
    if c["op"] == "rope":
        moved = 2 * x + (2 * tokens * c["H_kv"] * c["D"] if c["cap"] else 0)
        return {"bytes": e * moved + 4 * c["axes"] * tokens, "flops": 7.0 * x}
    return {"bytes": e * (3 if c["norm"] else 2) * x + 4 * c["axes"] * tokens, "flops": 13.0 * x}


# ---------------------------------------------------------------- inputs

def _normal(g, shape, dtype, mean=0.0, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std + mean).to(dtype)


def _prepare_rope(c, g):
    B, H, H_kv, S, D, R = (c[k] for k in ("B", "H", "H_kv", "S", "D", "R"))
    dt = DTYPES[c["dtype"]]
    st = dict(case=c)
    # projections as they leave a matrix product: tokens first, heads beside each other
    st["q"] = _normal(g, (B, S, H, D), dt).transpose(1, 2)
    st["k"] = _normal(g, (B, S, H_kv, D), dt).transpose(1, 2)
    half = R // 2
    st["freqs"] = (10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).to(torch.float32)
    if c["axes"] == 1:
        first = torch.randint(0, 100000, (B, 1), generator=g, device="cuda")
        pos = first + torch.arange(S, device="cuda")[None]
        st["pair_axis"] = None
        st["positions"] = pos[None].to(torch.int32).contiguous()
    else:
        # a grid of patches in raster order, behind a text of another length for each seed
        side = max(1, int(math.isqrt(S) // 2))
        t = torch.arange(S, device="cuda")
        grid = [t // (side * side), (t // side) % side, t % side][:c["axes"]]
        first = torch.randint(0, 5000, (B, 1), generator=g, device="cuda")
        st["positions"] = torch.stack([first + a[None] for a in grid]).to(torch.int32).contiguous()
        cut = [half * i // c["axes"] for i in range(c["axes"] + 1)]
        st["pair_axis"] = tuple(a for a in range(c["axes"]) for _ in range(cut[a], cut[a + 1]))
    st["axis"] = torch.tensor(st["pair_axis"] or (0,) * half, device="cuda", dtype=torch.int64)
    st["eps"] = EPS if c["norm"] else None
    st["q_weight"] = _normal(g, (D,), dt, 1.0, 0.1) if c["norm"] else None
    st["k_weight"] = _normal(g, (D,), dt, 1.0, 0.1) if c["norm"] else None
    if c["op"] == "rope_bwd":
        st["dq_out"] = _normal(g, (B, H, S, D), dt)
        st["dk_out"] = _normal(g, (B, H_kv, S, D), dt)
    if c["cap"]:
        cap = c["cap"]
        st["v"] = _normal(g, (B, S, H_kv, D), dt).transpose(1, 2)
        st["k_cache"] = _normal(g, (B, H_kv, cap, D), dt)
        st["v_cache"] = _normal(g, (B, H_kv, cap, D), dt)
        st["kv_len"] = torch.randint(S, cap + 1, (B,), generator=g, device="cuda").to(torch.int32)
    return st


def _prepare_attn(c, g):
    B, H, H_kv, S_q, S_p, cap = (c[k] for k in ("B", "H", "H_kv", "S_q", "S_p", "cap"))
    dt = DTYPES[c["dtype"]]
    return dict(case=c,
                q=_normal(g, (B, H, S_q, c["D_qk"]), dt),
                k_prefix=_normal(g, (H_kv, S_p, c["D_qk"]), dt),
                v_prefix=_normal(g, (H_kv, S_p, c["D_v"]), dt),
                # rows from a sequence's length on hold what earlier sequences left there
                k_cache=_normal(g, (B, H_kv, cap, c["D_qk"]), dt),
                v_cache=_normal(g, (B, H_kv, cap, c["D_v"]), dt),
                kv_len=torch.randint(c["lo"], c["hi"] + 1, (B,), generator=g, device="cuda").to(torch.int32),
                scale=float(c["D_qk"]) ** -0.5)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return _prepare_attn(case, g) if case["op"] == "attn" else _prepare_rope(case, g)


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"rope": _plain_rope, "rope_bwd": _plain_rope_bwd, "attn": _plain_attn}[op](state)


def _own(st, op):
    import scaled_dot_product_vt_gb300 as vt
    if op == "attn":
        return vt.attn_fwd_prefix(st["q"], st["k_prefix"], st["v_prefix"], st["k_cache"], st["v_cache"], st["kv_len"],
                                  scale=st["scale"], return_lse=True)
    form = dict(pair_axis=st["pair_axis"], interleaved=st["case"]["interleaved"], eps=st["eps"],
                q_weight=st["q_weight"], k_weight=st["k_weight"])
    if op == "rope":
        if "k_cache" in st:
            q, k = vt.qk_rope(st["q"], st["k"], st["freqs"], st["positions"], v=st["v"], k_out=st["k_cache"],
                              v_out=st["v_cache"], kv_len=st["kv_len"], **form)
            return q, k, st["v_cache"]
        return vt.qk_rope(st["q"], st["k"], st["freqs"], st["positions"], **form)
    dq, dk, dqw, dkw = vt.qk_rope_bwd(st["dq_out"], st["dk_out"], st["freqs"], st["positions"], q=st["q"], k=st["k"],
                                      **form)
    return (dq, dk, dqw, dkw) if st["case"]["norm"] else (dq, dk)


def _angles(st):
    """cos and sin [B, 1, S, R/2] in 32 bits of angles formed in 64: far positions keep their phase."""
    a = st["positions"].index_select(0, st["axis"]).to(torch.float64) * st["freqs"].to(torch.float64)[:, None, None]
    a = a.permute(1, 2, 0).unsqueeze(1)
    return torch.cos(a).to(torch.float32), torch.sin(a).to(torch.float32)


def _turn(x, cos, sin, interleaved):
    half = cos.shape[-1]
    y = x.clone()
    if interleaved:
        lo, hi = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2] = lo * cos - hi * sin
        y[..., 1:2 * half:2] = lo * sin + hi * cos
    else:
        lo, hi = x[..., :half], x[..., half:2 * half]
        y[..., :half] = lo * cos - hi * sin
        y[..., half:2 * half] = lo * sin + hi * cos
    return y


def _plain_rope(st):
    cos, sin = _angles(st)
    out = []
    for x, w in ((st["q"], st["q_weight"]), (st["k"], st["k_weight"])):
        y = x.to(torch.float32)
        if st["eps"] is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + st["eps"]) * w.to(torch.float32)
        out.append(_turn(y, cos, sin, st["case"]["interleaved"]).to(x.dtype))
    if "k_cache" not in st:
        return tuple(out)
    S = st["case"]["S"]
    rows = st["kv_len"].to(torch.int64)[:, None] - S + torch.arange(S, device="cuda")
    at = torch.arange(rows.shape[0], device="cuda")[:, None]
    st["k_cache"].transpose(1, 2)[at, rows] = out[1].transpose(1, 2)
    st["v_cache"].transpose(1, 2)[at, rows] = st["v"].transpose(1, 2)
    return out[0], st["k_cache"], st["v_cache"]


def _plain_rope_bwd(st):
    cos, sin = _angles(st)
    grads, weights = [], []
    for x, g, w in ((st["q"], st["dq_out"], st["q_weight"]), (st["k"], st["dk_out"], st["k_weight"])):
        u = _turn(g.to(torch.float32), cos, -sin, st["case"]["interleaved"])
        if st["eps"] is not None:
            f = x.to(torch.float32)
            r = torch.rsqrt((f * f).mean(-1, keepdim=True) + st["eps"])
            n = f * r
            weights.append((u * n).sum((0, 1, 2), dtype=torch.float64).to(torch.float32))
            u = u * w.to(torch.float32)
            u = r * (u - n * (u * n).mean(-1, keepdim=True))
        grads.append(u.to(x.dtype))
    return tuple(grads + weights)


def _plain_attn(st):
    c = st["case"]
    B, H, H_kv, S_q, S_p, cap = (c[k] for k in ("B", "H", "H_kv", "S_q", "S_p", "cap"))
    G = H // H_kv
    f = torch.float32
    q = st["q"].to(f).reshape(B, H_kv, G * S_q, c["D_qk"]) * st["scale"]
    qp = q.transpose(0, 1).reshape(H_kv, B * G * S_q, c["D_qk"])
    sp = (qp @ st["k_prefix"].to(f).transpose(1, 2)).reshape(H_kv, B, G * S_q, S_p).transpose(0, 1)
    sc = (q @ st["k_cache"].to(f).transpose(2, 3)).reshape(B, H_kv, G, S_q, cap)
    last = st["kv_len"].to(torch.int64)[:, None] - S_q + torch.arange(S_q, device="cuda")
    seen = torch.arange(cap, device="cuda") <= last[..., None]  # [B, S_q, cap]
    sc = torch.where(seen[:, None, None], sc, torch.full((), -math.inf, device="cuda")).reshape(B, H_kv, G * S_q, cap)
    top = torch.maximum(sp.amax(-1), sc.amax(-1))[..., None]
    sp, sc = torch.exp(sp - top), torch.exp(sc - top)
    total = sp.sum(-1, keepdim=True) + sc.sum(-1, keepdim=True)
    o = (sp.transpose(0, 1).reshape(H_kv, B * G * S_q, S_p) @ st["v_prefix"].to(f))
    o = o.reshape(H_kv, B, G * S_q, c["D_v"]).transpose(0, 1) + sc @ st["v_cache"].to(f)
    o = (o / total).reshape(B, H, S_q, c["D_v"]).to(st["q"].dtype)
    return o, (top + torch.log(total)).reshape(B, H, S_q)


# ---------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return _exact_attn(st) if case["op"] == "attn" else _exact_rope(st)


def _phases(st):
    p = st["positions"].to(torch.float64)
    f = st["freqs"].to(torch.float64)
    a = torch.stack([p[int(ax)] * f[i] for i, ax in enumerate(st["axis"].tolist())], -1)
    return torch.polar(torch.ones_like(a), a)[:, None]  # [B, 1, S, R/2], complex


def _rotated(x, phase, interleaved):
    half = phase.shape[-1]
    body, rest = x[..., :2 * half], x[..., 2 * half:]
    pairs = body.unflatten(-1, (half, 2)) if interleaved else body.unflatten(-1, (2, half)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * phase)
    z = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, rest], -1)


def _exact_rope(st):
    c = st["case"]
    d = torch.float64
    phase = _phases(st)
    D = c["D"]
    if c["op"] == "rope":
        res = []
        for x, w in (("q", "q_weight"), ("k", "k_weight")):
            y = st[x].to(d)
            if st["eps"] is not None:
                y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / D + st["eps"]) * st[w].to(d)
            res.append(_rotated(y, phase, c["interleaved"]))
        if not c["cap"]:
            return tuple(res)
        kc, vc = st["k_cache"].to(d), st["v_cache"].to(d)
        for b, n in enumerate(st["kv_len"].tolist()):
            kc[b, :, n - c["S"]:n] = res[1][b]
            vc[b, :, n - c["S"]:n] = st["v"][b].to(d)
        return res[0], kc, vc
    grads, weights = [], []
    for x, g, w in (("q", "dq_out", "q_weight"), ("k", "dk_out", "k_weight")):
        u = _rotated(st[g].to(d), phase.conj(), c["interleaved"])
        if st["eps"] is not None:
            y = st[x].to(d)
            s = torch.sqrt(y.square().sum(-1, keepdim=True) / D + st["eps"])
            weights.append((u * y / s).flatten(0, 2).sum(0))
            wu = u * st[w].to(d)
            u = wu / s - y * (wu * y).sum(-1, keepdim=True) / (D * s ** 3)
        grads.append(u)
    return tuple(grads + weights)


def _exact_attn(st):
    c = st["case"]
    d = torch.float64
    if work(c)["flops"] > 1.5e12:
        return None
    G = c["H"] // c["H_kv"]
    o = torch.empty((c["B"], c["H"], c["S_q"], c["D_v"]), dtype=d, device="cuda")
    lse = torch.empty((c["B"], c["H"], c["S_q"]), dtype=d, device="cuda")
    kp, vp = st["k_prefix"].to(d), st["v_prefix"].to(d)
    for b, n in enumerate(st["kv_len"].tolist()):
        key = torch.cat([kp, st["k_cache"][b, :, :n].to(d)], 1)
        val = torch.cat([vp, st["v_cache"][b, :, :n].to(d)], 1)
        own_at = torch.arange(key.shape[1], device="cuda") - c["S_p"]
        hidden = own_at[None] > (n - c["S_q"] + torch.arange(c["S_q"], device="cuda"))[:, None]
        for h in range(c["H"]):
            s = (st["q"][b, h].to(d) @ key[h // G].T * st["scale"]).masked_fill(hidden, -math.inf)
            lse[b, h] = torch.logsumexp(s, -1)
            o[b, h] = torch.exp(s - lse[b, h][:, None]) @ val[h // G]
    return o, lse
