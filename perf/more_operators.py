"""Workloads of the attention over packed sequences, of its gradients and of the attention for trees of drafted tokens:
what a pass takes, its plain form in elementary torch operations, and its value from the definition in 64 bits.

``packed``      attention of sequences of different lengths that lie behind each other in one tensor
``packed_bwd``  its gradients
``tree``        attention of each sequence's tree of drafted tokens over a shared prefix and its own cache
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a few short prompts that arrived together (latency)
        dict(name="packed_few_bf16", op="packed", dtype="bf16", N=4, H=16, H_kv=4, D_qk=128, D_v=128, lo=9, hi=100,
             past=0, mask="causal", window=0, empty=False),
        # the prompts of a batch, from a question to a long document, one of the places empty
        dict(name="packed_prompts_bf16", op="packed", dtype="bf16", N=16, H=32, H_kv=8, D_qk=128, D_v=128, lo=128,
             hi=8192, past=0, mask="causal", window=0, empty=True),
        # chunks of prompts behind what was read before, a sliding window, D_qk 96 and D_v 64
        dict(name="packed_chunks_bf16", op="packed", dtype="bf16", N=11, H=32, H_kv=32, D_qk=96, D_v=64, lo=65, hi=512,
             past=4096, mask="window", window=1024, empty=False),
        # single precision, width 72, queries over all the keys of their sequence (patches of images)
        dict(name="packed_f32", op="packed", dtype="f32", N=5, H=8, H_kv=2, D_qk=72, D_v=72, lo=100, hi=1000, past=0,
             mask="none", window=0, empty=False),
        # a small step of training on short texts (latency)
        dict(name="packed_bwd_few_bf16", op="packed_bwd", dtype="bf16", N=6, H=16, H_kv=4, D_qk=128, D_v=128, lo=20,
             hi=333, past=0, mask="causal", window=0, empty=False),
        # a step of training on texts packed to a fixed number of tokens
        dict(name="packed_bwd_texts_bf16", op="packed_bwd", dtype="bf16", N=16, H=32, H_kv=8, D_qk=128, D_v=128, lo=128,
             hi=4096, past=0, mask="causal", window=0, empty=True),
        # images of different sizes, every patch sees every other, no grouped heads, width 64
        dict(name="packed_bwd_images_bf16", op="packed_bwd", dtype="bf16", N=9, H=16, H_kv=16, D_qk=64, D_v=64, lo=256,
             hi=2048, past=0, mask="none", window=0, empty=False),
        # single precision, an odd width, a window
        dict(name="packed_bwd_f32", op="packed_bwd", dtype="f32", N=3, H=8, H_kv=2, D_qk=72, D_v=72, lo=77, hi=500,
             past=0, mask="window", window=128, empty=False),
        # eight drafted tokens for each of four sequences just begun (latency)
        dict(name="tree_few_bf16", op="tree", dtype="bf16", B=4, H=16, H_kv=4, nodes=8, D_qk=128, D_v=128, S_p=333,
             cap=256, lo=9, hi=100),
        # trees of 25 drafted tokens for 32 sequences behind a system prompt
        dict(name="tree_batch_bf16", op="tree", dtype="bf16", B=32, H=32, H_kv=8, nodes=25, D_qk=128, D_v=128, S_p=8192,
             cap=1024, lo=25, hi=1024),
        # full trees of 64 for sequences of different lengths, without a prefix
        dict(name="tree_long_bf16", op="tree", dtype="bf16", B=16, H=32, H_kv=8, nodes=64, D_qk=128, D_v=128, S_p=0,
             cap=8192, lo=64, hi=8192),
        # single precision, width 72, an odd tree
        dict(name="tree_f32", op="tree", dtype="f32", B=8, H=8, H_kv=2, nodes=13, D_qk=72, D_v=72, S_p=1000, cap=333,
             lo=13, hi=333),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {}
    for c in listed():
        most.setdefault((c["op"], c["dtype"]), []).append(work(c))
    while True:
        op = rng.choice(["packed", "packed_bwd", "tree"])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        H_kv = rng.choice([1, 2, 4, 8])
        D = rng.choice([64, 72, 96, 128])
        c = dict(op=op, dtype=dtype, H=H_kv * rng.choice([1, 2, 3, 4, 8]), H_kv=H_kv, D_qk=D, D_v=rng.choice([D, 64, 128]))
        if op == "tree":
            nodes = _between(rng, 1, 64)
            cap = _between(rng, nodes, 8192)
            c.update(B=_between(rng, 1, 64), nodes=nodes, S_p=rng.choice([0, _between(rng, 1, 16384)]), cap=cap, lo=nodes,
                     hi=cap)
        else:
            hi = _between(rng, 16, 4096)
            mask = rng.choice(["causal", "causal", "window", "none"])
            c.update(N=_between(rng, 1, 64), lo=_between(rng, 1, hi), hi=hi, past=rng.choice([0, 0, _between(rng, 1, 4096)]),
                     mask=mask, window=_between(rng, 1, 2048) if mask == "window" else 0, empty=rng.random() < 0.3)
        w = work(c)
        if all(w[k] <= max(m[k] for m in most[op, dtype]) for k in ("bytes", "flops")):
            return c


def _spread(n, lo, hi):
    """n whole numbers from hi down to lo, evenly over their logarithm."""
    return [int(round(hi * (lo / hi) ** (i / max(n - 1, 1)))) for i in range(n)]


def _lengths(c):
    """(queries, keys) of every sequence; the keys are those of the queries behind some of earlier chunks."""
    queries = _spread(c["N"], c["lo"], c["hi"])
    past = _spread(c["N"], 1, c["past"])[::-1] if c["past"] else [0] * c["N"]
    pairs = [(n, n + p) for n, p in zip(queries, past)]
    return pairs + [(0, 0)] if c["empty"] else pairs


def _seen(c, n, m):
    """Pairs of a query and a key it sees in a sequence of n queries and m keys."""
    if c["mask"] == "none":
        return n * m
    first, last = m - n + 1, m  # keys up to the first and the last query's own
    if c["mask"] == "window":
        w = c["window"]
        full = max(0, min(n, last - max(first, w) + 1))  # queries with a whole window
        return full * w + sum(range(first, last - full + 1))
    return (first + last) * n // 2


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    D_qk, D_v = c["D_qk"], c["D_v"]
    if c["op"] == "tree":
        keys = (c["lo"] + c["hi"]) / 2
        rows = c["B"] * c["H"] * c["nodes"]
        kv = c["H_kv"] * (c["S_p"] + c["B"] * keys) * (D_qk + D_v)
        return {"bytes": e * (kv + rows * (D_qk + D_v)) + 4 * rows + 8 * c["B"] * c["nodes"],
                "flops": 2.0 * rows * (c["S_p"] + keys) * (D_qk + D_v)}
    q_rows = c["H"] * sum(n for n, _ in _lengths(c))
    k_rows = c["H_kv"] * sum(m for _, m in _lengths(c))
    pairs = float(c["H"] * sum(_seen(c, n, m) for n, m in _lengths(c)))
    if c["op"] == "packed":
        return {"bytes": e * (q_rows + k_rows) * (D_qk + D_v) + 4 * q_rows, "flops": 2.0 * pairs * (D_qk + D_v)}
    return {"bytes": 2 * e * (q_rows + k_rows) * (D_qk + D_v) + 4 * q_rows, "flops": 2.0 * pairs * (3 * D_qk + 2 * D_v)}


# ---------------------------------------------------------------- inputs

def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _prepare_packed(c, g):
    dt = DTYPES[c["dtype"]]
    H, H_kv, D_qk, D_v = (c[k] for k in ("H", "H_kv", "D_qk", "D_v"))
    lengths = _lengths(c)
    # the sequences in another order for each seed
    lengths = [lengths[i] for i in torch.randperm(len(lengths), generator=g, device="cuda").tolist()]
    ends_q = [sum(n for n, _ in lengths[:i]) for i in range(len(lengths) + 1)]
    ends_k = [sum(m for _, m in lengths[:i]) for i in range(len(lengths) + 1)]
    T_q, T_k = ends_q[-1], ends_k[-1]
    # projections as they leave a matrix product: tokens first, heads beside each other
    st = dict(case=c, ends_q=ends_q, ends_k=ends_k, scale=float(D_qk) ** -0.5,
              q=_normal(g, (T_q, H, D_qk), dt).transpose(0, 1),
              k=_normal(g, (T_k, H_kv, D_qk), dt).transpose(0, 1),
              v=_normal(g, (T_k, H_kv, D_v), dt).transpose(0, 1),
              cu_q=torch.tensor(ends_q, dtype=torch.int32, device="cuda"),
              cu_k=torch.tensor(ends_k, dtype=torch.int32, device="cuda"))
    if c["op"] == "packed_bwd":
        st["do"] = _normal(g, (T_q, H, D_v), dt).transpose(0, 1)
        st["o"], st["lse"] = _plain_packed(st)  # what the forward pass left
    return st


def _prepare_tree(c, g):
    B, H, H_kv, S, S_p, cap = (c[k] for k in ("B", "H", "H_kv", "nodes", "S_p", "cap"))
    dt = DTYPES[c["dtype"]]
    st = dict(case=c, scale=float(c["D_qk"]) ** -0.5,
              q=_normal(g, (B, H, S, c["D_qk"]), dt),
              # rows from a sequence's length on hold what earlier sequences left there
              k_cache=_normal(g, (B, H_kv, cap, c["D_qk"]), dt),
              v_cache=_normal(g, (B, H_kv, cap, c["D_v"]), dt),
              kv_len=torch.randint(c["lo"], c["hi"] + 1, (B,), generator=g, device="cuda").to(torch.int32))
    st["k_prefix"] = _normal(g, (H_kv, S_p, c["D_qk"]), dt) if S_p else None
    st["v_prefix"] = _normal(g, (H_kv, S_p, c["D_v"]), dt) if S_p else None
    # node 0 is the last accepted token, every other one continues an earlier node
    at = torch.arange(S, device="cuda")
    parents = (torch.rand((B, S), generator=g, device="cuda") * at).to(torch.int64).clamp(max=(at - 1).clamp(min=0))
    parents[:, 0] = -1
    st["parents"] = parents.to(torch.int32)
    return st


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return _prepare_tree(case, g) if case["op"] == "tree" else _prepare_packed(case, g)


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"packed": _plain_packed, "packed_bwd": _plain_packed_bwd, "tree": _plain_tree}[op](state)


def _own(st, op):
    import scaled_dot_product_vt_gb300 as vt
    if op == "tree":
        return vt.attn_fwd_tree(st["q"], st["k_prefix"], st["v_prefix"], st["k_cache"], st["v_cache"], st["parents"],
                                st["kv_len"], scale=st["scale"], return_lse=True)
    form = dict(scale=st["scale"], mask=st["case"]["mask"], window=st["case"]["window"])
    if op == "packed":
        return vt.attn_fwd_packed(st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"], return_lse=True, **form)
    return vt.attn_bwd_packed(st["do"], st["q"], st["k"], st["v"], st["o"], st["lse"], st["cu_q"], st["cu_k"], **form)


def _parts(st):
    """(queries, keys, query heads, key/value heads) of the pieces that a pass takes at once: a whole sequence, or the
    heads that share keys where all of them would take too much memory."""
    c = st["case"]
    H, H_kv = c["H"], c["H_kv"]
    for i in range(len(st["ends_q"]) - 1):
        rows, keys = slice(*st["ends_q"][i:i + 2]), slice(*st["ends_k"][i:i + 2])
        if rows.stop == rows.start or keys.stop == keys.start:
            continue
        step = H_kv if H * (rows.stop - rows.start) * (keys.stop - keys.start) <= 1 << 28 else 1
        for a in range(0, H_kv, step):
            yield rows, keys, slice(a * (H // H_kv), (a + step) * (H // H_kv)), slice(a, a + step)


def _hidden(c, n, m):
    """Pairs of n queries and m keys of one sequence that the mask leaves out, or None."""
    if c["mask"] == "none":
        return None
    own_key = torch.arange(n, device="cuda")[:, None] + (m - n)
    key = torch.arange(m, device="cuda")
    hidden = key > own_key
    return hidden | (key <= own_key - c["window"]) if c["mask"] == "window" else hidden


def _scores(st, rows, keys, heads, kv):
    """exp(score - max), its sum and the max of a piece, [kv heads, group, rows, keys]."""
    f = torch.float32
    q = st["q"][heads, rows].to(f).unflatten(0, (kv.stop - kv.start, -1))
    s = (q * st["scale"]) @ st["k"][kv, keys].to(f).transpose(1, 2).unsqueeze(1)
    hidden = _hidden(st["case"], s.shape[2], s.shape[3])
    if hidden is not None:
        s.masked_fill_(hidden, -math.inf)
    top = s.amax(-1, keepdim=True)
    s = s.sub_(top).exp_()
    return s, s.sum(-1, keepdim=True), top


def _plain_packed(st):
    f = torch.float32
    o = torch.zeros((st["q"].shape[1], st["q"].shape[0], st["v"].shape[2]), dtype=st["q"].dtype, device="cuda").transpose(0, 1)
    lse = torch.full(o.shape[:2], -math.inf, dtype=f, device="cuda")
    for rows, keys, heads, kv in _parts(st):
        p, total, top = _scores(st, rows, keys, heads, kv)
        o[heads, rows] = ((p @ st["v"][kv, keys].to(f).unsqueeze(1)) / total).flatten(0, 1).to(o.dtype)
        lse[heads, rows] = (top + torch.log(total)).flatten(0, 1).squeeze(-1)
    return o, lse


def _plain_packed_bwd(st):
    f = torch.float32
    dq, dk, dv = (torch.zeros((x.shape[1], x.shape[0], x.shape[2]), dtype=x.dtype, device="cuda").transpose(0, 1)
                  for x in (st["q"], st["k"], st["v"]))
    for rows, keys, heads, kv in _parts(st):
        p, total, _ = _scores(st, rows, keys, heads, kv)
        p /= total
        n_kv = kv.stop - kv.start
        do = st["do"][heads, rows].to(f).unflatten(0, (n_kv, -1))
        v = st["v"][kv, keys].to(f).unsqueeze(1)
        dv[kv, keys] = (p.transpose(2, 3) @ do).sum(1).to(dv.dtype)
        ds = do @ v.transpose(2, 3)
        ds = ds.sub_((ds * p).sum(-1, keepdim=True)).mul_(p).mul_(st["scale"])
        dq[heads, rows] = (ds @ st["k"][kv, keys].to(f).unsqueeze(1)).flatten(0, 1).to(dq.dtype)
        q = st["q"][heads, rows].to(f).unflatten(0, (n_kv, -1))
        dk[kv, keys] = (ds.transpose(2, 3) @ q).sum(1).to(dk.dtype)
    return dq, dk, dv


def _plain_tree(st):
    c = st["case"]
    B, H, H_kv, S, S_p, cap = (c[k] for k in ("B", "H", "H_kv", "nodes", "S_p", "cap"))
    G = H // H_kv
    f = torch.float32
    # what every node sees of the tree: itself and, in log steps, its ancestors
    at = torch.arange(S, device="cuda")
    up = ((st["parents"].to(torch.int64)[..., None] == at) | (at[:, None] == at)).to(f)
    for _ in range(max(1, (S - 1).bit_length())):
        up = ((up @ up) > 0).to(f)
    # and of the cache: all before the tree, and the nodes' own rows
    first = st["kv_len"].to(torch.int64)[:, None] - S
    key = torch.arange(cap, device="cuda")[None]
    node = (key - first).clamp(0, S - 1)
    seen = torch.gather(up > 0, 2, node[:, None].expand(B, S, cap)) | (key < first)[:, None]
    seen &= (key < first + S)[:, None]
    q = st["q"].to(f).reshape(B, H_kv, G * S, c["D_qk"]) * st["scale"]
    s = (q @ st["k_cache"].to(f).transpose(2, 3)).reshape(B, H_kv, G, S, cap)
    s = s.masked_fill(~seen[:, None, None], -math.inf).reshape(B, H_kv, G * S, cap)
    top = s.amax(-1)
    if S_p:
        qp = q.transpose(0, 1).reshape(H_kv, B * G * S, c["D_qk"])
        sp = (qp @ st["k_prefix"].to(f).transpose(1, 2)).reshape(H_kv, B, G * S, S_p).transpose(0, 1)
        top = torch.maximum(top, sp.amax(-1))
    s = torch.exp(s - top[..., None])
    total = s.sum(-1, keepdim=True)
    o = s @ st["v_cache"].to(f)
    if S_p:
        sp = torch.exp(sp - top[..., None])
        total = total + sp.sum(-1, keepdim=True)
        op = sp.transpose(0, 1).reshape(H_kv, B * G * S, S_p) @ st["v_prefix"].to(f)
        o = o + op.reshape(H_kv, B, G * S, c["D_v"]).transpose(0, 1)
    o = (o / total).reshape(B, H, S, c["D_v"]).to(st["q"].dtype)
    return o, (top[..., None] + torch.log(total)).reshape(B, H, S)


# ---------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return _exact_tree(st) if case["op"] == "tree" else _exact_packed(st)


def _exact_packed(st):
    c = st["case"]
    d = torch.float64
    G = c["H"] // c["H_kv"]
    back = c["op"] == "packed_bwd"
    if sum(n * m for n, m in _lengths(c)) * c["H"] * 2.0 * (c["D_qk"] + c["D_v"]) * (2.5 if back else 1) > 5e12:
        return None
    q, k, v = (st[x].to(d) for x in ("q", "k", "v"))
    res = [torch.zeros_like(x) for x in (q, k, v)] if back else [
        torch.zeros((*q.shape[:2], c["D_v"]), dtype=d, device="cuda"),
        torch.full(q.shape[:2], -math.inf, dtype=d, device="cuda")]
    for i in range(len(st["ends_q"]) - 1):
        (a, b), (s, e) = st["ends_q"][i:i + 2], st["ends_k"][i:i + 2]
        if a == b or s == e:
            continue
        where = torch.arange(e - s, device="cuda") - torch.arange(a + (e - s) - b, e - s, device="cuda")[:, None]
        out = where > 0 if c["mask"] != "none" else torch.zeros_like(where, dtype=torch.bool)
        if c["mask"] == "window":
            out = out | (where <= -c["window"])
        for h in range(c["H"]):
            x = (q[h, a:b] @ k[h // G, s:e].T * st["scale"]).masked_fill(out, -math.inf)
            p = torch.softmax(x, -1)
            if not back:
                res[0][h, a:b] = p @ v[h // G, s:e]
                res[1][h, a:b] = torch.logsumexp(x, -1)
                continue
            g = st["do"][h, a:b].to(d)
            mean = (g * (p @ v[h // G, s:e])).sum(-1, keepdim=True)
            ds = p * (g @ v[h // G, s:e].T - mean) * st["scale"]
            res[0][h, a:b] = ds @ k[h // G, s:e]
            res[1][h // G, s:e] += ds.T @ q[h, a:b]
            res[2][h // G, s:e] += p.T @ g
    return tuple(res)


def _exact_tree(st):
    c = st["case"]
    d = torch.float64
    S, G = c["nodes"], c["H"] // c["H_kv"]
    if work(c)["flops"] > 1.5e12:
        return None
    o = torch.empty((c["B"], c["H"], S, c["D_v"]), dtype=d, device="cuda")
    lse = torch.empty((c["B"], c["H"], S), dtype=d, device="cuda")
    for b, (n, parents) in enumerate(zip(st["kv_len"].tolist(), st["parents"].tolist())):
        rows = []  # the keys every node leaves out
        for s in range(S):
            out = [True] * S
            at = s
            while at >= 0:
                out[at] = False
                at = parents[at]
            rows.append(out)
        hidden = torch.tensor([[False] * (c["S_p"] + n - S) + r for r in rows], device="cuda")
        for h in range(c["H"]):
            key, val = st["k_cache"][b, h // G, :n].to(d), st["v_cache"][b, h // G, :n].to(d)
            if c["S_p"]:
                key = torch.cat([st["k_prefix"][h // G].to(d), key])
                val = torch.cat([st["v_prefix"][h // G].to(d), val])
            x = (st["q"][b, h].to(d) @ key.T * st["scale"]).masked_fill(hidden, -math.inf)
            lse[b, h] = torch.logsumexp(x, -1)
            o[b, h] = torch.exp(x - lse[b, h][:, None]) @ val
    return o, lse
