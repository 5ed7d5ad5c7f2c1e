"""Timed cases of the language-model operators: sliding-window attention with sinks, the norm and
rotation of queries and keys, and the paged key/value cache (plan, append, decode).

``run`` makes one pass through an operator.  With ``own`` false it computes the plain form with
elementary torch operations; with ``own`` true it makes the calls a user makes of the package.
``exact`` computes the same outputs in 64 bits from the definitions.

Operators (a case's "op"):
  window_fwd  O and lse of attention where query i, at position p = q_start + i, sees the keys
              j <= p with j > p - window (window 0: no limit) or j < sinks; query heads share key
              heads in groups; rows at or past lens[b] are padding (O = 0, lse = -inf).
  window_bwd  dQ, dK, dV of it from the saved O and lse.
  rope_fwd    per-head RMS norm of queries and keys, then the rotation by position.
  rope_bwd    the gradients of that: dq, dk and the two norm weights'.
  append      rope_fwd on packed new tokens, with keys and values stored into cache pages.
  plan        block tables and slot maps of one serving step, from the requests' lengths.
  decode      one query token per request against its pages, with window and sinks.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"


# ---- cases ------------------------------------------------------------------------------------
def listed():
    return [
        # one short prompt through one layer: the smallest attention call, where latency counts
        {"name": "window_fwd_n197", "op": "window_fwd", "batch": 1, "heads": 8, "kv": 2, "nq": 197, "nk": 197,
         "d": 64, "window": 64, "sinks": 4, "dtype": "fp16", "ragged": False},
        # the text benchmark's sequence length, shared key heads, a window of 1024 and one run of sinks
        {"name": "window_fwd_n12288", "op": "window_fwd", "batch": 2, "heads": 16, "kv": 4, "nq": 12288,
         "nk": 12288, "d": 128, "window": 1024, "sinks": 16, "dtype": "bf16", "ragged": False},
        # a padded training batch of the small model: one key head per query head, odd length
        {"name": "window_bwd_n4099_ragged", "op": "window_bwd", "batch": 4, "heads": 8, "kv": 8, "nq": 4099,
         "nk": 4099, "d": 64, "window": 256, "sinks": 4, "dtype": "fp16", "ragged": True},
        # the gradient of the text-length layer
        {"name": "window_bwd_n12288", "op": "window_bwd", "batch": 2, "heads": 16, "kv": 4, "nq": 12288,
         "nk": 12288, "d": 128, "window": 1024, "sinks": 16, "dtype": "bf16", "ragged": False},
        # queries and keys of the text-length layer, far positions, scaled by parts, the half layout
        {"name": "rope_fwd_n12288", "op": "rope_fwd", "batch": 2, "heads": 16, "kv": 4, "n": 12288, "d": 128,
         "rot": 128, "interleaved": False, "scaling": "yarn", "factor": 16.0, "start": 500000, "norm": True,
         "dtype": "bf16"},
        # its gradient on an odd length, interleaved pairs on part of the head
        {"name": "rope_bwd_n8195", "op": "rope_bwd", "batch": 2, "heads": 16, "kv": 4, "n": 8195, "d": 128,
         "rot": 64, "interleaved": True, "scaling": "none", "factor": 1.0, "start": 0, "norm": True,
         "dtype": "bf16"},
        # a chunk of prompts entering the cache
        {"name": "append_t8192", "op": "append", "tokens": 8192, "live": 8000, "heads": 32, "kv": 8, "d": 128,
         "page": 64, "pages": 512, "rot": 128, "interleaved": False, "scaling": "linear", "factor": 4.0,
         "norm": True, "dtype": "bf16"},
        # one decode step's plan: 64 requests, a token each
        {"name": "plan_r64", "op": "plan", "requests": 64, "page": 16, "max_pages": 512, "pages": 40000,
         "tokens": 64, "most_new": 1, "most_len": 8000},
        # a mixed step of many requests: single tokens and prompt chunks
        {"name": "plan_r4096", "op": "plan", "requests": 4096, "page": 64, "max_pages": 1024, "pages": 300000,
         "tokens": 65536, "most_new": 30, "most_len": 8000},
        # one user, a short chat: the smallest decode call
        {"name": "decode_r1_len300", "op": "decode", "requests": 1, "heads": 16, "kv": 4, "d": 64, "page": 16,
         "most_len": 300, "fixed_len": True, "window": 0, "sinks": 0, "dtype": "fp16"},
        # one user, a long document, the whole past visible
        {"name": "decode_r1_len131072", "op": "decode", "requests": 1, "heads": 32, "kv": 8, "d": 128, "page": 64,
         "most_len": 131072, "fixed_len": True, "window": 0, "sinks": 0, "dtype": "bf16"},
        # a full batch of mixed lengths behind a window with sinks
        {"name": "decode_r200_ragged", "op": "decode", "requests": 200, "heads": 32, "kv": 8, "d": 128, "page": 32,
         "most_len": 12288, "fixed_len": False, "window": 4096, "sinks": 16, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window_fwd", "window_bwd", "rope_fwd", "rope_bwd", "append", "plan", "decode"])
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 4, 6])
    d = rng.choice([64, 128])
    if op in ("window_fwd", "window_bwd"):
        window = rng.choice([0, _log(rng, 1, 2000), _log(rng, 1, 2000)])
        n = _log(rng, 1, 8192 if 0 < window <= 1024 else 4000)
        more = rng.choice([0, 0, _log(rng, 1, 2000)]) if op == "window_fwd" else 0
        return {"op": op, "batch": rng.choice([1, 2]), "heads": min(heads, 16), "kv": kv if heads <= 16 else 1,
                "nq": n, "nk": n + more, "d": d, "window": window, "sinks": rng.choice([0, 1, 4, 16, _log(rng, 1, 300)]),
                "dtype": rng.choice(["bf16", "fp16"]), "ragged": rng.random() < 0.4}
    if op in ("rope_fwd", "rope_bwd"):
        d = rng.choice([64, 80, 96, 128, 256])
        batch, dtype = rng.choice([1, 2, 3]), rng.choice(["bf16", "fp16", "fp32"])
        heads, kv = (heads, kv) if heads <= 16 else (16, 1)
        most = 2 * 20 * 8192 * 128 // (batch * (heads + kv) * d * (2 if dtype == "fp32" else 1))
        return {"op": op, "batch": batch, "heads": heads, "kv": kv, "n": _log(rng, 1, min(8192, most)), "d": d,
                "rot": rng.choice([16, 32, 64, d]), "interleaved": rng.random() < 0.5,
                "scaling": rng.choice(["none", "linear", "ntk", "yarn"]), "factor": rng.choice([2.0, 4.0, 16.0]),
                "start": rng.choice([0, rng.randrange(1 << 20)]), "norm": rng.random() < 0.8, "dtype": dtype}
    if op == "append":
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        live = _log(rng, 1, 8000 * 48 * 128 // ((heads + 2 * kv) * d * (2 if dtype == "fp32" else 1)))
        live = min(live, 8000)
        page = rng.choice([16, 32, 64])
        return {"op": op, "tokens": live + rng.choice([0, rng.randrange(150)]), "live": live, "heads": heads,
                "kv": kv, "d": d, "page": page, "pages": -(-live // page) + 1 + rng.randrange(50),
                "rot": rng.choice([32, d]), "interleaved": rng.random() < 0.5,
                "scaling": rng.choice(["none", "linear", "ntk", "yarn"]), "factor": rng.choice([2.0, 8.0]),
                "norm": rng.random() < 0.8, "dtype": dtype}
    if op == "plan":
        r = _log(rng, 1, 4096)
        most_new = _log(rng, 1, 65536 // r) if rng.random() < 0.7 else 1
        page = rng.choice([16, 32, 64, 128])
        return {"op": op, "requests": r, "page": page, "max_pages": rng.choice([128, 512, 777]),
                "pages": r * (8000 // page + 3), "tokens": min(65536, r * most_new), "most_new": most_new,
                "most_len": _log(rng, 1, 8000)}
    r = _log(rng, 1, 200)
    return {"op": op, "requests": r, "heads": heads, "kv": kv, "d": d, "page": rng.choice([16, 32, 64, 128]),
            "most_len": _log(rng, 1, max(2, min(131072, 1200000 // r))), "fixed_len": rng.random() < 0.3,
            "window": rng.choice([0, 0, _log(rng, 1, 5000)]), "sinks": rng.choice([0, 4, 16, 100]),
            "dtype": rng.choice(["bf16", "fp16"])}


# ---- inputs -----------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _lens(case, seed):
    """Lengths of a padded batch: one of one token, one full, the others anywhere between."""
    rng = np.random.default_rng(seed)
    x = rng.integers(1, case["nk"] + 1, size=case["batch"])
    x[0] = case["nk"]
    if case["batch"] > 2:
        x[-1] = 1
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    op = case["op"]
    g = _gen(seed)
    st = {"case": case, "op": op}
    if op in ("window_fwd", "window_bwd"):
        dt = DTYPES[case["dtype"]]
        B, H, KV, nq, nk, d = (case[k] for k in ("batch", "heads", "kv", "nq", "nk", "d"))
        st["q"], st["k"], st["v"] = (_randn(g, (B, h, n, d), dt) for h, n in ((H, nq), (KV, nk), (KV, nk)))
        st["lens"] = _lens(case, seed) if case["ragged"] else None
        if op == "window_bwd":
            st["do"] = _randn(g, (B, H, nq, d), dt)
            st["o"], st["lse"] = _window_fwd_plain(st)
        if own:
            import block_sparse_factorized_b200 as bsf
            st["layout"] = bsf.WindowLayout(H, KV, case["window"], case["sinks"]).upload()
    elif op in ("rope_fwd", "rope_bwd"):
        dt = DTYPES[case["dtype"]]
        B, H, KV, n, d = (case[k] for k in ("batch", "heads", "kv", "n", "d"))
        # projections leave [batch, n, heads, d]; attention reads [batch, heads, n, d]
        st["q"] = _randn(g, (B, n, H, d), dt).transpose(1, 2)
        st["k"] = _randn(g, (B, n, KV, d), dt).transpose(1, 2)
        _rope_state(st, g)
        if op == "rope_bwd":
            st["gq"], st["gk"] = _randn(g, (B, H, n, d), dt), _randn(g, (B, KV, n, d), dt)
    elif op == "append":
        dt = DTYPES[case["dtype"]]
        T, live, H, KV, d, ps, P = (case[k] for k in ("tokens", "live", "heads", "kv", "d", "page", "pages"))
        qkv = _randn(g, (T, H + 2 * KV, d), dt)  # one fused projection
        st["q"], st["k"], st["v"] = qkv[:, :H], qkv[:, H:H + KV], qkv[:, H + KV:]
        _rope_state(st, g)
        rng = np.random.default_rng(seed)
        slots = np.full(T, -1, dtype=np.int32)
        off = int(rng.integers(0, ps))  # the first page is partly filled
        order = rng.permutation(P)
        t = np.arange(live) + off
        slots[:live] = order[t // ps] * ps + t % ps
        st["slots"] = torch.tensor(slots, device=DEV)
        st["positions"] = torch.tensor(np.arange(T) + int(rng.integers(0, 100000)), dtype=torch.int32, device=DEV)
        st["k_pages"], st["v_pages"] = (torch.zeros((P, KV, ps, d), dtype=dt, device=DEV) for _ in range(2))
        st["q_out"] = torch.zeros((T, H, d), dtype=dt, device=DEV)
    elif op == "plan":
        R, ps, MP, P = (case[k] for k in ("requests", "page", "max_pages", "pages"))
        rng = np.random.default_rng(seed)
        lens = rng.integers(0, min(case["most_len"], MP * ps - 1) + 1, size=R)
        new = rng.integers(1, case["most_new"] + 1, size=R) if case["most_new"] > 1 else np.ones(R, dtype=np.int64)
        if case["most_new"] > 1:
            new[rng.random(R) < 0.5] = 1  # half of the requests decode
        order = rng.permutation(P)
        held = -(-lens // ps)
        table = np.full((R, MP), -1, dtype=np.int32)
        at = np.concatenate([[0], np.cumsum(held)])
        for r in range(R):
            table[r, :held[r]] = order[at[r]:at[r + 1]]
        st["lens"], st["new"] = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in (lens, new))
        st["table"] = torch.tensor(table, device=DEV)
        st["free"] = torch.tensor(order[at[-1]:], dtype=torch.int32, device=DEV)
        st["count"] = torch.tensor([P - int(at[-1])], dtype=torch.int32, device=DEV)
        if own:
            import block_sparse_factorized_b200 as bsf
            st["plan"] = bsf.PagedPlan(R, case["tokens"], DEV)
    else:
        dt = DTYPES[case["dtype"]]
        R, H, KV, d, ps = (case[k] for k in ("requests", "heads", "kv", "d", "page"))
        rng = np.random.default_rng(seed)
        lens = np.full(R, case["most_len"]) if case["fixed_len"] else rng.integers(1, case["most_len"] + 1, size=R)
        held = -(-lens // ps)
        MP, P = -(-case["most_len"] // ps), int(held.sum()) + 7
        order = rng.permutation(P)
        table = np.full((R, MP), -1, dtype=np.int32)
        at = np.concatenate([[0], np.cumsum(held)])
        for r in range(R):
            table[r, :held[r]] = order[at[r]:at[r + 1]]
        st["q"] = _randn(g, (R, H, d), dt)
        st["k_pages"], st["v_pages"] = (_randn(g, (P, KV, ps, d), dt) for _ in range(2))
        st["table"] = torch.tensor(table, device=DEV)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        if own:
            import block_sparse_factorized_b200 as bsf
            st["layout"] = bsf.WindowLayout(H, KV, case["window"], case["sinks"]).upload()
            nb = bsf.st_paged_decode_workspace_bytes(st["q"], st["layout"])
            st["workspace"] = torch.empty(nb, dtype=torch.uint8, device=DEV)
    return st


def _rope_state(st, g):
    """Norm weights and the rotation's frequencies, which a program makes once per model."""
    case = st["case"]
    d = case["d"]
    st["wq"] = st["wk"] = None
    if case["norm"]:
        st["wq"], st["wk"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV) for _ in range(2))
    if own:
        import block_sparse_factorized_b200 as bsf
        st["rope"] = bsf.RopeTable(case["rot"], base=10000.0, scaling=case["scaling"], factor=case["factor"],
                                   original=8192, interleaved=case["interleaved"], device=DEV)
    else:
        st["freqs"], st["mscale"] = _freqs_plain(case)


EPS = 1e-6


# ---- one pass ---------------------------------------------------------------------------------
def run(st):
    return _own(st) if own else _PLAIN[st["op"]](st)


def _own(st):
    import block_sparse_factorized_b200 as bsf
    op, case = st["op"], st["case"]
    if op == "window_fwd":
        return bsf.st_window_fwd(st["q"], st["k"], st["v"], st["layout"], lens=st["lens"])
    if op == "window_bwd":
        return bsf.st_window_bwd(st["q"], st["k"], st["v"], st["o"], st["lse"], st["do"], st["layout"],
                                 lens=st["lens"])
    if op == "rope_fwd":
        return bsf.st_qk_norm_rope(st["q"], st["k"], st["rope"], wq=st["wq"], wk=st["wk"], eps=EPS,
                                   start=case["start"])
    if op == "rope_bwd":
        out = bsf.st_qk_norm_rope_bwd(st["q"], st["k"], st["gq"], st["gk"], st["rope"], wq=st["wq"], wk=st["wk"],
                                      eps=EPS, start=case["start"])
        return [t for t in out if t is not None]
    if op == "append":
        bsf.st_paged_append(st["q"], st["k"], st["v"], st["rope"], st["slots"], st["positions"], st["k_pages"],
                            st["v_pages"], wq=st["wq"], wk=st["wk"], eps=EPS, q_out=st["q_out"])
        return st["q_out"], st["k_pages"], st["v_pages"]
    if op == "plan":
        p = bsf.st_paged_plan(st["lens"], st["new"], st["table"], st["free"], st["count"], case["page"],
                              case["tokens"], plan=st["plan"])
        return p.lens, p.free_left, p.offsets, p.slots, p.positions, p.status, st["table"]
    return bsf.st_paged_decode(st["q"], st["k_pages"], st["v_pages"], st["table"], st["lens"], st["layout"],
                               workspace=st["workspace"])


# ---- plain forms ------------------------------------------------------------------------------
ROWS = 1024  # query rows a plain pass takes at a time


def _blocks(case):
    """Row blocks (r0, r1), with the key columns that any of their rows may see."""
    nq, nk, w, s = case["nq"], case["nk"], case["window"], case["sinks"]
    start = nk - nq
    for r0 in range(0, nq, ROWS):
        r1 = min(nq, r0 + ROWS)
        lo = max(0, start + r0 - w + 1) if w else 0
        s1 = min(s, lo)
        cols = torch.cat([torch.arange(s1, device=DEV), torch.arange(lo, start + r1, device=DEV)])
        rows = torch.arange(start + r0, start + r1, device=DEV)
        see = cols[None, :] <= rows[:, None]
        if w:
            see &= (cols[None, :] > rows[:, None] - w) | (cols[None, :] < s)
        yield r0, r1, cols, rows, see


def _window_fwd_plain(st):
    case = st["case"]
    q, k, v, lens = st["q"], st["k"], st["v"], st["lens"]
    B, H, KV, d = case["batch"], case["heads"], case["kv"], case["d"]
    G = H // KV
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=DEV)
    for b in range(B):
        for r0, r1, cols, rows, see in _blocks(case):
            if lens is not None:
                see = see & (rows[:, None] < lens[b])
            for h in range(KV):
                qs = q[b, h * G:(h + 1) * G, r0:r1].float()
                ks, vs = k[b, h][cols].float(), v[b, h][cols].float()
                s = (qs @ ks.T) * (1 / math.sqrt(d))
                s = s.masked_fill(~see, float("-inf"))
                m = s.amax(-1, keepdim=True)
                m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
                p = torch.exp(s - m)
                l = p.sum(-1, keepdim=True)
                o[b, h * G:(h + 1) * G, r0:r1] = ((p @ vs) / torch.where(l == 0, torch.ones_like(l), l)).to(o.dtype)
                lse[b, h * G:(h + 1) * G, r0:r1] = (m + torch.log(l))[..., 0]
    return o, lse


def _window_bwd_plain(st):
    case = st["case"]
    q, k, v, o, lse, do, lens = (st[x] for x in ("q", "k", "v", "o", "lse", "do", "lens"))
    B, H, KV, d = case["batch"], case["heads"], case["kv"], case["d"]
    G = H // KV
    scale = 1 / math.sqrt(d)
    dq = torch.empty_like(q)
    dk, dv = (torch.zeros(k.shape, dtype=torch.float32, device=DEV) for _ in range(2))
    for b in range(B):
        for r0, r1, cols, rows, see in _blocks(case):
            if lens is not None:
                see = see & (rows[:, None] < lens[b])
            for h in range(KV):
                hs = slice(h * G, (h + 1) * G)
                qs, dos, os = q[b, hs, r0:r1].float(), do[b, hs, r0:r1].float(), o[b, hs, r0:r1].float()
                ks, vs = k[b, h][cols].float(), v[b, h][cols].float()
                s = (qs @ ks.T) * scale
                p = torch.exp(s - lse[b, hs, r0:r1, None]).masked_fill(~see, 0.0)
                ds = p * (dos @ vs.T - (dos * os).sum(-1, keepdim=True)) * scale
                ds = ds.masked_fill(~see, 0.0)
                dq[b, hs, r0:r1] = (ds @ ks).to(dq.dtype)
                dk[b, h].index_add_(0, cols, torch.einsum("gij,gid->jd", ds, qs))
                dv[b, h].index_add_(0, cols, torch.einsum("gij,gid->jd", p, dos))
    return dq, dk.to(k.dtype), dv.to(v.dtype)


def _freqs_plain(case):
    """Rotation frequencies (radians per position, in 64 bits) and the scale of cos and sin."""
    rot, base, f = case["rot"], 10000.0, case["factor"]
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    if case["scaling"] == "ntk":
        base = base * f ** (rot / (rot - 2))
    w = base ** (-2 * i / rot)
    m = 1.0
    if case["scaling"] == "linear":
        w = w / f
    elif case["scaling"] == "yarn":  # by parts: turns over the original context between 1 and 32
        turns = 8192 * w / (2 * math.pi)
        keep = ((turns - 1) / (32 - 1)).clamp(0, 1)
        w = w / f * (1 - keep) + w * keep
        m = 0.1 * math.log(f) + 1
    return w, m


def _rotate(x, cos, sin, rot, interleaved):
    a = x[..., :rot]
    if interleaved:
        x0, x1 = a[..., 0::2], a[..., 1::2]
        y = torch.stack([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1).flatten(-2)
    else:
        x0, x1 = a[..., :rot // 2], a[..., rot // 2:]
        y = torch.cat([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _cos_sin(st, pos):
    ang = pos.double()[..., None] * st["freqs"]
    return (torch.cos(ang) * st["mscale"]).float(), (torch.sin(ang) * st["mscale"]).float()


def _norm_rope(x, w, cos, sin, case):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w
    return _rotate(y, cos, sin, case["rot"], case["interleaved"]).to(x.dtype)


def _rope_fwd_plain(st):
    case = st["case"]
    cos, sin = _cos_sin(st, torch.arange(case["n"], device=DEV) + case["start"])
    return (_norm_rope(st["q"], st["wq"], cos, sin, case).contiguous(),
            _norm_rope(st["k"], st["wk"], cos, sin, case).contiguous())


def _rope_bwd_plain(st):
    case = st["case"]
    cos, sin = _cos_sin(st, torch.arange(case["n"], device=DEV) + case["start"])
    dx, dw = [], []
    for x, gr, w in ((st["q"], st["gq"], st["wq"]), (st["k"], st["gk"], st["wk"])):
        gr = _rotate(gr.float(), cos, -sin, case["rot"], case["interleaved"])
        if w is None:
            dx.append(gr.to(x.dtype).contiguous())
            continue
        xf = x.float()
        r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + EPS)
        xh = xf * r
        dw.append((gr * xh).double().sum((0, 1, 2)).float())
        gw = gr * w
        dx.append((r * (gw - xh * (gw * xh).mean(-1, keepdim=True))).to(x.dtype).contiguous())
    return dx + dw


def _append_plain(st):
    case = st["case"]
    ps = case["page"]
    live = torch.nonzero(st["slots"] >= 0)[:, 0]
    cos, sin = _cos_sin(st, st["positions"][live])
    cos, sin = cos[:, None], sin[:, None]
    slot = st["slots"][live].long()
    st["q_out"][live] = _norm_rope(st["q"][live], st["wq"], cos, sin, case)
    st["k_pages"][slot // ps, :, slot % ps] = _norm_rope(st["k"][live], st["wk"], cos, sin, case)
    st["v_pages"][slot // ps, :, slot % ps] = st["v"][live]
    return st["q_out"], st["k_pages"], st["v_pages"]


def _plan_plain(st):
    case = st["case"]
    ps, T, table, free = case["page"], case["tokens"], st["table"], st["free"]
    R, MP = table.shape
    lens, new, count = st["lens"].long(), st["new"].long(), st["count"].long()
    offsets = torch.cat([new.new_zeros(1), new.cumsum(0)])
    held, want = (lens + ps - 1) // ps, (lens + new + ps - 1) // ps
    fits = (want <= MP) & (offsets[1:] <= T)
    need = torch.where(fits, want - held, torch.zeros_like(want))
    upto = need.cumsum(0)
    served = fits & ((need == 0) | (upto <= count))
    got = torch.where(served, need, torch.zeros_like(need))
    first = upto - need
    col = torch.arange(MP, device=DEV)[None, :]
    take = (col >= held[:, None]) & (col < (held + got)[:, None])
    idx = count - 1 - (first[:, None] + col - held[:, None])
    r_i, c_i = torch.nonzero(take, as_tuple=True)
    table[r_i, c_i] = free[idx[r_i, c_i]]
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(offsets[1:].contiguous(), t, right=True)
    live = r < R
    r = r.clamp(max=R - 1)
    pos = lens[r] + t - offsets[r]
    live &= served[r]
    page = table[r, (pos // ps).clamp(0, MP - 1)].long()
    slots = torch.where(live & (page >= 0), page * ps + pos % ps, torch.full_like(pos, -1))
    positions = torch.where(live, pos, torch.full_like(pos, -1))
    i32 = torch.int32
    return ((lens + torch.where(served, new, torch.zeros_like(new))).to(i32), (count - got.sum()).to(i32),
            offsets.to(i32), slots.to(i32), positions.to(i32), (~served).to(i32), table)


def _decode_plain(st):
    case = st["case"]
    q, kp, vp, table, lens = (st[x] for x in ("q", "k_pages", "v_pages", "table", "lens"))
    R, H, d = q.shape
    P, KV, ps, _ = kp.shape
    cap, G, w, s = table.shape[1] * ps, H // KV, case["window"], case["sinks"]
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=DEV)
    col = torch.arange(cap, device=DEV)[None, :]
    step = max(1, (1 << 29) // (cap * KV * d))
    for r0 in range(0, R, step):
        t = table[r0:r0 + step].long()
        ln = lens[r0:r0 + step].long()[:, None]
        see = col < ln
        if w:
            see = see & ((col >= ln - w) | (col < s))
        see = see & (t >= 0).repeat_interleave(ps, 1)
        t = t.clamp(min=0)
        k = kp[t].float().transpose(1, 2).reshape(-1, KV, cap, d)
        sc = (q[r0:r0 + step].float().view(-1, KV, G, d) @ k.transpose(2, 3)) * (1 / math.sqrt(d))
        sc = sc.masked_fill(~see[:, None, None], float("-inf"))
        m = sc.amax(-1, keepdim=True)
        m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
        p = torch.exp(sc - m)
        l = p.sum(-1, keepdim=True)
        v = vp[t].float().transpose(1, 2).reshape(-1, KV, cap, d)
        x = (p @ v) / torch.where(l == 0, torch.ones_like(l), l)
        o[r0:r0 + step] = x.reshape(-1, H, d).to(o.dtype)
        lse[r0:r0 + step] = (m + torch.log(l)).reshape(-1, H)
    return o, lse


_PLAIN = {"window_fwd": _window_fwd_plain, "window_bwd": _window_bwd_plain, "rope_fwd": _rope_fwd_plain,
          "rope_bwd": _rope_bwd_plain, "append": _append_plain, "plan": _plan_plain, "decode": _decode_plain}


# ---- the definitions in 64 bits ---------------------------------------------------------------
def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return _EXACT[case["op"]](st)


def _masked_attention(q, k, v, see):
    """softmax(q k^T / sqrt d) v over the allowed keys (dense, 64 bits); rows without a key give 0."""
    s = torch.where(see, q @ k.transpose(-1, -2) / q.shape[-1] ** 0.5, float("-inf"))
    empty = ~see.any(-1, keepdim=True)
    p = torch.softmax(torch.where(empty, 0.0, s), -1)
    return torch.where(empty, 0.0, p @ v), torch.logsumexp(s, -1)


def _see_dense(case, length):
    p = torch.arange(case["nk"] - case["nq"], case["nk"], device=DEV)[:, None]
    j = torch.arange(case["nk"], device=DEV)[None, :]
    near = torch.ones_like(j, dtype=torch.bool) if case["window"] == 0 else p - j < case["window"]
    return (j <= p) & (near | (j < case["sinks"])) & (p < length)


def _window_exact(st):
    case = st["case"]
    bwd = case["op"] == "window_bwd"
    q, k, v = st["q"], st["k"], st["v"]
    G = case["heads"] // case["kv"]
    outs = [torch.zeros(t.shape, dtype=torch.float64, device=DEV)
            for t in ((q, k, v) if bwd else (q, q[..., 0]))]
    for b in range(case["batch"]):
        see = _see_dense(case, case["nk"] if st["lens"] is None else int(st["lens"][b]))
        for h in range(case["heads"]):
            qs, ks, vs = q[b, h].double(), k[b, h // G].double(), v[b, h // G].double()
            if not bwd:
                outs[0][b, h], outs[1][b, h] = _masked_attention(qs, ks, vs, see)
                continue
            leaves = [t.requires_grad_() for t in (qs, ks, vs)]
            y, _ = _masked_attention(*leaves, see)
            gq, gk, gv = torch.autograd.grad(y, leaves, st["do"][b, h].double())
            outs[0][b, h] = gq
            outs[1][b, h // G] += gk
            outs[2][b, h // G] += gv
    return outs


def _rope_of(case, x, w, pos):
    """The definition as complex numbers: pair (x0, x1) times mscale e^(i pos freq)."""
    if w is not None:
        x = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + EPS) * w.double()
    freqs, m = _freqs_exact(case)
    rot = case["rot"]
    a = x[..., :rot]
    z = a.unflatten(-1, (rot // 2, 2)) if case["interleaved"] else a.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    z = torch.view_as_complex(z.contiguous())
    z = torch.view_as_real(z * torch.polar(torch.full_like(freqs, m), pos.double()[..., None] * freqs))
    y = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _freqs_exact(case):
    rot, s = case["rot"], case["factor"]
    out = []
    for i in range(rot // 2):
        base = 10000.0 * (s ** (rot / (rot - 2)) if case["scaling"] == "ntk" else 1.0)
        w = math.exp(-2.0 * i / rot * math.log(base))
        if case["scaling"] == "linear":
            w /= s
        if case["scaling"] == "yarn":
            keep = min(1.0, max(0.0, (8192 * w / (2 * math.pi) - 1.0) / 31.0))
            w = keep * w + (1.0 - keep) * w / s
        out.append(w)
    m = 0.1 * math.log(s) + 1.0 if case["scaling"] == "yarn" else 1.0
    return torch.tensor(out, dtype=torch.float64, device=DEV), m


def _rope_exact(st):
    case = st["case"]
    pos = torch.arange(case["start"], case["start"] + case["n"], device=DEV)
    bwd = case["op"] == "rope_bwd"
    out, dws = [], []
    for x, w, gname in ((st["q"], st["wq"], "gq"), (st["k"], st["wk"], "gk")):
        xd = x.double().contiguous()
        if not bwd:
            out.append(_rope_of(case, xd, w, pos))
            continue
        leaves = [xd.requires_grad_()]
        if w is not None:
            leaves.append(w.double().requires_grad_())
        y = _rope_of(case, leaves[0], leaves[1] if w is not None else None, pos)
        gr = torch.autograd.grad(y, leaves, st[gname].double())
        out.append(gr[0])
        dws += gr[1:]
    return out + dws


def _append_exact(st):
    case = st["case"]
    ps = case["page"]
    outs = [st[x].double() for x in ("q_out", "k_pages", "v_pages")]
    live = st["slots"] >= 0
    slot, pos = st["slots"][live].long(), st["positions"][live][:, None]
    outs[0][live] = _rope_of(case, st["q"][live].double(), st["wq"], pos)
    rows = [t.transpose(1, 2).contiguous().flatten(0, 1) for t in outs[1:]]
    rows[0][slot] = _rope_of(case, st["k"][live].double(), st["wk"], pos)
    rows[1][slot] = st["v"][live].double()
    return [outs[0]] + [t.unflatten(0, (-1, ps)).transpose(1, 2).contiguous() for t in rows]


def _plan_exact(st):
    case = st["case"]
    ps, T = case["page"], case["tokens"]
    lens, new, free, table = (st[x].cpu().numpy() for x in ("lens", "new", "free", "table"))
    R, MP = table.shape
    left = start = int(st["count"][0])
    asked = 0
    offsets, status, after = [0], [], []
    slots, positions = np.full(T, -1, dtype=np.int32), np.full(T, -1, dtype=np.int32)
    for r in range(R):
        a, b, o = int(lens[r]), int(new[r]), offsets[-1]
        offsets.append(o + b)
        held, want = -(-a // ps), -(-(a + b) // ps)
        ok = want <= MP and o + b <= T
        if ok:
            asked += want - held
            ok = want == held or asked <= start
        status.append(0 if ok else 1)
        after.append(a + b if ok else a)
        if not ok:
            continue
        for i in range(held, want):
            table[r, i] = free[start - 1 - (asked - (want - held) + i - held)]
        left -= want - held
        p = np.arange(a, a + b)
        pg = table[r, p // ps]
        slots[o:o + b] = np.where(pg >= 0, pg * ps + p % ps, -1)
        positions[o:o + b] = p
    dev = [torch.tensor(np.asarray(x, dtype=np.int32), device=DEV)
           for x in (after, [left], offsets, slots, positions, status, table)]
    return dev


def _decode_exact(st):
    case = st["case"]
    R, H, d = st["q"].shape
    KV, ps = case["kv"], case["page"]
    G = H // KV
    o = torch.zeros((R, H, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((R, H), dtype=torch.float64, device=DEV)
    lens, table = st["lens"].tolist(), st["table"].cpu()
    for r in range(R):
        n = lens[r]
        keys = torch.arange(n, device=DEV)
        if case["window"]:
            keys = keys[(keys >= n - case["window"]) | (keys < case["sinks"])]
        pg = table[r].to(DEV).long()[keys // ps]
        k, v = (st[x][pg, :, keys % ps].double().transpose(0, 1) for x in ("k_pages", "v_pages"))
        q = st["q"][r].double().view(KV, G, d)
        y, z = _masked_attention(q, k, v, torch.ones((1, len(keys)), dtype=torch.bool, device=DEV))
        o[r], lse[r] = y.reshape(H, d), z.reshape(H)
    return o, lse


_EXACT = {"window_fwd": _window_exact, "window_bwd": _window_exact, "rope_fwd": _rope_exact,
          "rope_bwd": _rope_exact, "append": _append_exact, "plan": _plan_exact, "decode": _decode_exact}


# ---- what a pass cannot do without ------------------------------------------------------------
def _pairs(case):
    """Allowed (row, key) pairs of one head of a full-length sequence."""
    p = np.arange(case["nk"] - case["nq"], case["nk"], dtype=np.int64)
    if not case["window"]:
        return int((p + 1).sum())
    near = np.minimum(p + 1, case["window"])
    return int((near + np.minimum(case["sinks"], p + 1 - near)).sum())


def work(case):
    op = case["op"]
    e = 4 if case.get("dtype") == "fp32" else 2
    if op in ("window_fwd", "window_bwd"):
        B, H, KV, nq, nk, d = (case[k] for k in ("batch", "heads", "kv", "nq", "nk", "d"))
        q, kv, pairs = B * H * nq * d * e, B * KV * nk * d * e, B * H * _pairs(case)
        if case["ragged"]:  # lengths are spread evenly: about half of the pairs and rows live
            pairs //= 2
        lse = B * H * nq * 4
        if op == "window_fwd":
            return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * d * pairs}
        return {"bytes": 4 * q + 4 * kv + lse, "flops": 10 * d * pairs}
    if op in ("rope_fwd", "rope_bwd"):
        x = case["batch"] * (case["heads"] + case["kv"]) * case["n"] * case["d"]
        passes = 2 if op == "rope_fwd" else 3
        return {"bytes": passes * x * e, "flops": (8 if op == "rope_fwd" else 20) * x}
    if op == "append":
        x = case["live"] * (case["heads"] + 2 * case["kv"]) * case["d"]
        return {"bytes": 2 * x * e + 8 * case["tokens"], "flops": 8 * x}
    if op == "plan":
        return {"bytes": 16 * case["requests"] + 8 * case["tokens"], "flops": 10 * case["tokens"]}
    n = case["most_len"] if case["fixed_len"] else (case["most_len"] + 1) // 2
    if case["window"]:
        span = np.arange(1, case["most_len"] + 1) if not case["fixed_len"] else np.array([case["most_len"]])
        near = np.minimum(span, case["window"])
        n = int((near + np.minimum(case["sinks"], span - near)).mean())
    R, H, KV, d = (case[k] for k in ("requests", "heads", "kv", "d"))
    return {"bytes": 2 * R * KV * n * d * e + 2 * R * H * d * e, "flops": 4 * R * H * n * d}
