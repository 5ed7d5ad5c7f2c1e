"""Plain 64-bit forms of the language-model operators, shared by their tests, and the error bounds
that the kernels' roundings allow.

u(t) = finfo(t).eps / 2 is the half step of a rounding.  The window kernels round the weights P (and
dS) once and the result once, everything else is fp32, so with A_i = sum_j P_ij |v_j|:
    |O - O_ref| <= u A + u |O| + F,
F covering the fp32 parts: products of 16-bit values are exact, a sum of n of them is off by n 2^-23
times the sum of magnitudes (twice the fp32 half step, as tensor cores may truncate), ex2 and lg2 by
2^-21.  The gradients likewise, with dS in P's place; where O and lse are the kernel's own instead of
given, D = dO . O carries u sum |dO O| as well.
"""
import math

import torch

F64 = torch.float64


def u(dtype):
    return torch.finfo(dtype).eps / 2


def see(nq, nk, window, sinks, q_start, length, device):
    p = torch.arange(nq, device=device)[:, None] + q_start
    j = torch.arange(nk, device=device)[None, :]
    near = torch.ones_like(j, dtype=torch.bool) if window == 0 else j > p - window
    return (j <= p) & (near | (j < sinks)) & (p < length) & (j < length)


def window_fwd(q, k, v, window, sinks, q_start=None, lens=None):
    """O, lse, and A = sum P |v|, S-magnitude bound; all fp64."""
    q, k, v = (torch.nan_to_num(t.to(F64), nan=0.0) for t in (q, k, v))
    B, H, nq, d = q.shape
    KV, nk = k.shape[1], k.shape[2]
    q_start = nk - nq if q_start is None else q_start
    g = H // KV
    o = torch.zeros_like(q)
    a = torch.zeros_like(q)
    lse = torch.full(q.shape[:3], -math.inf, dtype=F64, device=q.device)
    mag = torch.zeros(q.shape[:3], dtype=F64, device=q.device)
    for b in range(B):
        length = nk if lens is None else min(max(int(lens[b]), 0), nk)
        m = see(nq, nk, window, sinks, q_start, length, q.device)
        for h in range(H):
            s = q[b, h] @ k[b, h // g].T / math.sqrt(d)
            s = s.masked_fill(~m, -math.inf)
            top = s.amax(-1, keepdim=True)
            top = torch.where(torch.isinf(top), 0.0, top)
            p = torch.exp(s - top)
            l = p.sum(-1, keepdim=True)
            p = torch.where(l > 0, p / l, 0.0)
            o[b, h], a[b, h] = p @ v[b, h // g], p @ v[b, h // g].abs()
            lse[b, h] = (top + torch.log(l))[:, 0]
            mag[b, h] = ((q[b, h].abs() @ k[b, h // g].abs().T) / math.sqrt(d)).masked_fill(~m, 0.0).amax(-1)
    return o, lse, a, mag


def check_window_fwd(o, lse, q, k, v, window, sinks, q_start=None, lens=None):
    ref, ref_lse, a, mag = window_fwd(q, k, v, window, sinks, q_start, lens)
    d, n = q.shape[-1], k.shape[2]
    es = d * 2.0 ** -23 * mag                      # error of a score
    rel = 2 * es + (n + 4) * 2.0 ** -23 + 2.0 ** -20  # of a weight, and of their sum
    e = u(o.dtype)
    bound = (e * (1 + e) + 2 * rel[..., None]) * a + e * ref.abs() + 1e-30
    if o.dtype == torch.float16:                   # results and weights below 2^-14 are subnormal
        bound = bound + 2.0 ** -25 + 2.0 ** -24 * v.to(F64).nan_to_num().abs().amax()
    bad = (o.to(F64) - ref).abs() > bound
    assert not bad.any(), f"{int(bad.sum())} elements of O off, worst {((o.to(F64) - ref).abs() / bound).max():.3f} of the bound"
    empty = torch.isinf(ref_lse)
    assert torch.equal(torch.isneginf(lse), empty)
    err = (lse.to(F64) - ref_lse)[~empty].abs()
    lim = (es + rel + ref_lse.abs() * 2.0 ** -22)[~empty]
    assert (err <= lim).all(), f"lse off by {(err / lim).max():.3f} of the bound"


def window_grads(q, k, v, o, lse, do, window, sinks, q_start=None, lens=None, own_o=False):
    """dq, dk, dv by the formulas from the given o and lse, with each one's bound."""
    dt = q.dtype
    e = u(dt)
    q, k, v, o, lse, do = (t.to(F64) for t in (q, k, v, o, lse, do))
    B, H, nq, d = q.shape
    KV, nk = k.shape[1], k.shape[2]
    q_start = nk - nq if q_start is None else q_start
    g, scale = H // KV, 1 / math.sqrt(d)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    bq, bk, bv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for b in range(B):
        length = nk if lens is None else min(max(int(lens[b]), 0), nk)
        m = see(nq, nk, window, sinks, q_start, length, q.device)
        live = m.any(-1)
        for h in range(H):
            qs, os, ds_ = (torch.where(live[:, None], t[b, h], 0.0) for t in (q, o, do))
            n = min(length, nk)
            ks, vs = k[b, h // g].clone(), v[b, h // g].clone()
            ks[n:], vs[n:] = 0.0, 0.0
            s = qs @ ks.T * scale
            p = torch.exp(s - torch.where(live, lse[b, h], 0.0)[:, None]).masked_fill(~m, 0.0)
            dp = ds_ @ vs.T
            dd = (ds_ * os).sum(-1, keepdim=True)
            ds = p * (dp - dd) * scale
            # fp32 errors: of a score (in P's exponent), of dP and of D; own_o: D's rounding of O
            es = d * 2.0 ** -23 * (qs.abs() @ ks.abs().T) * scale + 2.0 ** -20 + 2.0 ** -21 * lse[b, h].nan_to_num(neginf=0.0).abs()[:, None]
            ep = p * es
            edp = d * 2.0 ** -23 * (ds_.abs() @ vs.abs().T + (ds_ * os).abs().sum(-1, keepdim=True))
            if own_o:
                edp = edp + 2 * e * (ds_.abs() * (os.abs() + p @ vs.abs())).sum(-1, keepdim=True)
                ep = ep + p * (2.0 ** -18)
            eds = ep * (dp - dd).abs() * scale + p * edp * scale
            if dt == torch.float16:  # subnormal steps of the scaled P (2^-14 of 1) and dS (2^-15 of its bound)
                ep = ep + 2.0 ** -38
                bound_ds = 2 * scale * ds_.norm(dim=-1).max() * vs.norm(dim=-1).max()
                eds = eds + 2.0 ** -38 * bound_ds
            acc = (nq * g + 4) * 2.0 ** -23
            dq[b, h] = ds @ ks
            bq[b, h] = (e * ds.abs() + eds + acc * ds.abs()) @ ks.abs()
            dk[b, h // g] += ds.T @ qs
            bk[b, h // g] += (e * ds.abs() + eds + acc * ds.abs()).T @ qs.abs()
            dv[b, h // g] += p.T @ ds_
            bv[b, h // g] += (e * p + ep + acc * p).T @ ds_.abs()
    tiny = 2.0 ** -25 if dt == torch.float16 else 0.0
    return [(x, 1.01 * y + e * x.abs() + tiny + 1e-30) for x, y in ((dq, bq), (dk, bk), (dv, bv))]


def check_grads(got, want):
    for name, x, (ref, bound) in zip(("dq", "dk", "dv"), got, want):
        err = (x.to(F64) - ref).abs()
        assert (err <= bound).all(), f"{name}: worst {(err / bound).max():.3f} of the bound"


def freqs(rot, base=10000.0, scaling="none", factor=1.0, original=8192):
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    out, m = [], 1.0
    for i in range(rot // 2):
        w = base ** (-2.0 * i / rot)
        if scaling == "linear":
            w /= factor
        elif scaling == "yarn":
            t = min(1.0, max(0.0, (original * w / (2 * math.pi) - 1) / 31))
            w = w * t + w / factor * (1 - t)
        out.append(w)
    if scaling == "yarn":
        m = 0.1 * math.log(factor) + 1
    return torch.tensor(out, dtype=F64), m


def norm_rope(x, w, pos, rot, interleaved, eps=1e-6, scaling="none", factor=1.0):
    """x: [..., n, d] fp64, pos [..., n]."""
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.to(F64)
    f, m = freqs(rot, scaling=scaling, factor=factor)
    ang = pos.to(F64)[..., None] * f.to(x.device)
    c, s = torch.cos(ang) * m, torch.sin(ang) * m
    a = x[..., :rot]
    if interleaved:
        x0, x1 = a[..., 0::2], a[..., 1::2]
        y = torch.stack([x0 * c - x1 * s, x1 * c + x0 * s], -1).flatten(-2)
    else:
        x0, x1 = a[..., :rot // 2], a[..., rot // 2:]
        y = torch.cat([x0 * c - x1 * s, x1 * c + x0 * s], -1)
    return torch.cat([y, x[..., rot:]], -1)


def plan(lens, new, table, free, count, page, tokens):
    """The serving plan by its definition, request by request; lists in, dict of lists out."""
    table = [list(r) for r in table]
    R, cols = len(lens), len(table[0])
    count = min(max(count, 0), len(free))
    out = {"lens": [], "offsets": [0], "status": [], "slots": [-1] * tokens, "positions": [-1] * tokens}
    asked = taken = 0
    for r in range(R):
        a, b, o = lens[r], max(new[r], 0), out["offsets"][-1]
        out["offsets"].append(o + b)
        held, want = -(-a // page), -(-(a + b) // page)
        ok = a >= 0 and new[r] >= 0 and want <= cols and o + b <= tokens and a + b < 2 ** 31
        need = want - held if ok else 0
        first, asked = asked, asked + need
        ok = ok and (need == 0 or asked <= count)
        out["status"].append(0 if ok else 1)
        out["lens"].append(a + b if ok else a)
        if not ok:
            continue
        taken += need
        for i in range(need):
            table[r][held + i] = free[count - 1 - (first + i)]
        for i in range(b):
            pos = a + i
            pg = table[r][pos // page]
            slot = pg * page + pos % page
            out["slots"][o + i] = slot if pg >= 0 and slot < 2 ** 31 else -1
            out["positions"][o + i] = pos
    out["free_left"], out["table"] = [count - taken], table
    return out


def paged_rows(pages, table_row, length, page):
    """[kv, length, d] rows of a request, fp64."""
    idx = torch.arange(length, device=pages.device)
    pg = table_row.to(pages.device).long()[idx // page]
    return pages[pg, :, idx % page].to(F64).transpose(0, 1)
