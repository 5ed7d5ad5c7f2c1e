"""The paged cache on the GPU: the plan against its definition request by request (equal numbers), the
append, decode against the 64-bit attention over the gathered rows, and all of it together over steps."""
import math

import numpy as np
import pytest
import torch

import lm_ref
from lm_ref import F64

pytestmark = pytest.mark.gpu

bsf = pytest.importorskip("block_sparse_factorized_b200")

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run_plan(lens, new, table, free, count, page, tokens, **kw):
    t = i32(table)
    p = bsf.st_paged_plan(i32(lens), i32(new), t, i32(free), i32([count]), page, tokens, **kw)
    torch.cuda.synchronize()
    want = lm_ref.plan(lens, new, table, free, count, page, tokens)
    for f in ("lens", "free_left", "offsets", "slots", "positions", "status"):
        assert getattr(p, f).tolist() == want[f], f
    assert t.tolist() == want["table"]
    return p


def random_state(R, page, cols, most_len, most_new, seed, spare=10):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, min(most_len, cols * page) + 1, R)
    new = rng.integers(0, most_new + 1, R)
    held = -(-lens // page)
    pages = rng.permutation(int(held.sum()) + spare)
    table, at = np.full((R, cols), -1), 0
    for r in range(R):
        table[r, :held[r]] = pages[at:at + held[r]]
        at += held[r]
    return lens.tolist(), new.tolist(), table.tolist(), pages[at:].tolist()


@pytest.mark.parametrize("R,page,cols,most_len,most_new,spare,tokens", [
    (1, 16, 4, 60, 1, 3, 1), (5, 16, 8, 100, 20, 40, 64), (64, 32, 16, 500, 1, 70, 64), (100, 1, 30, 29, 3, 400, 300),
    (257, 7, 50, 340, 9, 900, 2000), (1025, 64, 6, 380, 40, 700, 40000), (4096, 16, 20, 319, 12, 6000, 30000),
    (8192, 128, 3, 380, 2, 9000, 9000)])
def test_plan(R, page, cols, most_len, most_new, spare, tokens):
    for seed in range(2):
        lens, new, table, free = random_state(R, page, cols, most_len, most_new, seed, spare)
        run_plan(lens, new, table, free, len(free), page, tokens)
        run_plan(lens, new, table, free, len(free) // 9, page, tokens)          # pages run out
        run_plan(lens, new, table, free, len(free), page, max(1, tokens // 7))   # tokens run out


def test_plan_edges():
    t = [[3, 5, -1], [7, -1, -1], [-1, -1, -1], [2, 9, 1]]
    free = [10, 11, 12, 13]
    run_plan([17, 16, 0, 48], [1, 1, 0, 1], t, free, 4, 16, 8)          # within a page, a page's end, nothing, full table
    run_plan([17, -1, 5, 3], [1, 2, -3, 0], t, free, 4, 16, 8)          # lengths below zero are refused
    run_plan([17, 16, 0, 3], [40, 40, 40, 13], t, free, 4, 16, 500)     # too many pages for the table; one still served
    run_plan([0, 0, 0, 0], [40, 40, 40, 1], t, free, 4, 16, 500)        # the third asks too much, and so does the fourth
    run_plan([16, 3, 40, 20], [1, 2, 1, 1], t, free, 4, 16, 8)          # entries of -1 where a page should be: slot -1
    run_plan([0, 0, 0, 0], [1, 1, 1, 1], t, free, 100, 16, 8)           # more pages counted than listed
    run_plan([0, 0, 0, 0], [1, 1, 1, 1], t, free, -2, 16, 8)
    run_plan([2 ** 31 - 1, 2 ** 31 - 2, 0, 0], [1, 1, 1, 0], [[1] * 3] * 4, free, 4, 1 << 20, 8)
    run_plan([2 ** 31 - 2, 0], [1, 1], [[5] * 2048, [6] * 2048], free, 4, 1 << 20, 8)  # slots past 31 bits: -1


def test_plan_buffers_strides_and_graph():
    lens, new, table, free = random_state(50, 16, 12, 150, 30, 3, 200)
    wide = torch.full((50, 20), 77, dtype=torch.int32, device="cuda")
    wide[:, :12] = i32(table)
    plan = bsf.PagedPlan(50, 900, "cuda")
    a, b, f, c = i32(lens), i32(new), i32(free), i32([len(free)])
    bsf.st_paged_plan(a, b, wide[:, :12], f, c, 16, 900, plan=plan)
    want = lm_ref.plan(lens, new, table, free, len(free), 16, 900)
    assert wide[:, :12].tolist() == want["table"] and (wide[:, 12:] == 77).all()
    assert plan.slots.tolist() == want["slots"]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bsf.st_paged_plan(a, b, wide[:, :12], f, c, 16, 900, plan=plan)
    lens, new, table, free = random_state(50, 16, 12, 150, 30, 4, 200)
    a.copy_(i32(lens)), b.copy_(i32(new)), wide[:, :12].copy_(i32(table))
    f.fill_(0), f[:len(free)].copy_(i32(free)[:f.shape[0]]), c.fill_(min(len(free), f.shape[0]))
    fl, n = f.tolist(), int(c)
    g.replay()
    torch.cuda.synchronize()
    want = lm_ref.plan(lens, new, table, fl, n, 16, 900)
    assert plan.slots.tolist() == want["slots"] and plan.status.tolist() == want["status"]
    with pytest.raises(ValueError):
        bsf.st_paged_plan(a, b, wide[:, :12], f, c, 16, 800, plan=plan)
    with pytest.raises(ValueError):
        bsf.st_paged_plan(a.long(), b, wide[:, :12], f, c, 16, 900)


# ---- append -----------------------------------------------------------------------------------
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,H,KV,d,page,rot,inter,norm", [(1, 1, 1, 64, 16, 64, False, True), (37, 6, 2, 128, 32, 64, True, True),
                                                         (300, 4, 4, 64, 16, 32, False, False), (5, 48, 8, 96, 64, 96, False, True)])
def test_append(T, H, KV, d, page, rot, inter, norm, dt):
    """The same bits as the norm and rotation of the tokens as a batch, each in its slot; all else stays."""
    g = torch.Generator(device="cuda").manual_seed(T)
    qkv = torch.randn(T, H + 2 * KV, d, generator=g, device="cuda").to(DT[dt])
    q, k, v = qkv[:, :H], qkv[:, H:H + KV], qkv[:, H + KV:]
    w = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")) if norm else None
    t = bsf.RopeTable(rot, interleaved=inter, device="cuda")
    P = T // page + 3
    slots = torch.randperm(P * page, generator=g, device="cuda")[:T].int()
    skip = torch.rand(T, generator=g, device="cuda") < 0.2
    slots[skip] = -1
    if T > 2:
        slots[1] = P * page        # past the cache: skipped like -1
        slots[2] = -2 ** 31
        skip[1:3] = True
    pos = torch.randint(0, 100000, (T,), generator=g, device="cuda").int()
    kp = torch.full((P, page, KV, d), 7.0, dtype=DT[dt], device="cuda").transpose(1, 2)   # heads inside the rows
    vp = torch.full((P, KV, page, d), 7.0, dtype=DT[dt], device="cuda")
    qo = torch.full((T, H, d), 7.0, dtype=DT[dt], device="cuda")
    bsf.st_paged_append(q, k, v, t, slots, pos, kp, vp, wq=w, wk=w, q_out=qo)
    rq, rk = bsf.st_qk_norm_rope(q.transpose(0, 1)[None], k.transpose(0, 1)[None], t, wq=w, wk=w, positions=pos)
    live = ~skip
    assert torch.equal(qo[live], rq[0].transpose(0, 1)[live]) and (qo[skip] == 7).all()
    s = slots[live].long()
    assert torch.equal(kp[s // page, :, s % page], rk[0].transpose(0, 1)[live])
    assert torch.equal(vp[s // page, :, s % page], v[live])
    kp[s // page, :, s % page] = 7.0
    vp[s // page, :, s % page] = 7.0
    assert (kp == 7).all() and (vp == 7).all()


# ---- decode -----------------------------------------------------------------------------------
def cache(lens, KV, d, page, dt, seed=0, spare=3, layout="heads"):
    rng = np.random.default_rng(seed)
    held = [-(-n // page) for n in lens]
    P = sum(held) + spare
    order, at = rng.permutation(P), 0
    table = torch.full((len(lens), max(max(held), 1) + 1), -1, dtype=torch.int32)
    for r, h in enumerate(held):
        table[r, :h] = torch.tensor(order[at:at + h].astype(np.int32))
        at += h
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (P, KV, page, d) if layout == "heads" else (P, page, KV, d)
    kp, vp = (torch.randn(shape, generator=g, device="cuda").to(DT[dt]) for _ in range(2))
    if layout != "heads":
        kp, vp = kp.transpose(1, 2), vp.transpose(1, 2)
    return kp, vp, table.cuda(), i32(list(lens))


def check_decode(o, lse, q, kp, vp, table, lens, w, s, unseen=()):
    """unseen: (request, page column) whose keys do not count."""
    R, H, d = q.shape
    KV, page = kp.shape[1], kp.shape[2]
    e = lm_ref.u(q.dtype)
    for r, n in enumerate(lens):
        j = torch.arange(n, device="cuda")
        m = torch.ones(n, dtype=torch.bool, device="cuda") if w == 0 else (j >= n - w) | (j < s)
        for rr, c in unseen:
            if rr == r:
                m &= (j // page) != c
        if n == 0 or not bool(m.any()):
            assert (o[r] == 0).all() and torch.isneginf(lse[r]).all()
            continue
        row = table[r].clamp(min=0, max=kp.shape[0] - 1)
        k, v = (lm_ref.paged_rows(t, row, n, page)[:, m] for t in (kp, vp))
        qs = q[r].to(F64).view(KV, H // KV, d)
        sc = qs @ k.transpose(1, 2) / math.sqrt(d)
        p = torch.softmax(sc, -1)
        ref, a = (p @ v).view(H, d), (p @ v.abs()).view(H, d)
        mag = (qs.abs() @ k.abs().transpose(1, 2)).amax(-1).view(H) / math.sqrt(d)
        es = d * 2.0 ** -23 * mag
        rel = 2 * es + (n + 8) * 2.0 ** -23 + 2.0 ** -19
        bound = (e + 2 * rel[:, None]) * 1.01 * a + e * ref.abs() + (2.0 ** -24 * (1 + v.abs().max()) if q.dtype == torch.float16 else 1e-30)
        assert ((o[r].to(F64) - ref).abs() <= bound).all()
        zl = torch.logsumexp(sc, -1).view(H)
        assert ((lse[r].to(F64) - zl).abs() <= es + rel + zl.abs() * 2.0 ** -22).all()


@pytest.mark.parametrize("lens,H,KV,d,page,w,s,dt,layout", [
    ((1,), 1, 1, 64, 16, 0, 0, "bf16", "heads"), ((0, 1, 2, 16, 17), 4, 2, 128, 16, 0, 0, "fp16", "heads"),
    ((300, 31, 128, 0, 1), 8, 1, 64, 32, 50, 4, "bf16", "rows"), ((1000, 5, 700), 16, 2, 128, 64, 100, 70, "bf16", "heads"),
    ((513, 512, 511), 6, 6, 64, 128, 1, 0, "fp16", "rows"), ((200, 90), 24, 2, 128, 16, 33, 17, "bf16", "heads"),
    ((150, 3), 48, 3, 64, 48, 0, 0, "fp16", "heads"), ((130, 131), 64, 1, 128, 16, 129, 1, "bf16", "rows"),
    ((20000, 10, 6000), 4, 4, 128, 256, 0, 0, "bf16", "heads"), ((9000,), 32, 8, 128, 64, 4000, 40, "fp16", "heads"),
    (tuple(range(0, 400, 3)), 4, 2, 64, 16, 64, 4, "bf16", "heads")], ids=lambda x: str(x)[:40])
def test_decode(lens, H, KV, d, page, w, s, dt, layout):
    kp, vp, table, ln = cache(lens, KV, d, page, dt, seed=len(lens), layout=layout)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(len(lens), H, d, generator=g, device="cuda").to(DT[dt])
    lay = bsf.WindowLayout(H, KV, w, s).upload()
    o, lse = bsf.st_paged_decode(q, kp, vp, table, ln, lay, check=True)
    check_decode(o, lse, q, kp, vp, table, lens, w, s)
    again = bsf.st_paged_decode(q, kp, vp, table, ln, lay)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("d", [64, 128])
def test_decode_ignores_what_it_does_not_see(d):
    """NaN in pages of no request, behind the lengths and outside the window change nothing."""
    lens, H, KV, page, w, s = (100, 257, 16), 4, 2, 32, 40, 5
    kp, vp, table, ln = cache(lens, KV, d, page, "bf16", seed=2)
    q = torch.randn(3, H, d, device="cuda").bfloat16()
    lay = bsf.WindowLayout(H, KV, w, s).upload()
    want = bsf.st_paged_decode(q, kp, vp, table, ln, lay)
    seen = torch.zeros(kp.shape[0], page, dtype=torch.bool, device="cuda")
    for r, n in enumerate(lens):
        for j in range(n):
            if j >= n - w or j < s:
                seen[int(table[r, j // page]), j % page] = True
    for t in (kp, vp):
        t.masked_fill_(~seen[:, None, :, None], math.nan)
    got = bsf.st_paged_decode(q, kp, vp, table, ln, lay, check=True)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_decode_bad_pages_and_lengths():
    """Pages outside the cache are not read: their keys do not count and the check reports them.  The
    table's entries past a length are never looked at."""
    lens, H, KV, d, page = (100, 70, 40), 4, 2, 64, 16
    kp, vp, table, ln = cache(lens, KV, d, page, "bf16", seed=3)
    q = torch.randn(3, H, d, device="cuda").bfloat16()
    lay = bsf.WindowLayout(H, KV, 0, 0).upload()
    table[1, 2], table[0, 0], table[2, 3:] = kp.shape[0], -5, 2 ** 31 - 1
    o, lse = bsf.st_paged_decode(q, kp, vp, table, ln, lay)
    with pytest.raises(bsf.StError) as exc:
        lay.check()
    assert exc.value.status == bsf.ST_ERR_BAD_PAGE
    lay.check()  # reported once
    check_decode(o, lse, q, kp, vp, table, lens, 0, 0, unseen=((1, 2), (0, 0)))
    table[2, :3] = -1  # no page at all: nothing seen
    o, lse = bsf.st_paged_decode(q, kp, vp, table, ln, lay)
    assert (o[2] == 0).all() and torch.isneginf(lse[2]).all()
    with pytest.raises(bsf.StError):
        lay.check()
    kp, vp, table, _ = cache(lens, KV, d, page, "bf16", seed=3)
    cap = table.shape[1] * page
    a = bsf.st_paged_decode(q, kp, vp, table.clamp(min=0), i32([-7, 10 ** 9, 40]), lay, check=True)
    b = bsf.st_paged_decode(q, kp, vp, table.clamp(min=0), i32([0, cap, 40]), lay, check=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_far_pages():
    """Pages whose elements lie past 2^31."""
    KV, d, page, n = 8, 128, 64, 1000
    P = (2 ** 31) // (KV * d * page) + 200
    kp, vp = (torch.empty(P, KV, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert kp.numel() > 2 ** 31
    table = torch.arange(P - 16, P, device="cuda", dtype=torch.int32).flip(0)[None].contiguous()
    for t in (kp, vp):
        t[-16:] = torch.randn(16, KV, page, d, device="cuda").bfloat16()
    q = torch.randn(1, 16, d, device="cuda").bfloat16()
    lay = bsf.WindowLayout(16, KV, 0, 0).upload()
    o, lse = bsf.st_paged_decode(q, kp, vp, table, i32([n]), lay, check=True)
    check_decode(o, lse, q, kp, vp, table, (n,), 0, 0)


def test_decode_graph_streams_and_workspace():
    lens, H, KV, d, page = (900, 3, 250), 8, 2, 128, 32
    kp, vp, table, ln = cache(lens, KV, d, page, "bf16", seed=4)
    q = torch.randn(3, H, d, device="cuda").bfloat16()
    lay = bsf.WindowLayout(H, KV, 200, 4).upload()
    ws = torch.full((bsf.st_paged_decode_workspace_bytes(q, lay),), 255, dtype=torch.uint8, device="cuda")
    want = bsf.st_paged_decode(q, kp, vp, table, ln, lay)
    got = bsf.st_paged_decode(q, kp, vp, table, ln, lay, workspace=ws)  # whatever the workspace holds
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = bsf.st_paged_decode(q, kp, vp, table, ln, lay, workspace=ws)
    ln.copy_(i32([870, 2, 249]))
    q.copy_(torch.randn(3, H, d, device="cuda").bfloat16())
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    check_decode(*out, q, kp, vp, table, (870, 2, 249), 200, 4)
    outs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append(bsf.st_paged_decode(q, kp, vp, table, ln, lay))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, out))
    with pytest.raises(bsf.StError):
        bsf.st_paged_decode(q, kp, vp, table, ln, lay, workspace=ws[:256])


def test_serving_steps():
    """Prompts in chunks, then single tokens, with requests joining; every step's decode and the cache
    itself against the window forward over each request's own tokens."""
    H, KV, d, page, P, cols = 8, 2, 64, 16, 120, 24
    w, s = 48, 4
    lay, t = bsf.WindowLayout(H, KV, w, s).upload(), bsf.RopeTable(d, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(20)
    wq, wk = (1 + 0.1 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    kp, vp = (torch.full((P, KV, page, d), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    R, room = 4, 64
    table = torch.full((R, cols), -1, dtype=torch.int32, device="cuda")
    lens, free, count = i32([0] * R), torch.randperm(P, generator=g, device="cuda").int(), i32([P])
    said = [[] for _ in range(R)]
    steps = [(30, 0, 5, 17), (25, 20, 1, 1), (1, 30, 1, 20)] + [(1, 1, 1, 1)] * 20 + [(0, 1, 0, 1)]
    for new in steps:
        plan = bsf.st_paged_plan(lens, i32(list(new)), table, free, count, page, room)
        x = torch.randn(room, H + 2 * KV, d, generator=g, device="cuda").bfloat16()
        q = bsf.st_paged_append(x[:, :H], x[:, H:H + KV], x[:, H + KV:], t, plan.slots, plan.positions, kp, vp, wq=wq, wk=wk)
        lens, count = plan.lens.clone(), plan.free_left.clone()
        assert plan.status.tolist() == [0] * R
        off = plan.offsets.tolist()
        for r in range(R):
            said[r] += list(x[off[r]:off[r + 1]])
        if max(new) == 1:
            # requests of no new token keep their last: they have no query this step
            rows = [r for r in range(R) if new[r]]
            pick = torch.tensor(rows, device="cuda")
            qs = q[torch.tensor([off[r] for r in rows], device="cuda")]
            o, lse = bsf.st_paged_decode(qs, kp, vp, table[pick].contiguous(), lens[pick].contiguous(), lay, check=True)
            for i, r in enumerate(rows):
                y = torch.stack(said[r]).transpose(0, 1)[None]
                fq, fk = bsf.st_qk_norm_rope(y[:, :H], y[:, H:H + KV], t, wq=wq, wk=wk)
                ref = lm_ref.window_fwd(fq[:, :, -1:], fk, y[:, H + KV:], w, s)
                assert ((o[i].to(F64) - ref[0][0, :, 0]).abs() <= 2.0 ** -8 * (1.01 * ref[2][0, :, 0] + ref[0][0, :, 0].abs()) + 1e-5).all()
                assert ((lse[i].to(F64) - ref[1][0, :, 0]).abs() <= 1e-5).all()
    assert lens.tolist() == [len(x) for x in said]
    assert int(count) == P - sum(-(-len(x) // page) for x in said)


def test_append_on_a_given_stream():
    """The zeros of a q_out made by the call come before its rows, whatever the current stream does."""
    H, KV, d, page, n = 4, 2, 64, 16, 20
    g = torch.Generator(device="cuda").manual_seed(30)
    q, k, v = (torch.randn(n, h, d, generator=g, device="cuda").bfloat16() for h in (H, KV, KV))
    t = bsf.RopeTable(d, device="cuda")
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    slots[3] = -1
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    kp, vp = (torch.zeros(2, KV, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    want = bsf.st_paged_append(q, k, v, t, slots, pos, kp, vp)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)  # the current stream is busy
    got = bsf.st_paged_append(q, k, v, t, slots, pos, kp, vp, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and (got[3] == 0).all() and (got[4] != 0).any()


def test_append_in_place():
    H, KV, d, page, n = 4, 2, 128, 16, 33
    g = torch.Generator(device="cuda").manual_seed(31)
    q, k, v = (torch.randn(n, h, d, generator=g, device="cuda").bfloat16() for h in (H, KV, KV))
    wq, wk = (1 + 0.1 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    t = bsf.RopeTable(64, interleaved=True, device="cuda")
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    kp, vp = (torch.zeros(3, KV, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots[5] = -1
    want = bsf.st_paged_append(q, k, v, t, slots, slots, kp, vp, wq=wq, wk=wk)
    q5 = q[5].clone()
    bsf.st_paged_append(q, k, v, t, slots, slots, kp, vp, wq=wq, wk=wk, q_out=q)
    assert torch.equal(q[5], q5)
    want[5] = q5
    assert torch.equal(q, want)


def test_decode_refuses_outputs_that_are_inputs():
    kp, vp, table, ln = cache((20, 3), 2, 64, 16, "bf16", seed=32)
    q = torch.randn(2, 4, 64, device="cuda").bfloat16()
    lay = bsf.WindowLayout(4, 2, 0, 0).upload()
    with pytest.raises(bsf.StError):
        bsf.st_paged_decode(q, kp, vp, table, ln, lay, o=q)


@pytest.mark.parametrize("H,KV", [(4, 2), (24, 2)])  # 8 rows of a product, 16 rows
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_decode_shows_bad_values_it_sees(dt, d, H, KV):
    """A NaN, or a score of +inf, among the keys a request sees makes its O and lse NaN (an lse of -inf
    says that nothing was seen), whether its row is one CTA's or joined from parts."""
    lens, page, w, s = (40, 9000, 17, 9000, 33), 32, 0, 0
    kp, vp, table, ln = cache(lens, KV, d, page, dt, seed=40)
    q = torch.randn(len(lens), H, d, generator=torch.Generator(device="cuda").manual_seed(41), device="cuda").to(DT[dt])
    lay = bsf.WindowLayout(H, KV, w, s).upload()
    want = bsf.st_paged_decode(q, kp, vp, table, ln, lay)

    def row(r, j):
        return int(table[r, j // page]), j % page
    pg, at = row(0, 39)
    kp[pg, 1, at, 3] = math.nan              # request 0: one key head
    pg, at = row(1, 8000)
    kp[pg, 0, at, d - 1] = math.inf          # request 1: +inf for the heads whose query is above 0 there
    q[3, 2] = math.nan                       # request 3: one head
    pg, at = row(4, 5)
    vp[pg, 0, at, 7] = math.nan              # request 4: a value, O alone
    o, lse = bsf.st_paged_decode(q, kp, vp, table, ln, lay, check=True)
    for r, n in enumerate(lens):
        k = lm_ref.paged_rows(kp, table[r], n, page)
        sc = q[r].to(F64).view(KV, H // KV, d) @ k.transpose(1, 2)
        bad = (torch.isnan(sc) | (sc == math.inf)).any(-1).view(H)
        assert torch.equal(torch.isnan(lse[r]), bad) and torch.isnan(o[r][bad]).all(), r
        assert torch.equal(lse[r][~bad], want[1][r][~bad]) or r == 1  # (request 1: a key of -inf counts for nothing)
        assert not torch.isneginf(lse[r]).any()
    assert torch.isnan(lse[0]).any() and torch.isnan(lse[1]).any() and int(torch.isnan(lse[3]).sum()) == 1
    assert torch.isnan(o[4, :H // KV, 7]).all() and not torch.isnan(lse[4]).any()
    assert torch.equal(o[2], want[0][2]) and torch.equal(lse[2], want[1][2])


def test_plan_with_no_free_pages():
    """A full cache and an empty list: requests with room in their last page are served, others are not."""
    run_plan([17, 16, 0, 47], [1, 1, 0, 1], [[3, 5, -1], [7, -1, -1], [-1, -1, -1], [2, 9, 1]], [], 0, 16, 8)
    run_plan([17, 16, 0, 47], [1, 1, 0, 1], [[3, 5, -1], [7, -1, -1], [-1, -1, -1], [2, 9, 1]], [], 5, 16, 8)
    lens, new, table, _ = random_state(1500, 16, 6, 90, 3, 6)
    run_plan(lens, new, table, [], 0, 16, 5000)
