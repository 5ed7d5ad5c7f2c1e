"""Sliding-window attention with sinks on the GPU: forward and gradients against the 64-bit forms of
lm_ref.py, element by element within the roundings' bounds, and the calls a user may make of it:
strided views, padded batches with garbage in the padding, graphs, streams, extreme values."""
import math
import threading

import pytest
import torch

import lm_ref
from lm_ref import F64

pytestmark = pytest.mark.gpu

bsf = pytest.importorskip("block_sparse_factorized_b200")

# batch, heads, kv, nq, nk, d, window, sinks, dtype, lens
CASES = [
    (1, 1, 1, 1, 1, 64, 1, 0, "bf16", None), (1, 2, 1, 1, 1, 128, 0, 0, "fp16", None),
    (2, 4, 2, 2, 2, 64, 0, 0, "bf16", None), (1, 3, 3, 127, 127, 64, 5, 1, "fp16", None),
    (1, 4, 1, 128, 128, 128, 64, 4, "bf16", None), (2, 2, 2, 129, 129, 128, 128, 0, "fp16", None),
    (1, 6, 2, 200, 200, 64, 129, 3, "bf16", None), (1, 8, 2, 257, 257, 64, 0, 7, "fp16", None),
    (2, 4, 4, 300, 300, 128, 40, 130, "bf16", None), (1, 5, 1, 385, 385, 64, 1, 1, "bf16", None),
    (1, 12, 2, 130, 130, 128, 257, 300, "fp16", None), (1, 4, 2, 700, 700, 128, 200, 16, "bf16", None),
    (4, 4, 2, 260, 260, 64, 70, 4, "bf16", (260, 1, 131, 0)), (3, 3, 1, 300, 300, 128, 0, 0, "fp16", (129, 300, 128)),
    (2, 2, 1, 500, 500, 64, 16, 140, "bf16", (500, 255)), (1, 16, 1, 1000, 1000, 64, 100, 4, "fp16", None),
]
# queries that are not the keys' last: more keys than queries, explicit starts (rows past the keys: padding)
OFFSETS = [(1, 4, 2, 1, 400, 64, 50, 4, "bf16", None, None), (2, 2, 1, 130, 333, 128, 100, 0, "fp16", None, None),
           (1, 4, 4, 100, 300, 64, 0, 0, "bf16", None, 37), (1, 2, 1, 200, 150, 64, 30, 2, "fp16", None, 0),
           (2, 3, 3, 140, 300, 128, 64, 5, "bf16", (300, 180), 100), (1, 2, 2, 5, 128, 64, 8, 0, "bf16", None, 1000)]
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def inputs(B, H, KV, nq, nk, d, dt, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    mk = lambda h, n: torch.randn(B, h, n, d, generator=g, device="cuda")  # noqa: E731
    q, k, v, do = mk(H, nq), mk(KV, nk), mk(KV, nk), mk(H, nq)
    return (q * scale).to(dt), k.to(dt), v.to(dt), do.to(dt)


def lens_of(lens):
    return None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_forward_and_gradients(case):
    B, H, KV, nq, nk, d, w, s, dt, lens = case
    q, k, v, do = inputs(B, H, KV, nq, nk, d, DT[dt])
    lay, ln = bsf.WindowLayout(H, KV, w, s).upload(), lens_of(lens)
    o, lse = bsf.st_window_fwd(q, k, v, lay, lens=ln, check=True)
    lm_ref.check_window_fwd(o, lse, q, k, v, w, s, lens=lens)
    got = bsf.st_window_bwd(q, k, v, o, lse, do, lay, lens=ln, check=True)
    lm_ref.check_grads(got, lm_ref.window_grads(q, k, v, o, lse, do, w, s, lens=lens))
    # against the true gradient too, through autograd of the 64-bit forward
    leaves = [t.to(F64).requires_grad_() for t in (q, k, v)]
    ref = lm_ref.window_fwd(*leaves, w, s, lens=lens)[0]
    true = torch.autograd.grad((ref * do.to(F64)).sum(), leaves)
    bounds = lm_ref.window_grads(q, k, v, o, lse, do, w, s, lens=lens, own_o=True)
    lm_ref.check_grads(got, [(t, b) for t, (_, b) in zip(true, bounds)])


@pytest.mark.parametrize("case", OFFSETS, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_query_offsets(case):
    B, H, KV, nq, nk, d, w, s, dt, lens, start = case
    q, k, v, do = inputs(B, H, KV, nq, nk, d, DT[dt], seed=1)
    lay, ln = bsf.WindowLayout(H, KV, w, s).upload(), lens_of(lens)
    o, lse = bsf.st_window_fwd(q, k, v, lay, q_start=start, lens=ln, check=True)
    lm_ref.check_window_fwd(o, lse, q, k, v, w, s, q_start=start, lens=lens)
    got = bsf.st_window_bwd(q, k, v, o, lse, do, lay, q_start=start, lens=ln, check=True)
    lm_ref.check_grads(got, lm_ref.window_grads(q, k, v, o, lse, do, w, s, q_start=start, lens=lens))


def run_all(q, k, v, do, lay, ln=None):
    o, lse = bsf.st_window_fwd(q, k, v, lay, lens=ln)
    return (o, lse) + tuple(bsf.st_window_bwd(q, k, v, o, lse, do, lay, lens=ln))


@pytest.mark.parametrize("d", [64, 128])
def test_strided_views_and_determinism(d):
    """[batch, n, heads, d] views and slices of one fused projection: the same bits as contiguous."""
    B, H, KV, n = 2, 4, 2, 300
    g = torch.Generator(device="cuda").manual_seed(5)
    qkv = torch.randn(B, n, H + 2 * KV, d, generator=g, device="cuda").bfloat16()
    q, k, v = (t.transpose(1, 2) for t in (qkv[:, :, :H], qkv[:, :, H:H + KV], qkv[:, :, H + KV:]))
    do = torch.randn(B, n, H, d, generator=g, device="cuda").bfloat16().transpose(1, 2)
    lay = bsf.WindowLayout(H, KV, 90, 5).upload()
    a = run_all(q, k, v, do, lay)
    b = run_all(*(t.contiguous() for t in (q, k, v, do)), lay)
    c = run_all(q, k, v, do, lay)
    lay.check()
    assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(a, b, c))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_padding_is_never_used(d, dt):
    """NaN and infinities behind each sequence's end change nothing; padding rows get 0 (lse: -inf)."""
    B, H, KV, n, lens = 3, 4, 2, 333, (333, 130, 0)
    q, k, v, do = inputs(B, H, KV, n, n, d, DT[dt], seed=7)
    lay, ln = bsf.WindowLayout(H, KV, 100, 4).upload(), lens_of(lens)
    o, lse = bsf.st_window_fwd(q, k, v, lay, lens=ln)
    clean = (o, lse) + bsf.st_window_bwd(q, k, v, o, lse, do, lay, lens=ln)
    for b, m in enumerate(lens):
        for t, bad in ((q, math.nan), (k, math.inf), (v, math.nan), (do, math.nan)):
            t[b, :, m:] = bad
    o2, lse2 = bsf.st_window_fwd(q, k, v, lay, lens=ln)
    o_in, lse_in = o2.clone(), lse2.clone()
    for b, m in enumerate(lens):
        o_in[b, :, m:], lse_in[b, :, m:] = math.nan, math.nan
    dirty = (o2, lse2) + bsf.st_window_bwd(q, k, v, o_in, lse_in, do, lay, lens=ln)
    lay.check()
    for x, y in zip(clean, dirty):
        assert torch.equal(x, y)
    for b, m in enumerate(lens):
        assert torch.isneginf(lse2[b, :, m:]).all()
        assert all((t[b, :, m:] == 0).all() for t in (o2,) + dirty[2:])


def test_lengths_are_clamped():
    q, k, v, do = inputs(2, 2, 2, 140, 140, 64, torch.bfloat16, seed=8)
    lay = bsf.WindowLayout(2, 2, 30, 2).upload()
    a = run_all(q, k, v, do, lay, lens_of((-5, 1 << 30)))
    b = run_all(q, k, v, do, lay, lens_of((0, 140)))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
def test_growing_maxima(d, dt):
    """Scores that rise by far more than 2^8 from tile to tile, and fall again."""
    n = 520
    q, k, v, do = inputs(1, 2, 2, n, n, d, DT[dt], seed=9, scale=6.0)
    k = k * torch.linspace(0.1, 4.0, n, device="cuda").to(DT[dt])[:, None] * torch.where(
        torch.arange(n, device="cuda") < 400, 1.0, 0.05).to(DT[dt])[:, None]
    lay = bsf.WindowLayout(2, 2, 0, 0).upload()
    o, lse = bsf.st_window_fwd(q, k, v, lay, check=True)
    lm_ref.check_window_fwd(o, lse, q, k, v, 0, 0)
    got = bsf.st_window_bwd(q, k, v, o, lse, do, lay, check=True)
    lm_ref.check_grads(got, lm_ref.window_grads(q, k, v, o, lse, do, 0, 0))


@pytest.mark.parametrize("scale", [2.0 ** -12, 1.0, 2.0 ** 9])
def test_fp16_gradient_range(scale):
    """Loss-scaled gradients, large and small, keep their relative accuracy (dS is scaled in range)."""
    q, k, v, do = inputs(1, 4, 2, 1500, 1500, 64, torch.float16, seed=10)
    do = (do.float() * scale).half()
    lay = bsf.WindowLayout(4, 2, 0, 0).upload()
    o, lse = bsf.st_window_fwd(q, k, v, lay)
    got = bsf.st_window_bwd(q, k, v, o, lse, do, lay, check=True)
    lm_ref.check_grads(got, lm_ref.window_grads(q, k, v, o, lse, do, 0, 0))


def test_zero_gradient():
    q, k, v, do = inputs(1, 2, 1, 200, 200, 64, torch.float16, seed=11)
    lay = bsf.WindowLayout(2, 1, 50, 0).upload()
    o, lse = bsf.st_window_fwd(q, k, v, lay)
    for t in bsf.st_window_bwd(q, k, v, o, lse, torch.zeros_like(do), lay):
        assert (t == 0).all()


@pytest.mark.parametrize("d", [64, 128])
def test_nothing_else_is_written(d):
    """Outputs inside larger buffers: what lies around them stays."""
    B, H, KV, n = 1, 4, 2, 150
    q, k, v, do = inputs(B, H, KV, n, n, d, torch.bfloat16, seed=12)
    lay = bsf.WindowLayout(H, KV, 40, 3).upload()

    def guarded(h, m):
        buf = torch.full((B + 2, h + 2, m + 9, d + 16), 7.0, dtype=torch.bfloat16, device="cuda")
        return buf, buf[1:1 + B, 1:1 + h, 4:4 + m, 8:8 + d]
    bufs = [guarded(h, n) for h in (H, H, KV, KV)]
    lse = torch.full((3 * B * H * n,), 7.0, device="cuda")
    inner = lse[B * H * n:2 * B * H * n].view(B, H, n)
    o, _ = bsf.st_window_fwd(q, k, v, lay, o=bufs[0][1], lse=inner)
    bsf.st_window_bwd(q, k, v, o, inner, do, lay, dq=bufs[1][1], dk=bufs[2][1], dv=bufs[3][1], check=True)
    plain = run_all(q, k, v, do, lay)
    for (buf, view), want in zip(bufs, (plain[0],) + plain[2:]):
        assert torch.equal(view, want)
        view.fill_(7.0)
        assert (buf == 7.0).all()
    assert torch.equal(inner, plain[1]) and (lse[:B * H * n] == 7).all() and (lse[2 * B * H * n:] == 7).all()


def test_graph_streams_and_concurrent_calls():
    n = 700
    lay = bsf.WindowLayout(4, 2, 128, 4).upload()
    a, b = (inputs(2, 4, 2, n, n, 64, torch.bfloat16, seed=s) for s in (13, 14))
    want = [run_all(*x, lay) for x in (a, b)]
    # captured once, replayed on other inputs
    st = [t.clone() for t in a]
    run_all(*st, lay)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run_all(*st, lay)
    for x, w in ((a, want[0]), (b, want[1])):
        for t, y in zip(st, x):
            t.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, w))
    # two streams at a time, each with its own workspace (allocated by the call)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    res = [None, None]
    for i, s in enumerate((s1, s2)):
        with torch.cuda.stream(s):
            res[i] = run_all(*(a, b)[i], lay)
    torch.cuda.synchronize()
    # a stream given by hand, not the current one
    o, lse = bsf.st_window_fwd(*a[:3], lay, stream=s1)
    s1.synchronize()
    lay.check()
    assert torch.equal(o, want[0][0]) and torch.equal(lse, want[0][1])
    for r, w in zip(res, want):
        assert all(torch.equal(p, q) for p, q in zip(r, w))


def test_autograd():
    """The wrapper's gradients, through a strided projection and a summed loss (an expanded gradient)."""
    B, n, H, KV, d = 2, 190, 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(15)
    qkv = torch.randn(B, n, (H + 2 * KV) * d, generator=g, device="cuda").bfloat16().requires_grad_()
    lay = bsf.WindowLayout(H, KV, 60, 2).upload()
    x = qkv.view(B, n, H + 2 * KV, d).transpose(1, 2)
    q, k, v = x[:, :H], x[:, H:H + KV], x[:, H + KV:]
    o = bsf.WindowAttention.apply(q, k, v, lay)
    o.sum().backward()
    with torch.no_grad():
        of, lse = bsf.st_window_fwd(q, k, v, lay)
        want = bsf.st_window_bwd(q, k, v, of, lse, torch.ones_like(of), lay)
    got = qkv.grad.view(B, n, H + 2 * KV, d).transpose(1, 2)
    assert torch.equal(o, of)
    for a, b in zip((got[:, :H], got[:, H:H + KV], got[:, H + KV:]), want):
        assert torch.equal(a, b)


def test_long_sequence_rows():
    """n = 65536 with a window: sampled rows of O and lse, sampled keys' gradients by the formulas."""
    n, w, s = 65536, 4096, 64
    q, k, v, do = inputs(1, 2, 1, n, n, 128, torch.bfloat16, seed=16)
    lay = bsf.WindowLayout(2, 1, w, s).upload()
    o, lse = bsf.st_window_fwd(q, k, v, lay, check=True)
    dq, dk, dv = bsf.st_window_bwd(q, k, v, o, lse, do, lay, check=True)
    for r0 in (0, 4000, 32700, n - 100):
        rows = slice(r0, r0 + 100)
        sub = lm_ref.window_fwd(q[:, :, rows], k, v, w, s, q_start=r0)
        assert ((o[:, :, rows].to(F64) - sub[0]).abs() <= 2.0 ** -8 * (sub[2] * 1.01 + sub[0].abs()) + 1e-4 * sub[2]).all()
        assert ((lse[:, :, rows].to(F64) - sub[1]).abs() <= 1e-4).all()
    keys = torch.tensor([0, 5, 63, 64, 127, 20000, n - 1], device="cuda")  # sinks (seen by all), others
    p = torch.arange(n, device="cuda")[:, None]
    m = (keys <= p) & ((keys > p - w) | (keys < s))
    rk, rv = torch.zeros(len(keys), 128, dtype=F64, device="cuda"), torch.zeros(len(keys), 128, dtype=F64, device="cuda")
    bk, bv = rk.clone(), rv.clone()
    for h in range(2):
        qs, ds_, os = q[0, h].to(F64), do[0, h].to(F64), o[0, h].to(F64)
        pr = torch.exp(qs @ k[0, 0, keys].to(F64).T / math.sqrt(128) - lse[0, h].to(F64)[:, None]).masked_fill(~m, 0.0)
        ds = pr * (ds_ @ v[0, 0, keys].to(F64).T - (ds_ * os).sum(-1, keepdim=True)) / math.sqrt(128)
        rk += ds.T @ qs
        rv += pr.T @ ds_
        bk += ds.abs().T @ qs.abs()
        bv += pr.T @ ds_.abs()
    # half a step of P and of dS (2^-8), fp32 sums of 131072 terms and the weights' own errors (2^-6 of that)
    assert ((dk[0, 0, keys].to(F64) - rk).abs() <= 2.0 ** -8 * (bk * 1.02 + rk.abs())).all()
    assert ((dv[0, 0, keys].to(F64) - rv).abs() <= 2.0 ** -8 * (bv * 1.02 + rv.abs())).all()


def test_offsets_past_32_bits():
    """Tensors of over 2^31 elements: the last head's last rows."""
    B, H, n, d = 1, 9, 2_000_000, 128
    q = torch.zeros(B, H, n, d, dtype=torch.bfloat16, device="cuda")
    k, v = torch.zeros_like(q), torch.zeros_like(q)
    assert q.numel() > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(17)
    m = 700
    for t in (q, k, v):
        t[0, -1, -m:] = torch.randn(m, d, generator=g, device="cuda").bfloat16()
    lay = bsf.WindowLayout(H, H, 200, 0).upload()
    o, lse = bsf.st_window_fwd(q, k, v, lay, check=True)
    a, b, c = (t[:, -1:, -m:] for t in (q, k, v))
    ref = lm_ref.window_fwd(a, b, c, 200, 0)
    rows = slice(200, m)  # rows whose window lies inside the last m
    assert ((o[:, -1:, -m:].to(F64) - ref[0]).abs() <= 2.0 ** -8 * (1.01 * ref[2] + ref[0].abs()) + 1e-4 * ref[2])[:, :, rows].all()
    assert ((lse[:, -1:, -m:].to(F64) - ref[1]).abs() <= 1e-4)[:, :, rows].all()


def test_binding_refusals():
    q, k, v, do = inputs(1, 4, 2, 20, 20, 64, torch.bfloat16)
    lay = bsf.WindowLayout(4, 2, 8).upload()
    with pytest.raises(bsf.StError):
        bsf.st_window_fwd(q, k, v, bsf.WindowLayout(4, 2, 8))  # not uploaded
    with pytest.raises(ValueError):
        bsf.st_window_fwd(q[:, :3], k, v, lay)
    with pytest.raises(ValueError):
        bsf.st_window_fwd(q, k.half(), v, lay)
    with pytest.raises(ValueError):
        bsf.st_window_fwd(q, k[:, :, :5], v[:, :, :5], lay)  # more queries than keys and no q_start
    with pytest.raises(ValueError):
        bsf.st_window_fwd(q, k, v, lay, lens=torch.ones(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        bsf.st_window_fwd(q.transpose(2, 3), k, v, lay)
    with pytest.raises(bsf.StError):
        bsf.st_window_fwd(q, k[:1].expand(1, -1, -1, -1)[:, :1].expand(-1, 2, -1, -1), v, lay)  # stride 0
    with pytest.raises(bsf.StError):
        bsf.st_window_fwd(q.float(), k.float(), v.float(), lay)
    o, lse = bsf.st_window_fwd(q, k, v, lay)
    with pytest.raises(bsf.StError):
        bsf.st_window_bwd(q, k, v, o, lse, do, lay, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_refuses_outputs_that_are_inputs():
    q, k, v, do = inputs(1, 4, 4, 130, 130, 64, torch.bfloat16, seed=21)
    lay = bsf.WindowLayout(4, 4, 64, 2).upload()
    o, lse = bsf.st_window_fwd(q, k, v, lay)
    kept = [t.clone() for t in (q, k, v, o, do)]
    for call in (lambda: bsf.st_window_fwd(q, k, v, lay, o=q), lambda: bsf.st_window_fwd(q, k, v, lay, o=v),
                 lambda: bsf.st_window_bwd(q, k, v, o, lse, do, lay, dq=do), lambda: bsf.st_window_bwd(q, k, v, o, lse, do, lay, dk=k),
                 lambda: bsf.st_window_bwd(q, k, v, o, lse, do, lay, dk=o, dv=torch.empty_like(v)),
                 lambda: bsf.st_window_bwd(q, k, v, o, lse, do, lay, dq=kept[0], dv=kept[0])):
        with pytest.raises(bsf.StError):
            call()
    torch.cuda.synchronize()
    assert torch.equal(q, kept[0]) and all(torch.equal(a, b) for a, b in zip((k, v, o, do), kept[1:]))


def test_given_stream_owns_what_the_call_allocates():
    """On a stream given by hand that runs behind the current one, the call's workspace stays its own:
    the current stream's next allocation of that size must not be it."""
    x = inputs(1, 4, 2, 900, 900, 64, torch.bfloat16, seed=22)
    lay = bsf.WindowLayout(4, 2, 0, 0).upload()
    o, lse = bsf.st_window_fwd(*x[:3], lay)
    want = bsf.st_window_bwd(*x[:3], o, lse, x[3], lay)
    need = bsf.st_window_bwd_workspace_bytes(x[0], x[1], lay)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    got = bsf.st_window_bwd(*x[:3], o, lse, x[3], lay, stream=s)
    spoil = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    for _ in range(20):
        spoil[0].fill_(255)
    s.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    raw = bsf.st_window_bwd(*x[:3], o, lse, x[3], lay, stream=s.cuda_stream)  # the stream as a number
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(raw, want))


def test_no_second_derivative():
    q, k, v, _ = inputs(1, 4, 2, 40, 40, 64, torch.bfloat16, seed=23)
    q.requires_grad_()
    o = bsf.WindowAttention.apply(q, k, v, bsf.WindowLayout(4, 2, 0, 0).upload())
    gq, = torch.autograd.grad(o.float().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):
        gq.float().sum().backward()


@pytest.mark.parametrize("H,KV,d,w,s", [(2, 1, 64, 0, 0), (2, 1, 128, 200, 3), (1, 1, 64, 100, 0)])
def test_many_empty_sequences(H, KV, d, w, s):
    """A large batch with few live sequences: long runs of units with nothing to do between others.
    Live sequences equal themselves alone, bit for bit; all else is zeros."""
    B, n = 256, 1024
    lens = [0] * B
    for b, m in ((3, 1024), (40, 1), (41, 1000), (130, 513), (131, 128), (255, 1024)):
        lens[b] = m
    q, k, v, do = inputs(B, H, KV, n, n, d, torch.bfloat16, seed=24)
    lay = bsf.WindowLayout(H, KV, w, s).upload()
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = bsf.st_window_fwd(q, k, v, lay, lens=ln, check=True)
    grads = bsf.st_window_bwd(q, k, v, o, lse, do, lay, lens=ln, check=True)
    dead = torch.tensor([m == 0 for m in lens], device="cuda")
    assert (o[dead] == 0).all() and (lse[dead] == -math.inf).all() and all((g[dead] == 0).all() for g in grads)
    for b, m in enumerate(lens):
        if m == 0:
            continue
        one = [t[b:b + 1] for t in (q, k, v)]
        lb = ln[b:b + 1].contiguous()
        o1, lse1 = bsf.st_window_fwd(*one, lay, lens=lb, check=True)
        assert torch.equal(o1[0], o[b]) and torch.equal(lse1[0], lse[b]), b
        assert (o[b, :, m:] == 0).all() and (lse[b, :, m:] == -math.inf).all()
        g1 = bsf.st_window_bwd(*one, o1, lse1, do[b:b + 1], lay, lens=lb, check=True)
        for x, y in zip(g1, grads):
            # key tiles may be cut into other chunks: fp32 sums in another order, one rounding to bf16 each
            # (2^-8 of the value on either side; the rest is for sums that cancel)
            assert torch.allclose(x[0].float(), y[b].float(), rtol=2 ** -6, atol=2 ** -6)
            assert (y[b, :, m:] == 0).all()


@pytest.mark.parametrize("pair", [(4, 2), (3, 1)])  # units of two heads, of two row tiles
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_bad_values_in_live_rows_are_seen(d, dt, pair):
    """A NaN, or a score of +inf, makes the rows that see it NaN in O and lse (a zero row with an lse of
    -inf is a padding row's); the other batch elements keep their bits."""
    (H, KV), B, n, w, s, lens = pair, 4, 333, 100, 4, (333, 260, 333, 130)
    q, k, v, do = inputs(B, H, KV, n, n, d, DT[dt], seed=31)
    lay, ln = bsf.WindowLayout(H, KV, w, s).upload(), lens_of(lens)
    o, lse = bsf.st_window_fwd(q, k, v, lay, lens=ln)
    clean = (o, lse) + bsf.st_window_bwd(q, k, v, o, lse, do, lay, lens=ln)
    q[0, 1, 50] = math.nan                   # a query, one of its elements
    q[0, 0, 200, 3], q[0, 2, 332, d - 1] = math.inf, -math.inf
    k[0, 0, 120, 5] = math.nan               # a key that a hundred rows see
    k[1, KV - 1, 2, 7] = math.inf            # a sink
    v[2, 0, 150, 9] = math.nan               # a value: O alone
    o, lse = bsf.st_window_fwd(q, k, v, lay, lens=ln, check=True)
    grads = bsf.st_window_bwd(q, k, v, o, lse, do, lay, lens=ln, check=True)
    for b in range(3):
        m = lm_ref.see(n, n, w, s, 0, lens[b], "cuda")
        for h in range(H):
            sc = q[b, h].to(F64) @ k[b, h * KV // H].to(F64).T
            bad = (m & (torch.isnan(sc) | (sc == math.inf))).any(-1)
            assert torch.equal(torch.isnan(lse[b, h]), bad) and torch.isnan(o[b, h][bad]).all(), (b, h)
            same = ~bad & m.any(-1) & ~(m & torch.isneginf(sc)).any(-1)  # (a score of -inf counts for nothing)
            assert ((lse[b, h] - clean[1][b, h])[same].abs() <= 1e-4).all()
            assert torch.isnan(grads[0][b, h][bad]).all()
            worse = (m & torch.isnan(v[b, h * KV // H, :, 9])[None]).any(-1)
            assert torch.isnan(o[b, h, :, 9][worse]).all()
            dead = ~m.any(-1)
            assert (o[b, h][dead] == 0).all() and torch.isneginf(lse[b, h][dead]).all()
        assert torch.isnan(lse[b]).any() == (b < 2) and torch.isnan(o[b]).any()
    for x, y in zip(clean, (o, lse) + grads):
        assert torch.equal(x[3], y[3])


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("n,d", [(60, 64), (700, 128), (2500, 64)])
def test_backward_over_one_workspace(n, d, dt):
    """Calls behind one another on one workspace, whatever it held: each sees its own preparation (D, the
    maxima, the counters), in a graph's replays too."""
    lay = bsf.WindowLayout(4, 2, 90, 4).upload()
    calls, want = [], []
    for i in range(6):
        q, k, v, do = inputs(2, 4, 2, n, n, d, DT[dt], seed=50 + i)
        do = do * 4.0 ** i  # (fp16: another factor on dS each time)
        o, lse = bsf.st_window_fwd(q, k, v, lay)
        calls.append((q, k, v, o, lse, do))
        want.append(bsf.st_window_bwd(*calls[-1], lay))
    ws = torch.empty(bsf.st_window_bwd_workspace_bytes(calls[0][0], calls[0][1], lay), dtype=torch.uint8, device="cuda")
    for fill in (0, 1, 255):
        ws.fill_(fill)
        got = [bsf.st_window_bwd(*x, lay, workspace=ws) for x in calls for _ in range(3)]
        lay.check()
        assert all(torch.equal(a, b) for i, g in enumerate(got) for a, b in zip(g, want[i // 3]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = [bsf.st_window_bwd(*x, lay, workspace=ws) for x in calls]
    for _ in range(3):
        for x in out:
            for t in x:
                t.fill_(7.0)
        g.replay()
        lay.check()
        assert all(torch.equal(a, b) for x, w in zip(out, want) for a, b in zip(x, w))


def in_a_thread(f):
    """f() in a thread that has made no CUDA call: its result, or its exception raised here."""
    out = []

    def run():
        try:
            out.append((f(), None))
        except BaseException as e:  # noqa: BLE001
            out.append((None, e))
    t = threading.Thread(target=run)
    t.start()
    t.join()
    if out[0][1] is not None:
        raise out[0][1]
    return out[0][0]


def test_first_cuda_call_of_a_thread():
    """Each call as the first that its thread makes (as PyTorch's backward runs in a thread of its own):
    no context is current there yet."""
    q, k, v, do = inputs(1, 4, 4, 256, 256, 64, torch.bfloat16, seed=60)
    lay, t = bsf.WindowLayout(4, 4, 60, 2).upload(), bsf.RopeTable(64, device="cuda")
    fixed = bsf.Layout(bsf.ST_FIXED, bsf.ST_PER_HEAD_ALTERNATING, 4, 256, 128, 32).upload()
    o, lse = bsf.st_window_fwd(q, k, v, lay)
    fo, flse = bsf.st_attn_fwd(q, k, v, fixed)
    pages = [x[0].view(4, 16, 16, 64).transpose(0, 1).contiguous() for x in (k, v)]
    table, i = torch.arange(16, dtype=torch.int32, device="cuda")[None], torch.arange(256, dtype=torch.int32, device="cuda")
    tok = [x[0].transpose(0, 1) for x in (q, k, v)]
    calls = {
        "window_fwd": lambda: bsf.st_window_fwd(q, k, v, lay),
        "window_bwd": lambda: bsf.st_window_bwd(q, k, v, o, lse, do, lay),
        "rope": lambda: bsf.st_qk_norm_rope(q, k, t),
        "rope_bwd": lambda: bsf.st_qk_norm_rope_bwd(q, k, do, do, t)[:2],
        "plan": lambda: (bsf.st_paged_plan(i[:1], i[3:4], table.clone(), i, i[9:10], 16, 8).slots,),
        "append": lambda: (bsf.st_paged_append(*tok, t, i, i, *[x.clone() for x in pages]),),
        "decode": lambda: bsf.st_paged_decode(tok[0][-1:].contiguous(), *pages, table, i[255:], lay),
        "attn_fwd": lambda: bsf.st_attn_fwd(q, k, v, fixed),
        "attn_bwd": lambda: bsf.st_attn_bwd(q, k, v, fo, flse, do, fixed),
        "attn_decode": lambda: bsf.st_attn_decode(q[:, :, 255].contiguous(), k, v, fixed, 255),
    }
    for name, f in calls.items():
        want = f()
        torch.cuda.synchronize()
        kept = [x.clone() for x in want]
        del want  # its memory is there for the thread's call, which need not allocate
        torch.cuda.synchronize()
        got = in_a_thread(f)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, got)), name


def test_backward_offsets_past_32_bits():
    """The backward over tensors of more than 2^31 elements, with a sequence's end inside a tile: the last
    head's last rows."""
    B, H, n, d, w, m = 1, 9, 2_000_000, 128, 200, 700
    end = n - 50
    q = torch.zeros(B, H, n, d, dtype=torch.bfloat16, device="cuda")
    k, v, do = (torch.zeros_like(q) for _ in range(3))
    assert q.numel() > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(18)
    for t in (q, k, v, do):
        t[0, -1, -m:] = torch.randn(m, d, generator=g, device="cuda").bfloat16()
    lay = bsf.WindowLayout(H, H, w, 0).upload()
    ln = lens_of((end,))
    o, lse = bsf.st_window_fwd(q, k, v, lay, lens=ln, check=True)
    got = bsf.st_window_bwd(q, k, v, o, lse, do, lay, lens=ln, check=True)
    a = [t[:, -1:, -m:] for t in (q, k, v, o, lse, do)]
    want = lm_ref.window_grads(*a, w, 0, q_start=0, lens=(m - 50,))
    # every query that sees these keys is among these rows, so dK and dV are whole; dQ where the window is
    for i, (x, (ref, bound)) in enumerate(zip(got, want)):
        rows = slice(w if i == 0 else 0, m)
        err = (x[:, -1:, -m:].to(F64) - ref).abs()[:, :, rows]
        assert (err <= bound[:, :, rows]).all(), f"{i}: worst {(err / bound[:, :, rows]).max():.3f} of the bound"
        assert (x[:, -1:, -50:] == 0).all() and (x[:, :-1] == 0).all()


@pytest.mark.parametrize("H,KV,d,w,s", [(2, 1, 64, 0, 0), (2, 1, 128, 200, 3), (1, 1, 64, 100, 0)])
def test_gradients_among_many_empty_sequences(H, KV, d, w, s):
    """The live sequences of such a batch against the formulas, by the derived bounds."""
    B, n = 256, 1024
    lens = [0] * B
    for b, m in ((3, 1024), (40, 1), (41, 1000), (130, 513), (131, 128), (255, 1024)):
        lens[b] = m
    q, k, v, do = inputs(B, H, KV, n, n, d, torch.bfloat16, seed=25)
    lay = bsf.WindowLayout(H, KV, w, s).upload()
    ln = lens_of(lens)
    o, lse = bsf.st_window_fwd(q, k, v, lay, lens=ln, check=True)
    got = bsf.st_window_bwd(q, k, v, o, lse, do, lay, lens=ln, check=True)
    for b in [b for b in range(B) if lens[b]]:
        a = [t[b:b + 1] for t in (q, k, v, o, lse, do)]
        lm_ref.check_grads([t[b:b + 1] for t in got], lm_ref.window_grads(*a, w, s, lens=(lens[b],)))
