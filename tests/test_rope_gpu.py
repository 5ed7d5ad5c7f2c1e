"""Norm and rotation of queries and keys on the GPU, against the 64-bit forms of lm_ref.py.

Bounds: results are rounded once (u relative); the fp32 arithmetic before it has some ten operations
(2^-20 of the magnitudes that enter a pair), and the angle is off by 2^-24 turns and, for 16-bit rows,
2^-20 from the fast sine and cosine, times the pair's magnitude."""
import pytest
import torch

import lm_ref
from lm_ref import F64

pytestmark = pytest.mark.gpu

bsf = pytest.importorskip("block_sparse_factorized_b200")

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# batch, heads, kv, n, d, rot, interleaved, norm, scaling, start, dtype
CASES = [(1, 1, 1, 1, 16, 16, False, True, "none", 0, "fp32"), (2, 3, 1, 5, 32, 32, True, True, "none", 7, "bf16"),
         (1, 4, 2, 33, 64, 32, False, True, "linear", 100, "fp16"), (2, 2, 2, 129, 64, 64, True, False, "ntk", 0, "fp32"),
         (1, 8, 2, 70, 80, 48, False, True, "yarn", 5000, "bf16"), (1, 6, 6, 17, 96, 96, True, True, "yarn", 1 << 20, "fp32"),
         (3, 16, 4, 300, 128, 128, False, True, "yarn", 1 << 29, "bf16"), (1, 5, 1, 64, 256, 256, False, True, "none", 12345, "fp16"),
         (1, 48, 8, 3, 128, 64, True, True, "linear", 99, "bf16"), (2, 32, 8, 1, 128, 128, False, False, "none", 4000, "fp16"),
         (1, 2, 1, 4000, 240, 16, True, True, "none", 0, "fp32"), (1, 64, 64, 9, 112, 112, False, True, "ntk", 3, "bf16")]
IDS = lambda c: "-".join(map(str, c))  # noqa: E731


def make(case, seed=0):
    B, H, KV, n, d, rot, inter, norm, scaling, start, dt = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, k = (r(B, n, h, d).to(DT[dt]).transpose(1, 2) for h in (H, KV))
    gq, gk = (r(B, h, n, d).to(DT[dt]) for h in (H, KV))
    wq, wk = ((1 + 0.3 * r(d)), (1 + 0.3 * r(d))) if norm else (None, None)
    t = bsf.RopeTable(rot, scaling=scaling, factor=8.0, original=8192, interleaved=inter, device="cuda")
    return q, k, gq, gk, wq, wk, t


def forward(x, w, pos, case, eps=1e-6):
    return lm_ref.norm_rope(x.to(F64), w, pos, case[5], case[6], eps, case[8], 8.0)


def bound_of(ref, x, w, dt, rot, inter, half):
    """u of the result plus the fp32 part, from the magnitudes of each pair before the rotation."""
    mag = x.abs()
    a = mag[..., :rot]
    if inter:
        m = (a[..., 0::2] + a[..., 1::2]).repeat_interleave(2, -1)
    else:
        m = (a[..., :rot // 2] + a[..., rot // 2:]).repeat(*([1] * (a.dim() - 1)), 2)
    mag = torch.cat([m, mag[..., rot:]], -1)
    return lm_ref.u(dt) * ref.abs() + 1.4 * mag * (2.0 ** -20 + (2.0 ** -19 if half else 2.0 ** -21)) + (2.0 ** -25 if dt == torch.float16 else 1e-37)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    B, H, KV, n, d, rot, inter, norm, scaling, start, dt = case
    q, k, _, _, wq, wk, t = make(case)
    oq, ok = bsf.st_qk_norm_rope(q, k, t, wq=wq, wk=wk, start=start)
    pos = torch.arange(n, device="cuda") + start
    for x, w, y in ((q, wq, oq), (k, wk, ok)):
        ref = forward(x, w, pos, case)
        plain = x.to(F64)
        if w is not None:
            plain = plain / torch.sqrt((plain * plain).mean(-1, keepdim=True) + 1e-6) * w.to(F64)
        assert ((y.to(F64) - ref).abs() <= bound_of(ref, plain, w, DT[dt], rot, inter, dt != "fp32")).all()


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_gradients(case):
    B, H, KV, n, d, rot, inter, norm, scaling, start, dt = case
    q, k, gq, gk, wq, wk, t = make(case, seed=1)
    got = bsf.st_qk_norm_rope_bwd(q, k, gq, gk, t, wq=wq, wk=wk, start=start)
    again = bsf.st_qk_norm_rope_bwd(q, k, gq, gk, t, wq=wq, wk=wk, start=start)
    pos = torch.arange(n, device="cuda") + start
    for i, (x, w, gr) in enumerate(((q, wq, gq), (k, wk, gk))):
        leaves = [x.to(F64).contiguous().requires_grad_()] + ([w.to(F64).requires_grad_()] if norm else [])
        y = lm_ref.norm_rope(leaves[0], leaves[1] if norm else None, pos, rot, inter, 1e-6, scaling, 8.0)
        ref = torch.autograd.grad(y, leaves, gr.to(F64))
        r = 1 / torch.sqrt((leaves[0] ** 2).mean(-1, keepdim=True) + 1e-6) if norm else torch.ones_like(leaves[0][..., :1])
        wm = w.to(F64).abs().amax() if norm else 1.0
        # magnitudes: |w g'| r and x r^3 mean|w g' x| <= r max|w| max|g'| (1 + |xhat| |xhat| mean)
        xh = (leaves[0] * r).abs()
        mag = 1.4 * r * wm * gr.to(F64).abs().amax(-1, keepdim=True) * (2 + (xh * xh.mean(-1, keepdim=True) * 2 if norm else 0))
        f32 = 2.0 ** -18 if dt != "fp32" else 2.0 ** -19
        bound = lm_ref.u(DT[dt]) * ref[0].abs() + mag * f32 + (2.0 ** -25 if dt == "fp16" else 1e-37)
        assert ((got[i].to(F64) - ref[0]).abs() <= bound.detach()).all()
        if norm:
            mags = 2.8 * (gr.to(F64).abs().amax(-1, keepdim=True) * xh.detach()).sum((0, 1, 2))
            assert ((got[2 + i].to(F64) - ref[1]).abs() <= mags * 2.0 ** -18).all()
        else:
            assert got[2 + i] is None
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, again))


def test_gradient_against_differences():
    case = (1, 2, 1, 6, 64, 32, True, True, "yarn", 50, "fp32")
    q, k, gq, gk, wq, wk, t = make(case, seed=2)
    dq, dk, dwq, dwk = bsf.st_qk_norm_rope_bwd(q, k, gq, gk, t, wq=wq, wk=wk, start=50)
    pos = torch.arange(6, device="cuda") + 50
    g = torch.Generator(device="cuda").manual_seed(9)
    for x, w, gr, dx, dw in ((q, wq, gq, dq, dwq), (k, wk, gk, dk, dwk)):
        a, b = (torch.randn(s.shape, generator=g, device="cuda", dtype=F64) for s in (x, w))
        f = lambda e: (lm_ref.norm_rope(x.to(F64) + e * a, w.to(F64) + e * b, pos, 32, True, 1e-6, "yarn", 8.0) * gr.to(F64)).sum()  # noqa: E731
        num = float((f(1e-6) - f(-1e-6)) / 2e-6)
        ana = float((dx.to(F64) * a).sum() + (dw.to(F64) * b).sum())
        assert ana == pytest.approx(num, rel=1e-4, abs=1e-4)


def test_positions_in_place_and_weights_type():
    case = (2, 4, 2, 50, 64, 64, False, True, "none", 0, "bf16")
    q, k, gq, gk, wq, wk, t = make(case, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    pos = torch.randint(-1000, 1 << 30, (2, 50), generator=g, device="cuda", dtype=torch.int32)
    oq, ok = bsf.st_qk_norm_rope(q, k, t, wq=wq, wk=wk, positions=pos)
    for b in range(2):  # a row of positions alone: the same bits
        q1, k1 = bsf.st_qk_norm_rope(q[b:b + 1], k[b:b + 1], t, wq=wq, wk=wk, positions=pos[b])
        assert torch.equal(q1, oq[b:b + 1]) and torch.equal(k1, ok[b:b + 1])
    assert torch.equal(bsf.st_qk_norm_rope(q, k, t, wq=wq, wk=wk, start=5)[0],
                       bsf.st_qk_norm_rope(q, k, t, wq=wq, wk=wk, positions=torch.arange(5, 55, device="cuda", dtype=torch.int32))[0])
    dq, dk, _, _ = bsf.st_qk_norm_rope_bwd(q, k, gq, gk, t, wq=wq, wk=wk, positions=pos)
    bsf.st_qk_norm_rope_bwd(q, k, gq, gk, t, wq=wq, wk=wk, positions=pos, dq=gq, dk=gk)  # over the gradients
    assert torch.equal(gq, dq) and torch.equal(gk, dk)
    bsf.st_qk_norm_rope(q, k, t, wq=wq, wk=wk, positions=pos, q_out=q, k_out=k)          # over the inputs
    assert torch.equal(q, oq) and torch.equal(k, ok)
    w16 = wq.bfloat16()
    a = bsf.st_qk_norm_rope(oq, ok, t, wq=w16, wk=w16)
    b = bsf.st_qk_norm_rope(oq, ok, t, wq=w16.float(), wk=w16.float())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_extremes_guards_graph_and_streams():
    case = (1, 4, 2, 40, 96, 64, False, True, "none", 0, "bf16")
    q, k, gq, gk, wq, wk, t = make(case, seed=5)
    q[0, 0, 0] = 0.0                                     # a zero row: eps keeps it finite
    q[0, 1, 3] = float("nan")                            # a NaN stays in its row
    buf = torch.full((1, 6, 48, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    kb = torch.full((1, 4, 48, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    oq, ok = buf[:, 1:5, 4:44, 16:112], kb[:, 1:3, 4:44, 16:112]
    bsf.st_qk_norm_rope(q, k, t, wq=wq, wk=wk, q_out=oq, k_out=ok)
    want = bsf.st_qk_norm_rope(q, k, t, wq=wq, wk=wk)
    assert torch.equal(torch.nan_to_num(oq), torch.nan_to_num(want[0])) and torch.equal(ok, want[1])
    assert (oq[0, 0, 0] == 0).all() and torch.isnan(oq[0, 1, 3]).all() and int(torch.isnan(oq).sum()) == 96
    oq.fill_(7.0)
    ok.fill_(7.0)
    assert (buf == 7).all() and (kb == 7).all()
    q[0, 1, 3] = 1.0
    g = torch.cuda.CUDAGraph()
    bsf.st_qk_norm_rope_bwd(q, k, gq, gk, t, wq=wq, wk=wk)
    with torch.cuda.graph(g):
        out = bsf.st_qk_norm_rope(q, k, t, wq=wq, wk=wk) + bsf.st_qk_norm_rope_bwd(q, k, gq, gk, t, wq=wq, wk=wk)
    q.mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        want = bsf.st_qk_norm_rope(q, k, t, wq=wq, wk=wk) + bsf.st_qk_norm_rope_bwd(q, k, gq, gk, t, wq=wq, wk=wk)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_autograd():
    """Through the norm and rotation into the attention: gradients reach projections and weights."""
    B, n, H, KV, d = 2, 77, 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(B, n, (H + 2 * KV) * d, generator=g, device="cuda").bfloat16().requires_grad_()
    wq, wk = (torch.ones(d, device="cuda").bfloat16().requires_grad_() for _ in range(2))
    t, lay = bsf.RopeTable(d, device="cuda"), bsf.WindowLayout(H, KV, 20, 2).upload()
    y = x.view(B, n, H + 2 * KV, d).transpose(1, 2)
    q, k = bsf.QKNormRope.apply(y[:, :H], y[:, H:H + KV], wq, wk, t)
    o = bsf.WindowAttention.apply(q, k, y[:, H + KV:], lay)
    do = torch.randn(o.shape, generator=g, device="cuda").bfloat16()
    o.backward(do)
    with torch.no_grad():
        of, lse = bsf.st_window_fwd(q, k, y[:, H + KV:], lay)
        gq, gk, gv = bsf.st_window_bwd(q, k, y[:, H + KV:], of, lse, do, lay)
        dq, dk, dwq, dwk = bsf.st_qk_norm_rope_bwd(y[:, :H], y[:, H:H + KV], gq, gk, t, wq=wq, wk=wk)
    got = x.grad.view(B, n, H + 2 * KV, d).transpose(1, 2)
    for a, b in ((got[:, :H], dq), (got[:, H:H + KV], dk), (got[:, H + KV:], gv), (wq.grad, dwq.bfloat16()), (wk.grad, dwk.bfloat16())):
        assert torch.equal(a, b)


def test_autograd_of_a_concatenation():
    """Gradients that come as slices of a larger one, off a 16-byte boundary."""
    B, n, H, KV, d = 1, 33, 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(8)
    q, k, v = (torch.randn(B, h, n, d, generator=g, device="cuda").bfloat16().requires_grad_() for h in (H, KV, KV))
    t, lay = bsf.RopeTable(d, device="cuda"), bsf.WindowLayout(H, KV, 20, 2).upload()
    extra = torch.randn(3, generator=g, device="cuda").bfloat16()
    w = [torch.randn(3 + B * h * n * d, generator=g, device="cuda").bfloat16() for h in (H, H, KV)]

    def grads(head):
        qr, kr = bsf.QKNormRope.apply(q, k, None, None, t)
        o = bsf.WindowAttention.apply(qr, kr, v, lay)
        loss = sum((torch.cat([extra, x.flatten()]) * y).sum() if head else (x.flatten() * y[3:]).sum()
                   for x, y in zip((o, qr, kr), w))
        return torch.autograd.grad(loss, (q, k, v))
    for a, b in zip(grads(True), grads(False)):
        assert torch.equal(a, b)


def test_autograd_of_slices_alone():
    """The same for each operator by itself: its only gradient is such a slice."""
    g = torch.Generator(device="cuda").manual_seed(9)
    q, k = (torch.randn(1, h, 5, 64, generator=g, device="cuda").bfloat16().requires_grad_() for h in (2, 1))
    one = torch.zeros(1, device="cuda").bfloat16()
    t, lay = bsf.RopeTable(64, device="cuda"), bsf.WindowLayout(2, 1, 0, 0).upload()
    for f in (lambda: bsf.QKNormRope.apply(q, k, None, None, t)[0], lambda: bsf.WindowAttention.apply(q, k, k, lay)):
        w = torch.randn(2 * 5 * 64, generator=g, device="cuda").bfloat16()
        a = torch.autograd.grad(torch.cat([one, f().flatten()]), q, torch.cat([one, w]))[0]
        b = torch.autograd.grad(f(), q, w.view(1, 2, 5, 64))[0]
        assert torch.equal(a, b)
