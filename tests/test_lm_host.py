"""Language-model operators, host side (no GPU): what the C ABI and the binding refuse, with which
status, and the rotation speeds against their formulas."""
import ctypes as c
import math
import os
import re

import pytest
import torch

import lm_ref
from block_sparse_factorized_b200 import _abi, lm

bsf = pytest.importorskip("block_sparse_factorized_b200")

P = 0x10000  # an aligned address that no check reads
OK, INVALID, UNSUPPORTED, ALIGNMENT, NOT_UPLOADED, WORKSPACE = 0, 1, 2, 3, 4, 8
BF16, FP32, FP16 = _abi.ST_BF16, _abi.ST_FP32, _abi.ST_FP16


@pytest.fixture()
def lib():
    return _abi.load()


def window(lib, heads=4, kv=2, w=64, s=4):
    h = c.c_void_p()
    assert lib.st_window_create(heads, kv, w, s, c.byref(h)) == OK
    return h


def strides(B, H, n, d):
    return _abi.st_strides_t(H * n * d, n * d, d)


def window_desc(B=2, H=4, KV=2, nq=200, nk=200, d=64, dtype=BF16, q_start=0):
    x = _abi.st_window_desc_t(B, nq, nk, d, q_start, dtype, 0)
    for f in ("q", "o", "dout", "dq"):
        setattr(x, f, strides(B, H, nq, d))
    for f in ("k", "v", "dk", "dv"):
        setattr(x, f, strides(B, KV, nk, d))
    return x


@pytest.mark.parametrize("args", [(0, 1, 1, 0), (4, 0, 1, 0), (4, 3, 1, 0), (4, 2, -1, 0), (4, 2, 1, -1),
                                  (4, 2, (1 << 30) + 1, 0), (4, 2, 1, (1 << 30) + 1)])
def test_window_create_refuses(lib, args):
    h = c.c_void_p()
    assert lib.st_window_create(*args, c.byref(h)) == INVALID and not h.value
    with pytest.raises(bsf.StError):
        bsf.WindowLayout(*args)
    assert lib.st_window_create(4, 2, 1, 1, None) == INVALID


def fwd(lib, w, desc, q=P, o=P, lse=P, lens=None):
    return lib.st_window_fwd(q, P, P, lens, w, o, lse, c.byref(desc) if desc else None, None)


def bwd(lib, w, desc, ws=P, nbytes=1 << 40, q=P):
    return lib.st_window_bwd(q, P, P, P, P, P, None, w, P, P, P, ws, nbytes, c.byref(desc), None)


def test_window_refusals(lib):
    w = window(lib)
    assert fwd(lib, w, window_desc()) == NOT_UPLOADED
    assert bwd(lib, w, window_desc()) == NOT_UPLOADED
    assert fwd(lib, None, window_desc()) == INVALID
    assert fwd(lib, w, None) == INVALID
    for kw in ({"q": None}, {"o": None}, {"lse": None}):
        assert fwd(lib, w, window_desc(), **kw) == INVALID
    for kw in ({"B": 0}, {"nq": 0}, {"nk": 0}, {"d": 0}, {"q_start": -1}, {"dtype": 7}):
        x = window_desc()
        for f, v in kw.items():
            setattr(x, {"B": "batch"}.get(f, f), v)
        assert fwd(lib, w, x) == INVALID, kw
        assert bwd(lib, w, x) == INVALID, kw
        assert lib.st_window_bwd_workspace_bytes(c.byref(x), w) == 0
    for kw in ({"d": 32}, {"d": 96}, {"dtype": FP32}, {"nk": (1 << 30) + 1}, {"q_start": 1 << 30}):
        x = window_desc()
        for f, v in kw.items():
            setattr(x, f, v)
        assert fwd(lib, w, x) == UNSUPPORTED, kw
        assert bwd(lib, w, x) == UNSUPPORTED, kw
    assert fwd(lib, w, window_desc(), q=P + 8) == ALIGNMENT
    assert fwd(lib, w, window_desc(), lens=P + 2) == ALIGNMENT
    assert bwd(lib, w, window_desc(), q=P + 8) == ALIGNMENT
    for f, k, v, want in (("q", "row", 68, ALIGNMENT), ("k", "row", 0, INVALID), ("v", "head", -64, INVALID),
                          ("o", "row", 32, INVALID), ("q", "batch", 12, INVALID)):
        x = window_desc()
        setattr(getattr(x, f), k, v)
        assert fwd(lib, w, x) == want, (f, k)
    x = window_desc(B=1, H=4, KV=2, nq=1, nk=1)  # strides of dimensions of extent 1 are not read
    x.q.row = x.q.batch = -3
    x.k.row = x.k.batch = 0
    assert fwd(lib, w, x) == NOT_UPLOADED
    assert lib.st_window_check(w, None) == NOT_UPLOADED
    assert lib.st_window_upload(None, None) == INVALID
    lib.st_window_destroy(w)
    lib.st_window_destroy(None)


def rope_desc(B=2, H=4, KV=2, n=10, d=64, rot=64, inter=0, dtype=BF16, wdtype=BF16, eps=1e-6):
    x = _abi.st_rope_desc_t(B, H, KV, n, d, 0, 0, rot, inter, dtype, wdtype, eps, 1.0)
    for f in ("q", "q_out", "dq"):
        setattr(x, f, strides(B, H, n, d))
    for f in ("k", "k_out", "dk"):
        setattr(x, f, strides(B, KV, n, d))
    return x


def rope(lib, x, wq=P, wk=P, q=P, turns=P):
    return lib.st_qk_norm_rope(q, P, wq, wk, turns, None, P, P, c.byref(x), None)


def test_rope_refusals(lib):
    for kw, want in (({"batch": 0}, INVALID), ({"heads": 0}, INVALID), ({"rot": 0}, INVALID), ({"rot": 80}, INVALID),
                     ({"interleaved": 2}, INVALID), ({"dtype": 9}, INVALID), ({"wdtype": FP16}, INVALID),
                     ({"eps": -1.0}, INVALID), ({"eps": math.nan}, INVALID), ({"pos_batch": -1}, INVALID),
                     ({"rot": 24}, UNSUPPORTED), ({"d": 72}, UNSUPPORTED), ({"d": 272}, UNSUPPORTED)):
        x = rope_desc()
        for f, v in kw.items():
            setattr(x, f, v)
        assert rope(lib, x) == want, kw
        assert lib.st_qk_norm_rope_bwd_workspace_bytes(c.byref(x)) == 0
    assert rope(lib, rope_desc(), wk=None) == INVALID
    assert rope(lib, rope_desc(), turns=None) == INVALID
    assert rope(lib, rope_desc(), q=P + 4) == ALIGNMENT
    x = rope_desc()
    x.q_out.row = 68
    assert rope(lib, x) == ALIGNMENT
    x = rope_desc()
    args = [P] * 8 + [P, P, P, P]
    assert lib.st_qk_norm_rope_bwd(*args, None, 0, c.byref(x), None) == WORKSPACE
    args[10] = None  # dwq missing with weights
    assert lib.st_qk_norm_rope_bwd(*args, P, 1 << 30, c.byref(x), None) == INVALID


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
@pytest.mark.parametrize("rot", [16, 64, 128])
def test_rope_turns(scaling, rot):
    """turns / 2^64 is w / 2 pi to the 53 bits of the double formula."""
    t = bsf.RopeTable(rot, scaling=scaling, factor=8.0, original=8192, device="cpu")
    f, m = lm_ref.freqs(rot, scaling=scaling, factor=8.0)
    got = torch.tensor([x % 2 ** 64 / 2 ** 64 for x in t.turns.tolist()], dtype=torch.float64)
    assert torch.allclose(got, f / (2 * math.pi), rtol=1e-14, atol=2.0 ** -64)
    assert t.mscale == pytest.approx(m, rel=1e-7)


@pytest.mark.parametrize("kw", [{"rot": 1}, {"rot": 0}, {"base": 1.0}, {"base": math.inf}, {"scaling": "linear", "factor": 0.5},
                                {"scaling": "yarn", "factor": 2.0, "original": 0}, {"rot": 2, "scaling": "ntk", "factor": 2.0},
                                {"factor": math.nan}])
def test_rope_table_refuses(kw):
    with pytest.raises(bsf.StError):
        bsf.RopeTable(**{"rot": 64, "device": "cpu", **kw})


def test_rope_table_unknown_scaling():
    with pytest.raises(ValueError):
        bsf.RopeTable(64, scaling="dynamic", device="cpu")


def plan_args(lib, R=4, T=8, MP=6, page=16, F=20, stride=6, **over):
    sizes = {"lens": R, "new": R, "table": R * stride, "free": F, "count": 1, "lens_out": R, "left": 1, "offsets": R + 1,
             "slots": T, "positions": T, "status": R}
    at, ptr = P, {}
    for k, n in sizes.items():
        ptr[k] = at
        at += 4 * n
    ptr.update({k: v for k, v in over.items() if k in ptr})
    if "alias" in over:
        a, b, words = over["alias"]
        ptr[a] = ptr[b] + 4 * words
    d = _abi.st_plan_desc_t(R, T, MP, stride, page, F)
    for k, v in over.get("desc", {}).items():
        setattr(d, k, v)
    return lib.st_paged_plan(*ptr.values(), c.byref(d), None)


def test_plan_refusals(lib):
    for k in ("lens", "new", "table", "free", "count", "lens_out", "left", "offsets", "slots", "positions", "status"):
        assert plan_args(lib, **{k: None}) == INVALID
    for f, v in (("requests", 0), ("tokens", 0), ("max_pages", 0), ("page_size", 0), ("page_size", (1 << 20) + 1),
                 ("table_stride", 5), ("free_capacity", -1), ("tokens", (1 << 30) + 1), ("max_pages", (1 << 24) + 1)):
        assert plan_args(lib, desc={f: v}) == INVALID, f
    assert plan_args(lib, desc={"requests": 8193}) == UNSUPPORTED
    for a, b, words in (("lens_out", "lens", 0), ("lens_out", "lens", 3), ("slots", "table", 0), ("left", "count", 0),
                        ("positions", "slots", 7), ("status", "new", 1), ("offsets", "free", 19)):
        assert plan_args(lib, alias=(a, b, words)) == INVALID, (a, b)
    assert plan_args(lib, lens=P + 2) == ALIGNMENT


def paged_desc(R=3, d=64, MP=4, page=16, pages=9, KV=2, dtype=BF16):
    s = _abi.st_strides_t(KV * page * d, page * d, d)
    return _abi.st_paged_desc_t(R, d, MP, MP, dtype, 0, _abi.st_pages_t(pages, page, s, s))


def test_decode_refusals(lib):
    w = window(lib)

    def run(x, ws=P, n=1 << 40, q=P, wh=w):
        return lib.st_paged_decode(q, P, P, P, P, wh, P, P, ws, n, c.byref(x), None)
    assert run(paged_desc()) == NOT_UPLOADED
    assert run(paged_desc(), wh=None) == INVALID
    assert run(paged_desc(), q=None) == INVALID
    for f, v in (("requests", 0), ("max_pages", 0), ("d", 0), ("dtype", 8), ("table_stride", 3)):
        x = paged_desc()
        setattr(x, f, v)
        assert run(x) == INVALID, f
        assert lib.st_paged_decode_workspace_bytes(c.byref(x), w) == 0
    x = paged_desc()
    x.pages.num_pages = 1 << 28  # slots would pass 31 bits
    assert run(x) == INVALID
    assert run(paged_desc(page=24)) == UNSUPPORTED
    assert run(paged_desc(d=32)) == UNSUPPORTED
    assert run(paged_desc(dtype=FP32)) == UNSUPPORTED
    assert run(paged_desc(R=8193)) == UNSUPPORTED
    wide = window(lib, heads=130, kv=2)
    assert run(paged_desc(), wh=wide) == UNSUPPORTED
    assert run(paged_desc(), q=P + 2) == ALIGNMENT
    x = paged_desc()
    x.pages.k.row = 0
    assert run(x) == INVALID


def test_append_refusals(lib):
    s = _abi.st_strides_t(2 * 16 * 64, 16 * 64, 64)
    g = _abi.st_pages_t(5, 16, s, s)

    def run(x, slots=P, pages=g, v=P):
        vs = strides(1, 2, x.n, x.d)
        return lib.st_paged_append(P, P, v, P, P, P, P, slots, P, P, P, c.byref(vs), c.byref(pages), c.byref(x), None)
    assert run(rope_desc(B=1), slots=None) == INVALID
    assert run(rope_desc(B=2)) == INVALID
    assert run(rope_desc(B=1), v=P + 8) == ALIGNMENT
    bad = _abi.st_pages_t(5, 16, _abi.st_strides_t(2 * 16 * 64, 16 * 64, 60), s)
    assert run(rope_desc(B=1), pages=bad) == INVALID
    assert run(rope_desc(B=1), pages=_abi.st_pages_t(0, 16, s, s)) == INVALID


def test_binding_refuses_cpu_tensors():
    q, k = torch.zeros(1, 4, 8, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    win = bsf.WindowLayout(4, 2, 16)
    t = bsf.RopeTable(64, device="cpu")
    i = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: bsf.st_window_fwd(q, k, k, win),
                 lambda: bsf.st_qk_norm_rope(q, k, t),
                 lambda: bsf.st_paged_append(q[0].transpose(0, 1), k[0].transpose(0, 1), k[0].transpose(0, 1), t, i, i, k, k),
                 lambda: bsf.st_paged_plan(i, i, torch.zeros(3, 4, dtype=torch.int32), i, i[:1], 16, 8),
                 lambda: bsf.st_paged_decode(q[0], k, k, torch.zeros(4, 4, dtype=torch.int32), i, win)):
        with pytest.raises(ValueError):
            call()


def test_reference_gradient_against_differences():
    """The 64-bit formulas that the GPU tests compare with, against central differences."""
    g = torch.Generator().manual_seed(3)
    q, k, v, do = (torch.randn(1, h, 9, 8, generator=g, dtype=torch.float64) for h in (4, 2, 2, 4))
    for w, s in ((3, 1), (0, 0), (2, 4)):
        def f(q, k, v):
            return (lm_ref.window_fwd(q, k, v, w, s)[0] * do).sum()
        o, lse, _, _ = lm_ref.window_fwd(q, k, v, w, s)
        grads = lm_ref.window_grads(q, k, v, o, lse, do, w, s)
        for i, x in enumerate((q, k, v)):
            d = torch.randn(x.shape, generator=g, dtype=torch.float64)
            a, b = [q, k, v], [q, k, v]
            a[i], b[i] = x + 1e-6 * d, x - 1e-6 * d
            num = float((f(*a) - f(*b)) / 2e-6)
            assert float((grads[i][0] * d).sum()) == pytest.approx(num, rel=1e-6, abs=1e-7)


def test_rope_refuses_outputs_that_are_other_arrays(lib):
    """In place means the same layout, and one output is not the other's input."""
    at = [P + 0x100000 * i for i in range(12)]

    def run(q_out, k_out, wider=None):
        x = rope_desc()
        if wider:
            getattr(x, wider).row = 128
        return lib.st_qk_norm_rope(at[0], at[1], at[2], at[3], at[4], None, q_out, k_out, c.byref(x), None)
    for q_out, k_out in ((at[1], at[6]), (at[5], at[0]), (at[5], at[5]), (at[2], at[6]), (at[5], at[4])):
        assert run(q_out, k_out) == INVALID
    assert run(at[0], at[6], "q_out") == INVALID
    assert run(at[5], at[1], "k_out") == INVALID

    def bwd(dq=at[5], dk=at[6], dwq=at[7], dwk=at[8], ws=at[9]):
        x = rope_desc()
        return lib.st_qk_norm_rope_bwd(at[0], at[1], at[10], at[11], at[2], at[3], at[4], None, dq, dk, dwq, dwk, ws, 1 << 30,
                                       c.byref(x), None)
    for kw in ({"dq": at[0]}, {"dk": at[1]}, {"dq": at[11]}, {"dk": at[10]}, {"dq": at[6]}, {"dwq": at[8]}, {"dwk": at[5]},
               {"ws": at[10]}, {"ws": at[7]}):
        assert bwd(**kw) == INVALID, kw


def test_append_refuses_outputs_that_are_other_arrays(lib):
    at = [P + 0x100000 * i for i in range(12)]
    s = _abi.st_strides_t(2 * 16 * 64, 16 * 64, 64)
    g, vs = _abi.st_pages_t(5, 16, s, s), strides(1, 2, 10, 64)
    for q_out, kp, vp in ((at[1], at[9], at[10]), (at[8], at[9], at[9]), (at[8], at[8], at[10]), (at[8], at[0], at[10]),
                          (at[8], at[1], at[10]), (at[8], at[9], at[2]), (at[6], at[9], at[10])):
        assert lib.st_paged_append(at[0], at[1], at[2], at[3], at[4], at[5], at[6], at[7], q_out, kp, vp, c.byref(vs),
                                   c.byref(g), c.byref(rope_desc(B=1)), None) == INVALID


def test_window_backward_waits_steer_whole_warps():
    """The roles of the backward's kernels are whole warps that vote, elect and synchronise with full
    masks, so a bounded wait, which may run out for some lanes and not for others, must not steer lanes
    apart: its result is put to a vote, or ignored."""
    with open(os.path.join(os.path.dirname(_abi.__file__), "csrc", "window_bwd.cu")) as f:
        lines = [x.split("//")[0].strip() for x in f]
    waits = [x for x in lines if "mbar_wait(" in x]
    assert len(waits) > 10
    for x in waits:
        ignored = re.fullmatch(r"((if|for) \(.*\) )?mbar_wait\(.*, &never, err\);", x)
        assert ignored or x.count("mbar_wait(") == x.count("__all_sync(0xffffffffu, mbar_wait("), x


def test_plan_takes_an_empty_free_list(lib):
    """No free pages: NULL with a capacity of 0 (PyTorch's pointer to no elements) gets past the checks of
    pointers and overlaps, to the last refusal here; with a capacity it is refused."""
    assert plan_args(lib, F=0, free=None, status=P + 2) == ALIGNMENT
    assert plan_args(lib, F=1, free=None, status=P + 2) == INVALID
    assert plan_args(lib, F=0, free=None, alias=("lens_out", "lens", 0)) == INVALID
    assert plan_args(lib, F=0, free=None, lens=None) == INVALID
    assert plan_args(lib, F=0, alias=("free", "slots", 1), status=P + 2) == ALIGNMENT  # (no elements overlap nothing)


def test_gradients_are_brought_to_aligned_rows():
    """What PyTorch may hand a backward: slices that start off a 16-byte boundary though contiguous (the
    gradient of a concatenation), expanded and transposed ones; all come out as the kernels read them."""
    x = torch.arange(2 * 3 * 5 * 64 + 8, dtype=torch.float32).bfloat16()
    odd = x[3:3 + 2 * 3 * 5 * 64].view(2, 3, 5, 64)
    assert odd.data_ptr() % 16 != 0 and odd.is_contiguous()
    even = x[:2 * 3 * 5 * 64].view(2, 3, 5, 64)
    one = x[1:65].view(1, 1, 1, 64)  # strides of dimensions of extent 1 are not read, the address is
    for t in (odd, even, one, even[:, :, :, :1].expand(2, 3, 5, 64), even[:, :1].expand(2, 3, 5, 64), even.transpose(1, 2),
              x[:2 * 3 * 5 * 64].view(2, 3, 64, 5).transpose(2, 3), x[:1].expand(2, 3, 5, 64)):
        y = lm._as_rows(t)
        assert torch.equal(y, t) and y.data_ptr() % 16 == 0 and y.stride(-1) == 1
        assert all(n == 1 or (s >= 64 and s % 8 == 0) for n, s in zip(y.shape[:-1], y.stride()))
    assert lm._as_rows(even) is even and lm._as_rows(even.transpose(1, 2)).data_ptr() == even.data_ptr()


def test_rope_table_under_a_default_device():
    """The speeds are written on the host, whatever device new tensors have by default."""
    want = bsf.RopeTable(64, scaling="yarn", factor=4.0, device="cpu")
    with torch.device("meta"):
        got = bsf.RopeTable(64, scaling="yarn", factor=4.0, device="cpu")
    assert got.turns.device.type == "cpu" and torch.equal(got.turns, want.turns) and got.mscale == want.mscale
