"""ep_swiglu and its gradient against binary64, on the GPU.

Tolerances (relative to the exact value unless said otherwise): exp(-g) is off by
(|g| + 2) 2^-23 (the rounded argument and one ulp of the instruction), 1 / (1 + e) by
no more than that and 2^-23; every further product by 2^-24; bf16 by 2^-8; E4M3 by 2^-4
of the value or 2^-10 of the block's scale.  Values below 2^-126 of gate * up may come
out as zero.  The checkpoint's codes are those of ep_quantize_fp8, bit for bit."""
import pytest
import torch

import combine_ep_layout_08_amd as ep
from tests import layer_ref as ref
from tests.gpu_util import needs_gpu, say

pytestmark = [pytest.mark.gpu, needs_gpu]


def _case(T, K, E, A, inter, empty, seed, spread=2.0, max_tokens=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    idx = ref.ids(T, K, E, gen, "cuda", empty)
    h = ep.Handle(max_tokens or T, K, E, A)
    h.layout(idx)
    gu = (torch.randn((h.capacity, 2 * inter), generator=gen, device="cuda") * spread).bfloat16()
    w = torch.rand(h.capacity, generator=gen, device="cuda")
    grad = torch.randn((h.capacity, inter), generator=gen, device="cuda").bfloat16()
    rows = ref.rows_of(h, idx)[0]
    # rows without a slot hold values that would spoil any sum
    gap = torch.ones(h.capacity, dtype=torch.bool, device="cuda")
    gap[rows] = False
    gu[gap], grad[gap], w[gap] = float("nan"), float("inf"), float("nan")
    return h, rows, gu, w, grad


CASES = [  # T, K, E, A, inter, empty slots
    (1, 1, 1, 1, 8, 0.0),
    (1, 8, 64, 1, 2048, 0.0),
    (33, 4, 16, 8, 136, 0.3),
    (64, 4, 16, 1, 256, 0.1),
    (100, 4, 16, 8, 640, 0.2),
    (128, 8, 256, 128, 512, 0.0),
    (5, 2, 4, 16, 4224, 0.5),
    (3, 2, 4, 1, 32768, 0.0),
    (700, 8, 32, 64, 1024, 0.0),
]


def _exact(gu, w):
    e = ref.swiglu(gu, w)
    g = gu.double().chunk(2, 1)[0].abs()
    tiny = (gu.double().chunk(2, 1)[1].abs() * g + 1.0) * 2.0 ** -125
    return e, e.abs() * (g + 6) * 2.0 ** -23 + tiny


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("T,K,E,A,inter,empty", CASES)
def test_forward_bf16(T, K, E, A, inter, empty, weighted):
    say("swiglu", T, K, E, A, inter, empty, weighted)
    h, rows, gu, w, _ = _case(T, K, E, A, inter, empty, T + inter)
    out = ref.poisoned((h.capacity, inter), torch.bfloat16)
    got, sf, saved, saved_sf = h.swiglu(gu, row_weights=w if weighted else None, out=out)
    assert got is out and sf is None and saved is None and saved_sf is None
    want, tol = _exact(gu[rows], w[rows] if weighted else None)
    ref.assert_close(out[rows], want, want.abs() * ref.BF16 + tol, "h")
    assert ref.untouched(out, rows)


@pytest.mark.parametrize("ckpt", ["f32", "ue8m0"])
@pytest.mark.parametrize("fmt", [None, "f32", "ue8m0"])
@pytest.mark.parametrize("T,K,E,A,inter,empty", [c for c in CASES if c[4] % 128 == 0])
def test_forward_eight_bits(T, K, E, A, inter, empty, fmt, ckpt):
    say("swiglu eight bits", T, K, E, A, inter, empty, fmt, ckpt)
    h, rows, gu, w, _ = _case(T, K, E, A, inter, empty, T + 2 * inter)
    cap = h.capacity
    packs = lambda c, f: ep.ep_sf_packs(c, 0 if f == "f32" else 1)  # noqa: E731
    dt = {"f32": torch.float32, "ue8m0": torch.int32}
    out = ref.poisoned((cap, inter), torch.bfloat16 if fmt is None else torch.uint8)
    out_sf = None if fmt is None else ref.poisoned((cap, packs(inter, fmt)), dt[fmt])
    saved = ref.poisoned((cap, 2 * inter), torch.uint8)
    saved_sf = ref.poisoned((cap, packs(2 * inter, ckpt)), dt[ckpt])
    h.swiglu(gu, row_weights=w, scale_format=fmt, out=out, out_sf=out_sf, checkpoint=ckpt,
             saved=saved, saved_sf=saved_sf)
    want, tol = _exact(gu[rows], w[rows])
    if fmt is None:
        ref.assert_close(out[rows], want, want.abs() * ref.BF16 + tol, "h")
    else:
        s = ref.scale_values(out_sf[rows], inter // 128)
        amax = want.abs().reshape(len(rows), -1, 128).amax(2)
        most = torch.clamp(amax, min=1e-12) / 448.0
        room = (tol.reshape(len(rows), -1, 128).amax(2) / 448.0) + most * 4 * ref.F32
        if fmt == "f32":
            ref.assert_close(s, most, room, "scales")
        else:       # the power of two above, unless the block's maximum is next to one
            low = torch.exp2(torch.ceil(torch.log2(most - room)))
            high = torch.exp2(torch.ceil(torch.log2(most + room)))
            assert bool(((s >= low) & (s <= high)).all())
        step = want.abs() * 2.0 ** -4 + s.repeat_interleave(128, 1) * 2.0 ** -10
        ref.assert_close(ref.code_values(out[rows], out_sf[rows]), want, step + tol, "codes")
        assert ref.untouched(out, rows) and ref.untouched(out_sf, rows)
    if len(rows):
        q, sf = ep.quantize_fp8(gu[rows].contiguous(), ckpt)
        assert torch.equal(saved[rows], q)
        assert torch.equal(saved_sf[rows].view(torch.int32), sf.view(torch.int32))
    assert ref.untouched(saved, rows) and ref.untouched(saved_sf, rows)


def test_strided_scales():
    """Column-major scales of h and a strided view for the checkpoint's."""
    h, rows, gu, _, grad = _case(40, 4, 8, 4, 384, 0.1, 5)
    want = h.swiglu(gu, scale_format="ue8m0", checkpoint="f32")
    wide = torch.zeros((h.capacity, 13), dtype=torch.float32, device="cuda")
    got = h.swiglu(gu, scale_format="ue8m0", checkpoint="f32", col_major_sf=True,
                   saved_sf=wide[:, 2:8])
    assert got[1].stride(0) == 1
    for a, b in zip(got, want):
        assert torch.equal(a[rows], b[rows])
    assert bool((wide[:, :2] == 0).all()) and bool((wide[:, 8:] == 0).all())
    a = h.swiglu_backward(grad, want[2], want[3])[0]
    b = h.swiglu_backward(grad, got[2], got[3])[0]
    assert torch.equal(a[rows], b[rows])


def test_extremes():
    """Gates far out on both sides, zeros, infinities and NaN stay in their elements."""
    inter = 128
    idx = torch.zeros((1, 1), dtype=torch.int64, device="cuda")
    h = ep.Handle(1, 1, 1, 1)
    h.layout(idx)
    gu = torch.ones((1, 2 * inter), device="cuda")
    vals = [0.0, -0.0, 100.0, -100.0, 3e38, -3e38, float("inf"), float("nan"), -88.0, 88.0, -1e-30]
    gu[0, :len(vals)] = torch.tensor(vals, device="cuda")
    gu = gu.bfloat16()
    out = h.swiglu(gu)[0].float()[0]
    want = ref.swiglu(gu)[0]
    assert bool(out[7].isnan()) and float(out[6]) == float("inf")
    assert float(out[3]) == 0.0 and float(out[5]) == 0.0
    fine = [i for i in range(inter) if i not in (6, 7)]
    ref.assert_close(out[fine], want[fine], want[fine].abs() * (ref.BF16 + 2.0 ** -16) + 2.0 ** -118,
                     "h")
    g = torch.ones((1, inter), device="cuda").bfloat16()
    gg = h.swiglu_backward(g, gu)[0].float()[0]
    assert float(gg[3]) == 0.0 and float(gg[5]) == 0.0          # slope far left
    assert float(gg[2]) == 1.0 and float(gg[4]) == 1.0          # and far right
    assert int(gg[:inter].isnan().sum()) == 2                   # the infinity's and the NaN's
    _, _, saved, sf = h.swiglu(gu, checkpoint="f32")
    assert int(saved[0, 7]) == 0x7F and int(saved[0, 6]) == 0x7F and bool(torch.isinf(sf[0, 0]))


def _grad_exact(gu, grad, w):
    g, u = gu.double().chunk(2, 1)
    gh = grad.double()
    s = torch.sigmoid(g)
    ww = torch.ones_like(g[:, :1]) if w is None else w.double()[:, None]
    slope = s * (1 + g * (1 - s))
    gg, gu_ = ww * gh * u * slope, ww * gh * g * s
    err = (g.abs() + 6) * 2.0 ** -23
    tiny = (1 + u.abs()) * (1 + g.abs()) * gh.abs() * 2.0 ** -124
    # the slope's two terms may cancel: its error is that of s (1 + |g|)
    size = (ww * gh * u).abs() * s * (1 + g.abs())
    whole = g * s * u
    return (torch.cat((gg, gu_), 1),
            torch.cat((gg.abs() * ref.BF16 + 2 * size * err + tiny,
                       gu_.abs() * (ref.BF16 + err) + tiny), 1),
            # a lane's chain of inter / 64 products, then the wave's and the block's sums
            (gh * whole).sum(1),
            ((gh * whole).abs() * (err + (g.shape[1] / 64 + 40) * ref.F32)).sum(1) + 1e-30,
            ww * whole, (ww * whole).abs() * (ref.BF16 + err) + tiny + 2.0 ** -120)


@pytest.mark.parametrize("saved_kind", ["bf16", "f32", "ue8m0"])
@pytest.mark.parametrize("T,K,E,A,inter,empty", CASES)
def test_backward(T, K, E, A, inter, empty, saved_kind):
    if saved_kind != "bf16" and inter % 128:
        pytest.skip("E4M3 rows come in blocks of 128 channels")
    say("swiglu gradient", T, K, E, A, inter, empty, saved_kind)
    h, rows, gu, w, grad = _case(T, K, E, A, inter, empty, T + 5 * inter)
    cap = h.capacity
    saved, sf, values = gu, None, gu
    if saved_kind != "bf16":
        _, _, saved, sf = h.swiglu(gu, checkpoint=saved_kind)
        values = torch.zeros((cap, 2 * inter), dtype=torch.float64, device="cuda")
        values[rows] = ref.code_values(saved[rows], sf[rows])
    ggu = ref.poisoned((cap, 2 * inter), torch.bfloat16)
    gw = ref.poisoned((cap,), torch.float32)
    again = ref.poisoned((cap, inter), torch.bfloat16)
    h.swiglu_backward(grad, saved, sf, row_weights=w, grad_gate_up=ggu, grad_row_weights=gw,
                      out=again)
    want, tol, want_w, tol_w, want_h, tol_h = _grad_exact(values[rows], grad[rows], w[rows])
    ref.assert_close(ggu[rows], want, tol, "grad_gate_up")
    ref.assert_close(gw[rows], want_w, tol_w, "grad_row_weights")
    ref.assert_close(again[rows], want_h, tol_h, "h again")
    for t in (ggu, gw[:, None], again):
        assert ref.untouched(t, rows)
    # without weights, and only what is asked for
    plain, none_w, none_h = h.swiglu_backward(grad, saved, sf)
    assert none_w is None and none_h is None
    want, tol, *_ = _grad_exact(values[rows], grad[rows], None)
    ref.assert_close(plain[rows], want, tol, "grad_gate_up, no weights")


def test_backward_in_place():
    """grad_gate_up over a bf16 gate_up, h over grad_h."""
    h, rows, gu, w, grad = _case(60, 4, 8, 4, 520, 0.1, 6)
    want = h.swiglu_backward(grad, gu, row_weights=w, want_grad_weights=True, want_h=True)
    got = h.swiglu_backward(grad, gu, row_weights=w, want_grad_weights=True, grad_gate_up=gu,
                            out=grad)
    assert got[0] is gu and got[2] is grad
    for a, b in zip(got, want):
        assert torch.equal(a[rows], b[rows])


def test_gradient_against_differences():
    h, rows, gu, w, grad = _case(6, 2, 4, 2, 128, 0.0, 7, spread=1.0)
    ggu, gw, _ = h.swiglu_backward(grad, gu, row_weights=w, want_grad_weights=True)
    x, g, ww = gu[rows].double(), grad[rows].double(), w[rows].double()
    gen = torch.Generator(device="cuda").manual_seed(1)

    def loss(x, ww):
        return float((ref.swiglu(x) * ww[:, None] * g).sum())

    for _ in range(4):
        d = torch.randn(x.shape, generator=gen, device="cuda", dtype=torch.float64)
        e = torch.randn(ww.shape, generator=gen, device="cuda", dtype=torch.float64)
        s = 1e-5
        dx = (loss(x + s * d, ww) - loss(x - s * d, ww)) / (2 * s)
        dw = (loss(x, ww + s * e) - loss(x, ww - s * e)) / (2 * s)
        gx = ggu[rows].double() * d
        assert abs(float(gx.sum()) - dx) <= float(gx.abs().sum()) * ref.BF16 * 2 + 1e-6
        ge = gw[rows].double() * e
        assert abs(float(ge.sum()) - dw) <= float(ge.abs().sum()) * 1e-5 + 1e-6


def test_void_layout_writes_nothing():
    """After a capacity error on the handle the calls leave every buffer as it was."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    idx = ref.ids(32, 4, 8, gen, "cuda")
    h = ep.Handle(32, 4, 8, 1, capacity=64)              # 128 rows are needed
    h.layout(idx)
    assert h.read_counts(check=False)["status"] == ep.EP_ERR_CAPACITY
    gu = torch.ones((64, 256), device="cuda").bfloat16()
    out = ref.poisoned((64, 128), torch.bfloat16)
    saved, sf = ref.poisoned((64, 256), torch.uint8), ref.poisoned((64, 2), torch.float32)
    h.swiglu(gu, out=out, checkpoint="f32", saved=saved, saved_sf=sf)
    ggu, gw = ref.poisoned((64, 256), torch.bfloat16), ref.poisoned((64, 1), torch.float32)
    h.swiglu_backward(gu[:, :128].contiguous(), gu, grad_gate_up=ggu, grad_row_weights=gw.view(-1))
    for t in (out, saved, sf, ggu, gw):
        assert ref.untouched(t, [])


def test_no_tokens():
    h = ep.Handle(4, 2, 4, 8)
    h.layout(torch.empty((0, 2), dtype=torch.int64, device="cuda"))
    out = ref.poisoned((h.capacity, 128), torch.bfloat16)
    h.swiglu(torch.zeros((h.capacity, 256), device="cuda").bfloat16(), out=out)
    assert ref.untouched(out, [])


@pytest.mark.parametrize("fmt", ["f32", "ue8m0"])
def test_row_weights_of_any_size(fmt):
    """Weights above one, below zero, zero and not finite: each in its own row, with
    and without a checkpoint beside the E4M3 rows."""
    h, rows, gu, w, _ = _case(9, 1, 1, 1, 256, 0.0, 8)
    w[:] = torch.tensor([3.5, -2.0, 0.0, 1e30, 1.0, -1.0, float("inf"), float("nan"), 0.3],
                        device="cuda")[torch.argsort(rows)]
    a = h.swiglu(gu, row_weights=w, scale_format=fmt)
    b = h.swiglu(gu, row_weights=w, scale_format=fmt, checkpoint="f32")
    assert torch.equal(a[0], b[0]) and torch.equal(a[1].view(torch.int32), b[1].view(torch.int32))
    fine = torch.isfinite(w)
    want, tol = _exact(gu, w)
    s = ref.scale_values(a[1], 2).repeat_interleave(128, 1)
    got = ref.code_values(a[0], a[1])
    tol = want.abs() * 2.0 ** -4 + s * 2.0 ** -10 + tol * (1 + w.double().abs()[:, None])
    ref.assert_close(got[fine], want[fine], tol[fine], "h")
    assert bool((a[0][w.isnan()] == 0x7F).all()) and bool((a[0][w.isinf()] == 0x7F).all())


def test_products_that_overflow():
    """Finite factors whose product is not: the recipe's codes for an infinity, the other
    values of its block 0, other blocks as ever."""
    h = ep.Handle(1, 1, 1, 1)
    h.layout(torch.zeros((1, 1), dtype=torch.int64, device="cuda"))
    gu = torch.ones((1, 512), device="cuda").bfloat16()
    gu[0, 3] = gu[0, 256 + 3] = 3e38
    for ckpt in (None, "f32"):
        q, sf, _, _ = h.swiglu(gu, scale_format="f32", checkpoint=ckpt)
        assert int(q[0, 3]) == 0x7F and bool(torch.isinf(sf[0, 0]))
        assert bool((q[0, :3] == 0).all()) and bool((q[0, 4:128] == 0).all())
        assert bool((q[0, 128:] == 0x7E).all())


def test_offsets_past_32_bits():
    """Rows behind the first 4 GiB of gate_up, and of its checkpoint."""
    T, inter = 150_000, 16384
    h = ep.Handle(T, 1, 1, 1)
    h.layout(torch.zeros((T, 1), dtype=torch.int32, device="cuda"))
    gen = torch.Generator(device="cuda").manual_seed(3)
    gu = torch.ones((T, 2 * inter), dtype=torch.bfloat16, device="cuda")
    gu[-20:] = torch.randn((20, 2 * inter), generator=gen, device="cuda").bfloat16()
    say("swiglu offsets", T, inter)
    out, _, saved, sf = h.swiglu(gu, checkpoint="ue8m0")
    want, tol = _exact(gu[-20:], None)
    ref.assert_close(out[-20:], want, want.abs() * ref.BF16 + tol, "h")
    q, s = ep.quantize_fp8(gu[-20:].contiguous(), "ue8m0")
    assert torch.equal(saved[-20:], q) and torch.equal(sf[-20:], s)
    ggu, _, again = h.swiglu_backward(out, saved, sf, want_h=True)
    want, tol, _, _, want_h, tol_h = _grad_exact(ref.code_values(q, s), out[-20:], None)
    ref.assert_close(ggu[-20:], want, tol, "grad_gate_up")
    ref.assert_close(again[-20:], want_h, tol_h, "h again")


def test_graph():
    """Forward with a checkpoint and backward from it, captured; every replay on new
    rows and routing equals the eager calls."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    T, K, E, inter = 24, 2, 8, 256
    idx = ref.ids(T, K, E, gen, "cuda")
    h = ep.Handle(T, K, E, 4)
    lay = h.bind_layout(idx)
    lay()
    gu = torch.randn((h.capacity, 2 * inter), generator=gen, device="cuda").bfloat16()
    grad = torch.randn((h.capacity, inter), generator=gen, device="cuda").bfloat16()
    w = torch.rand(h.capacity, generator=gen, device="cuda")

    def step():
        lay()
        a = h.swiglu(gu, row_weights=w, scale_format="ue8m0", checkpoint="f32")
        return (*a, *h.swiglu_backward(grad, a[2], a[3], row_weights=w, want_grad_weights=True,
                                       want_h=True))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        idx.copy_(ref.ids(T, K, E, gen, "cuda", 0.2))
        gu.copy_(torch.randn(gu.shape, generator=gen, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        want = step()
        rows = ref.rows_of(h, idx)[0]
        for a, b in zip(kept, want):
            assert torch.equal(a[rows].view(torch.uint8), b[rows].view(torch.uint8))


def test_more_slots_than_waves():
    """More slots than the waves of one launch (2^24): the waves walk the rest."""
    T, inter = (1 << 24) + 1000, 8
    gen = torch.Generator(device="cuda").manual_seed(41)
    idx = torch.randint(0, 3, (T, 1), generator=gen, device="cuda", dtype=torch.int32)
    h = ep.Handle(T, 1, 3, 1)
    say("swiglu slots", T, inter)
    h.layout(idx)
    assert h.read_counts()["num_expanded"] == T
    rows = h.dst_slot.reshape(-1).long()
    gu = torch.randn((T, 2 * inter), generator=gen, device="cuda").bfloat16()
    w = torch.rand(T, generator=gen, device="cuda")
    out = ref.poisoned((T, inter), torch.bfloat16)
    h.swiglu(gu, row_weights=w, out=out)
    for part in (rows[:1000], rows[(1 << 24) - 1000:]):
        want, tol = _exact(gu[part], w[part])
        ref.assert_close(out[part], want, want.abs() * ref.BF16 + tol, "h")
    g = torch.randn((T, inter), generator=gen, device="cuda").bfloat16()
    ggu = ref.poisoned((T, 2 * inter), torch.bfloat16)
    gw = ref.poisoned((T,), torch.float32)
    again = ref.poisoned((T, inter), torch.bfloat16)
    h.swiglu_backward(g, gu, row_weights=w, grad_gate_up=ggu, grad_row_weights=gw, out=again)
    ok = torch.isfinite(gw) & (gw.view(torch.int32) != 0x5A5A5A5A)
    assert bool(ok.all()) and torch.equal(again.view(torch.int16), out.view(torch.int16))
    part = rows[(1 << 24) - 1000:]
    a, b = gu[part].double().chunk(2, 1)
    s = torch.sigmoid(a)
    want = torch.cat((b * s * (1.0 + a * (1.0 - s)), a * s), 1) * g[part].double().repeat(1, 2)
    want *= w[part].double()[:, None]
    # as in the forward pass; the slope's two terms may cancel, so relative to their sizes
    size = torch.cat((b.abs() * s * (1.0 + a.abs()), (a * s).abs()), 1) * g[part].double().abs().repeat(1, 2)
    ref.assert_close(ggu[part], want, want.abs() * ref.BF16 + size * (a.abs().repeat(1, 2) + 8) *
                     2.0 ** -23, "gradient")
