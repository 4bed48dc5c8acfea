"""ep_quantize_i8, ep_expert_i8, ep_expert_ffn and its gradients against binary64, on
the GPU.

Tolerances.  A rounding to bf16 is off by at most 2^-8 of the value, one to binary32 by 2^-24.
A bf16 product of K channels adds up K products in binary32: at most K roundings inside the matrix
instructions and one for each accumulation of 32, each of a partial sum that the sum of
|x w| bounds.  int8 sums are exact; turned into binary32 and scaled twice they are rounded three
times.  sigmoid(g) has its argument's rounding (|g| 2^-24, twice with the constant's) and two
hardware functions within 2^-23, so silu's relative error is at most (6 + 2 |g|) 2^-24, and an
error d of the gate moves silu by at most 1.1 |d|.  Each step is checked from what the step before
it left in memory, so no rounding counts twice.  Norms are held tighter than elements:
errors of many sums do not all point one way."""
import pytest
import torch

import combine_ep_layout_08_amd as ep
from tests import layer_ref as ref
from tests.gpu_util import needs_gpu, say

pytestmark = [pytest.mark.gpu, needs_gpu]
BF16, F32 = ref.BF16, ref.F32
TINY = 1e-37             # what flushing the quotient of a far negative gate leaves out


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(shape, gen, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).bfloat16()


def _laid_out(T, K, E, A, gen, empty=0.0, dtype=torch.int64):
    idx = ref.ids(T, K, E, gen, "cuda", empty).to(dtype)
    h = ep.Handle(T, K, E, A)
    h.layout(idx)
    return h, idx


def _spoil(x, rows, value=float("nan")):
    """What no slot holds would spoil any sum that it got into."""
    gap = torch.ones(x.shape[0], dtype=torch.bool, device=x.device)
    gap[rows] = False
    x[gap] = value
    return x


def _norm_close(got, want, bound, what):
    n = float(want.norm())
    if want.numel() > 64 and n > 0:
        off = float((got.double() - want).norm())
        assert off <= bound * n, f"{what}: {off / n} of the norm"


def _sum_tol(K):
    return (K + K // 32 + 1) * F32


# ---------------------------------------------------------------- quantiser

def _codes64(x):
    """The recipe, divisions in binary32 as it says."""
    f = x.float()
    s = torch.clamp(f.abs().amax(1), min=1e-12)
    s = s / torch.full_like(s, 127.0)
    return torch.round(f / s[:, None]).to(torch.int8), s


@pytest.mark.parametrize("T,C", [(1, 16), (1, 7168), (3, 48), (5, 1024), (7, 1040), (64, 2048),
                                 (33, 4096), (9, 4112), (17, 8192), (2, 8208), (3, 32768)])
def test_quantiser(T, C):
    say("quantize_i8", T, C)
    gen = _gen(T + C)
    x = _randn((T, C), gen)
    x[0, C // 2] = 40.0
    q, s = ep.quantize_i8(x)
    wq, ws = _codes64(x)
    assert torch.equal(s, ws) and torch.equal(q, wq)
    # and the recipe against binary64: half a step, and the quotient's rounding
    exact = x.double() / (x.double().abs().amax(1, keepdim=True) / 127.0)
    assert float((q.double() - exact).abs().max()) <= 0.5 + 127 * 3 * F32


def test_quantiser_every_magnitude():
    """Rows over bf16's whole range of exponents, ties among the quotients, zeros."""
    rows = []
    for e in range(-133, 127, 4):
        v = torch.arange(256, dtype=torch.float64) - 127.5
        rows.append(v * 2.0 ** (e - 8 if e > -120 else e))
    x = torch.stack(rows).float().bfloat16().cuda().contiguous()
    x[3] = 0.0
    x[4, :128] = 0.0
    q, s = ep.quantize_i8(x)
    wq, ws = _codes64(x)
    assert torch.equal(s, ws) and torch.equal(q, wq)
    assert bool((q[3] == 0).all()) and float(s[3]) > 0


def test_quantiser_ties_to_even():
    x = torch.zeros((1, 16), device="cuda")
    x[0, :6] = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5, -2.5])
    q, s = ep.quantize_i8(x.bfloat16())
    assert float(s[0]) == 1.0 and q[0, :6].tolist() == [127, 0, 2, 2, 0, -2]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_quantiser_marks_rows_that_have_no_codes(bad):
    x = _randn((4, 256), _gen(1))
    want = ep.quantize_i8(x)
    x[2, 77] = bad
    q, s = ep.quantize_i8(x)
    keep = [0, 1, 3]
    assert torch.equal(q[keep], want[0][keep]) and torch.equal(s[keep], want[1][keep])
    assert bool(s[2].isnan()) and bool((q[2] == 0).all())


@pytest.mark.parametrize("T,K,E,A,C,empty", [(1, 1, 1, 1, 16, 0.0), (100, 4, 16, 8, 640, 0.2),
                                             (33, 2, 5, 64, 2048, 0.1), (7, 3, 6, 1, 1040, 0.3)])
def test_quantiser_of_expert_rows(T, K, E, A, C, empty):
    say("quantize_i8 rows", T, K, E, A, C, empty)
    gen = _gen(T * C)
    h, idx = _laid_out(T, K, E, A, gen, empty)
    rows = ref.rows_of(h, idx)[0]
    x = _randn((h.capacity, C), gen)
    q, s = ref.poisoned((h.capacity, C), torch.int8), ref.poisoned((h.capacity,), torch.float32)
    assert h.quantize_i8(x, out_q=q, out_scale=s) == (q, s)
    wq, ws = _codes64(x[rows])
    assert torch.equal(q[rows], wq) and torch.equal(s[rows], ws)
    assert ref.untouched(q, rows) and ref.untouched(s[:, None], rows)


# ---------------------------------------------------------------- int8 products

def _i8_case(h, E, rows_n, k, n, gen):
    x = torch.randint(-127, 128, (rows_n, k), generator=gen, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (E, n, k), generator=gen, device="cuda", dtype=torch.int8)
    xs = torch.rand(rows_n, generator=gen, device="cuda") * 0.02 + 1e-3
    ws = (torch.rand((E, n), generator=gen, device="cuda") + 0.1) * k ** -0.5 * 0.02
    return x, xs, w, ws


def _silu(g):
    return g * torch.sigmoid(g)


def _check_i8(h, idx, x, xs, w, ws, gated, rw, out, token_rows, what):
    rows, expert, token = ref.rows_of(h, idx)
    for e in torch.unique(expert).tolist():
        mine = expert == e
        src = token[mine] if token_rows else rows[mine]
        v = (x[src].double() @ w[e].double().t()) * xs[src].double()[:, None] * ws[e].double()
        tol = v.abs() * 4 * F32
        if gated:
            g, u = v.chunk(2, 1)
            dg, du = tol.chunk(2, 1)
            f = 1.0 if rw is None else rw[rows[mine]].double()[:, None]
            v = _silu(g) * u * f
            tol = (1.1 * dg * u.abs() + _silu(g).abs() * du) * f + \
                v.abs() * (10 + 2 * g.abs()) * F32 + TINY * u.abs()
        tol = tol + v.abs() * BF16 + 1e-38
        ref.assert_close(out[rows[mine]], v, tol, f"{what}, expert {e}")
        _norm_close(out[rows[mine]], v, BF16, what)
    assert ref.untouched(out, rows)


I8_CASES = [  # T, K, E, A, k, n, gated, weights, token rows, empty
    (1, 1, 1, 1, 16, 16, False, False, False, 0.0),
    (1, 1, 1, 1, 16, 16, True, True, True, 0.0),
    (1, 8, 64, 1, 7168, 512, True, False, True, 0.0),
    (1, 8, 16, 1, 2048, 264, False, False, False, 0.0),
    (2, 2, 5, 1, 144, 24, False, False, True, 0.0),
    (7, 3, 6, 8, 400, 48, True, True, False, 0.2),
    (16, 1, 1, 1, 640, 136, False, False, False, 0.0),
    (17, 1, 1, 4, 896, 272, True, False, True, 0.0),
    (64, 4, 16, 128, 256, 520, False, False, False, 0.1),
    (33, 2, 2, 1, 528, 104, False, False, True, 0.1),
    (100, 8, 8, 1, 768, 96, True, True, False, 0.0),
    (130, 2, 2, 1, 272, 8, False, False, True, 0.2),
    (200, 2, 2, 64, 1040, 512, True, True, False, 0.1),
    (300, 1, 1, 1, 384, 784, False, False, False, 0.0),
    (513, 2, 3, 16, 320, 528, True, False, True, 0.0),
    (600, 3, 4, 8, 128, 1032, False, False, False, 0.1),
    (96, 8, 300, 8, 256, 64, False, False, False, 0.1),
    (3, 2, 1000, 1, 128, 16, True, True, True, 0.0),
    (5, 2, 4, 1, 32768, 32, False, False, False, 0.0),
    # tiles of 32 rows, of 64, of 256 (more outputs fill the card), and weights of more than 64 MB
    # read past the caches in tiles of 16, 32 and 64 rows
    (40, 4, 16, 1, 80, 4112, False, False, True, 0.1),
    (40, 4, 16, 1, 80, 4112, True, True, False, 0.1),
    (130, 4, 16, 8, 144, 4104, False, False, False, 0.1),
    (130, 4, 16, 1, 144, 4112, True, False, True, 0.0),
    (700, 2, 3, 8, 208, 9528, False, False, True, 0.0),
    (700, 2, 3, 1, 336, 9552, True, True, False, 0.1),
    (3, 2, 4, 1, 5136, 4096, False, False, True, 0.0),
    (20, 4, 8, 1, 2064, 8208, True, True, True, 0.1),
    (60, 4, 8, 1, 1040, 8200, False, False, False, 0.1),
]


@pytest.mark.parametrize("T,K,E,A,k,n,gated,weights,token_rows,empty", I8_CASES)
def test_i8_product(T, K, E, A, k, n, gated, weights, token_rows, empty):
    say("expert_i8", T, K, E, A, k, n, gated, weights, token_rows, empty)
    gen = _gen(T + k + n)
    h, idx = _laid_out(T, K, E, A, gen, empty)
    x, xs, w, ws = _i8_case(h, E, T if token_rows else h.capacity, k, n, gen)
    if not token_rows:
        _spoil(xs, ref.rows_of(h, idx)[0])
    rw = torch.rand(h.capacity, generator=gen, device="cuda") if weights else None
    if weights:
        _spoil(rw, ref.rows_of(h, idx)[0])
    cols = n // 2 if gated else n
    out = ref.poisoned((h.capacity, cols), torch.bfloat16)
    got = h.expert_i8(x, xs, w, ws, gated=gated, row_weights=rw, token_rows=token_rows, out=out)
    assert got is out
    _check_i8(h, idx, x, xs, w, ws, gated, rw, out, token_rows, "int8")
    again = ref.poisoned((h.capacity, cols), torch.bfloat16)
    h.expert_i8(x, xs, w, ws, gated=gated, row_weights=rw, token_rows=token_rows, out=again)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("T", [1, 20, 100, 400])
def test_i8_every_channel_and_extreme_sums(T):
    """One-hot rows read single weights back; rows of -127 and weights of -128 reach the largest
    sums (exact: scales are powers of two and bf16 holds the codes)."""
    k, n = 272, 144
    w = (torch.arange(n * k, device="cuda").reshape(1, n, k) * 7 % 256 - 128).to(torch.int8)
    ws = torch.exp2((torch.arange(n, device="cuda") % 5).float())[None].contiguous()
    x = torch.zeros((T, k), dtype=torch.int8, device="cuda")
    at = torch.arange(T, device="cuda") * 13 % k
    x[torch.arange(T, device="cuda"), at] = 1
    xs = torch.full((T,), 0.5, device="cuda")
    h = ep.Handle(T, 1, 1, 1)
    h.layout(torch.zeros((T, 1), dtype=torch.int64, device="cuda"))
    y = h.expert_i8(x, xs, w, ws)
    want = w[0].double()[:, at].t() * ws[0].double() * 0.5
    assert torch.equal(y.double(), want)
    big = 32768
    w = torch.full((1, 16, big), -128, dtype=torch.int8, device="cuda")
    x = torch.full((T, big), -128, dtype=torch.int8, device="cuda")
    y = h.expert_i8(x, xs, w, torch.ones((1, 16), device="cuda"))
    assert bool((y.double() == big * 16384 * 0.5).all())


def test_i8_rows_without_codes_are_nan_and_alone():
    gen = _gen(8)
    h, idx = _laid_out(40, 2, 4, 1, gen)
    x = _randn((40, 256), gen)
    w, ws = ep.quantize_i8(_randn((4 * 64, 256), gen))
    w, ws = w.reshape(4, 64, 256), ws.reshape(4, 64)
    want = h.expert_i8(*ep.quantize_i8(x), w, ws, token_rows=True)
    x[7, 3] = float("inf")
    got = h.expert_i8(*ep.quantize_i8(x), w, ws, token_rows=True)
    rows, _, token = ref.rows_of(h, idx)
    bad = rows[token == 7]
    assert bool(got[bad].isnan().all())
    assert torch.equal(got[rows[token != 7]], want[rows[token != 7]])


# ---------------------------------------------------------------- the block

class Block:
    def __init__(self, T, K, E, A, H, I, token_rows, weights, empty, seed, dtype=torch.int64):
        gen = _gen(seed)
        self.h, self.idx = _laid_out(T, K, E, A, gen, empty, dtype)
        self.rows, self.expert, self.token = ref.rows_of(self.h, self.idx)
        cap = self.h.capacity
        self.E, self.H, self.I, self.token_rows = E, H, I, token_rows
        self.x = _randn((T if token_rows else cap, H), gen)
        self.w13 = _randn((E, 2 * I, H), gen, 1.5 * H ** -0.5)
        self.w2 = _randn((E, H, I), gen, I ** -0.5)
        self.rw = torch.rand(cap, generator=gen, device="cuda") if weights else None
        self.grad = _randn((cap, H), gen, 0.1)
        if not token_rows:
            _spoil(self.x, self.rows)
        if weights:
            _spoil(self.rw, self.rows)
        _spoil(self.grad, self.rows)

    def segments(self):
        for e in range(self.E):
            mine = self.expert == e
            rows = self.rows[mine]
            yield e, rows, self.token[mine] if self.token_rows else rows

    def weight(self, rows):
        return 1.0 if self.rw is None else self.rw[rows].double()[:, None]

    def forward(self, saved=True, **more):
        cap = self.h.capacity
        h = ref.poisoned((cap, self.I), torch.bfloat16)
        gu = ref.poisoned((cap, 2 * self.I), torch.bfloat16) if saved else None
        y = ref.poisoned((cap, self.H), torch.bfloat16)
        got = self.h.expert_ffn(self.x, self.w13, self.w2, row_weights=self.rw,
                                token_rows=self.token_rows, out_h=h, saved=gu, out=y)
        assert got[0] is y and got[1] is h and got[2] is gu
        return y, h, gu

    def check_forward(self, y, h, gu):
        for e, rows, src in self.segments():
            if not rows.numel():
                continue
            x, w = self.x[src].double(), self.w13[e].double()
            v = x @ w.t()
            d = (x.abs() @ w.abs().t()) * _sum_tol(self.H)
            if gu is not None:
                ref.assert_close(gu[rows], v, d + v.abs() * BF16 + 1e-38, f"gate_up {e}")
                _norm_close(gu[rows], v, BF16, "gate_up")
            (g, u), (dg, du), f = v.chunk(2, 1), d.chunk(2, 1), self.weight(rows)
            want = _silu(g) * u * f
            tol = (1.1 * dg * u.abs() + _silu(g).abs() * du) * f + TINY * u.abs() + \
                want.abs() * (BF16 + (10 + 2 * g.abs()) * F32) + 1e-38
            ref.assert_close(h[rows], want, tol, f"h {e}")
            _norm_close(h[rows], want, BF16, "h")
            hk, w2 = h[rows].double(), self.w2[e].double()
            want = hk @ w2.t()
            tol = (hk.abs() @ w2.abs().t()) * _sum_tol(self.I) + want.abs() * BF16 + 1e-38
            ref.assert_close(y[rows], want, tol, f"y {e}")
            _norm_close(y[rows], want, BF16, "y")
        for t in (y, h, gu):
            assert t is None or ref.untouched(t, self.rows)

    def backward(self, saved, h, dtype=torch.bfloat16, remake=False, alias=False, **more):
        cap = self.h.capacity
        gx = ref.poisoned((cap, self.H), torch.bfloat16)
        ggu = saved if alias else ref.poisoned((cap, 2 * self.I), torch.bfloat16)
        grw = ref.poisoned((cap,), torch.float32) if self.rw is not None else None
        g13 = ref.poisoned(tuple(self.w13.shape), dtype)
        g2 = ref.poisoned(tuple(self.w2.shape), dtype)
        if remake:
            h = ref.poisoned((cap, self.I), torch.bfloat16)
        got = self.h.expert_ffn_backward(
            self.grad, self.x, self.w13, self.w2, saved, h, row_weights=self.rw,
            token_rows=self.token_rows, remake_h=remake, grad_gate_up=ggu, grad_x=gx, grad_w13=g13,
            grad_w2=g2, grad_row_weights=grw, **more)
        assert [a is b for a, b in zip(got, (gx, g13, g2, grw, ggu))] == [True] * 5
        return gx, g13, g2, grw, ggu, h

    def check_backward(self, saved, given_h, out, remake):
        gx, g13, g2, grw, ggu, h = out
        I, low = self.I, BF16 if g13.dtype == torch.bfloat16 else F32
        for e, rows, src in self.segments():
            gy, w2 = self.grad[rows].double(), self.w2[e].double()
            g, u = saved[rows].double().chunk(2, 1)
            gh = gy @ w2
            d = (gy.abs() @ w2.abs()) * _sum_tol(self.H)
            s, f = torch.sigmoid(g), self.weight(rows)
            slope = s * (1 + g * (1 - s))
            whole = g * s * u
            # the slope's terms are added up: their own roundings, not the sum's
            dslope = s * (1 + g.abs() * (1 - s)) * (12 + 4 * g.abs()) * F32
            want = torch.cat((f * gh * u * slope, f * gh * g * s), 1)
            tol = torch.cat((f * u.abs() * (d * slope.abs() + gh.abs() * dslope),
                             f * (d * (g * s).abs())), 1)
            tol = tol + want.abs() * (BF16 + 16 * F32) + \
                torch.cat((g, g), 1).abs() * want.abs() * 4 * F32 + TINY
            if rows.numel():
                ref.assert_close(ggu[rows], want, tol, f"grad gate_up {e}")
                _norm_close(ggu[rows], want, BF16, "grad gate_up")
            if grw is not None and rows.numel():
                want = (gh * whole).sum(1)
                tol = (whole.abs() * d).sum(1) + \
                    ((gh * whole).abs() * (10 + 2 * g.abs())).sum(1) * F32 + \
                    (gh * whole).abs().sum(1) * (I + 8) * F32 + TINY
                ref.assert_close(grw[rows], want, tol, f"grad row weights {e}")
            if remake and rows.numel():
                want = whole * f
                ref.assert_close(h[rows], want, want.abs() * (BF16 + (10 + 2 * g.abs()) * F32) +
                                 TINY * u.abs() + 1e-38, f"h again {e}")
            kept = h if remake else given_h
            gk, w13 = ggu[rows].double(), self.w13[e].double()
            if rows.numel():
                want = gk @ w13
                ref.assert_close(gx[rows], want, (gk.abs() @ w13.abs()) * _sum_tol(2 * I) +
                                 want.abs() * BF16 + 1e-38, f"grad x {e}")
                _norm_close(gx[rows], want, BF16, "grad x")
            n = rows.numel()
            for name, got, p, q in (("w13", g13, gk, self.x[src].double()),
                                    ("w2", g2, gy, kept[rows].double())):
                want = p.t() @ q
                tol = (p.abs().t() @ q.abs()) * _sum_tol(n) + want.abs() * low + 1e-38
                ref.assert_close(got[e], want, tol, f"grad {name} {e}")
                _norm_close(got[e], want, max(low, 1e-5), name)
        for t in (gx, ggu if ggu is not saved else None, h if remake else None,
                  None if grw is None else grw[:, None]):
            assert t is None or ref.untouched(t, self.rows)


FFN_CASES = [  # T, K, E, A, H, I, token rows, weights, empty
    (1, 1, 1, 1, 8, 8, False, False, 0.0),
    (1, 1, 1, 1, 16, 8, True, True, 0.0),
    (1, 8, 64, 1, 1024, 264, True, True, 0.0),
    (3, 2, 5, 1, 72, 40, False, True, 0.0),
    (7, 3, 6, 8, 200, 136, True, False, 0.2),
    (17, 1, 1, 4, 136, 256, False, True, 0.0),
    (64, 4, 16, 128, 264, 128, False, True, 0.1),
    (100, 4, 16, 8, 648, 360, False, True, 0.2),
    (33, 2, 2, 1, 520, 104, True, True, 0.1),
    (130, 2, 2, 1, 272, 320, False, False, 0.2),
    (300, 1, 1, 16, 264, 392, True, True, 0.0),
    (520, 2, 3, 8, 384, 144, False, True, 0.1),
    (600, 3, 4, 1, 136, 264, True, False, 0.0),
    (40, 4, 300, 2, 64, 24, False, True, 0.1),
    # tiles of 32, 64 and 256 rows, for one of the products each; large tiles of the weights' gradients;
    # weights of more than 64 MB, read past the caches
    (40, 4, 16, 1, 72, 2056, True, True, 0.1),
    (130, 4, 16, 8, 4104, 40, False, True, 0.1),
    (130, 4, 16, 1, 88, 2064, False, False, 0.0),
    (700, 2, 3, 8, 72, 8200, False, True, 0.1),
    (700, 2, 3, 1, 9528, 40, True, False, 0.0),
    (3, 2, 4, 1, 2056, 4104, True, True, 0.0),
    (30, 4, 8, 1, 1032, 4104, False, True, 0.1),
    (60, 4, 8, 1, 8200, 520, True, False, 0.1),
]


@pytest.mark.parametrize("T,K,E,A,H,I,token_rows,weights,empty", FFN_CASES)
def test_block(T, K, E, A, H, I, token_rows, weights, empty):
    say("ffn", T, K, E, A, H, I, token_rows, weights, empty)
    b = Block(T, K, E, A, H, I, token_rows, weights, empty, T + H + I)
    out = b.forward()
    b.check_forward(*out)
    again = b.forward(saved=False)
    for p, q in zip(again[:2], out[:2]):
        assert torch.equal(p.view(torch.int16), q.view(torch.int16))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K,E,A,H,I,token_rows,weights,empty", FFN_CASES)
def test_block_gradients(T, K, E, A, H, I, token_rows, weights, empty, dtype):
    say("ffn gradients", T, K, E, A, H, I, token_rows, weights, empty, dtype)
    b = Block(T, K, E, A, H, I, token_rows, weights, empty, T + H + I)
    y, h, saved = b.forward()
    remake = dtype == torch.float32
    _spoil(saved, b.rows)
    _spoil(h, b.rows)
    out = b.backward(saved, h, dtype, remake)
    b.check_backward(saved, h, out, remake)
    again = b.backward(saved.clone(), h, dtype, remake)
    for p, q in zip(again, out):
        assert p is None or torch.equal(p.view(torch.uint8), q.view(torch.uint8))


def test_gradients_over_the_saved_rows():
    """grad_gate_up written over `saved` gives the same as into a buffer of its own."""
    b = Block(60, 3, 4, 4, 264, 136, False, True, 0.1, 3)
    y, h, saved = b.forward()
    want = b.backward(saved.clone(), h)
    over = saved.clone()
    got = b.backward(over, h, alias=True)
    for p, q in zip(got[:4], want[:4]):
        assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))
    assert torch.equal(over[b.rows], want[4][b.rows])


def test_what_is_not_wanted_stays_away():
    b = Block(50, 2, 4, 1, 136, 72, True, True, 0.1, 4)
    y, h, saved = b.forward()
    all_of = b.backward(saved, h)
    none = b.h.expert_ffn_backward(b.grad, None, b.w13, b.w2, saved, row_weights=b.rw,
                                   token_rows=True, want_grad_x=False, want_grad_w=False)
    assert none[:4] == (None, None, None, None)
    assert torch.equal(none[4][b.rows], all_of[4][b.rows])
    some = b.h.expert_ffn_backward(b.grad, b.x, b.w13, b.w2, saved, h, row_weights=b.rw,
                                   token_rows=True, want_grad_x=False)
    assert some[0] is None and torch.equal(some[1], all_of[1]) and torch.equal(some[2], all_of[2])
    only = b.h.expert_ffn(b.x, b.w13, None, row_weights=b.rw, token_rows=True)
    assert only[0] is None and only[2] is None and torch.equal(only[1][b.rows], h[b.rows])


def test_gradients_against_differences():
    """Along a direction of x, of each weight and of the row weights, the gradients against
    central differences of the block in binary64.  The kernel's roundings to bf16 (gate_up, its
    gradient, the results) move a product with a random direction by less than 2^-7 of what
    the norms allow."""
    T, K, E, H, I = 24, 2, 3, 64, 40
    b = Block(T, K, E, 1, H, I, False, True, 0.0, 5)
    gen = _gen(6)

    def loss(x, w13, w2, rw):
        total = torch.zeros((), dtype=torch.float64, device="cuda")
        for e, rows, _ in b.segments():
            g, u = (x[rows] @ w13[e].t()).chunk(2, 1)
            y = (_silu(g) * u * rw[rows][:, None]) @ w2[e].t()
            total = total + (y * b.grad[rows].double()).sum()
        return total

    at = [b.x.double(), b.w13.double(), b.w2.double(), b.rw.double()]
    y, h, saved = b.forward()
    gx, g13, g2, grw, _, _ = b.backward(saved, h, torch.float32)
    for i, got in enumerate((gx, g13, g2, grw)):
        d = torch.randn(at[i].shape, generator=gen, device="cuda", dtype=torch.float64)
        live = torch.zeros_like(d)
        if i in (0, 3):
            live[b.rows] = 1.0
        else:
            live += 1.0
        d = d * live
        step = 1e-5
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + step * d, at[i] - step * d
        slope = float(loss(*up) - loss(*down)) / (2 * step)
        kept = torch.where(live > 0, got.double(), torch.zeros_like(d))
        mine = float((kept * d).sum())
        assert abs(mine - slope) <= 2.0 ** -7 * float(kept.norm()) * 3 + 1e-9, (i, mine, slope)


def test_all_rows_on_one_expert_and_none():
    for popular in (0, 3, 7):
        gen = _gen(popular)
        T, E, H, I = 300, 8, 136, 72
        b = Block(T, 1, E, 16, H, I, False, True, 0.0, 7)
        idx = torch.full((T, 1), popular, dtype=torch.int64, device="cuda")
        b.h.layout(idx)
        b.idx = idx
        b.rows, b.expert, b.token = ref.rows_of(b.h, idx)
        b.x, b.grad = _randn(b.x.shape, gen), _randn(b.grad.shape, gen)
        b.rw = torch.rand(b.rw.shape, generator=gen, device="cuda")
        y, h, saved = b.forward()
        b.check_forward(y, h, saved)
        b.check_backward(saved, h, b.backward(saved, h), False)
    # a batch whose slots are all empty: nothing is written but zeros for the weights
    b.h.layout(torch.full((T, 1), -1, dtype=torch.int64, device="cuda"))
    out = b.backward(saved, h)
    assert bool((out[1] == 0).all()) and bool((out[2] == 0).all())
    for t in (out[0], out[4]):
        assert ref.untouched(t, torch.zeros(0, dtype=torch.long, device="cuda"))
    y, h2, gu = b.forward()
    for t in (y, h2, gu):
        assert ref.untouched(t, torch.zeros(0, dtype=torch.long, device="cuda"))


def test_no_tokens():
    b = Block(4, 2, 3, 1, 64, 32, False, False, 0.0, 8)
    b.h.layout(torch.zeros((0, 2), dtype=torch.int64, device="cuda"))
    b.forward()
    saved, h = _randn((b.h.capacity, 64), _gen(1)), _randn((b.h.capacity, 32), _gen(2))
    out = b.backward(saved, h)
    assert bool((out[1] == 0).all()) and bool((out[2] == 0).all())


def test_rows_with_infinities_and_nan_reach_no_other_row():
    b = Block(90, 2, 3, 8, 200, 72, True, False, 0.0, 9)
    want = b.forward()
    b.x[11, 5], b.x[40, 199] = float("inf"), float("nan")
    got = b.forward()
    keep = b.rows[(b.token != 11) & (b.token != 40)]
    for p, q in zip(got, want):
        assert torch.equal(p[keep], q[keep])
    bad = b.rows[b.token == 40]
    assert bool(got[0][bad].isnan().all())


def test_same_expert_twice_in_a_token():
    idx = torch.tensor([[1, 1, 0], [2, 1, 1]], device="cuda")
    b = Block(2, 3, 3, 4, 72, 40, True, True, 0.0, 10)
    b.h = ep.Handle(2, 3, 3, 4, capacity=24)
    b.h.layout(idx)
    b.idx = idx
    b.rows, b.expert, b.token = ref.rows_of(b.h, idx)
    b.rw = torch.rand(24, generator=_gen(1), device="cuda")
    b.grad = _randn((24, 72), _gen(2))
    y, h, saved = b.forward()
    b.check_forward(y, h, saved)
    b.check_backward(saved, h, b.backward(saved, h), False)


def test_after_a_capacity_error_nothing_is_written():
    gen = _gen(11)
    T, K, E, H, I = 32, 2, 4, 64, 32
    h = ep.Handle(T, K, E, 1, capacity=20)
    h.layout(ref.ids(T, K, E, gen, "cuda"))
    assert h.read_counts(check=False)["error_bits"] & ep.EP_ERRBIT_CAPACITY
    b = Block(T, K, E, 1, H, I, False, True, 0.0, 12)
    b.h, b.rows = h, torch.zeros(0, dtype=torch.long, device="cuda")
    cut = lambda t: t[:20].contiguous()  # noqa: E731
    b.x, b.grad, b.rw = _randn((20, H), gen), _randn((20, H), gen), cut(b.rw)
    for t in b.forward():
        assert ref.untouched(t, b.rows)
    saved = _randn((20, 2 * I), gen)
    out = b.backward(saved, _randn((20, I), gen))
    for t in out[:3] + out[4:5]:
        assert ref.untouched(t.reshape(-1, t.shape[-1]), b.rows)
    assert ref.untouched(out[3][:, None], b.rows)
    q, s = ref.poisoned((20, H), torch.int8), ref.poisoned((20,), torch.float32)
    h.quantize_i8(b.x, out_q=q, out_scale=s)
    assert ref.untouched(q, b.rows) and ref.untouched(s[:, None], b.rows)
    o = ref.poisoned((20, 16), torch.bfloat16)
    h.expert_i8(torch.ones((20, H), dtype=torch.int8, device="cuda"), torch.ones(20, device="cuda"),
                torch.ones((E, 16, H), dtype=torch.int8, device="cuda"),
                torch.ones((E, 16), device="cuda"), out=o)
    assert ref.untouched(o, b.rows)


# ---------------------------------------------------------------- far apart, and long

def test_offsets_past_32_bits_in_rows():
    """Segments 4.3 GB and more behind the buffers' start: rows of 32 KB, segments of 65536 rows."""
    T, E, A, H, I = 9, 3, 65536, 16384, 40
    idx = (torch.arange(T, device="cuda") % E)[:, None].contiguous()
    h = ep.Handle(T, 1, E, A)
    h.layout(idx)
    rows, expert, token = ref.rows_of(h, idx)
    assert int(rows.max()) * H * 2 > 2 ** 32 and h.capacity * H > 2 ** 31
    gen = _gen(21)
    b = Block.__new__(Block)
    b.h, b.idx, b.rows, b.expert, b.token = h, idx, rows, expert, token
    b.E, b.H, b.I, b.token_rows, b.rw = E, H, I, False, None
    b.w13, b.w2 = _randn((E, 2 * I, H), gen, H ** -0.5), _randn((E, H, I), gen, I ** -0.5)
    b.x = torch.zeros((h.capacity, H), dtype=torch.bfloat16, device="cuda")
    b.grad = torch.zeros_like(b.x)
    b.x[rows], b.grad[rows] = _randn((T, H), gen), _randn((T, H), gen, 0.1)
    y, hh, saved = h.expert_ffn(b.x, b.w13, b.w2, want_saved=True)
    gx, g13, g2, _, ggu = h.expert_ffn_backward(b.grad, b.x, b.w13, b.w2, saved, hh)
    far = int(rows.max())
    at = (rows == far).nonzero().item()
    e = int(expert[at])
    x64, w = b.x[far].double(), b.w13[e].double()
    v = w @ x64
    tol = (w.abs() @ x64.abs()) * _sum_tol(H) + v.abs() * BF16
    ref.assert_close(saved[far], v, tol, "far gate_up")
    want = b.w2[e].double() @ hh[far].double()
    tol = (b.w2[e].double().abs() @ hh[far].double().abs()) * _sum_tol(I) + want.abs() * BF16
    ref.assert_close(y[far], want, tol, "far y")
    want = ggu[far].double() @ w
    tol = (ggu[far].double().abs() @ w.abs()) * _sum_tol(2 * I) + want.abs() * BF16 + 1e-38
    ref.assert_close(gx[far], want, tol, "far grad x")
    mine = rows[expert == e]
    for got, p, q in ((g13[e], ggu[mine].double(), b.x[mine].double()),
                      (g2[e], b.grad[mine].double(), hh[mine].double())):
        want = p.t() @ q
        ref.assert_close(got, want, (p.abs().t() @ q.abs()) * _sum_tol(mine.numel()) +
                         want.abs() * BF16 + 1e-38, "far weight gradient")
    n = 16400
    q, s = h.quantize_i8(b.x)
    wq = torch.randint(-127, 128, (E, n, H), generator=gen, device="cuda", dtype=torch.int8)
    ws = torch.rand((E, n), generator=gen, device="cuda") * 0.01
    out = h.expert_i8(q, s, wq, ws)
    assert torch.equal(q[far], _codes64(b.x[far][None])[0][0])
    want = (wq[e].double() @ q[far].double()) * s[far].double() * ws[e].double()
    ref.assert_close(out[far], want, want.abs() * (BF16 + 4 * F32) + 1e-38, "far int8")


def test_offsets_past_32_bits_in_weights():
    """The widest block: 32768 channels of h, weights of 4.8 GB in both projections."""
    T, E, H, I = 5, 3, 12288, 32768
    gen = _gen(22)
    idx = torch.tensor([[2], [0], [2], [1], [2]], device="cuda")
    h = ep.Handle(T, 1, E, 1)
    h.layout(idx)
    rows, expert, token = ref.rows_of(h, idx)
    w13 = (torch.randn((E, 2 * I, H), generator=gen, device="cuda", dtype=torch.float32)
           .mul_(H ** -0.5).bfloat16())
    w2 = _randn((E, H, I), gen, I ** -0.5)
    assert w13.numel() * 2 > 2 ** 32
    x, grad = _randn((T, H), gen), _randn((h.capacity, H), gen, 0.1)
    y, hh, saved = h.expert_ffn(x, w13, w2, token_rows=True, want_saved=True)
    gx, g13, g2, _, ggu = h.expert_ffn_backward(grad, x, w13, w2, saved, hh, token_rows=True)
    e, mine = 2, expert == 2
    r, src = rows[mine], token[mine]
    for name, got, p, w in (("gate_up", saved, x[src], w13[e]), ("y", y, hh[r], w2[e])):
        for part in range(0, w.shape[0], 8192):
            wp = w[part:part + 8192].double()
            want = p.double() @ wp.t()
            tol = (p.double().abs() @ wp.abs().t()) * _sum_tol(w.shape[1]) + want.abs() * BF16 + 1e-38
            ref.assert_close(got[r, part:part + 8192], want, tol, f"{name} {part}")
    want, tol = torch.zeros((len(r), H), dtype=torch.float64, device="cuda"), 0
    for part in range(0, 2 * I, 8192):
        gp, wp = ggu[r, part:part + 8192].double(), w13[e, part:part + 8192].double()
        want += gp @ wp
        tol = tol + (gp.abs() @ wp.abs()) * _sum_tol(2 * I)
        full = gp.t() @ x[src].double()
        ref.assert_close(g13[e, part:part + 8192], full, full.abs() * BF16 +
                         (gp.abs().t() @ x[src].double().abs()) * _sum_tol(3) + 1e-38, f"w13 {part}")
    ref.assert_close(gx[r], want, tol + want.abs() * BF16 + 1e-38, "grad x")
    full = grad[r].double().t() @ hh[r].double()
    ref.assert_close(g2[e], full, full.abs() * BF16 + (grad[r].double().abs().t() @
                     hh[r].double().abs()) * _sum_tol(3) + 1e-38, "w2")


def test_many_tiles_a_block_and_few_rows_between_many():
    """Weight gradients of more tiles than blocks, experts of none, one and many rows in turns: a
    block goes from tiles of one chunk to tiles of many and back."""
    gen = _gen(23)
    E, H, I = 24, 520, 1032
    counts = [0, 1, 700, 2, 0, 64, 65, 1, 1, 63, 300, 0, 128, 3, 0, 0, 5, 200, 1, 64, 1, 1, 129, 0]
    ids = torch.repeat_interleave(torch.arange(E), torch.tensor(counts))
    idx = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(1))][:, None].cuda()
    for token_rows in (False, True):
        b = Block(len(ids), 1, E, 4, H, I, token_rows, True, 0.0, 24)
        b.h.layout(idx)
        b.idx = idx
        b.rows, b.expert, b.token = ref.rows_of(b.h, idx)
        b.grad = _spoil(_randn(b.grad.shape, gen, 0.1), b.rows)
        b.rw = _spoil(torch.rand(b.rw.shape, generator=gen, device="cuda"), b.rows)
        b.x = _randn(b.x.shape, gen)
        if not token_rows:
            _spoil(b.x, b.rows)
        y, h, saved = b.forward()
        b.check_forward(y, h, saved)
        for dtype in (torch.bfloat16, torch.float32):
            b.check_backward(saved, h, b.backward(saved, h, dtype), False)


def _popular(T, E, popular, every):
    """All tokens on one expert but every few, which go round the others."""
    idx = torch.full((T, 1), popular, dtype=torch.int64, device="cuda")
    idx[::every, 0] = torch.arange(len(range(0, T, every)), device="cuda") % E
    return idx


@pytest.mark.parametrize("T,E,k,n,gated", [(100, 8, 4112, 2056, False), (300, 32, 528, 4112, True),
                                           (700, 32, 528, 4112, False)])
def test_i8_popular_expert_beside_weights_past_the_caches(T, E, k, n, gated):
    """More than 64 MB of weights, few rows an expert on average, one expert with many row tiles of
    16, 32 and 64 rows and others with one or two."""
    say("expert_i8 popular", T, E, k, n, gated)
    gen = _gen(T)
    idx = _popular(T, E, 5, 4)
    h = ep.Handle(T, 1, E, 1)
    h.layout(idx)
    x, xs, w, ws = _i8_case(h, E, h.capacity, k, n, gen)
    out = ref.poisoned((h.capacity, n // 2 if gated else n), torch.bfloat16)
    h.expert_i8(x, xs, w, ws, gated=gated, out=out)
    _check_i8(h, idx, x, xs, w, ws, gated, None, out, False, "popular")


@pytest.mark.parametrize("token_rows", [False, True])
def test_block_popular_expert_beside_weights_past_the_caches(token_rows):
    T, E, H, I = 1400, 32, 520, 2056
    b = Block(T, 1, E, 1, H, I, token_rows, False, 0.0, 31)
    idx = _popular(T, E, 5, 20)
    b.h.layout(idx)
    b.idx = idx
    b.rows, b.expert, b.token = ref.rows_of(b.h, idx)
    gen = _gen(32)
    b.x, b.grad = _randn(b.x.shape, gen), _randn(b.grad.shape, gen, 0.1)
    y, h, saved = b.forward()
    b.check_forward(y, h, saved)
    b.check_backward(saved, h, b.backward(saved, h), False)


@pytest.mark.parametrize("rows", ["one chunk", "one or two", "one to three, some none"])
@pytest.mark.parametrize("token_rows", [False, True])
def test_weight_gradients_of_full_tiles_and_few_rows(rows, token_rows):
    """Weight gradients in full tiles, several a block, of so few rows that a tile is stored while the
    next ones' first rows are on their way."""
    say("weight gradients", rows, token_rows)
    E, H, I = 96, 1024, 512
    most = {"one chunk": 64, "one or two": 128}.get(rows, 192)
    gen = torch.Generator().manual_seed(most)
    counts = torch.randint(0 if most == 192 else 1, most + 1, (E,), generator=gen)
    if most == 192:
        counts[torch.rand(E, generator=gen) < 0.3] = 0
    ids = torch.repeat_interleave(torch.arange(E), counts)
    idx = ids[torch.randperm(len(ids), generator=gen)][:, None].cuda()
    b = Block(len(ids), 1, E, 1, H, I, token_rows, False, 0.0, most)
    b.h.layout(idx)
    b.idx = idx
    b.rows, b.expert, b.token = ref.rows_of(b.h, idx)
    dev = _gen(most)
    b.x, b.grad = _randn(b.x.shape, dev), _randn(b.grad.shape, dev, 0.1)
    y, h, saved = b.forward()
    for dtype in (torch.bfloat16, torch.float32):
        first = b.backward(saved, h, dtype)
        b.check_backward(saved, h, first, False)
        for _ in range(3):
            again = b.backward(saved, h, dtype)
            assert torch.equal(again[1], first[1]) and torch.equal(again[2], first[2])
