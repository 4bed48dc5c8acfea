"""ep_add_rmsnorm and its gradient against binary64, on the GPU.

Tolerances: a bf16 result is off by half a step (2^-8 relative) of a binary32
value that is itself off by a counted number of roundings (2^-24 each).
z, rstd's last bit aside, and the E4M3 rows are exact: the squares are summed
in binary64, so rstd is the correctly rounded one and y is two products."""
import pytest
import torch

import combine_ep_layout_08_amd as ep
from tests import layer_ref as ref
from tests.gpu_util import needs_gpu, say

pytestmark = [pytest.mark.gpu, needs_gpu]
EPS = 1e-6


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rows(T, H, gen, scale=1.0):
    x = torch.randn((T, H), generator=gen, device="cuda") * scale
    return (x * torch.where(torch.rand(H, generator=gen, device="cuda") < 0.01, 20.0,
                            1.0)).bfloat16()


def _weight(H, gen, dtype):
    return (1.0 + 0.3 * torch.randn(H, generator=gen, device="cuda")).to(dtype)


def _reference(x, residual, weight):
    z = x if residual is None else (x.float() + residual.float()).bfloat16()
    rstd = (1.0 / torch.sqrt(z.double().square().mean(1) + EPS)).float()
    y = z.float() * rstd[:, None] * weight.float()      # two rounded products
    return z, rstd, y


CASES = [  # T, H, residual, weight dtype, scale format
    (1, 8, False, torch.float32, None),
    (1, 7168, True, torch.bfloat16, "f32"),
    (3, 128, True, torch.float32, "ue8m0"),
    (5, 256, False, torch.bfloat16, "f32"),
    (64, 640, True, torch.bfloat16, "ue8m0"),
    (333, 1280, True, torch.float32, "f32"),
    (17, 4104, True, torch.bfloat16, None),
    (130, 5120, False, torch.float32, "ue8m0"),
    (2, 32768, True, torch.bfloat16, "f32"),
    (9, 16512, True, torch.float32, "ue8m0"),
    (4096, 7168, True, torch.bfloat16, "ue8m0"),
    (2500, 520, True, torch.bfloat16, None),
]


@pytest.mark.parametrize("T,H,residual,wdt,fmt", CASES)
def test_forward(T, H, residual, wdt, fmt):
    say("norm", T, H, residual, wdt, fmt)
    gen = _gen(T + H)
    x = _rows(T, H, gen)
    r = _rows(T, H, gen) if residual else None
    w = _weight(H, gen, wdt)
    z, rstd, y = _reference(x, r, w)
    got_y, got_z, q, sf, got_rstd = ep.add_rmsnorm(x, w, residual=r, eps=EPS, scale_format=fmt,
                                                   want_rstd=True)
    assert (got_z is None) == (r is None)
    if got_z is not None:
        assert torch.equal(got_z.view(torch.int16), z.view(torch.int16))
    ref.assert_close(got_rstd, rstd, ref.F32 * rstd.double() * 2, "rstd")
    y64 = z.double() / torch.sqrt(z.double().square().mean(1, keepdim=True) + EPS) * w.double()
    ref.assert_close(got_y, y64, y64.abs() * (ref.BF16 + 4 * ref.F32) + 1e-38, "y")
    if fmt:
        # the rows whose rstd is the correctly rounded one, as all but a few are
        same = got_rstd == rstd
        assert int((~same).sum()) <= 1
        want_q, want_sf = ref.quantise(y, fmt)
        assert torch.equal(q[same], want_q[same])
        assert torch.equal(sf.view(torch.int32)[same], want_sf.view(torch.int32)[same])


@pytest.mark.parametrize("fmt", ["f32", "ue8m0"])
def test_outputs_one_by_one_and_column_major_scales(fmt):
    gen = _gen(3)
    T, H = 37, 896
    x, r, w = _rows(T, H, gen), _rows(T, H, gen), _weight(H, gen, torch.bfloat16)
    y, z, q, sf, rstd = ep.add_rmsnorm(x, w, residual=r, scale_format=fmt, want_rstd=True)
    alone = ep.add_rmsnorm(x, w, residual=r, want_y=False, scale_format=fmt, col_major_sf=True)
    assert alone[0] is None and alone[4] is None and alone[3].stride(0) == 1
    assert torch.equal(alone[1], z) and torch.equal(alone[2], q)
    assert torch.equal(alone[3].contiguous(), sf)
    only_y = ep.add_rmsnorm(z, w)
    assert only_y[1] is None and torch.equal(only_y[0], y)
    only_rstd = ep.add_rmsnorm(z, w, want_y=False, want_rstd=True)
    assert torch.equal(only_rstd[4], rstd)


@pytest.mark.parametrize("target", ["x", "residual"])
def test_sum_in_place(target):
    gen = _gen(4)
    x, r, w = _rows(50, 2048, gen), _rows(50, 2048, gen), _weight(2048, gen, torch.float32)
    y, z, *_ = ep.add_rmsnorm(x, w, residual=r)
    z, y = z.clone(), y.clone()
    y2, z2, *_ = ep.add_rmsnorm(x, w, residual=r, out_z=x if target == "x" else r)
    assert z2 is (x if target == "x" else r)
    assert torch.equal(z2, z) and torch.equal(y2, y)


def test_rows_of_extremes():
    """Zero rows, rows whose squares overflow binary32, tiny rows, a NaN and an
    infinity: each stays in its own row, and the E4M3 recipe's special cases hold."""
    H = 512
    x = torch.ones((6, H), device="cuda").bfloat16()
    x[0] = 0
    x[1] = 2.0 ** 100
    x[2] = 2.0 ** -120
    x[3, 5] = float("nan")
    x[4, 200] = float("inf")
    w = torch.ones(H, device="cuda")
    y, _, q, sf, rstd = ep.add_rmsnorm(x, w, eps=EPS, scale_format="f32",
                                       want_rstd=True)
    assert torch.equal(y[0].float(), torch.zeros(H, device="cuda"))
    assert bool((q[0] == 0).all())
    ref.assert_close(y[1], torch.ones(H, device="cuda"), ref.BF16, "large")
    want = 2.0 ** -120 * 1e3
    ref.assert_close(y[2], torch.full((H,), want, device="cuda").double(), want * 2 ** -7, "tiny")
    assert bool(y[3].isnan().all()) and bool((q[3] == 0x7F).all())
    assert float(rstd[4]) == 0.0
    assert bool(y[4, 200].isnan()) and int(q[4, 200]) == 0x7F       # inf * 0
    assert int(y[4].isnan().sum()) == 1 and bool((q[4, :128] == 0).all())
    ref.assert_close(y[5], torch.ones(H, device="cuda"), ref.BF16, "ones")
    z, _, _, _, r0 = ep.add_rmsnorm(x[:1], w, eps=0.0, want_rstd=True)
    assert bool(torch.isinf(r0).all()) and bool(z.isnan().all())    # 0 * inf, as the formula says


def test_infinite_values_in_the_eight_bit_rows():
    """A weight that makes y infinite: the block's codes are those of the quantiser's
    recipe (scale inf, quotient NaN for the infinity, 0 for the finite values)."""
    x = torch.full((1, 256), 1.0, device="cuda").bfloat16()
    w = torch.ones(256, device="cuda")
    w[3] = float("inf")
    w[4] = float("nan")
    _, _, q, sf, _ = ep.add_rmsnorm(x, w, want_y=False, scale_format="f32")
    assert bool(torch.isinf(sf[0, 0])) and int(q[0, 3]) == 0x7F and int(q[0, 4]) == 0x7F
    assert int(q[0, 5]) == 0 and abs(float(sf[0, 1]) - 1 / 448) < 1e-6


def test_no_tokens():
    w = torch.ones(256, device="cuda")
    x = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    y, _, q, sf, rstd = ep.add_rmsnorm(x, w, scale_format="ue8m0", want_rstd=True)
    assert y.shape == (0, 256) and q.shape == (0, 256) and rstd.shape == (0,)
    gx, gw = ep.add_rmsnorm_backward(x, x, w, rstd)
    assert gx.shape == (0, 256) and bool((gw == 0).all())


GRAD_CASES = [  # T, H, residual gradient, weight dtype
    (1, 8, False, torch.float32),
    (1, 7168, True, torch.bfloat16),
    (3, 136, True, torch.float32),
    (333, 1280, False, torch.float32),
    (511, 264, True, torch.bfloat16),
    (513, 4104, True, torch.bfloat16),
    (1024, 520, True, torch.float32),
    (1025, 264, True, torch.bfloat16),
    (1500, 16512, False, torch.bfloat16),
    (2, 32768, True, torch.float32),
    (4096, 7168, True, torch.bfloat16),
    (9000, 256, False, torch.float32),
]


def _grad_reference(g, z, w, rstd, gz):
    g, z, w, r = g.double(), z.double(), w.double(), rstd.double()[:, None]
    n = z * r
    c = (g * w * n).mean(1, keepdim=True)
    gx = r * (g * w - n * c)
    size = r * ((g * w).abs() + n.abs() * (g * w * n).abs().mean(1, keepdim=True))
    if gz is not None:
        gx, size = gx + gz.double(), size + gz.double().abs()
    return gx, (g * n).sum(0), size, (g * n).abs().sum(0)


@pytest.mark.parametrize("T,H,residual,wdt", GRAD_CASES)
def test_backward(T, H, residual, wdt):
    say("norm gradient", T, H, residual, wdt)
    gen = _gen(T + 3 * H)
    z, w = _rows(T, H, gen), _weight(H, gen, wdt)
    g = _rows(T, H, gen, 1e-2)
    gz = _rows(T, H, gen, 1e-2) if residual else None
    rstd = (1.0 / torch.sqrt(z.double().square().mean(1) + EPS)).float()
    gx, gw = ep.add_rmsnorm_backward(g, z, w, rstd, grad_residual=gz)
    want_x, want_w, size, size_w = _grad_reference(g, z, w, rstd, gz)
    # the row's mean: a chain of at most 32 products a thread, then 4 + 4 + 16
    # sums over lanes and waves; then six roundings of terms no larger than size
    ref.assert_close(gx, want_x, want_x.abs() * ref.BF16 + 72 * ref.F32 * size, "grad_x")
    # every sum is at most T + 64 long, each product rounded twice
    ref.assert_close(gw, want_w, (T + 66) * ref.F32 * size_w, "grad_weight")
    rel = float((gw.double() - want_w).norm() / want_w.norm())
    assert rel < 1e-6, rel
    again = ep.add_rmsnorm_backward(g, z, w, rstd, grad_residual=gz)
    assert torch.equal(again[0], gx) and torch.equal(again[1], gw)
    only_x = ep.add_rmsnorm_backward(g, z, w, rstd, grad_residual=gz, want_grad_weight=False)
    only_w = ep.add_rmsnorm_backward(g, z, w, rstd, grad_residual=gz, want_grad_x=False)
    assert only_x[1] is None and torch.equal(only_x[0], gx)
    assert only_w[0] is None and torch.equal(only_w[1], gw)


@pytest.mark.parametrize("target", ["grad_y", "grad_residual"])
def test_backward_in_place(target):
    gen = _gen(8)
    T, H = 700, 1024
    z, w = _rows(T, H, gen), _weight(H, gen, torch.bfloat16)
    g, gz = _rows(T, H, gen), _rows(T, H, gen)
    rstd = ep.add_rmsnorm(z, w, want_rstd=True)[4]
    want = ep.add_rmsnorm_backward(g, z, w, rstd, grad_residual=gz)
    want = (want[0].clone(), want[1].clone())
    out = g if target == "grad_y" else gz
    got = ep.add_rmsnorm_backward(g, z, w, rstd, grad_residual=gz, grad_x=out)
    assert got[0] is out and torch.equal(out, want[0]) and torch.equal(got[1], want[1])


def test_gradient_against_differences():
    """Directional differences of the binary64 loss sum(y * g) along random
    directions of z and of the weight."""
    gen = _gen(9)
    T, H = 5, 256
    z, w, g = _rows(T, H, gen), _weight(H, gen, torch.float32), _rows(T, H, gen)
    rstd = ep.add_rmsnorm(z, w, eps=EPS, want_rstd=True)[4]
    gx, gw = ep.add_rmsnorm_backward(g, z, w, rstd)

    def loss(zz, ww):
        r = 1.0 / torch.sqrt(zz.square().mean(1, keepdim=True) + EPS)
        return float((zz * r * ww * g.double()).sum())

    for k in range(4):
        d = torch.randn((T, H), generator=gen, device="cuda", dtype=torch.float64)
        e = torch.randn(H, generator=gen, device="cuda", dtype=torch.float64)
        h = 1e-4
        dz = (loss(z.double() + h * d, w.double()) - loss(z.double() - h * d, w.double())) / (2 * h)
        dw = (loss(z.double(), w.double() + h * e) - loss(z.double(), w.double() - h * e)) / (2 * h)
        # bf16 gradients: half a step each, along the direction
        tol = float((gx.double() * d).abs().sum()) * ref.BF16 * 2 + 1e-6 * abs(dz)
        assert abs(float((gx.double() * d).sum()) - dz) <= tol
        assert abs(float((gw.double() * e).sum()) - dw) <= 1e-5 * float((gw.double() * e).abs().sum())


@pytest.mark.parametrize("T,H", [(64, 1024), (2048, 640)])
def test_bound_call_and_graph(T, H):
    """A bound call and a captured pair (norm, gradient) follow their tensors' new
    contents; each replay is compared with the eager calls."""
    gen = _gen(10)
    x, r, w = _rows(T, H, gen), _rows(T, H, gen), _weight(H, gen, torch.bfloat16)
    g = _rows(T, H, gen)
    call = ep.bind_add_rmsnorm(x, w, residual=r, scale_format="f32", want_rstd=True)
    call()
    y, z, q, sf, rstd = call()
    ep.add_rmsnorm_backward(g, z, w, rstd)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        gx, gw = ep.add_rmsnorm_backward(g, z, w, rstd, grad_residual=g)
    for k in range(3):
        x.copy_(_rows(T, H, gen))
        g.copy_(_rows(T, H, gen))
        graph.replay()
        torch.cuda.synchronize()
        want = ep.add_rmsnorm(x, w, residual=r, scale_format="f32", want_rstd=True)
        for a, b in zip((y, z, q, sf, rstd), want):
            assert torch.equal(a, b)
        wx, ww = ep.add_rmsnorm_backward(g, want[1], w, want[4], grad_residual=g)
        assert torch.equal(gx, wx) and torch.equal(gw, ww)


def test_offsets_past_32_bits():
    """Rows behind the first 4 GiB."""
    T, H = 140_000, 16384
    gen = _gen(12)
    x = torch.ones((T, H), dtype=torch.bfloat16, device="cuda")
    x[-50:] = _rows(50, H, gen)
    w = _weight(H, gen, torch.float32)
    say("norm offsets", T, H)
    y, _, q, sf, rstd = ep.add_rmsnorm(x, w, eps=EPS, scale_format="f32", want_rstd=True)
    last = ep.add_rmsnorm(x[-50:].contiguous(), w, eps=EPS, scale_format="f32", want_rstd=True)
    for a, b in zip((y, q, sf, rstd), (last[0], *last[2:])):
        assert torch.equal(a[-50:], b)
    gx, gw = ep.add_rmsnorm_backward(y, x, w, rstd)
    lx, _ = ep.add_rmsnorm_backward(last[0], x[-50:].contiguous(), w, last[4])
    # another number of rows sums in another order: a step of bf16 at most
    ref.assert_close(gx[-50:], lx, lx.double().abs() * 2 * ref.BF16 + 1e-4, "gradient")
    assert bool(torch.isfinite(gw).all())


def test_two_streams():
    """Forward and backward of two batches at once, each with its own buffers."""
    gen = _gen(13)
    sets = []
    for T, H in ((1500, 2048), (700, 4096)):
        x, r, g = _rows(T, H, gen), _rows(T, H, gen), _rows(T, H, gen)
        sets.append((x, r, g, _weight(H, gen, torch.bfloat16)))

    def step(x, r, g, w):
        y, z, q, sf, rstd = ep.add_rmsnorm(x, w, residual=r, scale_format="f32", want_rstd=True)
        return (y, q, sf, *ep.add_rmsnorm_backward(g, z, w, rstd, grad_residual=g))

    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = []
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(step(*s))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for u, v in zip(a, b):
                assert torch.equal(u, v)


@pytest.mark.parametrize("T", [3, 700, 1500])
def test_backward_over_z(T):
    gen = _gen(14)
    H = 1024
    z, w = _rows(T, H, gen), _weight(H, gen, torch.bfloat16)
    g = _rows(T, H, gen)
    rstd = ep.add_rmsnorm(z, w, want_rstd=True)[4]
    want = ep.add_rmsnorm_backward(g, z, w, rstd)
    got = ep.add_rmsnorm_backward(g, z, w, rstd, grad_x=z)
    assert got[0] is z and torch.equal(z, want[0]) and torch.equal(got[1], want[1])


def test_weight_gradient_past_32_bits():
    """grad_weight over rows on both sides of the first 4 GiB (row 131072).  Of a channel's
    sum each of the 512 blocks adds up 274 rows in turn, then 4 of its 128 groups and 18 more
    sums join them, and a term is two rounded products: 298 roundings.  The last rows weigh
    enough for each of them to show."""
    T, H, last = 140_000, 16384, 50
    gen = _gen(31)
    z = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    g = torch.empty_like(z)
    rstd = torch.empty(T, device="cuda")
    w = _weight(H, gen, torch.bfloat16)
    want = torch.zeros(H, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    say("norm weight gradient offsets", T, H)
    for a in range(0, T, 4000):
        z[a:a + 4000] = _rows(4000, H, gen)
        g[a:a + 4000] = _rows(4000, H, gen, 1e-2)
        if a + 4000 == T:
            z[-last:] = torch.where(z[-last:] < 0, -1.0, 1.0)
            g[-last:] = 1.0
        rstd[a:a + 4000] = (1.0 / torch.sqrt(z[a:a + 4000].double().square().mean(1) + EPS)).float()
        term = g[a:a + 4000].double() * z[a:a + 4000].double() * rstd[a:a + 4000].double()[:, None]
        want += term.sum(0)
        size += term.abs().sum(0)
    tol = 298 * ref.F32 * size
    assert float(tol.max()) < 0.5 * float(term[-last:].abs().min())
    gx, gw = ep.add_rmsnorm_backward(g, z, w, rstd)
    ref.assert_close(gw, want, tol, "grad_weight")
    del gx
    only = ep.add_rmsnorm_backward(g, z, w, rstd, want_grad_x=False)[1]
    assert torch.equal(only, gw)


@pytest.mark.parametrize("T,H,residual,fmt", [(262_844, 1024, True, "ue8m0"),
                                              (262_844, 256, False, None)])
def test_more_rows_than_blocks(T, H, residual, fmt):
    """More rows than a launch has blocks (2^18): the blocks walk the rest, with the sums of
    two waves in turn, and with the rows stored past the caches."""
    test_forward(T, H, residual, torch.bfloat16, fmt)


@pytest.mark.parametrize("fmt", [None, "f32", "ue8m0"])
@pytest.mark.parametrize("T,H", [(13_000, 2048), (4000, 7168), (1700, 16384)])
def test_rows_stored_past_the_caches(T, H, fmt):
    """106 to 144 MB of rows, one, two and four vectors a thread: every form of the kernel
    that stores past the caches."""
    test_forward(T, H, True, torch.float32, fmt)
