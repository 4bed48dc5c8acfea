"""ep_expert_w4 and ep_w4_pack against binary64, on the GPU.

Tolerance: one rounding to bf16 (2^-8 of the value), and binary32 sums: a
matrix instruction adds 32 products to its accumulator, at most 33 roundings of
partial sums, and the steps' sums follow.  The partial sums are bounded by the
sum of |x w|; with EP_W4_INT4 the codes enter as 128 + code and 136 is taken off,
so there they are bounded by the sum of 136 |x scale| within the group."""
import pytest
import torch

import combine_ep_layout_08_amd as ep
from tests import layer_ref as ref
from tests.gpu_util import needs_gpu, say

pytestmark = [pytest.mark.gpu, needs_gpu]
INT4, MX = ep.EP_W4_INT4, ep.EP_W4_MXFP4


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _x(rows, k, kind, gen):
    x = torch.randn((rows, k), generator=gen, device="cuda").bfloat16()
    if kind == "bf16":
        return x, None, x.double()
    if rows == 0:
        return x.view(torch.uint8)[:, :k], None, x.double()
    q, sf = ep.quantize_fp8(x, kind)
    return q, sf, ref.code_values(q, sf)


def _check(h, idx, x64, w64, scale64, out, token_rows, what):
    """Rows of ``out`` against x64 . w64, others untouched."""
    rows, expert, token = ref.rows_of(h, idx)
    for e in torch.unique(expert).tolist():
        mine = expert == e
        src = x64[token[mine] if token_rows else rows[mine]]
        want = src @ w64[e].t()
        size = src.abs() @ (w64[e].abs() if scale64 is None else scale64[e] * 136.0).t()
        tol = want.abs() * ref.BF16 + size * 66 * ref.F32 + 1e-38
        got = out[rows[mine]]
        ref.assert_close(got, want, tol, f"{what}, expert {e}")
        norm = float(want.norm())
        if norm > 0 and want.numel() > 64:
            assert float((got.double() - want).norm()) < ref.BF16 * norm
    assert ref.untouched(out, rows)


def _scales64(scales, group, fmt):
    return scales.double().abs().repeat_interleave(group, 2) if fmt == INT4 else None


CASES = [  # T, K, E, A, k, n, format, group, x, token rows, empty
    (1, 1, 1, 1, 128, 8, INT4, 128, "bf16", False, 0.0),
    (1, 1, 1, 1, 128, 16, MX, 32, "bf16", True, 0.0),
    (1, 8, 64, 1, 7168, 512, INT4, 128, "bf16", True, 0.0),
    (1, 8, 16, 1, 2048, 264, MX, 32, "f32", False, 0.0),
    (2, 2, 5, 1, 256, 24, INT4, 64, "bf16", False, 0.0),
    (7, 3, 6, 8, 384, 40, INT4, 32, "bf16", True, 0.2),
    (16, 1, 1, 1, 640, 72, INT4, 64, "f32", False, 0.0),
    (17, 1, 1, 4, 896, 136, MX, 32, "bf16", False, 0.0),
    (64, 4, 16, 1, 256, 512, INT4, 32, "bf16", False, 0.1),
    (64, 4, 16, 128, 1152, 200, INT4, 128, "ue8m0", False, 0.1),
    (33, 2, 2, 1, 512, 104, INT4, 64, "ue8m0", True, 0.1),
    (65, 1, 1, 16, 1024, 48, MX, 32, "ue8m0", True, 0.0),
    (100, 8, 8, 1, 768, 96, INT4, 128, "f32", False, 0.0),
    (130, 2, 2, 1, 256, 8, MX, 32, "f32", True, 0.2),
    (200, 4, 4, 64, 128, 24, INT4, 32, "f32", True, 0.0),
    (128, 8, 64, 128, 2048, 1024, MX, 32, "f32", False, 0.0),
    (96, 8, 300, 8, 256, 64, INT4, 64, "bf16", False, 0.1),
    (3, 2, 1000, 1, 128, 16, INT4, 128, "bf16", True, 0.0),
    (5, 2, 4, 1, 32768, 32, INT4, 128, "f32", False, 0.0),
    (300, 1, 3, 1, 1920, 80, INT4, 64, "bf16", False, 0.0),
]


@pytest.mark.parametrize("T,K,E,A,k,n,fmt,group,kind,token_rows,empty", CASES)
def test_product(T, K, E, A, k, n, fmt, group, kind, token_rows, empty):
    say("w4", T, K, E, A, k, n, fmt, group, kind, token_rows, empty)
    gen = _gen(T + k + n)
    idx = ref.ids(T, K, E, gen, "cuda", empty)
    h = ep.Handle(T, K, E, A)
    h.layout(idx)
    codes, scales = ref.random_w4(E, n, k, fmt, group, gen, "cuda")
    w64 = ref.w4_values(codes, scales, group)
    rows = T if token_rows else h.capacity
    x, sf, x64 = _x(rows, k, kind, gen)
    if not token_rows:                       # what no slot holds would spoil any sum
        gap = torch.ones(rows, dtype=torch.bool, device="cuda")
        gap[ref.rows_of(h, idx)[0]] = False
        if kind == "bf16":
            x[gap] = float("nan")
        else:
            x[gap] = 0x7F
    packed = ep.pack_w4(codes, scales)
    assert (packed.num_experts, packed.n, packed.k, packed.group) == (E, n, k, group)
    out = ref.poisoned((h.capacity, n), torch.bfloat16)
    got = h.expert_w4(x, packed, sf=sf, token_rows=token_rows, out=out)
    assert got is out
    _check(h, idx, x64, w64, _scales64(scales, group, fmt), out, token_rows, "product")
    again = ref.poisoned((h.capacity, n), torch.bfloat16)
    h.expert_w4(x, packed, sf=sf, token_rows=token_rows, out=again)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("fmt,group", [(INT4, 32), (INT4, 64), (INT4, 128), (MX, 32)])
def test_every_code_and_channel(fmt, group):
    """One-hot rows read single weights back: every code value at every channel's
    place, through every lane and record (exact: one product, a power of two)."""
    k, n, T = 384, 40, 384
    codes = (torch.arange(n * k, device="cuda").reshape(1, n, k) * 7 % 16).to(torch.uint8)
    both = (codes[..., 0::2] | (codes[..., 1::2] << 4)).contiguous()
    if fmt == INT4:
        scales = torch.exp2((torch.arange(n * k // group, device="cuda") % 5).float()).reshape(
            1, n, -1).bfloat16()
    else:
        scales = (120 + torch.arange(n * k // group, device="cuda") % 11).reshape(
            1, n, -1).to(torch.uint8)
    w64 = ref.w4_values(both, scales, group)
    idx = torch.zeros((T, 1), dtype=torch.int64, device="cuda")
    h = ep.Handle(T, 1, 1, 1)
    h.layout(idx)
    x = torch.eye(k, device="cuda").bfloat16()
    y = h.expert_w4(x, ep.pack_w4(both, scales))
    assert torch.equal(y.double(), w64[0].t().contiguous())


def test_mxfp4_exponents():
    """The whole range of exponents that bf16 holds, and 255, which makes NaN."""
    k, n = 128, 256
    codes = torch.full((1, n, k // 2), 0x22, dtype=torch.uint8, device="cuda")      # ones
    e = torch.arange(256, device="cuda").reshape(1, n, 1).expand(1, n, 4)
    scales = e.to(torch.uint8).contiguous()
    h = ep.Handle(1, 1, 1, 1)
    h.layout(torch.zeros((1, 1), dtype=torch.int32, device="cuda"))
    x = torch.zeros((1, k), device="cuda").bfloat16()
    x[0, 40] = 1.0
    y = h.expert_w4(x, ep.pack_w4(codes, scales.view(torch.float8_e8m0fnu)))[0].double()
    want = torch.exp2(torch.arange(255, device="cuda").double() - 127.0)
    normal = torch.arange(255, device="cuda") >= 1
    assert torch.equal(y[:255][normal], want[normal])
    assert float(y[0]) in (0.0, 2.0 ** -127) and bool(y[255].isnan())


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_rows_with_infinities_and_nan(kind):
    """A row that holds an infinity or a NaN does not reach the other rows."""
    T, k, n = 20, 256, 32
    gen = _gen(4)
    codes, scales = ref.random_w4(2, n, k, INT4, 64, gen, "cuda")
    idx = torch.zeros((T, 1), dtype=torch.int64, device="cuda")
    h = ep.Handle(T, 1, 2, 1)
    h.layout(idx)
    x = torch.randn((T, k), generator=gen, device="cuda").bfloat16()
    packed = ep.pack_w4(codes, scales)
    q, sf = (x, None) if kind == "bf16" else ep.quantize_fp8(x, kind)
    want = h.expert_w4(q, packed, sf=sf, token_rows=True)
    bad = q.clone()
    if kind == "bf16":
        bad[3, 100] = float("inf")
        bad[9, 7] = float("nan")
    else:
        bad[3, 100] = bad[9, 7] = 0x7F
    got = h.expert_w4(bad, packed, sf=sf, token_rows=True)
    keep = [t for t in range(T) if t not in (3, 9)]
    assert torch.equal(got[keep], want[keep])
    assert bool(got[3].isnan().all()) and bool(got[9].isnan().all())


def test_same_expert_twice_in_a_token():
    gen = _gen(5)
    idx = torch.tensor([[1, 1, 0], [2, 1, 1]], device="cuda")
    h = ep.Handle(2, 3, 3, 4, capacity=24)
    h.layout(idx)
    codes, scales = ref.random_w4(3, 48, 256, MX, 32, gen, "cuda")
    x, sf, x64 = _x(2, 256, "bf16", gen)
    out = ref.poisoned((24, 48), torch.bfloat16)
    h.expert_w4(x, ep.pack_w4(codes, scales), token_rows=True, out=out)
    _check(h, idx, x64, ref.w4_values(codes, scales, 32), None, out, True, "twice")


@pytest.mark.parametrize("popular", [0, 3, 7])
def test_all_rows_on_one_expert(popular):
    """Skewed as far as it goes, the experts before and behind it empty."""
    T, E, k, n = 150, 8, 512, 56
    gen = _gen(6)
    idx = torch.full((T, 1), popular, dtype=torch.int32, device="cuda")
    h = ep.Handle(T, 1, E, 16)
    h.layout(idx)
    codes, scales = ref.random_w4(E, n, k, INT4, 128, gen, "cuda")
    x, sf, x64 = _x(h.capacity, k, "f32", gen)
    out = ref.poisoned((h.capacity, n), torch.bfloat16)
    h.expert_w4(x, ep.pack_w4(codes, scales), sf=sf, out=out)
    _check(h, idx, x64, ref.w4_values(codes, scales, 128), _scales64(scales, 128, INT4), out,
           False, "one expert")


def test_strided_scale_rows():
    gen = _gen(7)
    T, k, n = 30, 1152, 64
    idx = ref.ids(T, 2, 4, gen, "cuda")
    h = ep.Handle(T, 2, 4, 8)
    h.layout(idx)
    codes, scales = ref.random_w4(4, n, k, INT4, 32, gen, "cuda")
    packed = ep.pack_w4(codes, scales)
    x = torch.randn((T, k), generator=gen, device="cuda").bfloat16()
    for kind in ("f32", "ue8m0"):
        q, sf = ep.quantize_fp8(x, kind)
        ex, esf, _ = h.dispatch(q, sf=sf, col_major_sf=True)
        assert esf.stride(0) == 1
        a = h.expert_w4(ex, packed, sf=esf)
        b = h.expert_w4(q, packed, sf=sf, token_rows=True)
        rows = ref.rows_of(h, idx)[0]
        assert torch.equal(a[rows], b[rows])


def test_void_layout_and_no_tokens_write_nothing():
    gen = _gen(8)
    codes, scales = ref.random_w4(8, 16, 128, MX, 32, gen, "cuda")
    packed = ep.pack_w4(codes, scales)
    h = ep.Handle(32, 4, 8, 1, capacity=64)
    h.layout(ref.ids(32, 4, 8, gen, "cuda"))
    out = ref.poisoned((64, 16), torch.bfloat16)
    h.expert_w4(torch.ones((64, 128), device="cuda").bfloat16(), packed, out=out)
    assert ref.untouched(out, [])
    h.layout(torch.empty((0, 4), dtype=torch.int64, device="cuda"))
    h.expert_w4(torch.ones((64, 128), device="cuda").bfloat16(), packed, out=out)
    assert ref.untouched(out, [])
    h.layout(torch.full((9, 4), -1, dtype=torch.int64, device="cuda"))
    h.expert_w4(torch.ones((64, 128), device="cuda").bfloat16(), packed, out=out)
    assert ref.untouched(out, [])


def test_bound_call_and_graph():
    """Bound and captured, the product follows new routing and new rows; every
    replay is compared with the eager calls."""
    gen = _gen(9)
    T, K, E, k, n = 24, 4, 16, 512, 96
    codes, scales = ref.random_w4(E, n, k, INT4, 64, gen, "cuda")
    packed = ep.pack_w4(codes, scales)
    idx = ref.ids(T, K, E, gen, "cuda")
    x = torch.randn((T, k), generator=gen, device="cuda").bfloat16()
    h, ref_h = ep.Handle(T, K, E, 8), ep.Handle(T, K, E, 8)
    lay = h.bind_layout(idx)
    lay()
    out = torch.zeros((h.capacity, n), dtype=torch.bfloat16, device="cuda")
    call = h.bind_expert_w4(x, packed, token_rows=True, out=out)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lay()
        call()
    for _ in range(3):
        idx.copy_(ref.ids(T, K, E, gen, "cuda", 0.2))
        x.copy_(torch.randn((T, k), generator=gen, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        ref_h.layout(idx)
        want = ref_h.expert_w4(x, packed, token_rows=True)
        rows = ref.rows_of(ref_h, idx)[0]
        assert torch.equal(out[rows], want[rows])


@pytest.mark.parametrize("fmt,group", [(INT4, 32), (INT4, 128), (MX, 32)])
@pytest.mark.parametrize("rows", [256, 7])
def test_every_e4m3_code(fmt, group, rows):
    """One-hot FP8 rows of every code (subnormal ones, zeros of both signs and NaN among
    them), the hot channel going round: exact, as code times weight has 7 bits at most."""
    k, n = 256, 24
    gen = _gen(11)
    codes, _ = ref.random_w4(1, n, k, fmt, group, gen, "cuda")
    if fmt == INT4:
        scales = torch.ones((1, n, k // group), device="cuda").bfloat16()
    else:
        scales = torch.full((1, n, k // group), 127, dtype=torch.uint8, device="cuda")
    w64 = ref.w4_values(codes, scales, group)[0]
    code = torch.arange(256, device="cuda").to(torch.uint8)[-rows:]
    ch = torch.arange(rows, device="cuda") * 37 % k
    q = torch.zeros((rows, k), dtype=torch.uint8, device="cuda")
    q[torch.arange(rows, device="cuda"), ch] = code
    h = ep.Handle(rows, 1, 1, 1)
    h.layout(torch.zeros((rows, 1), dtype=torch.int64, device="cuda"))
    sf = torch.ones((rows, k // 128), device="cuda")
    y = h.expert_w4(q, ep.pack_w4(codes, scales), sf=sf).double()
    x = code.view(torch.float8_e4m3fn).double()
    want = x[:, None] * w64.t()[ch]
    nan = x.isnan()
    assert bool(y[nan].isnan().all()) and torch.equal(y[~nan], want[~nan])


def test_more_passes_than_one_launch_takes():
    T, E, k, n = 1_100_000, 4, 128, 8
    gen = _gen(12)
    idx = torch.randint(0, E, (T, 1), generator=gen, device="cuda", dtype=torch.int32)
    h = ep.Handle(T, 1, E, 1)
    h.layout(idx)
    codes, scales = ref.random_w4(E, n, k, INT4, 128, gen, "cuda")
    x = torch.randn((T, k), generator=gen, device="cuda").bfloat16()
    say("w4 passes", T)
    y = h.expert_w4(x, ep.pack_w4(codes, scales), token_rows=True)
    w64 = ref.w4_values(codes, scales, 128)
    s64 = _scales64(scales, 128, INT4)
    rows, expert, token = ref.rows_of(h, idx)
    for e in range(E):
        mine = expert == e
        xe = x[token[mine]].double()
        want = xe @ w64[e].t()
        tol = want.abs() * ref.BF16 + xe.abs() @ (s64[e] * 136.0).t() * 66 * ref.F32
        ref.assert_close(y[rows[mine]], want, tol, f"expert {e}")


def test_offsets_past_32_bits():
    """Rows behind the first 4 GiB of x and of the product."""
    rows, k, n = 300_000, 8192, 8192
    h = ep.Handle(rows, 1, 2, 1)
    idx = torch.zeros((rows, 1), dtype=torch.int32, device="cuda")
    idx[-40:] = 1
    h.layout(idx)
    gen = _gen(13)
    codes, scales = ref.random_w4(2, n, k, MX, 32, gen, "cuda")
    x = torch.zeros((rows, k), dtype=torch.bfloat16, device="cuda")
    x[-90:] = torch.randn((90, k), generator=gen, device="cuda").bfloat16()
    say("w4 offsets", rows, k, n)
    y = h.expert_w4(x, ep.pack_w4(codes, scales))
    w64 = ref.w4_values(codes, scales, 32)
    for e, part in ((0, slice(rows - 90, rows - 40)), (1, slice(rows - 40, rows))):
        x64 = x[part].double()
        want = x64 @ w64[e].t()
        tol = want.abs() * ref.BF16 + x64.abs() @ w64[e].abs().t() * 66 * ref.F32
        ref.assert_close(y[part], want, tol, f"expert {e}")
    assert not bool(y[:rows - 90].any())


FEW = [  # T, K, E, k, n, format, group, x, token rows, all on one expert
    (1, 8, 64, 640, 2064, INT4, 128, "bf16", True, False),
    (1, 8, 64, 512, 2064, MX, 32, "bf16", True, False),
    (1, 8, 64, 896, 2064, MX, 32, "f32", True, False),
    (2, 4, 16, 1152, 104, INT4, 64, "f32", False, False),
    (4, 4, 16, 768, 24, INT4, 32, "ue8m0", True, False),
    (4, 4, 16, 1280, 8, MX, 32, "ue8m0", False, False),
    (16, 1, 16, 640, 40, INT4, 32, "bf16", False, True),
    (13, 1, 13, 1664, 40, MX, 32, "f32", False, True),
    (13, 1, 13, 640, 2064, MX, 32, "bf16", True, True),
    (32, 1, 16, 512, 1040, INT4, 128, "bf16", True, False),
    (4, 1, 4, 8064, 16, INT4, 128, "bf16", False, True),
    (4, 1, 4, 8192, 16, INT4, 128, "bf16", False, True),
    (1, 1, 2, 32768, 16, MX, 32, "f32", True, False),
    (2, 1, 2, 30592, 16, MX, 32, "f32", True, False),
    (2, 1, 2, 32768, 16, MX, 32, "f32", True, True),
    (1, 1, 1, 32640, 24, INT4, 64, "bf16", True, False),
]


@pytest.mark.parametrize("T,K,E,k,n,fmt,group,kind,token_rows,one", FEW)
def test_few_rows(T, K, E, k, n, fmt, group, kind, token_rows, one):
    """A row or two an expert, more on some of them; rows as long as may be held and
    longer; step counts that four waves do not share evenly."""
    say("few", T, K, E, k, n, fmt, group, kind, token_rows, one)
    gen = _gen(T + k + n)
    idx = ref.ids(T, K, E, gen, "cuda", 0.0)
    if one:
        idx = torch.full_like(idx, E - 1)
    h = ep.Handle(T, K, E, 1)
    h.layout(idx)
    codes, scales = ref.random_w4(E, n, k, fmt, group, gen, "cuda")
    x, sf, x64 = _x(T if token_rows else h.capacity, k, kind, gen)
    out = ref.poisoned((h.capacity, n), torch.bfloat16)
    h.expert_w4(x, ep.pack_w4(codes, scales), sf=sf, token_rows=token_rows, out=out)
    _check(h, idx, x64, ref.w4_values(codes, scales, group), _scales64(scales, group, fmt), out,
           token_rows, "few rows")


@pytest.mark.parametrize("fmt,group,kind", [(INT4, 128, "bf16"), (INT4, 32, "f32"),
                                            (MX, 32, "bf16"), (MX, 32, "f32")])
def test_few_rows_with_nan(fmt, group, kind):
    """Rows of one pass, one of them spoilt, and an expert whose weights are."""
    T, E, k, n = 6, 8, 640, 48
    gen = _gen(12)
    codes, scales = ref.random_w4(E, n, k, fmt, group, gen, "cuda")
    idx = torch.tensor([[2], [2], [2], [2], [2], [5]], device="cuda")
    h = ep.Handle(T, 1, E, 1)
    h.layout(idx)
    x, sf, _ = _x(T, k, kind, gen)
    want = h.expert_w4(x, ep.pack_w4(codes, scales), sf=sf, token_rows=True)
    bad = x.clone()
    bad[1, 600] = float("nan") if kind == "bf16" else 0x7F
    scales = scales.clone()
    scales[5, :, -1] = float("nan") if fmt == INT4 else 255
    got = h.expert_w4(bad, ep.pack_w4(codes, scales), sf=sf, token_rows=True)
    assert torch.equal(got[[0, 2, 3, 4]], want[[0, 2, 3, 4]])
    assert bool(got[1].isnan().all()) and bool(got[5].isnan().all())


SPLITS = [  # T, K, E, k, n, format, group, x: every tile and split that the sizes may choose
    (20, 4, 8, 2304, 1248, INT4, 32, "bf16"),       # two waves a group
    (20, 4, 8, 2304, 304, INT4, 64, "f32"),         # four waves a group
    (24, 3, 6, 2048, 904, MX, 32, "ue8m0"),
    (64, 2, 8, 1152, 6200, INT4, 32, "ue8m0"),      # one wave a group, 16 and 32 rows
    (128, 2, 8, 1152, 6200, INT4, 32, "f32"),
    (128, 2, 8, 1152, 6200, MX, 32, "f32"),
    (64, 2, 16, 4224, 6184, INT4, 64, "bf16"),      # 64 outputs a wave
    (130, 2, 16, 4224, 6184, INT4, 64, "f32"),
    (130, 2, 16, 4224, 6184, MX, 32, "bf16"),
    (9, 4, 4, 640, 72, INT4, 128, "f32"),           # a small grid, rows held
    (4, 6, 8, 1024, 72, MX, 32, "f32"),             # few tokens, more rows an expert than one
]


@pytest.mark.parametrize("T,K,E,k,n,fmt,group,kind", SPLITS)
def test_tiles_and_splits(T, K, E, k, n, fmt, group, kind):
    say("splits", T, K, E, k, n, fmt, group, kind)
    gen = _gen(T + k + n)
    idx = ref.ids(T, K, E, gen, "cuda", 0.0)
    h = ep.Handle(T, K, E, 8)
    h.layout(idx)
    codes, scales = ref.random_w4(E, n, k, fmt, group, gen, "cuda")
    x, sf, x64 = _x(h.capacity, k, kind, gen)
    out = ref.poisoned((h.capacity, n), torch.bfloat16)
    h.expert_w4(x, ep.pack_w4(codes, scales), sf=sf, out=out)
    _check(h, idx, x64, ref.w4_values(codes, scales, group), _scales64(scales, group, fmt), out,
           False, "splits")


@pytest.mark.parametrize("fmt,group,kind", [(INT4, 128, "bf16"), (INT4, 32, "f32"),
                                            (MX, 32, "bf16"), (MX, 32, "f32")])
def test_few_rows_captured(fmt, group, kind):
    """A decode step of three tokens captured once: new routing (all rows on one expert,
    empty slots, the same expert twice in a token) and new rows at every replay."""
    gen = _gen(15)
    T, K, E, k, n = 3, 4, 16, 1152, 264
    codes, scales = ref.random_w4(E, n, k, fmt, group, gen, "cuda")
    packed = ep.pack_w4(codes, scales)
    w64, s64 = ref.w4_values(codes, scales, group), _scales64(scales, group, fmt)
    idx = ref.ids(T, K, E, gen, "cuda")
    x, sf, x64 = _x(T, k, kind, gen)
    h = ep.Handle(T, K, E, 1)
    lay = h.bind_layout(idx)
    lay()
    out = torch.zeros((h.capacity, n), dtype=torch.bfloat16, device="cuda")
    call = h.bind_expert_w4(x, packed, sf=sf, token_rows=True, out=out)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lay()
        call()
    routes = [ref.ids(T, K, E, gen, "cuda"), torch.full_like(idx, 7), torch.full_like(idx, -1),
              torch.tensor([[5, 5, -1, 15], [-1, -1, -1, -1], [0, 5, 5, 5]], device="cuda")]
    for route in routes:
        idx.copy_(route)
        q, s, x64 = _x(T, k, kind, gen)
        x.copy_(q)
        if sf is not None:
            sf.copy_(s)
        out.copy_(ref.poisoned((h.capacity, n), torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        _check(h, idx, x64, w64, s64, out, True, "captured")


@pytest.mark.parametrize("fmt,group,kind", [(INT4, 32, "bf16"), (INT4, 128, "f32"),
                                            (MX, 32, "bf16"), (MX, 32, "f32"), (MX, 32, "ue8m0")])
@pytest.mark.parametrize("T,k", [(1, 128), (1, 640), (3, 896), (20, 128), (20, 640), (40, 640)])
def test_small_products_beside_large_ones(fmt, group, kind, T, k):
    """Two large products that cancel and a small one: whatever the order, each partial sum
    has 24 bits at most (MXFP4: 448 * 6 = 21 * 2^7 and 2^-9 * 0.5, 22 bits; INT4: up to
    2 * 279 * 28 < 2^14 and multiples of 2^-6, 20 bits), so binary32 sums are exact."""
    say("w4 small", fmt, group, kind, T, k)
    n = 40
    large, small, c_large, c_small, w_small = ((28.0, 2.0 ** -6, 15, 9, 1.0) if fmt == INT4 else
                                               (448.0, 2.0 ** -9, 7, 1, 0.5))
    code = torch.full((1, n, k), c_large, dtype=torch.uint8, device="cuda")
    code[..., ::4] = c_small
    codes = (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous()
    if fmt == INT4:
        scales = torch.ones((1, n, k // group), device="cuda").bfloat16()
    else:
        scales = torch.full((1, n, k // group), 127, dtype=torch.uint8, device="cuda")
    packed = ep.pack_w4(codes, scales)
    h = ep.Handle(T, 1, 1, 1)
    h.layout(torch.zeros((T, 1), dtype=torch.int64, device="cuda"))
    rows = torch.arange(T, device="cuda")
    for far in (1, 2, 18, 50, 125):                     # places of the three within the row
        at = (rows * 37 + far * 4) % (k // 4) * 4
        x = torch.zeros((T, k), device="cuda")
        x[rows, at] = small
        x[rows, (at + 1) % k] = large
        other = (at + 1 + far) % k
        x[rows, torch.where(other % 4 == 0, (other + 1) % k, other)] = -large
        if kind == "bf16":
            q, sf = x.bfloat16(), None
        else:
            q = x.to(torch.float8_e4m3fn).view(torch.uint8)
            sf = (torch.ones((T, k // 128), device="cuda") if kind == "f32" else
                  torch.full((T, (k // 128 + 3) // 4), 0x7F7F7F7F, dtype=torch.int32,
                             device="cuda"))
        assert bool((x.sum(1) == small).all())
        y = h.expert_w4(q, packed, sf=sf, token_rows=True)
        assert torch.equal(y.double(), torch.full((T, n), small * w_small, device="cuda",
                                                  dtype=torch.float64)), far


@pytest.mark.parametrize("fmt,group", [(INT4, 64), (MX, 32)])
@pytest.mark.parametrize("T,k", [(4, 640), (40, 256)])       # rows held whole, and streamed
def test_layout_content_stays_in_the_buffers(fmt, group, T, k):
    """Segments and source slots outside the buffers (here written into the handle's
    workspace) reach no row outside them.  The buffers lie inside larger ones, whose rest
    must stay untouched and unread."""
    say("w4 bounds", fmt, group, T, k)
    gen = _gen(21)
    n, cap = 40, 2 * T
    codes, scales = ref.random_w4(2, n, k, fmt, group, gen, "cuda")
    packed = ep.pack_w4(codes, scales)
    h = ep.Handle(T, 1, 2, 1, capacity=cap)
    h.layout(torch.ones((T, 1), dtype=torch.int64, device="cuda"))
    whole_x = torch.full((3 * cap, k), float("nan"), device="cuda").bfloat16()
    whole_x[cap:2 * cap] = torch.randn((cap, k), generator=gen, device="cuda").bfloat16()
    whole = ref.poisoned((3 * cap, n), torch.bfloat16)
    x, out = whole_x[cap:2 * cap], whole[cap:2 * cap]
    w64, s64 = ref.w4_values(codes, scales, group)[1], _scales64(scales, group, fmt)

    def close(got, x64, what):
        want = x64 @ w64.t()
        size = x64.abs() @ (w64.abs() if s64 is None else s64[1] * 136.0).t()
        ref.assert_close(got, want, want.abs() * ref.BF16 + size * 66 * ref.F32 + 1e-38, what)

    inside = T // 2
    h.psum[1] = cap - inside                            # the segment's second half lies behind
    h.expert_w4(x, packed, out=out)
    close(out[cap - inside:], x[cap - inside:].double(), "last rows")
    assert ref.untouched(whole, torch.arange(2 * cap - inside, 2 * cap, device="cuda"))
    whole.copy_(ref.poisoned(whole.shape, whole.dtype))
    for start in (-inside, cap):
        h.psum[1] = start
        h.expert_w4(x, packed, out=out)                 # what lies inside may be written
        assert ref.untouched(whole, torch.arange(cap, 2 * cap, device="cuda"))

    h.psum[1] = 0                                       # tokens before and behind the batch
    h.src_meta[:T] = torch.arange(T, device="cuda", dtype=torch.int32)
    h.src_meta[1], h.src_meta[2] = -3, T + 1
    tokens = whole_x[cap:cap + T]
    whole_x[cap + T:] = float("nan")
    h.expert_w4(tokens, packed, token_rows=True, out=out)
    at = torch.arange(T, device="cuda")
    at[1], at[2] = 0, T - 1
    close(out[:T], tokens[at].double(), "tokens")


def test_a_copied_handle_of_fewer_tokens():
    """What a captured call sees after a layout of a larger batch: rows of its own tokens
    are right, and no row behind its batch is read."""
    gen = _gen(22)
    T, K, E, k, n = 12, 2, 4, 384, 24
    codes, scales = ref.random_w4(E, n, k, INT4, 128, gen, "cuda")
    packed = ep.pack_w4(codes, scales)
    w64 = ref.w4_values(codes, scales, 128)
    s64 = _scales64(scales, 128, INT4)
    h = ep.Handle(2 * T, K, E, 1)
    few, many = ref.ids(T, K, E, gen, "cuda"), ref.ids(2 * T, K, E, gen, "cuda")
    h.layout(few)
    old = ep.ep_handle.from_buffer_copy(h.h)
    whole = torch.full((2 * T, k), float("nan"), device="cuda").bfloat16()
    whole[:T] = torch.randn((T, k), generator=gen, device="cuda").bfloat16()
    out = ref.poisoned((h.capacity, n), torch.bfloat16)
    h.layout(many)
    say("w4 copied handle")
    status = ep.ep_expert_w4(old, whole.data_ptr(), ep.EP_BF16, 1, k, None, 0, 0, 0,
                             packed.codes.data_ptr(), packed.scales.data_ptr(), INT4, 128, n,
                             out.data_ptr(), ep._stream())
    assert status == ep.EP_OK
    rows, expert, token = ref.rows_of(h, many)
    written = (out[rows].view(torch.int16) != 0x5A5A).any(1)
    assert not bool(out[rows][written].isnan().any())
    mine = written & (token < T)
    assert bool(mine.any())
    x64 = whole[token[mine]].double()
    want = torch.stack([x64[i] @ w64[e].t() for i, e in enumerate(expert[mine].tolist())])
    size = torch.stack([x64[i].abs() @ (s64[e] * 136.0).t()
                        for i, e in enumerate(expert[mine].tolist())])
    ref.assert_close(out[rows[mine]], want, want.abs() * ref.BF16 + size * 66 * ref.F32, "own")


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,k", [(1, 128), (2, 640), (20, 256), (40, 640)])
def test_int4_range_of_a_groups_sum(group, T, k):
    """Partial sums reach 136 times a group's sum of |x|.  With channels of one sign and
    a sum of 1.75 * 2^120 (238 * 2^120 < 2^128) every product is right; with four times
    as much the row is infinite or NaN, never a wrong finite number."""
    say("w4 range", group, T, k)
    gen = _gen(23)
    n = 40
    codes, _ = ref.random_w4(1, n, k, INT4, group, gen, "cuda")
    scales = torch.full((1, n, k // group), 2.0 ** -20, device="cuda").bfloat16()
    packed = ep.pack_w4(codes, scales)
    h = ep.Handle(T, 1, 1, 1)
    idx = torch.zeros((T, 1), dtype=torch.int64, device="cuda")
    h.layout(idx)
    sign = torch.where(torch.arange(T, device="cuda") % 2 == 0, 1.0, -1.0)
    x = (sign[:, None] * torch.full((T, k), 1.75 * 2.0 ** 120 / group, device="cuda")).bfloat16()
    y = h.expert_w4(x, packed, token_rows=True)
    assert bool(torch.isfinite(y).all())
    _check(h, idx, x.double(), ref.w4_values(codes, scales, group),
           _scales64(scales, group, INT4), y, True, "range")
    y = h.expert_w4(x * 4, packed, token_rows=True)
    assert not bool(torch.isfinite(y).any())


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,k", [(1, 128), (1, 640), (20, 128), (20, 640)])
@pytest.mark.parametrize("x,code,weight,sf", [(1.0, 0x22, 1.0, 1.0), (2.0 ** -9, 0x11, 0.5, 2.0 ** 20),
                                              (448.0, 0x77, 6.0, 2.0 ** -20)])
def test_mxfp4_every_exponent(kind, T, k, x, code, weight, sf):
    """Every exponent byte in both kinds of rows: byte 0 is 2^-127, products below the
    normal range are kept, and what leaves binary32 before x's scale is infinite: a product,
    or a weight (6 * 2^126 and up), which times the row's zeros is NaN."""
    n = 256
    codes = torch.full((1, n, k // 2), code, dtype=torch.uint8, device="cuda")
    e = torch.arange(256, device="cuda").reshape(1, n, 1).expand(1, n, k // 32)
    h = ep.Handle(T, 1, 1, 1)
    h.layout(torch.zeros((T, 1), dtype=torch.int32, device="cuda"))
    say("w4 exponents", kind, T, k, x)
    row = torch.zeros((T, k), device="cuda")
    row[torch.arange(T, device="cuda"), (torch.arange(T, device="cuda") * 37 + 40) % k] = x
    packed = ep.pack_w4(codes, e.to(torch.uint8).contiguous())
    if kind == "bf16":
        sf, y = 1.0, h.expert_w4(row.bfloat16(), packed, token_rows=True)
    else:
        y = h.expert_w4(row.to(torch.float8_e4m3fn).view(torch.uint8), packed, token_rows=True,
                        sf=torch.full((T, k // 128), sf, device="cuda"))
    before = x * weight * torch.exp2(torch.arange(255, device="cuda").double() - 127.0)
    want = torch.where(before >= 2.0 ** 128, float("inf"), before * sf)
    want = want.float().bfloat16().double()         # 1, 1/2 and 21 * 2^7 times powers of two
    fits = int((before / x < 2.0 ** 128).sum())
    assert torch.equal(y[:, :fits].double(), want[:fits].expand(T, fits))
    assert fits == (253 if weight == 6.0 else 255) and bool(y[:, fits:].isnan().all())
