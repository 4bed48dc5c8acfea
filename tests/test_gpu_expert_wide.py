"""The widest block, on the GPU: 32768 channels in and between, so that one expert's up and gate
weights are 4 GiB and the places of their rows go past 31 bits of the expert's own start.  Only
the second expert has rows: whatever lies before its weights is the first one's."""
import pytest
import torch

import combine_ep_layout_08_amd as ep
from tests import layer_ref as ref
from tests.gpu_util import needs_gpu, say

pytestmark = [pytest.mark.gpu, needs_gpu]
BF16, F32 = ref.BF16, ref.F32
WIDE = 32768
PART = 2048


def _sum_tol(K):
    """Of the sum of |x w|: K roundings inside the matrix instructions, one for each of their sums."""
    return (K + K // 32 + 1) * F32


def _weights(shape, gen):
    w = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for e in range(shape[0]):
        for p in range(0, shape[1], 8192):
            w[e, p:p + 8192] = torch.randn((8192, shape[2]), generator=gen, device="cuda") \
                .mul_(shape[2] ** -0.5).bfloat16()
    return w


@pytest.mark.parametrize("token_rows", [True, False])
def test_widest_block(token_rows):
    say("widest block", token_rows)
    T, E, H, I = 5, 2, WIDE, WIDE  # noqa: E741
    gen = torch.Generator(device="cuda").manual_seed(51)
    h = ep.Handle(T, 1, E, 1)
    idx = torch.ones((T, 1), dtype=torch.int64, device="cuda")
    h.layout(idx)
    rows = ref.rows_of(h, idx)[0]
    w13, w2 = _weights((E, 2 * I, H), gen), _weights((E, H, I), gen)
    assert w13[0].numel() * 2 == 2 ** 32
    x = torch.randn((T if token_rows else h.capacity, H), generator=gen, device="cuda").bfloat16()
    gy = (torch.randn((h.capacity, H), generator=gen, device="cuda") * 0.1).bfloat16()
    y, hh, saved = h.expert_ffn(x, w13, w2, token_rows=token_rows, want_saved=True)
    gx, g13, g2, _, ggu = h.expert_ffn_backward(gy, x, w13, w2, saved, hh, token_rows=token_rows)
    src = x.double() if token_rows else x[rows].double()
    low = ggu[rows].double()
    want_x = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    size_x = torch.zeros_like(want_x)
    for p in range(0, 2 * I, PART):
        w = w13[1, p:p + PART].double()
        want = src @ w.t()
        ref.assert_close(saved[rows, p:p + PART], want, (src.abs() @ w.abs().t()) * _sum_tol(H) +
                         want.abs() * BF16 + 1e-38, f"gate_up {p}")
        want_x += low[:, p:p + PART] @ w
        size_x += low[:, p:p + PART].abs() @ w.abs()
        want = low[:, p:p + PART].t() @ src
        size = low[:, p:p + PART].abs().t() @ src.abs()
        ref.assert_close(g13[1, p:p + PART], want, size * _sum_tol(T) + want.abs() * BF16 + 1e-38,
                         f"gradient of w13 {p}")
    ref.assert_close(gx[rows], want_x, size_x * _sum_tol(2 * I) + want_x.abs() * BF16 + 1e-38,
                     "gradient of x")
    act, g = hh[rows].double(), gy[rows].double()
    gh, size_h = torch.zeros((T, I), dtype=torch.float64, device="cuda"), 0
    for p in range(0, H, PART):
        w = w2[1, p:p + PART].double()
        want = act @ w.t()
        ref.assert_close(y[rows, p:p + PART], want, (act.abs() @ w.abs().t()) * _sum_tol(I) +
                         want.abs() * BF16 + 1e-38, f"y {p}")
        gh += g[:, p:p + PART] @ w
        size_h = size_h + g[:, p:p + PART].abs() @ w.abs()
        want = g[:, p:p + PART].t() @ act
        size = g[:, p:p + PART].abs().t() @ act.abs()
        ref.assert_close(g2[1, p:p + PART], want, size * _sum_tol(T) + want.abs() * BF16 + 1e-38,
                         f"gradient of w2 {p}")
    # gradient of up: gh silu(gate), sigmoid within (6 + 2 |gate|) 2^-24
    gate = saved[rows, :I].double()
    silu = gate * torch.sigmoid(gate)
    want = gh * silu
    ref.assert_close(ggu[rows, I:], want, size_h * _sum_tol(H) * silu.abs() +
                     want.abs() * (BF16 + (16 + 6 * gate.abs()) * F32) + 1e-37, "gradient of up")
    assert bool((g13[0] == 0).all()) and bool((g2[0] == 0).all())


def test_widest_int8_product():
    """65536 outputs of 32768 channels: 2 GiB of codes an expert."""
    T, E, k, n = 3, 2, WIDE, 2 * WIDE
    say("widest int8 product", T, E, k, n)
    gen = torch.Generator(device="cuda").manual_seed(52)
    h = ep.Handle(T, 1, E, 1)
    idx = torch.ones((T, 1), dtype=torch.int64, device="cuda")
    h.layout(idx)
    rows = ref.rows_of(h, idx)[0]
    w = torch.randint(-128, 128, (E, n, k), generator=gen, device="cuda", dtype=torch.int8)
    ws = torch.rand((E, n), generator=gen, device="cuda") * 1e-3 + 1e-4
    x = torch.randint(-127, 128, (T, k), generator=gen, device="cuda", dtype=torch.int8)
    xs = torch.rand(T, generator=gen, device="cuda") * 0.02 + 1e-3
    out = h.expert_i8(x, xs, w, ws, token_rows=True)
    for p in range(0, n, PART):
        v = x.double() @ w[1, p:p + PART].double().t()
        want = v * xs.double()[:, None] * ws[1, p:p + PART].double()
        ref.assert_close(out[rows, p:p + PART], want, want.abs() * (BF16 + 4 * F32) + 1e-38,
                         f"int8 {p}")
