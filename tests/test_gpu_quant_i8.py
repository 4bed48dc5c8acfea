"""The int8 quantiser's forms for many rows, on the GPU: codes and scales equal to the recipe's,
s = max(max |row|, 1e-12) / 127 and rint(x / s), both divisions in binary32."""
import pytest
import torch

import combine_ep_layout_08_amd as ep
from tests import layer_ref as ref
from tests.gpu_util import needs_gpu, say

pytestmark = [pytest.mark.gpu, needs_gpu]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rows(T, C, gen):
    """Rows whose sizes differ by up to 2^16, so that a row's scale is its own."""
    size = torch.exp2(torch.randint(-8, 9, (T, 1), generator=gen, device="cuda").float())
    return (torch.randn((T, C), generator=gen, device="cuda") * size).bfloat16()


def _recipe(x):
    f = x.float()
    s = torch.clamp(f.abs().amax(1), min=1e-12)
    s = s / torch.full_like(s, 127.0)
    return torch.round(f / s[:, None]).to(torch.int8), s


def test_more_slots_than_a_launch_has_rows():
    """2^24 + 8 slots, nearly all of them empty, of rows that four waves share: the routed ones
    lie at both ends and on both sides of every 2^22nd slot."""
    T, K, E, C = 2 ** 21 + 1, 8, 4, 4112
    say("quantize_i8 rows, many slots", T, K, E, C)
    idx = torch.full((T, K), -1, dtype=torch.int32, device="cuda")
    at = [0, T * K - 1] + [i * 2 ** 22 + d for i in range(1, 5) for d in (-1, 0, 1)]
    idx.view(-1)[torch.tensor(at, device="cuda")] = \
        (torch.arange(len(at), device="cuda") % E).to(torch.int32)
    h = ep.Handle(T, K, E, 2, capacity=32)
    h.layout(idx)
    rows = ref.rows_of(h, idx)[0]
    assert rows.numel() == len(at)
    x = _rows(h.capacity, C, _gen(41))
    q, s = ref.poisoned((h.capacity, C), torch.int8), ref.poisoned((h.capacity,), torch.float32)
    h.quantize_i8(x, out_q=q, out_scale=s)
    wq, ws = _recipe(x[rows])
    assert torch.equal(q[rows], wq) and torch.equal(s[rows], ws)
    assert ref.untouched(q, rows) and ref.untouched(s[:, None], rows)
