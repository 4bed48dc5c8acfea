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


# on both sides of every number of channels at which a row's form changes
CHANNELS = [16, 496, 512, 528, 1024, 1040, 2048, 2064, 4096, 4112, 8192, 8208, 32752, 32768]


@pytest.mark.parametrize("C", CHANNELS)
@pytest.mark.parametrize("T", [2047, 2048, 2051])
def test_many_rows(T, C):
    say("quantize_i8", T, C)
    x = _rows(T, C, _gen(T + C))
    x[5] = 0.0
    x[T - 1, C - 1] = 2.0 ** 12            # the last channel of all has the row's largest value
    for r, bad in ((0, float("nan")), (1027, float("inf")), (T - 2, -float("inf"))):
        x[r, (r * 7) % C] = bad
    q, s = ref.poisoned((T, C), torch.int8), ref.poisoned((T,), torch.float32)
    assert ep.quantize_i8(x, out_q=q, out_scale=s) == (q, s)
    bad = torch.tensor([0, 1027, T - 2], device="cuda")
    fine = torch.ones(T, dtype=torch.bool, device="cuda")
    fine[bad] = False
    wq, ws = _recipe(x[fine])
    assert torch.equal(s[fine], ws) and torch.equal(q[fine], wq)
    assert bool(s[bad].isnan().all()) and bool((q[bad] == 0).all())


@pytest.mark.parametrize("C", CHANNELS)
@pytest.mark.parametrize("T,K,E,A,empty", [(682, 3, 7, 16, 0.2), (683, 3, 7, 16, 0.2),
                                           (2049, 1, 5, 1, 0.3)])
def test_many_expert_rows(T, K, E, A, empty, C):
    """2046 slots and 2049 of them, some empty; rows without a slot hold what would show."""
    say("quantize_i8 rows", T, K, E, A, C)
    gen = _gen(T + C)
    idx = ref.ids(T, K, E, gen, "cuda", empty)
    h = ep.Handle(T, K, E, A)
    h.layout(idx)
    rows = ref.rows_of(h, idx)[0]
    x = _rows(h.capacity, C, gen)
    bad = rows[torch.tensor([0, rows.numel() // 2, rows.numel() - 1], device="cuda")]
    x[bad, torch.tensor([0, C // 2, C - 1], device="cuda")] = \
        torch.tensor([float("inf"), float("nan"), -float("inf")], device="cuda").bfloat16()
    q, s = ref.poisoned((h.capacity, C), torch.int8), ref.poisoned((h.capacity,), torch.float32)
    h.quantize_i8(x, out_q=q, out_scale=s)
    fine = rows[~torch.isin(rows, bad)]
    wq, ws = _recipe(x[fine])
    assert torch.equal(s[fine], ws) and torch.equal(q[fine], wq)
    assert bool(s[bad].isnan().all()) and bool((q[bad] == 0).all())
    assert ref.untouched(q, rows) and ref.untouched(s[:, None], rows)


def test_many_rows_of_every_magnitude():
    """Rows over bf16's whole range of exponents, with ties among their quotients, as often as
    the form for many rows takes."""
    rows = []
    for e in range(-133, 127):
        v = torch.arange(256, dtype=torch.float64) - 127.5
        rows.append(v * 2.0 ** (e - 8 if e > -120 else e))
    few = torch.stack(rows).float().bfloat16().cuda()
    x = few.repeat(8, 1).contiguous()
    assert x.shape[0] >= 2048
    q, s = ep.quantize_i8(x)
    wq, ws = _recipe(x)
    assert torch.equal(s, ws) and torch.equal(q, wq)
