"""Bound calls of the gated feed-forward block, on the GPU: every call works on what the bound
tensors hold when it is made, and gives what the method gives, bit for bit."""
import pytest
import torch

import combine_ep_layout_08_amd as ep
from tests import layer_ref as ref
from tests.gpu_util import needs_gpu, say

pytestmark = [pytest.mark.gpu, needs_gpu]


def _randn(shape, gen, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).bfloat16()


@pytest.mark.parametrize("token_rows,weights,saved,down", [(True, False, False, True),
                                                           (False, True, True, True),
                                                           (True, True, True, False)])
@pytest.mark.parametrize("T,K,E,A,H,I", [(24, 2, 8, 8, 256, 64), (130, 3, 5, 16, 264, 136)])
def test_block(T, K, E, A, H, I, token_rows, weights, saved, down):  # noqa: E741
    say("bound ffn", T, K, E, A, H, I, token_rows, weights, saved, down)
    gen = torch.Generator(device="cuda").manual_seed(T + H)
    h = ep.Handle(T, K, E, A)
    idx = ref.ids(T, K, E, gen, "cuda", 0.1)
    h.layout(idx)
    rows_in = T if token_rows else h.capacity
    x = _randn((rows_in, H), gen)
    w13, w2 = _randn((E, 2 * I, H), gen, H ** -0.5), _randn((E, H, I), gen, I ** -0.5)
    w2 = w2 if down else None
    rw = torch.rand(h.capacity, generator=gen, device="cuda") if weights else None
    call = ep.bind_expert_ffn(h, x, w13, w2, row_weights=rw, token_rows=token_rows,
                              want_saved=saved)
    before = None
    for turn in range(3):
        x.copy_(_randn(x.shape, gen))
        w13.copy_(_randn(w13.shape, gen, H ** -0.5))
        if weights:
            rw.copy_(torch.rand(rw.shape, generator=gen, device="cuda"))
        idx.copy_(ref.ids(T, K, E, gen, "cuda", 0.1 * turn))
        h.layout(idx)
        rows = ref.rows_of(h, idx)[0]
        for t in call._result:
            if t is not None:
                t.view(torch.uint8).fill_(ref.POISON)
        got = call()
        want = h.expert_ffn(x, w13, w2, row_weights=rw, token_rows=token_rows, want_saved=saved)
        assert [t is None for t in got] == [not down, False, not saved]
        for a, b in zip(got, want):
            assert (a is None) == (b is None)
            if a is not None:
                assert bool(b[rows].isfinite().all()) and float(b[rows].float().abs().max()) > 0
                assert torch.equal(a[rows].view(torch.int16), b[rows].view(torch.int16))
                assert ref.untouched(a, rows)
        kept = got[1][rows].clone()
        assert before is None or kept.shape != before.shape or not torch.equal(kept, before)
        before = kept
