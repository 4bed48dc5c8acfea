"""The layer operators together with layout, dispatch, combine and their
gradients, as a serving step and a training step use them."""
import pytest
import torch

import combine_ep_layout_08_amd as ep
from tests import layer_ref as ref
from tests.gpu_util import needs_gpu, say

pytestmark = [pytest.mark.gpu, needs_gpu]
EPS = 1e-6


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(shape, gen, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).bfloat16()


class Serving:
    """A decode layer: norm, layout, dispatch in FP8, two 4-bit products around
    the activation, combine.  All buffers are made once."""

    def __init__(self, T, H, inter, E, K, A, gen, fmt):
        self.H, self.inter, self.E, self.K, self.fmt = H, inter, E, K, fmt
        up = ref.random_w4(E, 2 * inter, H, ep.EP_W4_MXFP4, 32, gen, "cuda")
        down = ref.random_w4(E, H, inter, ep.EP_W4_INT4, 64, gen, "cuda")
        self.up64 = ref.w4_values(*up, 32)
        self.down64 = ref.w4_values(*down, 64)
        self.up, self.down = ep.pack_w4(*up), ep.pack_w4(*down)
        self.norm_w = _randn((H,), gen, 0.1) + 1.0
        self.x, self.residual = _randn((T, H), gen), _randn((T, H), gen)
        self.idx = ref.ids(T, K, E, gen, "cuda", 0.1)
        self.w = torch.rand((T, K), generator=gen, device="cuda")
        self.h = ep.Handle(T, K, E, A)

    def step(self):
        h = self.h
        y, z, q, sf, _ = ep.add_rmsnorm(self.x, self.norm_w, residual=self.residual, eps=EPS,
                                        scale_format=self.fmt)
        h.layout(self.idx)
        ex, esf, _ = h.dispatch(q, sf=sf)
        gu = h.expert_w4(ex, self.up, sf=esf)
        a, asf, _, _ = h.swiglu(gu, scale_format=self.fmt)
        o = h.expert_w4(a, self.down, sf=asf)
        return z, y, gu, a, asf, o, h.combine(o, topk_weights=self.w)


@pytest.mark.parametrize("fmt", ["f32", "ue8m0"])
def test_serving_step(fmt):
    """Each step against binary64 from what the step before left, and the step as a
    whole: two roundings to E4M3 (2^-4 each) and five to bf16 on the way."""
    say("serving step", fmt)
    s = Serving(48, 512, 256, 16, 4, 16, _gen(1), fmt)
    z, y, gu, a, asf, o, out = s.step()
    rows, expert, token = ref.rows_of(s.h, s.idx)
    z64 = s.x.double() + s.residual.double()
    n64 = z64 / torch.sqrt(z64.square().mean(1, keepdim=True) + EPS) * s.norm_w.double()
    g64 = torch.stack([n64[t] @ s.up64[e].t() for e, t in zip(expert.tolist(), token.tolist())])
    a64 = ref.swiglu(g64)
    o64 = torch.stack([a64[i] @ s.down64[e].t() for i, e in enumerate(expert.tolist())])
    slot = s.h.src_meta[rows].long()
    want = torch.zeros_like(z64).index_add_(0, token, o64 * s.w.reshape(-1)[slot].double()[:, None])
    rel = lambda p, q: float((p.double() - q).norm() / q.norm())  # noqa: E731
    # a rounding of every element by at most 2^-4 moves a row's norm by no more,
    # and a random product of it by as much
    assert rel(gu[rows], g64) < 2.0 ** -4
    # in slope and value the activation carries gate's and up's errors
    assert rel(ref.code_values(a[rows], asf[rows]), a64) < 3 * 2.0 ** -4
    assert rel(o[rows], o64) < 3 * 2.0 ** -4
    assert rel(out, want) < 3 * 2.0 ** -4
    assert bool((out[0] == 0).all())                        # the token without a slot


def test_tokens_own_rows_give_what_dispatch_gives():
    gen = _gen(2)
    T, K, E, k, n = 40, 4, 16, 640, 72
    idx = ref.ids(T, K, E, gen, "cuda", 0.2)
    h = ep.Handle(T, K, E, 32)
    h.layout(idx)
    packed = ep.pack_w4(*ref.random_w4(E, n, k, ep.EP_W4_INT4, 128, gen, "cuda"))
    x = _randn((T, k), gen)
    rows = ref.rows_of(h, idx)[0]
    a = h.expert_w4(x, packed, token_rows=True)
    b = h.expert_w4(h.dispatch(x)[0], packed)
    assert torch.equal(a[rows], b[rows])


def test_serving_step_in_a_graph():
    """The whole step captured; every replay on new inputs equals the eager step."""
    s = Serving(16, 256, 128, 8, 2, 8, _gen(3), "f32")
    gen = _gen(4)
    s.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = s.step()
    for k in range(3):
        s.x.copy_(_randn(s.x.shape, gen))
        s.idx.copy_(ref.ids(16, 2, 8, gen, "cuda", 0.1 * k))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        want = s.step()
        rows = ref.rows_of(s.h, s.idx)[0]
        for i, (a, b) in enumerate(zip(kept, want)):
            if i in (2, 3, 4, 5):
                a, b = a[rows], b[rows]
            assert torch.equal(a, b), i


def test_two_streams():
    """Two steps on two streams, with their own handles and buffers, give what each
    gives alone."""
    steps = [Serving(32, 512, 256, 16, 4, 8, _gen(5 + i), "f32") for i in range(2)]
    want = [s.step() for s in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(steps):
            streams[i].wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(streams[i]):
                got[i] = s.step()
    torch.cuda.synchronize()
    for s, a, b in zip(steps, got, want):
        rows = ref.rows_of(s.h, s.idx)[0]
        assert torch.equal(a[-1], b[-1]) and torch.equal(a[2][rows], b[2][rows])


def _experts(x, weights, rows, expert):
    """The caller's own products with full weights, fp32, rounded to bf16."""
    out = torch.zeros((x.shape[0], weights.shape[1]), dtype=torch.bfloat16, device=x.device)
    for e in torch.unique(expert).tolist():
        r = rows[expert == e]
        out[r] = (x[r].float() @ weights[e].float().t()).bfloat16()
    return out


@pytest.mark.parametrize("checkpoint", [None, "f32", "ue8m0"])
def test_training_step(checkpoint):
    """Forward and backward of a layer against binary64 autograd.  Without a
    checkpoint a dozen bf16 roundings of 2^-8 lie on the way (a product's norm
    moves by no more than its factors'); the E4M3 one adds 2^-4 to what the
    activation's gradients are taken from, and none to the forward pass."""
    say("training step", checkpoint)
    gen = _gen(9)
    T, H, inter, E, K, A = 64, 256, 128, 8, 2, 8
    x, residual = _randn((T, H), gen), _randn((T, H), gen)
    nw = torch.randn(H, generator=gen, device="cuda") * 0.1 + 1.0
    w1, w2 = _randn((E, 2 * inter, H), gen, H ** -0.5), _randn((E, H, inter), gen, inter ** -0.5)
    idx = ref.ids(T, K, E, gen, "cuda", 0.1)
    topw = torch.rand((T, K), generator=gen, device="cuda") + 0.2
    gout, gz = _randn((T, H), gen), _randn((T, H), gen)

    h = ep.Handle(T, K, E, A)
    y, z, _, _, rstd = ep.add_rmsnorm(x, nw, residual=residual, eps=EPS, want_rstd=True)
    h.layout(idx)
    ex, _, ew = h.dispatch(y, topk_weights=topw, want_weights=True)
    rows, expert, token = ref.rows_of(h, idx)
    gu = _experts(ex, w1, rows, expert)
    a, _, saved, ssf = h.swiglu(gu, row_weights=ew, checkpoint=checkpoint)
    out = h.combine(_experts(a, w2, rows, expert))
    go, _, _ = h.combine_backward(gout)
    ga = _experts(go, w2.transpose(1, 2).contiguous(), rows, expert)
    ggu, gew, again = h.swiglu_backward(ga, gu if saved is None else saved, ssf, row_weights=ew,
                                        want_grad_weights=True, want_h=True)
    gex = _experts(ggu, w1.transpose(1, 2).contiguous(), rows, expert)
    gy, gtopw = h.dispatch_backward(gex, grad_out_w=gew, want_grad_weights=True)
    gx, gnw = ep.add_rmsnorm_backward(gy, z, nw, rstd, grad_residual=gz)
    gw2 = torch.stack([go[r].float().t() @ again[r].float()
                       for r in (rows[expert == e] for e in range(E))])

    leaf = [t.double().requires_grad_() for t in (x, nw, topw, w2)]
    x6, nw6, tw6, w26 = leaf
    z6 = x6 + residual.double()
    y6 = z6 / torch.sqrt(z6.square().mean(1, keepdim=True) + EPS) * nw6
    slot = h.src_meta[rows].long()
    g6 = torch.stack([w1[e].double() @ y6[t] for e, t in zip(expert.tolist(), token.tolist())])
    gate, up = g6.chunk(2, 1)
    a6 = gate * torch.sigmoid(gate) * up * tw6.reshape(-1)[slot][:, None]
    o6 = torch.stack([w26[e] @ a6[i] for i, e in enumerate(expert.tolist())])
    out6 = torch.zeros((T, H), dtype=torch.float64, device="cuda").index_add(0, token, o6)
    ((out6 * gout.double()).sum() + (z6 * gz.double()).sum()).backward()
    rel = lambda p, q: float((p.double() - q).norm() / q.norm())  # noqa: E731
    plain = 12 * ref.BF16
    eight = plain + (0 if checkpoint is None else 2 * 2.0 ** -4)
    assert rel(out, out6.detach()) < plain
    assert rel(gx, x6.grad) < eight
    assert rel(gnw, nw6.grad) < eight
    assert rel(gtopw, tw6.grad) < eight
    assert rel(gw2, w26.grad) < eight
    assert bool((gtopw[idx < 0] == 0).all())
