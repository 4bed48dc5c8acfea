"""The experts' products together with layout, dispatch, combine and their gradients, as a
serving step in 8 bits and a training step use them: against binary64, captured, and on two
streams at once."""
import subprocess
import sys

import pytest
import torch

import combine_ep_layout_08_amd as ep
from tests import layer_ref as ref
from tests.gpu_util import needs_gpu, say

pytestmark = [pytest.mark.gpu, needs_gpu]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(shape, gen, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).bfloat16()


def _rel(p, q):
    return float((p.double() - q.double()).norm() / q.double().norm())


def _bits(t):
    return t.contiguous().view(torch.uint8)


class Int8Serving:
    """A layer that serves in 8 bits: norm, int8 rows, both products on them, combine."""

    def __init__(self, T, H, inter, E, K, A, gen):
        self.E, self.K, self.T = E, K, T
        self.w13, self.s13 = ep.quantize_i8(_randn((E * 2 * inter, H), gen, H ** -0.5))
        self.w2, self.s2 = ep.quantize_i8(_randn((E * H, inter), gen, inter ** -0.5))
        self.w13, self.s13 = self.w13.reshape(E, 2 * inter, H), self.s13.reshape(E, 2 * inter)
        self.w2, self.s2 = self.w2.reshape(E, H, inter), self.s2.reshape(E, H)
        self.norm_w = _randn((H,), gen, 0.1) + 1.0
        self.x, self.residual = _randn((T, H), gen), _randn((T, H), gen)
        self.idx = ref.ids(T, K, E, gen, "cuda", 0.1 if T > 1 else 0.0)
        self.w = torch.rand((T, K), generator=gen, device="cuda")
        self.h = ep.Handle(T, K, E, A)

    def step(self):
        h = self.h
        y, z, _, _, _ = ep.add_rmsnorm(self.x, self.norm_w, residual=self.residual)
        h.layout(self.idx)
        q, s = ep.quantize_i8(y)
        act = h.expert_i8(q, s, self.w13, self.s13, gated=True, token_rows=True)
        aq, as_ = h.quantize_i8(act)
        o = h.expert_i8(aq, as_, self.w2, self.s2)
        return z, y, q, s, act, aq, as_, o, h.combine(o, topk_weights=self.w)


@pytest.mark.parametrize("T,H,inter,E,K,A", [(48, 512, 256, 16, 4, 16), (1, 1040, 80, 8, 8, 1),
                                             (200, 272, 528, 4, 2, 8)])
def test_int8_serving_step(T, H, inter, E, K, A):
    """The whole step against binary64 on the int8 weights' values.  A code is off by half a step
    at most, amax / 254: its row by sqrt(channels) amax / 254 at most, which is taken in terms of
    the row's norm (sqrt(channels) / 254 of it at most, as amax is no more than the norm); the product
    of an error with random weights is as large as the product itself times that.  Two such
    roundings, and the first's error in gate and up twice."""
    say("int8 serving", T, H, inter, E, K, A)
    s = Int8Serving(T, H, inter, E, K, A, _gen(T))
    z, y, q, sc, act, aq, as_, o, out = s.step()
    rows, expert, token = ref.rows_of(s.h, s.idx)
    w13, w2 = s.w13.double() * s.s13.double()[..., None], s.w2.double() * s.s2.double()[..., None]
    most = lambda t: float((t.double().abs().amax(1) * t.shape[1] ** 0.5 / 254 /  # noqa: E731
                            t.double().norm(dim=1)).max())
    first, second = most(y), most(act[rows])
    assert first <= H ** 0.5 / 254 and second <= inter ** 0.5 / 254
    a64 = torch.empty((len(rows), inter), dtype=torch.float64, device="cuda")
    o64 = torch.empty((len(rows), H), dtype=torch.float64, device="cuda")
    for i, (e, t) in enumerate(zip(expert.tolist(), token.tolist())):
        g, u = (w13[e] @ y[t].double()).chunk(2)
        a64[i] = g * torch.sigmoid(g) * u
        o64[i] = w2[e] @ a64[i]
    assert _rel(act[rows], a64) < 3 * first
    assert _rel(o[rows], o64) < 3 * first + second + 2 * ref.BF16
    slot = s.h.src_meta[rows].long()
    want = torch.zeros((T, H), dtype=torch.float64, device="cuda").index_add_(
        0, token, o64 * s.w.reshape(-1)[slot].double()[:, None])
    if bool((want != 0).any()):
        assert _rel(out, want) < 3 * first + second + 3 * ref.BF16


class Training:
    """Dispatch, the block, combine, and back."""

    def __init__(self, T, H, inter, E, K, A, gen, weights_in_rows):
        self.x, self.gy = _randn((T, H), gen), _randn((T, H), gen, 0.1)
        self.w13 = _randn((E, 2 * inter, H), gen, H ** -0.5)
        self.w2 = _randn((E, H, inter), gen, inter ** -0.5)
        self.idx = ref.ids(T, K, E, gen, "cuda", 0.1)
        self.w = torch.rand((T, K), generator=gen, device="cuda") + 0.25
        self.h = ep.Handle(T, K, E, A)
        self.in_rows = weights_in_rows           # the router's weights: in the block, or in combine

    def step(self):
        h = self.h
        h.layout(self.idx)
        ex, _, ew = h.dispatch(self.x, topk_weights=self.w, want_weights=True)
        rw = ew if self.in_rows else None
        y, hh, saved = h.expert_ffn(ex, self.w13, self.w2, row_weights=rw, want_saved=True)
        out = h.combine(y, topk_weights=None if self.in_rows else self.w)
        gy, gw, _ = h.combine_backward(self.gy, topk_weights=None if self.in_rows else self.w, y=y,
                                       want_grad_weights=not self.in_rows)
        gx, g13, g2, grw, ggu = h.expert_ffn_backward(
            gy, ex, self.w13, self.w2, saved, hh, row_weights=rw, want_grad_weights=self.in_rows,
            grad_dtype=torch.float32)
        grad_x, gtw = h.dispatch_backward(gx, grad_out_w=grw, want_grad_weights=self.in_rows)
        return out, grad_x, g13, g2, gtw if self.in_rows else gw


@pytest.mark.parametrize("in_rows", [True, False])
@pytest.mark.parametrize("T,H,inter,E,K,A", [(64, 264, 136, 8, 2, 16), (17, 72, 40, 3, 3, 1),
                                             (300, 136, 264, 4, 1, 8)])
def test_training_step(T, H, inter, E, K, A, in_rows):
    """The layer's output and all its gradients against binary64's own differentiation.  Six
    roundings to bf16 on the way, 2^-8 each, are the most that any of them meets; where terms
    cancel the error stays and the sum shrinks, less than by half in these norms."""
    say("training", T, H, inter, E, K, A, in_rows)
    s = Training(T, H, inter, E, K, A, _gen(H), in_rows)
    got = s.step()
    leaves = [t.double().requires_grad_(True) for t in (s.x, s.w13, s.w2, s.w)]
    x, w13, w2, w = leaves
    out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for e in range(E):
        t, k = torch.nonzero(s.idx == e, as_tuple=True)
        g, u = (x[t] @ w13[e].t()).chunk(2, 1)
        y = (g * torch.sigmoid(g) * u) @ w2[e].t()
        out = out.index_add(0, t, y * w[t, k][:, None])
    want = torch.autograd.grad((out * s.gy.double()).sum(), leaves)
    for name, p, q in zip(("out", "x", "w13", "w2", "w"), got, (out.detach(), *want)):
        assert _rel(p, q) < 2 * 6 * ref.BF16, (name, _rel(p, q))


def test_tokens_own_rows_give_what_dispatch_gives():
    gen = _gen(2)
    T, K, E, H, inter = 90, 4, 16, 328, 72
    idx = ref.ids(T, K, E, gen, "cuda", 0.2)
    h = ep.Handle(T, K, E, 32)
    h.layout(idx)
    x = _randn((T, H), gen)
    w13, w2 = _randn((E, 2 * inter, H), gen, H ** -0.5), _randn((E, H, inter), gen, inter ** -0.5)
    rows = ref.rows_of(h, idx)[0]
    ex = h.dispatch(x)[0]
    a = h.expert_ffn(x, w13, w2, token_rows=True, want_saved=True)
    b = h.expert_ffn(ex, w13, w2, want_saved=True)
    for p, q in zip(a, b):
        assert torch.equal(p[rows], q[rows])
    g = _randn((h.capacity, H), gen)
    ga = h.expert_ffn_backward(g, x, w13, w2, a[2], a[1], token_rows=True)
    gb = h.expert_ffn_backward(g, ex, w13, w2, b[2], b[1])
    assert torch.equal(ga[1], gb[1]) and torch.equal(ga[2], gb[2])


@pytest.mark.parametrize("make", [
    lambda gen: Int8Serving(24, 256, 128, 8, 2, 8, gen),
    lambda gen: Training(40, 264, 72, 8, 2, 8, gen, True),
    lambda gen: Training(700, 136, 72, 4, 2, 1, gen, False),
], ids=["int8", "training", "training, many rows"])
def test_steps_in_a_graph(make):
    """The whole step captured; every replay on new inputs and routing, with eager work between the
    replays, equals the eager step."""
    s, gen = make(_gen(3)), _gen(4)
    s.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = s.step()
    T, K = s.idx.shape
    for k in range(4):
        s.x.copy_(_randn(s.x.shape, gen))
        s.idx.copy_(ref.ids(T, K, s.h.h.num_experts, gen, "cuda", 0.1 * k))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        want = s.step()
        rows = ref.rows_of(s.h, s.idx)[0]
        for i, (a, b) in enumerate(zip(kept, want)):
            if a.shape[0] == s.h.capacity and a.shape[0] != T:
                a, b = a[rows], b[rows]
            assert torch.equal(_bits(a), _bits(b)), (k, i)


@pytest.mark.parametrize("make", [
    lambda i: Int8Serving(32, 512, 256, 16, 4, 8, _gen(5 + i)),
    lambda i: Training(200, 264, 136, 8, 2, 8, _gen(7 + i), True),
], ids=["int8", "training"])
def test_two_streams(make):
    """Two steps on two streams, with their own handles and buffers, give what each gives alone."""
    steps = [make(i) for i in range(2)]
    want = [s.step() for s in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    got = [None, None]
    for _ in range(3):
        for i, (s, stream) in enumerate(zip(steps, streams)):
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                got[i] = s.step()
    torch.cuda.synchronize()
    for s, p, q in zip(steps, got, want):
        rows = ref.rows_of(s.h, s.idx)[0]
        for i, (a, b) in enumerate(zip(p, q)):
            if a.shape[0] == s.h.capacity and a.shape[0] != s.idx.shape[0]:
                a, b = a[rows], b[rows]
            assert torch.equal(_bits(a), _bits(b)), i


def test_bound_calls_give_what_the_methods_give():
    gen = _gen(9)
    s = Int8Serving(24, 256, 128, 8, 2, 8, gen)
    s.step()
    h = s.h
    y = _randn((24, 256), gen)
    quant = ep.bind_quantize_i8(y)
    q, sc = quant()
    up = ep.bind_expert_i8(h, q, sc, s.w13, s.s13, gated=True, token_rows=True)
    rows_q = ep.bind_quantize_i8(up(), handle=h)
    down = ep.bind_expert_i8(h, *rows_q(), s.w2, s.s2)
    block = ep.bind_expert_ffn(h, y, _randn((8, 128, 256), gen, 0.1), _randn((8, 256, 64), gen, 0.1),
                              token_rows=True)
    for _ in range(2):
        y.copy_(_randn(y.shape, gen))
        for call in (quant, up, rows_q):
            call()
        out = down()
        rows = ref.rows_of(h, s.idx)[0]
        q2, s2 = ep.quantize_i8(y)
        a = h.expert_i8(q2, s2, s.w13, s.s13, gated=True, token_rows=True)
        assert torch.equal(out[rows], h.expert_i8(*h.quantize_i8(a), s.w2, s.s2)[rows])
        got = block()
        assert got[2] is None and bool(got[0][rows].isfinite().all())


def test_one_handle_two_streams():
    """Calls on one laid out handle only read it: two streams with their own buffers may use it at
    once."""
    gen = _gen(11)
    T, K, E, H, I = 200, 2, 8, 264, 136
    h = ep.Handle(T, K, E, 8)
    h.layout(ref.ids(T, K, E, gen, "cuda", 0.1))
    w13, w2 = _randn((E, 2 * I, H), gen, H ** -0.5), _randn((E, H, I), gen, I ** -0.5)
    x = [_randn((T, H), gen) for _ in range(2)]
    gy = [_randn((h.capacity, H), gen, 0.1) for _ in range(2)]
    rw = torch.rand(h.capacity, generator=gen, device="cuda")

    def step(i):
        y, a, saved = h.expert_ffn(x[i], w13, w2, row_weights=rw, token_rows=True, want_saved=True)
        gx, g13, g2, grw, _ = h.expert_ffn_backward(gy[i], x[i], w13, w2, saved, a, row_weights=rw,
                                                    token_rows=True, want_grad_weights=True)
        return (y, gx, grw), (g13, g2)

    want = [step(i) for i in range(2)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [None, None]
    for _ in range(3):
        for i, stream in enumerate(streams):
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                got[i] = step(i)
    torch.cuda.synchronize()
    rows = ref.rows_of(h, h.topk_idx)[0]
    for (p, pw), (q, qw) in zip(got, want):
        assert all(torch.equal(a[rows], b[rows]) for a, b in zip(p, q))
        assert all(torch.equal(a, b) for a, b in zip(pw, qw))


def test_imported_layout_gives_what_its_own_gives():
    """A layout that came from the host, with gaps between the segments."""
    gen = _gen(12)
    T, K, E, H, I = 60, 3, 6, 136, 80
    a = ep.Handle(T, K, E, 16)
    idx = ref.ids(T, K, E, gen, "cuda", 0.1)
    a.layout(idx)
    own = a.read_counts()
    b = ep.Handle(T, K, E, 16)
    n = own["num_expanded"]
    b.import_layout(idx, own["counts"], own["psum"], a.dst_slot.cpu().numpy(),
                    a.src_meta[:n].cpu().numpy(), own["num_recv_tokens"])
    w13, w2 = _randn((E, 2 * I, H), gen, H ** -0.5), _randn((E, H, I), gen, I ** -0.5)
    x, gy = _randn((T, H), gen), _randn((a.capacity, H), gen, 0.1)
    rows = ref.rows_of(a, idx)[0]
    got = []
    for h in (a, b):
        y, act, saved = h.expert_ffn(x, w13, w2, token_rows=True, want_saved=True)
        q, s = h.quantize_i8(act)
        gx, g13, g2, _, _ = h.expert_ffn_backward(gy, x, w13, w2, saved, act, token_rows=True)
        got.append((y[rows], q[rows], s[rows], gx[rows], g13, g2))
    assert all(torch.equal(p, q) for p, q in zip(*got))


FIRST_CALLS = """
import torch, combine_ep_layout_08_amd as ep
T, K, E, H, I = 40, 2, 4, 264, 136
g = torch.Generator(device="cuda").manual_seed(1)
new = lambda *s: torch.randn(s, generator=g, device="cuda").mul_(0.1).bfloat16()
idx = torch.randint(0, E, (T, K), generator=g, device="cuda")
x, w13, w2 = new(T, H), new(E, 2 * I, H), new(E, H, I)
i13 = torch.randint(-127, 128, (E, 2 * I, H // 16 * 16), generator=g, device="cuda", dtype=torch.int8)
s13 = torch.rand((E, 2 * I), generator=g, device="cuda")
h = ep.Handle(T, K, E, 8)
h.layout(idx)
gy = new(h.capacity, H)
def step():
    q, s = ep.quantize_i8(x[:, :256].contiguous())
    act = h.expert_i8(q, s, i13[:, :, :256].contiguous(), s13, gated=True, token_rows=True)
    y, a, saved = h.expert_ffn(x, w13, w2, token_rows=True, want_saved=True)
    return act, y, *h.expert_ffn_backward(gy, x, w13, w2, saved, a, token_rows=True)[:3]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
for _ in range(3):
    graph.replay()
    torch.cuda.synchronize()
    kept = [t.clone() for t in got]
    rows = h.dst_slot.reshape(-1).long()
    rows = rows[rows >= 0]
    for p, q in zip(kept, step()):
        if p.shape[0] == h.capacity:
            p, q = p[rows], q[rows]
        assert torch.equal(p, q)
print("same")
"""


def test_first_calls_of_a_process_inside_a_capture():
    """Whatever a kernel needs once a device (its LDS limit) may be asked for while a graph is
    captured."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], capture_output=True, text=True,
                       timeout=110)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
