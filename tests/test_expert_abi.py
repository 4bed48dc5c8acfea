"""The C entries of the experts' products and their binding on the CPU: exported functions,
sizes, and every refusal, none of which reaches a HIP runtime function; and the binding's
arguments, with a fake library in place of the real one."""
import gc
import os
import re
import weakref

import pytest
import torch

import combine_ep_layout_08_amd as ep
from tests.test_abi import A16, _fake_handle
from tests.test_binding_contract import STREAM, FakeLib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# places far apart: nothing of these sizes reaches from one to the next
P = [A16 + (i << 28) for i in range(16)]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(ep.LIB_PATH):
        from combine_ep_layout_08_amd import build
        build.build()
    return ep.lib()


def _empty():
    h = _fake_handle()
    h.num_tokens = 0
    return h


def test_every_declared_function_is_exported():
    text = open(os.path.join(ROOT, "include", "ep_expert.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(ep_[a-z0-9_]+)\s*\(", text)))
    assert len(names) == 6, names
    for n in names:
        assert hasattr(ep.lib(), n) and n in ep._SIGNATURES and n in ep.__all__, n


# Every refusal of the pointers a call takes: (argument, what it does misaligned, what it does
# missing).  None: it may be missing.
def _pointer_cases(call, sixteen, four, needed):
    for name in sixteen:
        assert call(**{name: P[0] + 8}) == ep.EP_ERR_MISALIGNED, name
    for name in four:
        assert call(**{name: P[0] + 2}) == ep.EP_ERR_MISALIGNED, name
    for name in needed:
        assert call(**{name: None}) == ep.EP_ERR_NULL, name


def quant(x=P[0], rows=4, channels=256, q=P[1], s=P[2]):
    return ep.ep_quantize_i8(x, rows, channels, q, s, None)


def quant_rows(h=None, x=P[0], channels=256, q=P[1], s=P[2]):
    return ep.ep_quantize_i8_rows(h or _fake_handle(), x, channels, q, s, None)


def test_quantiser_refusals():
    assert quant(rows=-1) == ep.EP_ERR_SHAPE
    for call in (quant, quant_rows):
        assert call(channels=0) == ep.EP_ERR_SHAPE and call(channels=-16) == ep.EP_ERR_SHAPE
        assert call(channels=24) == ep.EP_ERR_MISALIGNED
        assert call(channels=32784) == ep.EP_ERR_UNSUPPORTED
        _pointer_cases(call, ("x", "q"), ("s",), ("x", "q", "s"))
        assert call(q=P[0]) == ep.EP_ERR_UNSUPPORTED and call(s=P[1]) == ep.EP_ERR_UNSUPPORTED
        assert call(s=P[0] + 1024) == ep.EP_ERR_UNSUPPORTED
    assert quant(rows=0, x=None, q=None, s=None) == ep.EP_OK
    assert quant_rows(h=_empty(), x=None, q=None, s=None) == ep.EP_OK
    assert quant_rows(h=_fake_handle(laid_out=0)) == ep.EP_ERR_NOT_LAID_OUT
    assert quant_rows(h=ep.ep_handle()) == ep.EP_ERR_WORKSPACE
    assert ep.lib().ep_quantize_i8_rows(None, P[0], 256, P[1], P[2], None) == ep.EP_ERR_NULL


def i8(h=None, x=P[0], xs=P[1], tokens=0, k=256, w=P[2], ws=P[3], n=64, gated=0, rw=None,
       out=P[4]):
    return ep.ep_expert_i8(h or _fake_handle(), x, xs, tokens, k, w, ws, n, gated, rw, out, None)


def test_i8_refusals():
    assert i8(h=_fake_handle(laid_out=0)) == ep.EP_ERR_NOT_LAID_OUT
    assert i8(h=ep.ep_handle()) == ep.EP_ERR_WORKSPACE
    assert ep.lib().ep_expert_i8(None, P[0], P[1], 0, 256, P[2], P[3], 64, 0, None, P[4],
                                 None) == ep.EP_ERR_NULL
    assert i8(tokens=2) == ep.EP_ERR_UNSUPPORTED and i8(gated=2) == ep.EP_ERR_UNSUPPORTED
    assert i8(rw=P[5]) == ep.EP_ERR_UNSUPPORTED             # weights of a product that has none
    assert i8(k=0) == ep.EP_ERR_SHAPE and i8(n=-8) == ep.EP_ERR_SHAPE
    assert i8(k=264) == ep.EP_ERR_MISALIGNED and i8(n=12) == ep.EP_ERR_MISALIGNED
    assert i8(n=24, gated=1) == ep.EP_ERR_MISALIGNED
    assert i8(k=32784) == ep.EP_ERR_UNSUPPORTED and i8(n=65552) == ep.EP_ERR_UNSUPPORTED
    _pointer_cases(i8, ("x", "w", "ws", "out"), ("xs",), ("x", "xs", "w", "ws", "out"))
    assert i8(gated=1, rw=P[5] + 2) == ep.EP_ERR_MISALIGNED
    for other in (P[0], P[1], P[2], P[3]):
        assert i8(out=other) == ep.EP_ERR_UNSUPPORTED
    assert i8(gated=1, rw=P[4] + 16) == ep.EP_ERR_UNSUPPORTED
    assert i8(h=_empty(), x=None, xs=None, out=None) == ep.EP_OK


def ffn(h=None, x=P[0], tokens=0, hidden=128, w13=P[1], w2=P[2], inter=64, rw=P[3], oh=P[4],
        saved=P[5], y=P[6]):
    return ep.ep_expert_ffn(h or _fake_handle(), x, tokens, hidden, w13, w2, inter, rw, oh, saved,
                            y, None)


def test_ffn_refusals():
    assert ffn(h=_fake_handle(laid_out=0)) == ep.EP_ERR_NOT_LAID_OUT
    assert ffn(h=ep.ep_handle()) == ep.EP_ERR_WORKSPACE
    assert ep.lib().ep_expert_ffn(None, P[0], 0, 128, P[1], P[2], 64, None, P[4], None, P[6],
                                  None) == ep.EP_ERR_NULL
    assert ffn(tokens=-1) == ep.EP_ERR_UNSUPPORTED
    for size in ("hidden", "inter"):
        assert ffn(**{size: 0}) == ep.EP_ERR_SHAPE and ffn(**{size: 12}) == ep.EP_ERR_MISALIGNED
        assert ffn(**{size: 32776}) == ep.EP_ERR_UNSUPPORTED
    _pointer_cases(ffn, ("x", "w13", "w2", "oh", "saved", "y"), ("rw",),
                   ("x", "w13", "w2", "oh", "y"))
    outs, ins = dict(oh=P[4], saved=P[5], y=P[6]), (P[0], P[1], P[2], P[3])
    for name, place in outs.items():
        for other in ins + tuple(p for p in outs.values() if p != place):
            assert ffn(**{name: other}) == ep.EP_ERR_UNSUPPORTED, name
    assert ffn(h=_empty(), x=None, oh=None, y=None) == ep.EP_OK


def grads(h=None, gy=P[0], x=P[1], tokens=0, hidden=128, w13=P[2], w2=P[3], inter=64, rw=P[4],
          saved=P[5], rows_h=P[6], remake=0, ggu=P[7], gx=P[8], dtype=ep.EP_BF16, g13=P[9],
          g2=P[10], grw=P[11], ws=P[12], nbytes=1 << 20):
    return ep.ep_expert_ffn_backward(h or _fake_handle(), gy, x, tokens, hidden, w13, w2, inter,
                                     rw, saved, rows_h, remake, ggu, gx, dtype, g13, g2, grw, ws,
                                     nbytes, None)


def test_ffn_gradient_refusals():
    assert grads(h=_fake_handle(laid_out=0)) == ep.EP_ERR_NOT_LAID_OUT
    assert grads(h=ep.ep_handle()) == ep.EP_ERR_WORKSPACE
    assert grads(dtype=ep.EP_FP8_E4M3) == ep.EP_ERR_DTYPE
    assert grads(tokens=3) == ep.EP_ERR_UNSUPPORTED and grads(remake=2) == ep.EP_ERR_UNSUPPORTED
    for size in ("hidden", "inter"):
        assert grads(**{size: -8}) == ep.EP_ERR_SHAPE
        assert grads(**{size: 20}) == ep.EP_ERR_MISALIGNED
        assert grads(**{size: 40000}) == ep.EP_ERR_UNSUPPORTED
    _pointer_cases(grads, ("gy", "x", "w13", "w2", "saved", "rows_h", "ggu", "gx", "g13", "g2", "ws"),
                   ("rw", "grw"), ("gy", "x", "w13", "w2", "saved", "rows_h", "ggu"))
    assert grads(rows_h=None, g2=None, remake=1) == ep.EP_ERR_NULL
    need = ep.ep_expert_ffn_backward_workspace(_fake_handle(), 64)
    assert need >= 16 * 4
    assert grads(ws=None) == ep.EP_ERR_WORKSPACE and grads(nbytes=need - 1) == ep.EP_ERR_WORKSPACE
    outs = dict(gx=P[8], g13=P[9], g2=P[10], grw=P[11], ggu=P[7], ws=P[12])
    ins = dict(gy=P[0], x=P[1], w13=P[2], w2=P[3], rw=P[4], saved=P[5], rows_h=P[6])
    for name, place in outs.items():
        for other in tuple(ins.values()) + tuple(p for p in outs.values() if p != place):
            if (name, other) != ("ggu", ins["saved"]):
                assert grads(**{name: other}) == ep.EP_ERR_UNSUPPORTED, (name, hex(other))
    assert grads(ggu=P[5] + 16) == ep.EP_ERR_UNSUPPORTED
    for name in ("gy", "x", "w13", "w2", "rw", "saved"):     # h made over an input
        assert grads(remake=1, rows_h=ins[name]) == ep.EP_ERR_UNSUPPORTED, name


def test_ffn_gradient_workspace():
    h = _fake_handle()
    assert ep.ep_expert_ffn_backward_workspace(h, 12) == 0
    assert ep.ep_expert_ffn_backward_workspace(h, 40000) == 0
    assert ep.lib().ep_expert_ffn_backward_workspace(None, 64) == 0
    small, wide = (ep.ep_expert_ffn_backward_workspace(h, i) for i in (8, 2048))
    assert 16 * 4 <= small <= wide <= 16 * 4 * 64
    h.capacity = 1 << 33                                     # beyond 32 bits
    assert ep.ep_expert_ffn_backward_workspace(h, 2048) == (1 << 29) * wide


# ---------------------------------------------------------------- binding

@pytest.fixture
def fake(monkeypatch):
    class Lib(FakeLib):
        def __getattr__(self, name):
            call = super().__getattr__(name)
            if name != "ep_expert_ffn_backward_workspace":
                return call

            def counted(*args):
                call(*args)
                return 4096
            return counted

    lib = Lib()
    monkeypatch.setattr(ep, "lib", lambda: lib)
    monkeypatch.setattr(ep, "_stream", lambda: STREAM)
    monkeypatch.setattr(ep, "_dev", lambda t, name: ep._need(t.is_contiguous(),
                                                             f"{name} must be contiguous"))
    return lib


def _handle(T=16, K=4, E=8, A=4):
    h = ep.Handle(T, K, E, A, device="cpu")
    h.h.num_tokens, h.h.num_topk, h.h.num_experts, h.h.max_tokens = T, K, E, T
    return h


def _bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _i8(*shape):
    return torch.zeros(shape, dtype=torch.int8)


def test_binding_quantiser(fake):
    x = _bf16(6, 64)
    q, s = ep.quantize_i8(x)
    assert q.dtype == torch.int8 and q.shape == (6, 64) and s.shape == (6,)
    assert fake.last("ep_quantize_i8") == (x.data_ptr(), 6, 64, q.data_ptr(), s.data_ptr(), STREAM)
    assert ep.bind_quantize_i8(x, out_q=q, out_scale=s)() == (q, s)
    h = _handle()
    y = _bf16(h.capacity, 32)
    q, s = h.quantize_i8(y)
    assert fake.last("ep_quantize_i8_rows")[1:] == (y.data_ptr(), 32, q.data_ptr(), s.data_ptr(),
                                                    STREAM)
    assert ep.bind_quantize_i8(y, q, s, handle=h)() == (q, s)
    for bad in (lambda: ep.quantize_i8(x.float()), lambda: ep.quantize_i8(x[0]),
                lambda: ep.quantize_i8(x, out_q=_i8(6, 32)), lambda: ep.quantize_i8(x.t()),
                lambda: ep.quantize_i8(x, out_scale=torch.zeros(5)), lambda: h.quantize_i8(x)):
        with pytest.raises(ValueError):
            bad()


def test_binding_i8(fake):
    h = _handle()
    w, ws, x, xs = _i8(8, 32, 64), torch.ones(8, 32), _i8(16, 64), torch.ones(16)
    rw = torch.ones(h.capacity)
    out = h.expert_i8(x, xs, w, ws, gated=True, row_weights=rw, token_rows=True)
    assert out.shape == (h.capacity, 16) and out.dtype == torch.bfloat16
    assert fake.last("ep_expert_i8")[1:] == (
        x.data_ptr(), xs.data_ptr(), 1, 64, w.data_ptr(), ws.data_ptr(), 32, 1, rw.data_ptr(),
        out.data_ptr(), STREAM)
    cap = h.capacity
    x, xs = _i8(cap, 64), torch.ones(cap)
    call = ep.bind_expert_i8(h, x, xs, w, ws)
    assert call().shape == (cap, 32)
    a = fake.last("ep_expert_i8")
    assert a[3] == 0 and a[8:10] == (0, None)
    for bad in (lambda: h.expert_i8(x[:16], xs, w, ws), lambda: h.expert_i8(x, xs[:16], w, ws),
                lambda: h.expert_i8(x, xs, w[:4], ws), lambda: h.expert_i8(x, xs, w, ws[:, :16]),
                lambda: h.expert_i8(x.to(torch.uint8), xs, w, ws),
                lambda: h.expert_i8(x, xs, w, ws, row_weights=rw),
                lambda: h.expert_i8(x, xs, w, ws, out=_bf16(cap, 16)),
                lambda: h.expert_i8(x, xs, w, ws, gated=True, row_weights=torch.ones(3)),
                lambda: h.expert_i8(x, xs, _i8(8, 31, 64), torch.ones(8, 31), gated=True)):
        with pytest.raises(ValueError):
            bad()
    h.h.num_tokens = 3
    with pytest.raises(ValueError, match="bound for 16 tokens"):
        call()


def test_binding_ffn(fake):
    h = _handle()
    cap = h.capacity
    w13, w2, x, rw = _bf16(8, 48, 64), _bf16(8, 64, 24), _bf16(cap, 64), torch.ones(cap)
    y, hh, saved = h.expert_ffn(x, w13, w2, row_weights=rw, want_saved=True)
    assert y.shape == (cap, 64) and hh.shape == (cap, 24) and saved.shape == (cap, 48)
    assert fake.last("ep_expert_ffn")[1:] == (
        x.data_ptr(), 0, 64, w13.data_ptr(), w2.data_ptr(), 24, rw.data_ptr(), hh.data_ptr(),
        saved.data_ptr(), y.data_ptr(), STREAM)
    y, hh, none = ep.bind_expert_ffn(h, _bf16(16, 64), w13, None, token_rows=True)()
    a = fake.last("ep_expert_ffn")
    assert y is None and none is None and a[2] == 1 and a[5] is None and a[9:11] == (None, None)
    for bad in (lambda: h.expert_ffn(x, w13, w2, token_rows=True),
                lambda: h.expert_ffn(x, w13, w2[:, :32].contiguous()),
                lambda: h.expert_ffn(x, _bf16(8, 47, 64), w2),
                lambda: h.expert_ffn(x, w13.float(), w2), lambda: h.expert_ffn(x, w13, None, out=x),
                lambda: h.expert_ffn(x, w13, w2, row_weights=rw[:3]),
                lambda: h.expert_ffn(x, w13, w2, out_h=_bf16(cap, 64)),
                lambda: h.expert_ffn(x, w13.transpose(1, 2), w2)):
        with pytest.raises(ValueError):
            bad()


def test_binding_ffn_gradients(fake):
    h = _handle()
    cap = h.capacity
    w13, w2, x, rw = _bf16(8, 48, 64), _bf16(8, 64, 24), _bf16(cap, 64), torch.ones(cap)
    gy, saved, hh = _bf16(cap, 64), _bf16(cap, 48), _bf16(cap, 24)
    gx, g13, g2, grw, ggu = h.expert_ffn_backward(
        gy, x, w13, w2, saved, hh, row_weights=rw, want_grad_weights=True,
        grad_dtype=torch.float32)
    assert g13.dtype == g2.dtype == torch.float32 and g13.shape == w13.shape and g2.shape == w2.shape
    a = fake.last("ep_expert_ffn_backward")
    assert a[1:18] == (gy.data_ptr(), x.data_ptr(), 0, 64, w13.data_ptr(), w2.data_ptr(), 24,
                       rw.data_ptr(), saved.data_ptr(), hh.data_ptr(), 0, ggu.data_ptr(),
                       gx.data_ptr(), ep.EP_F32, g13.data_ptr(), g2.data_ptr(), grw.data_ptr())
    assert a[18] is not None and a[19:] == (4096, STREAM)
    got = h.expert_ffn_backward(gy, None, w13, w2, saved, want_grad_x=False, want_grad_w=False,
                                grad_gate_up=saved)
    assert got[:4] == (None,) * 4 and got[4] is saved
    assert fake.last("ep_expert_ffn_backward")[18:20] == (None, 0)
    h.expert_ffn_backward(gy, x, w13, w2, saved, remake_h=True, grad_w2=_bf16(8, 64, 24))
    assert fake.last("ep_expert_ffn_backward")[11] == 1
    for bad in (lambda: h.expert_ffn_backward(gy, None, w13, w2, saved, hh),
                lambda: h.expert_ffn_backward(gy, x, w13, w2, saved),
                lambda: h.expert_ffn_backward(gy, x, w13, w2, hh, hh),
                lambda: h.expert_ffn_backward(hh, x, w13, w2, saved, hh),
                lambda: h.expert_ffn_backward(gy, x, w13, None, saved, hh),
                lambda: h.expert_ffn_backward(gy, x, w13, w2, saved, hh, grad_dtype=torch.float16),
                lambda: h.expert_ffn_backward(gy, x, w13, w2, saved, hh, grad_w13=w13,
                                              grad_w2=w2.float()),
                lambda: h.expert_ffn_backward(gy, x, w13, w2, saved, hh, token_rows=True),
                lambda: h.expert_ffn_backward(gy, x, w13, w2, saved, hh, want_grad_weights=True,
                                              workspace=torch.zeros(64))):
        with pytest.raises(ValueError):
            bad()


def test_bound_calls_keep_the_handles_workspace(fake):
    """The kernels read counts, rows and the error word in the handle's workspace: a bound call
    that outlives the caller's handle holds it, and refuses another batch's size."""
    def calls(h):
        cap = h.capacity
        yield ep.bind_quantize_i8(_bf16(cap, 32), handle=h)
        yield ep.bind_expert_i8(h, _i8(cap, 64), torch.ones(cap), _i8(8, 32, 64), torch.ones(8, 32))
        yield ep.bind_expert_ffn(h, _bf16(cap, 64), _bf16(8, 48, 64), _bf16(8, 64, 24))

    for i in range(3):
        h = _handle()
        workspace = weakref.ref(h.workspace)
        call = list(calls(h))[i]
        del h
        gc.collect()
        assert workspace() is not None
        call()
        call._h.num_tokens = 3
        with pytest.raises(ValueError, match="bound for 16 tokens"):
            call()
        del call
        gc.collect()
        assert workspace() is None
