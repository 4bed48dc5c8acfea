"""The layer operators' C entries and binding on the CPU: exported functions,
sizes, and every refusal, none of which reaches a HIP runtime function; and the
binding's arguments, with a fake library in place of the real one."""
import os
import re

import pytest
import torch

import combine_ep_layout_08_amd as ep
from tests.test_abi import A16, _fake_handle
from tests.test_binding_contract import STREAM, FakeLib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F, U = ep.EP_SF_F32, ep.EP_SF_UE8M0


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(ep.LIB_PATH):
        from combine_ep_layout_08_amd import build
        build.build()
    return ep.lib()


def test_every_declared_function_is_exported():
    text = open(os.path.join(ROOT, "include", "ep_layer.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(ep_[a-z0-9_]+)\s*\(", text)))
    assert len(names) == 9, names
    for n in names:
        assert hasattr(ep.lib(), n) and n in ep._SIGNATURES and hasattr(ep, n), n
    enums = dict(re.findall(r"\b(EP_W4_[A-Z0-9]+) = (\d+)", text))
    assert enums and all(getattr(ep, k) == int(v) for k, v in enums.items())


def norm(x=A16, r=None, w=A16, wdt=ep.EP_BF16, eps=1e-6, T=4, H=256, z=None, y=A16, fmt=F, q=None,
         sf=None, ts=2, hs=1, rstd=None):
    return ep.ep_add_rmsnorm(x, r, w, wdt, eps, T, H, z, y, fmt, q, sf, ts, hs, rstd, None)


@pytest.mark.parametrize("status,args", [
    (ep.EP_ERR_DTYPE, dict(wdt=ep.EP_FP8_E4M3)),
    (ep.EP_ERR_SHAPE, dict(T=-1)),
    (ep.EP_ERR_SHAPE, dict(H=0)),
    (ep.EP_ERR_SHAPE, dict(eps=-1e-6)),
    (ep.EP_ERR_SHAPE, dict(eps=float("nan"))),
    (ep.EP_ERR_SHAPE, dict(eps=float("inf"))),
    (ep.EP_ERR_MISALIGNED, dict(H=252)),
    (ep.EP_ERR_MISALIGNED, dict(H=264, q=A16, sf=A16)),
    (ep.EP_ERR_UNSUPPORTED, dict(H=32776)),
    (ep.EP_ERR_DTYPE, dict(q=A16, sf=A16, fmt=2)),
    (ep.EP_ERR_SHAPE, dict(q=A16, sf=A16, ts=-1)),
    (ep.EP_ERR_NULL, dict(q=A16)),
    (ep.EP_ERR_NULL, dict(x=None)),
    (ep.EP_ERR_NULL, dict(w=None)),
    (ep.EP_ERR_NULL, dict(y=None)),
    (ep.EP_ERR_MISALIGNED, dict(x=A16 + 8)),
    (ep.EP_ERR_MISALIGNED, dict(r=A16 + 2)),
    (ep.EP_ERR_MISALIGNED, dict(w=A16 + 4)),
    (ep.EP_ERR_MISALIGNED, dict(z=A16 + 8)),
    (ep.EP_ERR_MISALIGNED, dict(y=A16 + 8)),
    (ep.EP_ERR_MISALIGNED, dict(q=A16 + 8, sf=A16)),
    (ep.EP_ERR_MISALIGNED, dict(q=A16, sf=A16 + 2)),
    (ep.EP_ERR_MISALIGNED, dict(rstd=A16 + 2)),
    (ep.EP_OK, dict(T=0, x=None, w=None, y=None)),
])
def test_norm_refusals(status, args):
    assert norm(**args) == status


def norm_grad(g=A16, z=A16, w=A16, wdt=ep.EP_F32, rstd=A16, gz=None, T=4, H=256, gx=A16, gw=A16,
              ws=A16, nbytes=1 << 30):
    return ep.ep_add_rmsnorm_backward(g, z, w, wdt, rstd, gz, T, H, gx, gw, ws, nbytes, None)


@pytest.mark.parametrize("status,args", [
    (ep.EP_ERR_DTYPE, dict(wdt=ep.EP_I32)),
    (ep.EP_ERR_SHAPE, dict(T=-1)),
    (ep.EP_ERR_SHAPE, dict(H=-8)),
    (ep.EP_ERR_MISALIGNED, dict(H=12)),
    (ep.EP_ERR_UNSUPPORTED, dict(H=40000)),
    (ep.EP_ERR_NULL, dict(g=None)),
    (ep.EP_ERR_NULL, dict(z=None)),
    (ep.EP_ERR_NULL, dict(w=None)),
    (ep.EP_ERR_NULL, dict(rstd=None)),
    (ep.EP_ERR_NULL, dict(gx=None, gw=None)),
    (ep.EP_ERR_WORKSPACE, dict(T=4096, ws=None)),
    (ep.EP_ERR_WORKSPACE, dict(T=4096, nbytes=4 * 256 - 1)),
    (ep.EP_ERR_MISALIGNED, dict(g=A16 + 8)),
    (ep.EP_ERR_MISALIGNED, dict(gz=A16 + 8)),
    (ep.EP_ERR_MISALIGNED, dict(gx=A16 + 8)),
    (ep.EP_ERR_MISALIGNED, dict(gw=A16 + 4)),
    (ep.EP_ERR_MISALIGNED, dict(ws=A16 + 4)),
    (ep.EP_ERR_MISALIGNED, dict(rstd=A16 + 2)),
    (ep.EP_OK, dict(T=0, g=None, z=None, w=None, rstd=None, gw=None)),
])
def test_norm_gradient_refusals(status, args):
    assert norm_grad(**args) == status


def test_norm_gradient_workspace():
    assert ep.ep_add_rmsnorm_backward_workspace(-1, 256) == 0
    assert ep.ep_add_rmsnorm_backward_workspace(4, 12) == 0
    assert ep.ep_add_rmsnorm_backward_workspace(4, 40000) == 0
    few, some, large = (ep.ep_add_rmsnorm_backward_workspace(t, 7168) for t in (1, 4096, 1 << 20))
    assert few == 0 and 4 * 7168 <= some <= large <= 4 * 7168 * 4096


def w4(h=None, x=A16, dt=ep.EP_BF16, tokens=0, k=256, sf=None, sfmt=F, ts=2, hs=1, codes=A16,
       scales=A16, fmt=ep.EP_W4_INT4, group=64, n=64, out=A16):
    return ep.ep_expert_w4(h or _fake_handle(), x, dt, tokens, k, sf, sfmt, ts, hs, codes, scales,
                           fmt, group, n, out, None)


FP8 = dict(dt=ep.EP_FP8_E4M3, sf=A16)


@pytest.mark.parametrize("status,args", [
    (ep.EP_ERR_NOT_LAID_OUT, dict(h=_fake_handle(laid_out=0))),
    (ep.EP_ERR_WORKSPACE, dict(h=ep.ep_handle())),
    (ep.EP_ERR_DTYPE, dict(dt=ep.EP_F32)),
    (ep.EP_ERR_DTYPE, dict(fmt=2)),
    (ep.EP_ERR_DTYPE, dict(sf=A16)),
    (ep.EP_ERR_UNSUPPORTED, dict(tokens=2)),
    (ep.EP_ERR_UNSUPPORTED, dict(group=16)),
    (ep.EP_ERR_UNSUPPORTED, dict(group=0)),
    (ep.EP_ERR_UNSUPPORTED, dict(fmt=ep.EP_W4_MXFP4, group=64)),
    (ep.EP_ERR_UNSUPPORTED, dict(k=32896)),
    (ep.EP_ERR_SHAPE, dict(k=0)),
    (ep.EP_ERR_SHAPE, dict(n=-8)),
    (ep.EP_ERR_MISALIGNED, dict(k=192)),
    (ep.EP_ERR_MISALIGNED, dict(n=12)),
    (ep.EP_ERR_NULL, dict(x=None)),
    (ep.EP_ERR_NULL, dict(out=None)),
    (ep.EP_ERR_NULL, dict(codes=None)),
    (ep.EP_ERR_NULL, dict(scales=None)),
    (ep.EP_ERR_NULL, dict(dt=ep.EP_FP8_E4M3)),
    (ep.EP_ERR_DTYPE, dict(FP8, sfmt=5)),
    (ep.EP_ERR_SHAPE, dict(FP8, hs=-1)),
    (ep.EP_ERR_MISALIGNED, dict(FP8, sf=A16 + 2)),
    (ep.EP_ERR_MISALIGNED, dict(x=A16 + 8)),
    (ep.EP_ERR_MISALIGNED, dict(out=A16 + 8)),
    (ep.EP_ERR_MISALIGNED, dict(codes=A16 + 8)),
    (ep.EP_ERR_MISALIGNED, dict(scales=A16 + 8)),
])
def test_w4_refusals(status, args):
    assert w4(**args) == status


def test_w4_null_handle_and_empty_batch():
    assert ep.lib().ep_expert_w4(None, A16, 0, 0, 256, None, 0, 0, 0, A16, A16, 0, 64, 64, A16,
                                 None) == ep.EP_ERR_NULL
    empty = _fake_handle()
    empty.num_tokens = 0
    assert w4(h=empty, x=None, out=None) == ep.EP_OK


def test_w4_sizes_and_pack_refusals():
    assert ep.ep_w4_code_bytes(4, 24, 256) == 4 * 32 * 128
    assert ep.ep_w4_scale_bytes(4, 24, 256, ep.EP_W4_INT4, 64) == 4 * 32 * 4 * 2
    assert ep.ep_w4_scale_bytes(4, 24, 256, ep.EP_W4_MXFP4, 32) == 4 * 32 * 8
    assert ep.ep_w4_code_bytes(1024, 8192, 32768) == 1024 * 8192 * 16384     # beyond 32 bits
    for bad in ((0, 8, 128), (1025, 8, 128), (4, 12, 128), (4, 8, 64), (4, 8, 32896), (4, -8, 128)):
        assert ep.ep_w4_code_bytes(*bad) == 0, bad
    assert ep.ep_w4_scale_bytes(4, 24, 256, ep.EP_W4_MXFP4, 64) == 0
    assert ep.ep_w4_scale_bytes(4, 24, 256, 7, 32) == 0

    def pack(c=A16, s=A16, E=4, n=8, k=128, fmt=0, group=32, oc=A16, os_=A16):
        return ep.ep_w4_pack(c, s, E, n, k, fmt, group, oc, os_, None)
    assert pack(E=0) == ep.EP_ERR_SHAPE and pack(fmt=3) == ep.EP_ERR_DTYPE
    assert pack(group=48) == ep.EP_ERR_UNSUPPORTED and pack(k=100) == ep.EP_ERR_MISALIGNED
    assert pack(c=None) == ep.EP_ERR_NULL and pack(os_=None) == ep.EP_ERR_NULL
    assert pack(c=A16 + 2) == ep.EP_ERR_MISALIGNED and pack(oc=A16 + 4) == ep.EP_ERR_MISALIGNED


def act(h=None, gu=A16, inter=128, w=None, hdt=ep.EP_BF16, out=A16, fmt=F, sf=None, ts=1, hs=1,
        saved=None, sfmt=F, ssf=None, sts=2, shs=1):
    return ep.ep_swiglu(h or _fake_handle(), gu, inter, w, hdt, out, fmt, sf, ts, hs, saved, sfmt,
                        ssf, sts, shs, None)


@pytest.mark.parametrize("status,args", [
    (ep.EP_ERR_NOT_LAID_OUT, dict(h=_fake_handle(laid_out=0))),
    (ep.EP_ERR_WORKSPACE, dict(h=ep.ep_handle())),
    (ep.EP_ERR_DTYPE, dict(hdt=ep.EP_F32)),
    (ep.EP_ERR_SHAPE, dict(inter=0)),
    (ep.EP_ERR_MISALIGNED, dict(inter=12)),
    (ep.EP_ERR_MISALIGNED, dict(inter=136, hdt=ep.EP_FP8_E4M3, sf=A16)),
    (ep.EP_ERR_MISALIGNED, dict(inter=136, saved=A16, ssf=A16)),
    (ep.EP_ERR_UNSUPPORTED, dict(inter=32776)),
    (ep.EP_ERR_NULL, dict(gu=None)),
    (ep.EP_ERR_NULL, dict(out=None)),
    (ep.EP_ERR_NULL, dict(hdt=ep.EP_FP8_E4M3)),
    (ep.EP_ERR_NULL, dict(saved=A16)),
    (ep.EP_ERR_NULL, dict(ssf=A16)),
    (ep.EP_ERR_DTYPE, dict(sf=A16)),
    (ep.EP_ERR_DTYPE, dict(saved=A16, ssf=A16, sfmt=9)),
    (ep.EP_ERR_SHAPE, dict(saved=A16, ssf=A16, sts=-1)),
    (ep.EP_ERR_MISALIGNED, dict(gu=A16 + 8)),
    (ep.EP_ERR_MISALIGNED, dict(out=A16 + 8)),
    (ep.EP_ERR_MISALIGNED, dict(w=A16 + 2)),
    (ep.EP_ERR_MISALIGNED, dict(saved=A16 + 8, ssf=A16)),
    (ep.EP_ERR_MISALIGNED, dict(saved=A16, ssf=A16 + 1)),
])
def test_swiglu_refusals(status, args):
    assert act(**args) == status


def act_grad(h=None, g=A16, inter=128, w=None, saved=A16, dt=ep.EP_BF16, fmt=F, sf=None, ts=2,
             hs=1, ggu=A16, gw=None, out=None):
    return ep.ep_swiglu_backward(h or _fake_handle(), g, inter, w, saved, dt, fmt, sf, ts, hs,
                                 ggu, gw, out, None)


@pytest.mark.parametrize("status,args", [
    (ep.EP_ERR_NOT_LAID_OUT, dict(h=_fake_handle(laid_out=0))),
    (ep.EP_ERR_DTYPE, dict(dt=ep.EP_F32)),
    (ep.EP_ERR_SHAPE, dict(inter=-128)),
    (ep.EP_ERR_MISALIGNED, dict(inter=12)),
    (ep.EP_ERR_MISALIGNED, dict(FP8, inter=136)),
    (ep.EP_ERR_UNSUPPORTED, dict(inter=65536)),
    (ep.EP_ERR_NULL, dict(g=None)),
    (ep.EP_ERR_NULL, dict(saved=None)),
    (ep.EP_ERR_NULL, dict(ggu=None)),
    (ep.EP_ERR_NULL, dict(dt=ep.EP_FP8_E4M3)),
    (ep.EP_ERR_DTYPE, dict(sf=A16)),
    (ep.EP_ERR_DTYPE, dict(FP8, fmt=4)),
    (ep.EP_ERR_SHAPE, dict(FP8, ts=-2)),
    (ep.EP_ERR_MISALIGNED, dict(g=A16 + 8)),
    (ep.EP_ERR_MISALIGNED, dict(saved=A16 + 8)),
    (ep.EP_ERR_MISALIGNED, dict(ggu=A16 + 8)),
    (ep.EP_ERR_MISALIGNED, dict(gw=A16 + 2)),
    (ep.EP_ERR_MISALIGNED, dict(out=A16 + 8)),
])
def test_swiglu_gradient_refusals(status, args):
    assert act_grad(**args) == status


# ---------------------------------------------------------------- binding

@pytest.fixture
def fake(monkeypatch):
    class Lib(FakeLib):
        def __getattr__(self, name):
            call = super().__getattr__(name)
            sized = {"ep_w4_code_bytes": 4096, "ep_w4_scale_bytes": 512,
                     "ep_add_rmsnorm_backward_workspace": 1 << 16}
            if name not in sized:
                return call

            def counted(*args):
                call(*args)
                return sized[name]
            return counted

    lib = Lib()
    monkeypatch.setattr(ep, "lib", lambda: lib)
    monkeypatch.setattr(ep, "_stream", lambda: STREAM)
    monkeypatch.setattr(ep, "_dev", lambda t, name: ep._need(t.is_contiguous(),
                                                             f"{name} must be contiguous"))
    monkeypatch.setattr(ep, "_dev_strided", lambda t, name: None)
    return lib


def _handle(T=16, K=4, E=8, A=4):
    h = ep.Handle(T, K, E, A, device="cpu")
    h.h.num_tokens, h.h.num_topk, h.h.num_experts, h.h.max_tokens = T, K, E, T
    return h


def _bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_binding_norm_arguments(fake):
    x, r, w = _bf16(6, 256), _bf16(6, 256), torch.ones(256)
    y, z, q, sf, rstd = ep.add_rmsnorm(x, w, residual=r, eps=0.5, scale_format="ue8m0",
                                       want_rstd=True)
    assert q.shape == (6, 256) and sf.shape == (6, 1) and sf.dtype == torch.int32
    assert fake.last("ep_add_rmsnorm") == (
        x.data_ptr(), r.data_ptr(), w.data_ptr(), ep.EP_F32, 0.5, 6, 256, z.data_ptr(),
        y.data_ptr(), U, q.data_ptr(), sf.data_ptr(), 1, 1, rstd.data_ptr(), STREAM)
    gx, gw = ep.add_rmsnorm_backward(y, x, w, rstd, grad_residual=r)
    a = fake.last("ep_add_rmsnorm_backward")
    assert a[:10] == (y.data_ptr(), x.data_ptr(), w.data_ptr(), ep.EP_F32, rstd.data_ptr(),
                      r.data_ptr(), 6, 256, gx.data_ptr(), gw.data_ptr())
    assert a[11] == 1 << 16 and a[12] == STREAM
    bound = ep.bind_add_rmsnorm(x, w.bfloat16(), want_y=True)
    assert bound()[1] is None and fake.last("ep_add_rmsnorm")[3] == ep.EP_BF16


def test_binding_norm_refusals(fake):
    x, w = _bf16(6, 256), torch.ones(256)
    for bad in (lambda: ep.add_rmsnorm(x.float(), w), lambda: ep.add_rmsnorm(x, w[:128]),
                lambda: ep.add_rmsnorm(x, w.half()), lambda: ep.add_rmsnorm(x[:, ::2], w[::2]),
                lambda: ep.add_rmsnorm(x, w, residual=_bf16(5, 256)),
                lambda: ep.add_rmsnorm(x, w, out_q=torch.zeros((6, 256), dtype=torch.uint8)),
                lambda: ep.add_rmsnorm(x, w, scale_format="int8"),
                lambda: ep.add_rmsnorm(x, w, scale_format="f32", out_sf=torch.zeros((6, 3))),
                lambda: ep.add_rmsnorm(x, w, out_rstd=torch.zeros(5)),
                lambda: ep.add_rmsnorm_backward(x, x, w, torch.zeros(5)),
                lambda: ep.add_rmsnorm_backward(_bf16(6, 128), x, w, torch.zeros(6)),
                lambda: ep.add_rmsnorm_backward(x, x, w, torch.zeros(6), grad_weight=w.bfloat16())):
        with pytest.raises(ValueError):
            bad()


def test_binding_w4_arguments(fake):
    h = _handle()
    codes = torch.zeros((8, 24, 128), dtype=torch.uint8)
    p = ep.pack_w4(codes, _bf16(8, 24, 4))
    assert (p.num_experts, p.n, p.k, p.format, p.group) == (8, 24, 256, ep.EP_W4_INT4, 64)
    assert fake.last("ep_w4_pack")[2:7] == (8, 24, 256, 0, 64)
    m = ep.pack_w4(codes, torch.zeros((8, 24, 8), dtype=torch.uint8))
    assert (m.format, m.group) == (ep.EP_W4_MXFP4, 32)
    x = _bf16(16, 256)
    out = h.expert_w4(x, p, token_rows=True)
    a = fake.last("ep_expert_w4")
    assert a[1:9] == (x.data_ptr(), ep.EP_BF16, 1, 256, None, F, 0, 0)
    assert a[9:] == (p.codes.data_ptr(), p.scales.data_ptr(), 0, 64, 24, out.data_ptr(), STREAM)
    q = torch.zeros((h.capacity, 256), dtype=torch.uint8)
    sf = torch.zeros((1, h.capacity), dtype=torch.int32).t()
    h.bind_expert_w4(q, m, sf=sf)()
    a = fake.last("ep_expert_w4")
    assert a[2:4] == (ep.EP_FP8_E4M3, 0) and a[5:9] == (sf.data_ptr(), U, 1, h.capacity)


def test_binding_w4_refusals(fake):
    h = _handle()
    codes = torch.zeros((8, 24, 128), dtype=torch.uint8)
    p = ep.pack_w4(codes, _bf16(8, 24, 4))
    q = torch.zeros((h.capacity, 256), dtype=torch.uint8)
    for bad in (lambda: ep.pack_w4(codes, torch.zeros((8, 24, 4))),
                lambda: ep.pack_w4(codes, _bf16(8, 24, 3)), lambda: ep.pack_w4(codes, _bf16(8, 8, 4)),
                lambda: ep.pack_w4(codes.int(), _bf16(8, 24, 4)),
                lambda: h.expert_w4(_bf16(16, 256), p), lambda: h.expert_w4(_bf16(h.capacity, 128), p),
                lambda: h.expert_w4(q, p), lambda: h.expert_w4(q.float(), p),
                lambda: h.expert_w4(q, p, sf=torch.zeros((h.capacity, 1))),
                lambda: h.expert_w4(_bf16(h.capacity, 256), p, sf=torch.zeros((h.capacity, 2))),
                lambda: h.expert_w4(_bf16(h.capacity, 256), p, out=_bf16(h.capacity, 32)),
                lambda: _handle(E=4).expert_w4(_bf16(28, 256), p)):
        with pytest.raises(ValueError):
            bad()


def test_binding_swiglu_arguments(fake):
    h = _handle()
    cap = h.capacity
    gu, w = _bf16(cap, 768), torch.ones(cap)
    out, sf, saved, ssf = h.swiglu(gu, row_weights=w, scale_format="f32", checkpoint="ue8m0")
    assert sf.shape == (cap, 3) and saved.shape == (cap, 768) and ssf.shape == (cap, 2)
    assert fake.last("ep_swiglu")[1:] == (
        gu.data_ptr(), 384, w.data_ptr(), ep.EP_FP8_E4M3, out.data_ptr(), F, sf.data_ptr(), 3, 1,
        saved.data_ptr(), U, ssf.data_ptr(), 2, 1, STREAM)
    g = _bf16(cap, 384)
    ggu, gw, again = h.swiglu_backward(g, saved, ssf, row_weights=w, want_grad_weights=True,
                                       want_h=True)
    assert fake.last("ep_swiglu_backward")[1:] == (
        g.data_ptr(), 384, w.data_ptr(), saved.data_ptr(), ep.EP_FP8_E4M3, U, ssf.data_ptr(), 2, 1,
        ggu.data_ptr(), gw.data_ptr(), again.data_ptr(), STREAM)
    h.bind_swiglu(gu)()
    a = fake.last("ep_swiglu")
    assert a[3:5] == (None, ep.EP_BF16) and a[6:8] == (F, None) and a[10] is None


def test_binding_swiglu_refusals(fake):
    h = _handle()
    cap = h.capacity
    gu, g = _bf16(cap, 768), _bf16(cap, 384)
    q = torch.zeros((cap, 768), dtype=torch.uint8)
    for bad in (lambda: h.swiglu(gu.float()), lambda: h.swiglu(_bf16(cap, 767)),
                lambda: h.swiglu(_bf16(cap - 1, 768)), lambda: h.swiglu(gu, row_weights=torch.ones(3)),
                lambda: h.swiglu(gu, out_sf=torch.zeros((cap, 3))), lambda: h.swiglu(gu, saved=q),
                lambda: h.swiglu(gu, scale_format="f32", out=g),
                lambda: h.swiglu(_bf16(cap, 128), checkpoint="f32"),
                lambda: h.swiglu(gu, checkpoint="f32", saved=gu),
                lambda: h.swiglu_backward(g, q), lambda: h.swiglu_backward(g, gu, torch.zeros((cap, 6))),
                lambda: h.swiglu_backward(g, q, torch.zeros((cap, 3))),
                lambda: h.swiglu_backward(_bf16(cap, 128), gu),
                lambda: h.swiglu_backward(g, gu, grad_row_weights=torch.zeros(3)),
                lambda: h.swiglu_backward(g, gu, out=gu)):
        with pytest.raises(ValueError):
            bad()


def test_bound_calls_refuse_another_batch(fake):
    h = _handle()
    call = h.bind_swiglu(_bf16(h.capacity, 256))
    call()
    h.h.num_tokens = 3
    with pytest.raises(ValueError, match="bound for 16 tokens"):
        call()


def test_status_becomes_an_error(fake):
    fake.status = ep.EP_ERR_HIP
    with pytest.raises(ep.EpError) as e:
        ep.add_rmsnorm(_bf16(2, 256), torch.ones(256))
    assert e.value.status == ep.EP_ERR_HIP


FAR = A16 + (1 << 30)                    # nothing of these sizes reaches from A16 to there


@pytest.mark.parametrize("call", [
    lambda: norm(y=A16),                                        # y over x
    lambda: norm(r=FAR, y=FAR),
    lambda: norm(y=FAR, z=FAR),
    lambda: norm(z=A16 + 16, y=None),                           # z over a part of x
    lambda: norm(y=None, q=A16 + 4 * 512 - 16, sf=FAR),         # codes over x's end
    lambda: norm(y=FAR, q=FAR + 4 * 512 - 16, sf=FAR),
    lambda: norm(z=FAR, y=None, q=FAR, sf=FAR),
    lambda: norm_grad(gx=A16 + 16),
    lambda: norm_grad(g=FAR, gx=FAR - 16),
    lambda: norm_grad(g=FAR, z=FAR, gz=A16 + 16),
    lambda: w4(),
    lambda: w4(**FP8),
    lambda: w4(tokens=1, x=A16 + 16),
    lambda: act(),
    lambda: act(hdt=ep.EP_FP8_E4M3, sf=FAR),
    lambda: act(out=FAR, saved=A16, ssf=FAR),
    lambda: act(out=FAR, saved=FAR, ssf=FAR),
    lambda: act_grad(),
    lambda: act_grad(saved=FAR, ggu=FAR + 16),
    lambda: act_grad(saved=FAR, ggu=FAR + (1 << 28), out=FAR),
    lambda: act_grad(saved=FAR, ggu=FAR, out=FAR),
    lambda: act_grad(saved=FAR, dt=ep.EP_FP8_E4M3, sf=A16, ggu=FAR),
])
def test_overlapping_rows_are_refused(call):
    assert call() == ep.EP_ERR_UNSUPPORTED


def test_packed_weights_of_other_sizes_are_refused(monkeypatch):
    """Weights put together by hand: the kernel reads as many bytes as the sizes say, so
    buffers of any other size are an error and not a read past their end."""
    monkeypatch.setattr(ep, "_dev", lambda t, name: ep._need(t.is_contiguous(),
                                                             f"{name} must be contiguous"))
    E, n, k = 3, 24, 256
    nc = ep.ep_w4_code_bytes(E, n, k)
    assert nc == E * 32 * k // 2
    for fmt, group, ns in ((ep.EP_W4_INT4, 64, E * 32 * 4 * 2), (ep.EP_W4_MXFP4, 32, E * 32 * 8)):
        assert ep.ep_w4_scale_bytes(E, n, k, fmt, group) == ns
        codes, scales = (torch.zeros(b, dtype=torch.uint8) for b in (nc, ns))
        w = ep.W4Weights(codes, scales, E, n, k, fmt, group)
        assert w.codes is codes and w.scales is scales
        for bad in ((codes[:-1], scales, E, n, k, fmt, group),
                    (codes, scales[:-1], E, n, k, fmt, group),
                    (codes, scales, E + 1, n, k, fmt, group),
                    (codes, scales, E, n + 16, k, fmt, group),
                    (codes, scales, E, n, 2 * k, fmt, group),
                    (codes, scales, E, n, k + 1, fmt, group),
                    (codes, scales, E, n, k, fmt, 48),
                    (torch.zeros(2 * nc, dtype=torch.uint8)[::2], scales, E, n, k, fmt, group)):
            with pytest.raises(ValueError):
                ep.W4Weights(*bad)
