"""Plain binary64 forms of the layer operators, and the 8- and 4-bit formats
they read and write, for the tests (torch on whatever device the inputs are)."""
import torch

import combine_ep_layout_08_amd as ep

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
E2M1 = torch.cat((E2M1, -E2M1))
BF16 = 2.0 ** -8          # half a step of bf16, relative
F32 = 2.0 ** -24          # half a step of binary32, relative
POISON = 0x5A


def scale_values(sf, blocks):
    """Scales [rows, blocks] as binary64, from fp32 scales or int32 packs of exponents."""
    if sf.dtype == torch.float32:
        return sf.double()
    e = torch.stack([(sf >> (8 * i)) & 255 for i in range(4)], -1).flatten(1)[:, :blocks]
    return torch.exp2(e.double() - 127.0)


def code_values(q, sf):
    """What E4M3 rows with scales of 128 channels stand for."""
    v = q.view(torch.float8_e4m3fn).double()
    return v * scale_values(sf, q.shape[1] // 128).repeat_interleave(128, 1)


def quantise(v, fmt):
    """The E4M3 recipe on fp32 rows of finite values: codes and scales."""
    b = v.reshape(v.shape[0], -1, 128)
    # a tensor as divisor: by a number, torch multiplies with its reciprocal on the GPU
    s = torch.clamp(b.abs().amax(2), min=1e-12)
    s = s / torch.full_like(s, 448.0)
    if fmt == "ue8m0":
        bits = s.view(torch.int32)
        e = (bits >> 23) + ((bits & 0x7FFFFF) != 0).int()
        s = (e << 23).view(torch.float32)
        e = torch.nn.functional.pad(e, (0, -e.shape[1] % 4)).reshape(e.shape[0], -1, 4)
        sf = e[..., 0] | (e[..., 1] << 8) | (e[..., 2] << 16) | (e[..., 3] << 24)
    else:
        sf = s
    q = (b / s[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.reshape(v.shape).view(torch.uint8), sf


def swiglu(gate_up, w=None):
    g, u = gate_up.double().chunk(2, 1)
    h = g * torch.sigmoid(g) * u
    return h if w is None else h * w.double()[:, None]


def w4_values(codes, scales, group):
    """Weights [E, n, k] in binary64."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(2).long()
    if scales.dtype == torch.bfloat16:
        v, s = (c - 8).double(), scales.double()
    else:
        v = E2M1.to(codes.device)[c]
        s = torch.exp2(scales.view(torch.uint8).double() - 127.0)
    return v * s.repeat_interleave(group, 2)


def random_w4(E, n, k, fmt, group, gen, device):
    """Codes over their whole range, scales of both small and large groups."""
    codes = torch.randint(0, 256, (E, n, k // 2), generator=gen, device=device, dtype=torch.uint8)
    s = torch.rand((E, n, k // group), generator=gen, device=device) + 0.5
    if fmt == ep.EP_W4_INT4:
        return codes, (s * 0.02).bfloat16()
    return codes, (118 + 6 * s).to(torch.uint8)


def ids(T, K, E, gen, device, empty=0.0):
    """Distinct experts for each token, some slots empty (all of them for token 0
    of a batch with empty slots)."""
    i = torch.rand((T, E), generator=gen, device=device).topk(K, dim=1).indices
    gone = torch.rand((T, K), generator=gen, device=device) < empty
    if empty:
        gone[:1] = True
    return i.masked_fill(gone, -1).contiguous()


def rows_of(handle, topk_idx):
    """Of every slot that holds a row: the row, its expert, its token."""
    dst = handle.dst_slot.reshape(-1).long()
    slot = torch.nonzero(dst >= 0).reshape(-1)
    return dst[slot], topk_idx.reshape(-1)[slot].long(), slot // topk_idx.shape[1]


def untouched(t, rows):
    """Whether every row of ``t`` but these still holds the poison."""
    left = torch.ones(t.shape[0], dtype=torch.bool, device=t.device)
    left[rows] = False
    return bool((t.contiguous().view(torch.uint8).reshape(t.shape[0], -1)[left] == POISON).all())


def poisoned(shape, dtype, device="cuda"):
    t = torch.empty(shape, dtype=dtype, device=device)
    t.view(torch.uint8).fill_(POISON)
    return t


def assert_close(got, want, tol, what):
    """|got - want| <= tol elementwise (binary64), NaN where want is NaN."""
    got, want = got.double(), want.double()
    bad = ~((got - want).abs() <= tol) & ~(got.isnan() & want.isnan()) & (got != want)
    if bool(bad.any()):
        at = torch.nonzero(bad)[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; at {at}: got "
                             f"{got[tuple(at)]}, want {want[tuple(at)]}")
