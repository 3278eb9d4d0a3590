"""Angles against 60 decimal digits.  x = (1, 0) in every pair, so y is
(cos, sin) itself.  fp32: sincospif is off by one unit of 2^-24 at most and the
correction of its argument rounds once (half a unit); the products with 1, 0
and mscale = 1 are exact.  The angle: the speed comes from a 64-bit power (one
unit of 2^-52), at most four more roundings and the product's: 8 * 2^-53 of
pos * f_i."""
import decimal
from decimal import Decimal as D

import numpy as np
import pytest
import torch

from conftest import cuda_ok
from long_context_decode_indexer_b200 import dsa
from long_context_decode_indexer_b200.batch import workspace

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

PI = D("3.14159265358979323846264338327950288419716939937510582097494459")


def turns60(rot, theta, scaling=0, factor=1.0, orig=0):
    """Turns per position of every pair, 60 digits (the YaRN ramp's ends are
    whole numbers, so 64 bits give them)."""
    base = D(theta)
    if scaling == 2:
        base *= (D(factor).ln() * rot / (rot - 2)).exp()
    if scaling == 3:
        edge = [rot * np.log(orig / (2 * np.pi * b)) / (2 * np.log(theta)) for b in (32.0, 1.0)]
        lo, hi = max(np.floor(edge[0]), 0.0), min(np.ceil(edge[1]), rot - 1.0)
    out = []
    for i in range(rot // 2):
        f = (base.ln() * D(-2 * i) / rot).exp()
        if scaling == 1:
            f /= D(factor)
        if scaling == 3:
            r = D(float(min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)))
            f = f * (1 - r) + f / D(factor) * r
        out.append(f / (2 * PI))
    return out


def cos_sin(pos, turn):
    """[len(pos), len(turn), 2] in 64 bits."""
    r = np.empty((len(pos), len(turn), 2))
    for i, p in enumerate(pos):
        for k, t in enumerate(turn):
            a = D(int(p)) * t
            a = float((a - a.to_integral_value()) * 2 * PI)
            r[i, k] = np.cos(a), np.sin(a)
    return r


SPECS = [dict(theta=10000.0), dict(theta=500000.0, scaling=1, factor=8.0), dict(theta=10000.0, scaling=2, factor=4.0),
         dict(theta=10000.0, scaling=3, factor=40.0, orig=4096), dict(theta=1.0)]


@pytest.mark.parametrize("spec", range(len(SPECS)))
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("rot", [64, 256, 2])
def test_sines_are_fp32_exact(spec, layout, rot):
    decimal.getcontext().prec = 60
    s = dict(SPECS[spec])
    rng = np.random.default_rng(spec)
    pos = np.unique(np.r_[0, 1, 2 ** 31 - 1, 2 ** 30 + 1, 2 ** 27, 2 ** 27 - 1, rng.integers(2, 5000, 30),
                          (2.0 ** rng.uniform(0, 31, 30)).astype(np.int64)])
    if s.get("scaling") == 2 and rot == 2:
        return      # one pair: its speed is 1 whatever the base
    turn = turns60(rot, **s)
    want = cos_sin(pos, turn)
    kw = dict(s)
    kw["orig_max_pos"] = kw.pop("orig", 0)
    rs = dsa.make_rope_spec(rope_dim=rot, layout=layout, **kw)
    x = torch.zeros((len(pos), 1, rot), device="cuda")
    first = x[..., 0::2] if layout == 0 else x[..., :rot // 2]
    first.fill_(1.0)
    p = torch.from_numpy(pos.astype(np.int32)).cuda()
    angle = np.abs(pos[:, None].astype(float) * np.array([float(t) for t in turn]) * 2 * np.pi)
    tol = (1.5 * 2.0 ** -24 + 8 * 2.0 ** -53 * angle)[..., None]
    assert np.all(tol[pos <= 2 ** 27] <= 4 * 2.0 ** -24)

    def parts(y):
        y = y.double().cpu().numpy()[:, 0]
        return np.stack((y[:, 0::2], y[:, 1::2]) if layout == 0 else (y[:, :rot // 2], y[:, rot // 2:]), -1)

    for d, begin in ((rot, 0), (rot + 3, 3)):            # by 16 bytes, and element by element
        full = torch.zeros((len(pos), 1, d), device="cuda")
        full[..., begin:] = x
        y = torch.full_like(full, 7.0)
        rp = dsa.make_rope_params(nt=len(pos), h=1, d=d, begin=begin, dtype=dsa.DTYPE_FP32)
        dsa.rope(rs, rp, full, p, y)
        assert np.all(np.abs(parts(y[..., begin:]) - want) <= tol)
        dsa.rope_backward(rs, rp, full, p, y)            # the inverse turn: (cos, -sin)
        assert np.all(np.abs(parts(y[..., begin:]) * (1, -1) - want) <= tol)
    rp = dsa.make_rope_params(nt=len(pos), h=3, x_heads=1, d=rot, dtype=dsa.DTYPE_FP32)
    dy, dx = torch.zeros((len(pos), 3, rot), device="cuda"), torch.empty_like(x)
    dy[:, 1] = x[:, 0]
    dsa.rope_backward(rs, rp, dy, p, dx)
    assert np.all(np.abs(parts(dx) * (1, -1) - want) <= tol)


@pytest.mark.parametrize("fp8", [False, True])
def test_angles_of_appended_rows(fp8):
    """bf16: half a step of the value on top of the above.  FP8: codes of
    values up to 1, the row's largest being 448 (scale 1)."""
    decimal.getcontext().prec = 60
    pos = np.array([2 ** 27, 2 ** 27 - 12345, 2 ** 20 + 3, 5])
    want = cos_sin(pos, turns60(64, 10000.0))
    n = len(pos)
    pe = torch.zeros((n, 64), device="cuda")
    pe[:, 0::2] = 1.0
    c = torch.zeros((n, 512), device="cuda")
    c[:, 0] = 448.0
    p, slots = (torch.from_numpy(np.asarray(a, np.int32)).cuda() for a in (pos, range(n)))
    ws, rs = workspace(dsa.WS_STATUS_BYTES), dsa.make_rope_spec()
    if not fp8:
        cache = torch.zeros((n, 576), dtype=torch.bfloat16, device="cuda")
        dsa.latent_append(rs, c.bfloat16(), pe.bfloat16(), p, slots, cache, ws)
        got = cache[:, 512:].double().cpu().numpy().reshape(n, 32, 2)
        assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 4 * 2.0 ** -24)
    else:
        cache = torch.zeros((n, 576), dtype=torch.uint8, device="cuda")
        sc = torch.zeros(n, device="cuda")
        dsa.latent_append_fp8(rs, c.bfloat16(), pe.bfloat16(), p, slots, cache, sc, ws)
        assert torch.all(sc == 1)
        code = torch.from_numpy(want.astype(np.float32)).to(torch.float8_e4m3fn)
        assert torch.equal(cache[:, 512:].cpu().view(n, 32, 2), code.view(torch.uint8))
    assert dsa.check_status(ws) == dsa.DSA_OK


# --------------------------------------------------- values that are not finite
@pytest.mark.parametrize("dtype", [dsa.DTYPE_BF16, dsa.DTYPE_FP16, dsa.DTYPE_FP32])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("xh,d,begin", [(6, 64, 0), (6, 70, 3), (1, 64, 0), (1, 70, 3)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_values_that_are_not_finite_stay_in_their_pair(dtype, layout, xh, d, begin, value):
    """They reach the two elements of their pair (every head's, where heads
    share it; the shared gradient's pair, where heads are summed) and nothing
    else; in a token that is padding they reach nothing."""
    dt = {dsa.DTYPE_BF16: torch.bfloat16, dsa.DTYPE_FP16: torch.float16, dsa.DTYPE_FP32: torch.float32}[dtype]
    nt, h, rot = 5, 6, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rs = dsa.make_rope_spec(rope_dim=rot, layout=layout)
    rp = dsa.make_rope_params(nt=nt, h=h, x_heads=xh, d=d, begin=begin, dtype=dtype)
    p = torch.tensor([3, 1000, -1, 77, 12345], dtype=torch.int32, device="cuda")
    pair = 9
    i0, i1 = (begin + 2 * pair, begin + 2 * pair + 1) if layout == 0 else (begin + pair, begin + pair + rot // 2)
    for backward in (False, True):
        heads_in, heads_out = (h, xh) if backward else (xh, h)
        x = torch.randn((nt, heads_in, d), generator=g, device="cuda").to(dt)
        fn = dsa.rope_backward if backward else dsa.rope
        want, got = (torch.zeros((nt, heads_out, d), dtype=dt, device="cuda") for _ in range(2))
        fn(rs, rp, x, p, want)
        x[1, heads_in - 1, i1] = value
        x[2, 0, i0] = value                      # padding
        if begin:
            x[3, 0, begin - 1] = value           # copied, not turned
        fn(rs, rp, x, p, got)
        touched = torch.zeros((nt, heads_out, d), dtype=torch.bool, device="cuda")
        touched[1, slice(None) if xh == 1 else h - 1, [i0, i1]] = True
        if begin:
            touched[3, slice(None) if xh == 1 else 0, begin - 1] = True
        assert torch.equal(got[~touched], want[~touched])
        assert not torch.isfinite(got[touched]).any()


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("h,xh,d,begin", [(6, 6, 64, 0), (6, 1, 64, 0), (6, 6, 70, 3), (6, 1, 70, 3), (1, 1, 70, 3)])
def test_sources_that_repeat_a_row(layout, h, xh, d, begin):
    """Strides of 0 on the side that is read (an expanded row, the gradient
    of a sum): the same bits as with the rows written out."""
    nt = 21
    p = torch.arange(-1, nt - 1, dtype=torch.int32, device="cuda") * 97
    rs = dsa.make_rope_spec(layout=layout)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    for backward in (False, True):
        heads_in, heads_out = (h, xh) if backward else (xh, h)
        for row in ((1, heads_in, d), (nt, 1, d), (1, 1, d)):
            x = torch.randn(row, generator=g, device="cuda").expand(nt, heads_in, d)
            st = x.stride()[:2]
            got = []
            for src in (x, x.contiguous()):
                kw = {} if src is not x else ({"y_strides": st} if backward else {"x_strides": st})
                rp = dsa.make_rope_params(nt=nt, h=h, x_heads=xh, d=d, begin=begin, dtype=dsa.DTYPE_FP32, **kw)
                dst = torch.full((nt, heads_out, d), 7.0, device="cuda")
                (dsa.rope_backward if backward else dsa.rope)(rs, rp, src, p, dst)
                got.append(dst)
            assert torch.equal(got[0], got[1])
