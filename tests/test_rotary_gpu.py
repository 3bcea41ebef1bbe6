"""Head norms and rotary positions against float64.

Tolerance per element, y the exact result, (a, b) the normed pair, u = eps / 2
of the output type:
  u |y|                         the rounding of the output
  (|a| + |b|) m e               e = (d / 2 + 8) 2^-24 for the norm (d squares
                                summed in fp32 under a root, rsqrt, products)
                                + 2^-21 for sine and cosine: their own error
                                (2 ulp) and the angle, one fp32 rounding of up
                                to one half turn (pi 2^-25)
channels outside the rotated part: the first two without the angle.
"""
import math

import pytest
import torch

import confidence_gated_kv_gb300 as ck

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def frequencies(rot, base, scaling, factor, length=4096, fast=32.0, slow=1.0):
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f, m = base ** (-2 * i / rot), 1.0
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        g = ((length * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        f, m = f * g + f / factor * (1 - g), 0.1 * math.log(factor) + 1
    return f, m


def reference(x, w, pos, rot, interleaved, f, m, eps):
    d = x.shape[2]
    x = x.double()
    if w is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    e = (d / 2 + 8) * 2.0 ** -24
    y, tol = x.clone(), x.abs() * e
    if rot:
        ia = torch.arange(0, rot, 2) if interleaved else torch.arange(0, rot // 2)
        ib = ia + 1 if interleaved else ia + rot // 2
        t = (pos.double()[:, None] * f)[:, None]
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = (a * t.cos() - b * t.sin()) * m, (b * t.cos() + a * t.sin()) * m
        tol[..., ia] = tol[..., ib] = (a.abs() + b.abs()) * m * (e + 2.0 ** -21 + pos.double().abs()[:, None, None] * 2.0 ** -50)
    return y, tol


def check(got, ref, tol):
    u = torch.finfo(got.dtype).eps / 2
    low = {F16: 2.0 ** -25, BF16: 2.0 ** -134, F32: 2.0 ** -150}[got.dtype]      # halves of the smallest steps
    off = (got.double() - ref).abs() - ((u * (ref.abs() + tol) + tol) * 1.001 + low)
    assert torch.isfinite(got).all()
    assert float(off.max()) <= 0, float(off.max())


def case(n, Hq, Hkv, d, rot, dtype, norm, interleaved, scaling="none", factor=1.0, first=0, outs=None, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    q, k = rand(n, Hq, d).to(dtype), (3 * rand(n, Hkv, d)).to(dtype)
    qw, kw = ((1 + 0.2 * rand(d)).to(dtype), (1 + 0.2 * rand(d)).to(dtype)) if norm else (None, None)
    pos = (torch.randint(0, 5000, (n,), generator=g, device="cuda") + first).int()
    r = ck.Rotary(rot, 10000.0, scaling, factor, interleaved=interleaved) if rot else None
    kwargs = {}
    if outs:
        kwargs = dict(q_out=torch.empty((n, Hq, d), dtype=outs[0], device="cuda"),
                      k_out=torch.empty((n, Hkv, d), dtype=outs[1], device="cuda"))
    f, m = frequencies(rot, 10000.0, scaling, factor) if rot else (None, 1.0)
    qo, ko = ck.qk_rotary(q, k, pos, r, qw, kw, eps=1e-6, **kwargs)
    check(qo, *reference(q, qw, pos, rot, interleaved, f, m, 1e-6))
    check(ko, *reference(k, kw, pos, rot, interleaved, f, m, 1e-6))


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("d, rot", [(64, 64), (128, 128), (128, 32), (256, 128), (64, 0), (128, 24), (80, 80),
                                    (96, 48), (6, 2), (511, 300)])
def test_layouts_and_types(d, rot, interleaved, norm, dtype):
    case(7, 10, 2, d, rot, dtype, norm, interleaved)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 1000, 5000])
@pytest.mark.parametrize("Hq, Hkv", [(1, 1), (12, 12), (40, 8)])
def test_lengths_and_heads(n, Hq, Hkv):
    case(n, Hq, Hkv, 64, 64, BF16, True, False, seed=n)


@pytest.mark.parametrize("scaling, factor", [("linear", 4.0), ("ntk", 8.0), ("yarn", 32.0), ("yarn", 1.0)])
@pytest.mark.parametrize("first", [0, 1000000, 2147478000, -2147483648])
def test_scalings_and_far_positions(scaling, factor, first):
    case(64, 4, 2, 128, 128, BF16, True, False, scaling, factor, first)
    case(64, 4, 2, 128, 64, F16, False, True, scaling, factor, first)


@pytest.mark.parametrize("outs", [(BF16, F16), (F16, F32), (F32, BF16)])
def test_outputs_of_other_types(outs):
    case(33, 10, 2, 128, 128, BF16, True, False, outs=outs)
    case(33, 10, 2, 96, 96, F32, True, True, outs=outs)


def test_rows_of_zeros_and_weights_for_one_tensor():
    q, k = torch.zeros((3, 2, 64), dtype=F16, device="cuda"), torch.ones((3, 1, 64), dtype=F16, device="cuda")
    pos, r = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), ck.Rotary(64)
    w = torch.full((64,), 2.0, dtype=F32, device="cuda")
    qo, ko = ck.qk_rotary(q, k, pos, r, q_weight=w)
    assert float(qo.abs().max()) == 0
    check(ko, *reference(k, None, pos, 64, False, *frequencies(64, 10000.0, "none", 1.0), 1e-6))
    qo, none = ck.qk_rotary(q + 1, None, pos, r, q_weight=w)
    assert none is None
    check(qo, *reference(q + 1, w, pos, 64, False, *frequencies(64, 10000.0, "none", 1.0), 1e-6))


@pytest.mark.parametrize("d, rot", [(128, 128), (128, 64), (80, 40)])
@pytest.mark.parametrize("interleaved", [True, False])
def test_in_place_strided_and_unaligned(d, rot, interleaved):
    n, Hq, Hkv = 50, 10, 2
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((n, Hq + 2 * Hkv, d), generator=g, device="cuda").to(BF16)
    pos, r = torch.arange(n, device="cuda").int() + 77, ck.Rotary(rot, interleaved=interleaved)
    w = torch.rand(d, generator=g, device="cuda")
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:].clone()
    want = ck.qk_rotary(q.contiguous(), k.contiguous(), pos, r, w, w)
    # rows that start off a 16-byte boundary
    wide = torch.zeros((n, Hq + 2 * Hkv, d + 3), dtype=BF16, device="cuda")
    wide[..., 1:d + 1] = x
    odd = ck.qk_rotary(wide[:, :Hq, 1:d + 1], wide[:, Hq:Hq + Hkv, 1:d + 1], pos, r, w, w)
    for a, b in zip(odd, want):      # the two forms sum squares in another order
        assert float((a.double() - b.double()).abs().max()) <= 2.0 ** -8 * 2 * float(b.abs().max())
    got = ck.qk_rotary(q, k, pos, r, w, w, q_out=q, k_out=k)
    assert got[0].data_ptr() == q.data_ptr()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(x[:, Hq + Hkv:], v)


def test_replayed_with_new_positions():
    q, k = torch.randn(2, 10, 128, device="cuda").to(BF16), torch.randn(2, 2, 128, device="cuda").to(BF16)
    pos, r = torch.tensor([5, 9], dtype=torch.int32, device="cuda"), ck.Rotary(128)
    qo, ko = torch.empty_like(q), torch.empty_like(k, dtype=F16)
    ck.qk_rotary(q, k, pos, r, q_out=qo, k_out=ko)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ck.qk_rotary(q, k, pos, r, q_out=qo, k_out=ko)
    for step in range(3):
        pos += 1
        graph.replay()
        a, b = ck.qk_rotary(q, k, pos, r, k_out=torch.empty_like(ko))
        assert torch.equal(qo, a) and torch.equal(ko, b)


def test_no_rows():
    q, k = torch.empty(0, 4, 64, dtype=F16, device="cuda"), torch.empty(0, 2, 64, dtype=F16, device="cuda")
    a, b = ck.qk_rotary(q, k, torch.empty(0, dtype=torch.int32, device="cuda"), ck.Rotary(64))
    assert a.shape == q.shape and b.shape == k.shape
