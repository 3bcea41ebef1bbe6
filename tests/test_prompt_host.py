"""Refusals and host arithmetic of the prompt operators (no GPU needed: every
refused call returns before anything is launched)."""
import ctypes
import math
import struct

import pytest
import torch

import confidence_gated_kv_gb300 as ck
from confidence_gated_kv_gb300 import binding, prompt

PTR = 1 << 20          # an aligned address that nothing reads


def attention_args(**kw):
    a = dict(B=1, Hq=8, Hkv=2, d=128, dtype=0, causal=1, total_q=10, total_k=10, scale=0.1, q=PTR, k=PTR, v=PTR,
             out=2 * PTR, lse=0, cu_q=PTR, cu_k=PTR, qs=(1024, 128), ks=(256, 128), vs=(256, 128), os=(1024, 128))
    a.update(kw)
    return prompt._PROMPT.pack(a["B"], a["Hq"], a["Hkv"], a["d"], a["dtype"], a["causal"], a["total_q"],
                               a["total_k"], a["scale"], a["q"], a["k"], a["v"], a["out"], a["lse"], a["cu_q"],
                               a["cu_k"], *a["qs"], *a["ks"], *a["vs"], *a["os"])


@pytest.mark.parametrize("bad", [
    dict(B=0), dict(Hq=0), dict(Hkv=0), dict(Hq=9), dict(Hq=258), dict(total_q=-1), dict(total_k=-1), dict(total_q=2 ** 31 - 1),
    dict(total_k=2 ** 31 - 100), dict(dtype=2),
    dict(dtype=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(q=0),
    dict(k=0), dict(v=0), dict(out=0), dict(cu_q=0), dict(cu_k=0), dict(cu_q=PTR + 2), dict(q=PTR + 8),
    dict(k=PTR + 2), dict(v=PTR + 4), dict(out=PTR + 8), dict(lse=PTR + 1), dict(qs=(1020, 128)),
    dict(qs=(1024, 120)), dict(ks=(256, 0)), dict(vs=(-256, 128)), dict(os=(64, 128)), dict(os=(128, 128)),
    dict(os=(512, 128)),
])
def test_attention_refusals(bad):
    assert ck.lib().confkv_prompt_attention(attention_args(**bad), None) == binding.EINVAL


def test_attention_head_sizes_and_empty_calls():
    L = ck.lib()
    for d in (32, 96, 256):
        assert L.confkv_prompt_attention(attention_args(d=d), None) == binding.ENOTIMPL
    assert L.confkv_prompt_attention(None, None) == binding.EINVAL
    assert L.confkv_prompt_attention(attention_args(total_q=0, q=0, out=0), None) == binding.OK
    assert L.confkv_prompt_status(None, None) == binding.EINVAL


def rotary_args(**kw):
    a = dict(n=4, Hq=8, Hkv=2, d=128, rot=128, inter=0, in_=0, w=0, qo_t=0, ko_t=0, eps=1e-6, mscale=1.0, q=PTR,
             k=PTR, qo=2 * PTR, ko=3 * PTR, qs=(1024, 128), ks=(256, 128), qos=(1024, 128), kos=(256, 128), qw=PTR,
             kw=PTR, pos=PTR, turns=PTR)
    a.update(kw)
    return prompt._ROTARY.pack(a["n"], a["Hq"], a["Hkv"], a["d"], a["rot"], a["inter"], a["in_"], a["w"], a["qo_t"],
                               a["ko_t"], a["eps"], a["mscale"], a["q"], a["k"], a["qo"], a["ko"], *a["qs"],
                               *a["ks"], *a["qos"], *a["kos"], a["qw"], a["kw"], a["pos"], a["turns"])


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(Hq=0), dict(Hkv=-1), dict(d=0, rot=0), dict(rot=3), dict(rot=130), dict(rot=-2), dict(in_=3),
    dict(w=7), dict(qo_t=-1), dict(ko_t=3), dict(eps=-1.0), dict(eps=math.nan), dict(mscale=math.inf), dict(q=0),
    dict(k=0), dict(qo=0), dict(ko=0), dict(pos=0), dict(turns=0), dict(pos=PTR + 2), dict(turns=PTR + 4),
    dict(q=PTR + 1), dict(qo=PTR + 1), dict(qw=PTR + 1),
    dict(qos=(1024, 64)), dict(qos=(512, 128)), dict(kos=(0, 128)),          # rows that overlap
    dict(qo=PTR, qos=(2048, 128)), dict(ko=PTR, ko_t=1),                     # in place, elsewhere or another type
])
def test_rotary_refusals(bad):
    assert ck.lib().confkv_qk_rotary(rotary_args(**bad), None) == binding.EINVAL


def test_rotary_sizes():
    L = ck.lib()
    assert L.confkv_qk_rotary(rotary_args(d=514, rot=0), None) == binding.ENOTIMPL
    assert L.confkv_qk_rotary(None, None) == binding.EINVAL
    assert L.confkv_qk_rotary(rotary_args(n=0, q=0, k=0), None) == binding.OK


def frequencies(rot, base=10000.0, kind=0, factor=1.0, length=4096.0, fast=32.0, slow=1.0):
    t, m = (ctypes.c_uint64 * max(1, rot // 2))(), ctypes.c_float()
    r = ck.lib().confkv_rotary_frequencies(rot, base, kind, factor, length, fast, slow, t, ctypes.byref(m))
    return r, [x / 2.0 ** 64 * 2 * math.pi for x in t][:rot // 2], m.value


def test_frequencies():
    rot = 64
    plain = [10000.0 ** (-2 * i / rot) for i in range(rot // 2)]
    r, f, m = frequencies(rot)
    assert r == 0 and m == 1.0 and f == pytest.approx(plain, rel=1e-15)
    assert frequencies(rot, kind=1, factor=4.0)[1] == pytest.approx([x / 4 for x in plain], rel=1e-15)
    base = 10000.0 * 8.0 ** (rot / (rot - 2))
    assert frequencies(rot, kind=2, factor=8.0)[1] == pytest.approx([base ** (-2 * i / rot) for i in range(rot // 2)],
                                                                   rel=1e-14)
    r, f, m = frequencies(rot, kind=3, factor=16.0, length=2048.0)
    assert m == pytest.approx(0.1 * math.log(16.0) + 1, rel=1e-7)
    turns = [2048.0 * x / (2 * math.pi) for x in plain]
    for got, x, n in zip(f, plain, turns):
        if n > 32:
            assert got == pytest.approx(x, rel=1e-15)               # many turns: kept
        elif n < 1:
            assert got == pytest.approx(x / 16, rel=1e-15)          # less than one: interpolated
        else:
            assert x / 16 < got <= x
    assert any(n > 32 for n in turns) and any(n < 1 for n in turns) and any(1 < n < 32 for n in turns)
    assert frequencies(0)[0] == 0


@pytest.mark.parametrize("bad", [
    dict(rot=3), dict(rot=-2), dict(base=1.0), dict(base=math.nan), dict(base=math.inf), dict(kind=4),
    dict(kind=-1), dict(kind=1, factor=0.5), dict(kind=3, factor=math.nan), dict(kind=3, factor=2.0, length=0.0),
    dict(kind=3, factor=2.0, fast=1.0, slow=1.0), dict(kind=3, factor=2.0, slow=-1.0), dict(rot=2, kind=2, factor=2.0),
])
def test_frequency_refusals(bad):
    assert frequencies(**dict(dict(rot=64), **bad))[0] == binding.EINVAL


def test_layer_calls_need_a_context():
    L = ck.lib()
    n = ctypes.c_int64()
    s = struct.pack("=2q", 256, 128)
    assert L.confkv_prefill_begin(None, s, None) == binding.EINVAL
    assert L.confkv_prefill_layer(None, 0, PTR, PTR, 0, s, s, None) == binding.EINVAL
    assert L.confkv_read_rows(None, ctypes.byref(n)) == binding.EINVAL
    assert L.confkv_read_layer(None, 0, 0, PTR, PTR, s, s, PTR, PTR, 10, None) == binding.EINVAL


def test_binding_refuses_unfit_tensors():
    q, k = torch.zeros(4, 8, 64), torch.zeros(4, 2, 64)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    for bad in (q, q[0], q.transpose(1, 2)):
        with pytest.raises(ValueError):
            ck.prompt_attention(bad, k, k, cu)
        with pytest.raises(ValueError):
            ck.qk_rotary(bad, k, None, None)
    with pytest.raises(ValueError):
        ck.Rotary(64, scaling="other", device="cpu")
    with pytest.raises(ck.ConfkvError):
        ck.Rotary(63, device="cpu")
    assert len(ck.Rotary(64, device="cpu").turns_host) == 32
