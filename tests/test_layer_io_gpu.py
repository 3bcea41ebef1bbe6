"""Prefill by layer and read-back: the same cache, bit for bit, as the
whole-cache prefill on the same values; read-back equal to code * scale
rounded once, before and after evictions."""
import numpy as np
import pytest
import torch

import confidence_gated_kv_gb300 as ck
from confidence_gated_kv_gb300 import binding
from workload import Workload

from _parity import step_inputs

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def config(lens, L=2, Hq=4, Hkv=2, d=128, W=32, cap=None, budget=None, **kw):
    cap = max(16, max(lens)) if cap is None else cap
    budget = cap if budget is None else budget
    return ck.make_config(L=L, Hq=Hq, Hkv=Hkv, d=d, V=1000, B=len(lens), cap=cap, W=W, P=1, n_high=[budget] * L,
                          n_low=[budget] * L, **kw)


def packed(lens, L, Hkv, d, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for _ in range(2 * L):
        x = torch.randn((sum(lens), Hkv, d), generator=g, device="cuda")
        x *= torch.exp(torch.randn((1, Hkv, d), generator=g, device="cuda"))      # unlike channel scales
        out.append(x.to(dtype))
    return out[:L], out[L:]


def padded(xs, lens):
    """[L][B][Hkv][T][d] fp16 of packed layers."""
    L, B, (_, H, d) = len(xs), len(lens), xs[0].shape
    y = torch.zeros((L, B, H, max(1, max(lens)), d), dtype=F16, device="cuda")
    for l, x in enumerate(xs):
        r = 0
        for b, n in enumerate(lens):
            y[l, b, :, :n] = x[r:r + n].to(F16).transpose(0, 1)
            r += n
    return y


def by_layer(cache, ks, vs, lens, order=None):
    cache.prefill_begin(lens)
    for l in order or range(len(ks)):
        cache.prefill_layer(l, ks[l], vs[l])


def same_unit(a, b):
    for key in a:
        np.testing.assert_array_equal(a[key], b[key], err_msg=key)


def rows_of_unit(u, d):
    """positions and dequantised K, V of an exported unit, in read order."""
    k8 = u["k8"].astype(np.float32) * u["sK"][None]
    v8 = u["v8"].astype(np.float32) * u["sV"][None]
    r = np.argsort(u["posR"], kind="stable")
    return (np.concatenate([u["pos8"], u["posR"][r]]),
            np.concatenate([k8, u["k16"][r].astype(np.float32)]), np.concatenate([v8, u["v16"][r].astype(np.float32)]))


def check_read(cache, dtype=F16):
    for l in range(cache.L):
        o = cache.read_layer(l, dtype=dtype)
        c = o["cu_seqlens"].tolist()
        assert c[0] == 0 and c[-1] <= cache.read_rows()
        for b in range(cache.B):
            p, k, v = rows_of_unit(cache.export_unit(b, l), cache.d)
            s = slice(c[b], c[b + 1])
            np.testing.assert_array_equal(o["positions"][s].cpu().numpy(), p)
            assert torch.equal(o["k"][s].cpu(), torch.from_numpy(k).to(dtype))
            assert torch.equal(o["v"][s].cpu(), torch.from_numpy(v).to(dtype))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens, W", [
    ([1], 1), ([16], 16), ([17], 16), ([600], 64), ([0, 5, 33], 32), ([100, 1, 259, 31], 100), ([2000, 3, 1500], 256),
])
def test_same_cache_as_the_whole_prefill(lens, W, d, dtype):
    L, Hkv = 2, 3
    ks, vs = packed(lens, L, Hkv, d, dtype)
    cfg = config(lens, L, 2 * Hkv, Hkv, d, W)
    a, b = ck.Cache(cfg), ck.Cache(cfg)
    a.workspace.fill_(0x7f)          # what an earlier use may have left: NaN as fp16 and fp32
    a.close()
    a = _over(cfg, a.workspace)
    b.prefill(padded(ks, lens), padded(vs, lens), lens)
    by_layer(a, ks, vs, lens, order=[1, 0])
    for l in range(L):
        for s in range(len(lens)):
            same_unit(a.export_unit(s, l), b.export_unit(s, l))
    assert a.get_clock() == b.get_clock()
    check_read(a, dtype)
    assert a.stats()["device_status"] == 0


def _over(cfg, workspace):
    c = ck.Cache(cfg)
    c.close()
    import ctypes
    h = ctypes.c_void_p()
    assert ck.lib().confkv_create(ctypes.byref(cfg), workspace.data_ptr(), workspace.numel(), ctypes.byref(h)) == 0
    c.workspace, c._h = workspace, h
    return c


def test_values_on_and_next_to_a_half_step():
    # x / s falls on k + 1/2 and next to it: codes as from the IEEE quotient
    n, d = 4000, 64
    k = torch.zeros((n, 1, d), dtype=F16, device="cuda")
    steps = (torch.arange(n - 1, device="cuda") % 254 - 127).float() + 0.5
    for c in range(d):
        s = 2.0 ** (c % 8 - 4) * (1 + c / 64)
        k[1:, 0, c] = (steps * s).half()
        k[0, 0, c] = 127 * s
    cfg = config([n], 1, 1, 1, d, 16)
    a, b = ck.Cache(cfg), ck.Cache(cfg)
    b.prefill(padded([k], [n]), padded([k], [n]), [n])
    by_layer(a, [k], [k], [n])
    same_unit(a.export_unit(0, 0), b.export_unit(0, 0))


def test_non_finite_values_as_in_the_whole_prefill():
    lens = [300]
    ks, vs = packed(lens, 1, 1, 64, F16, 3)
    ks[0][5, 0, 3], ks[0][7, 0, 4], vs[0][9, 0, 5] = float("nan"), float("inf"), -float("inf")
    cfg = config(lens, 1, 1, 1, 64, 16)
    a, b = ck.Cache(cfg), ck.Cache(cfg)
    b.prefill(padded(ks, lens), padded(vs, lens), lens)
    by_layer(a, ks, vs, lens)
    same_unit(a.export_unit(0, 0), b.export_unit(0, 0))


def test_strided_rows_and_rewritten_layer():
    lens = [120, 44]
    n, H, d = sum(lens), 2, 128
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((n, 2 * H + 5, d + 8), generator=g, device="cuda").to(BF16)
    k, v = x[:, 1:1 + H, :d], x[:, 1 + H:1 + 2 * H, :d]
    cfg = config(lens, 1, H, H, d, 32)
    a, b = ck.Cache(cfg), ck.Cache(cfg)
    by_layer(b, [k.contiguous()], [v.contiguous()], lens)
    a.prefill_begin(lens)
    with pytest.raises(ck.ConfkvError):
        a.read_layer(0)
    a.prefill_layer(0, k.transpose(0, 1).contiguous().transpose(0, 1), v)      # heads outermost
    for s in range(2):
        same_unit(a.export_unit(s, 0), b.export_unit(s, 0))
    wide = torch.full((n + 9, H + 1, d + 8), 7.0, dtype=F16, device="cuda")
    wide_v = wide.clone()
    pos = torch.full((n + 9,), -5, dtype=torch.int32, device="cuda")
    out = dict(k=wide[:, :H, :d], v=wide_v[:, :H, :d], positions=pos,
               cu_seqlens=torch.empty(3, dtype=torch.int32, device="cuda"))
    a.read_layer(0, out=out)
    want = b.read_layer(0)
    assert torch.equal(out["k"][:n], want["k"]) and torch.equal(out["v"][:n], want["v"])
    assert bool((wide[n:] == 7).all()) and bool((wide[:, H:] == 7).all()) and bool((wide[:, :, d:] == 7).all())
    assert bool((pos[n:] == -5).all())


def test_order_of_calls():
    lens = [40]
    ks, vs = packed(lens, 2, 2, 128, F16, 5)
    cache = ck.Cache(config(lens))
    with pytest.raises(ck.ConfkvError) as e:
        cache.prefill_layer(0, ks[0], vs[0])
    assert e.value.status == binding.ESTATE
    cache.prefill_begin(lens)
    cache.prefill_layer(0, ks[0], vs[0])
    cache.prefill_layer(0, ks[1], vs[1])          # written again before the last layer
    for call in (lambda: cache.read_layer(0), lambda: cache.set_clock(lens, 0),
                 lambda: cache.import_unit(0, 0, cache.export_unit(0, 0))):
        with pytest.raises(ck.ConfkvError) as e:
            call()
        assert e.value.status == binding.ESTATE
    cache.prefill_layer(1, ks[1], vs[1])
    with pytest.raises(ck.ConfkvError) as e:
        cache.prefill_layer(1, ks[1], vs[1])
    assert e.value.status == binding.ESTATE
    a, b = cache.read_layer(0), cache.read_layer(1)
    assert torch.equal(a["k"], b["k"]) and torch.equal(a["v"], b["v"])
    with pytest.raises(ck.ConfkvError) as e:
        cache.prefill_begin([5000])
    assert e.value.status == binding.ECAPACITY
    assert torch.equal(cache.read_layer(0)["k"], a["k"])          # the refused call changed nothing
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ck.ConfkvError) as e:
            cache.prefill_begin(lens)
        assert e.value.status == binding.ESTATE
        torch.zeros(1, device="cuda").add_(1)
    assert torch.equal(cache.read_layer(0)["k"], a["k"])


def test_too_few_rows_are_reported():
    lens = [50, 60]
    ks, vs = packed(lens, 1, 2, 128, F16, 6)
    cache = ck.Cache(config(lens, 1))
    by_layer(cache, ks, vs, lens)
    want = cache.read_layer(0)
    k = torch.full((70, 2, 128), 3.0, dtype=F16, device="cuda")
    out = dict(k=k[:64], v=torch.empty_like(k[:64]), positions=torch.empty(64, dtype=torch.int32, device="cuda"),
               cu_seqlens=torch.empty(3, dtype=torch.int32, device="cuda"))
    cache.read_layer(0, out=out)
    assert out["cu_seqlens"].tolist() == [0, 50, 110]
    assert torch.equal(k[:64], want["k"][:64]) and bool((k[64:] == 3).all())
    s = cache.stats(check=False)
    assert s["device_status"] == binding.STATUS_CAPACITY


def test_read_after_evictions_and_in_a_graph():
    w = Workload(name="read", B=3, L=2, Hq=8, Hkv=2, d=128, V=4000, T0=90, steps=40, n_high=(40, 48), n_low=(60, 52),
                 P=4, W=24, q_dtype="bf16")
    lens = [90, 33, 61]
    ks, vs = packed(lens, 2, 2, 128, BF16, 7)
    cache = ck.Cache(ck.config_from_workload(w))
    by_layer(cache, ks, vs, lens)
    for i in range(30):
        cache.step(*(x.cuda() for x in step_inputs(w, 5, i)))
        if i in (0, 1, 9, 29):
            check_read(cache)
    rows = cache.read_rows()
    assert rows < 3 * (90 + 30)
    x = [t.cuda() for t in step_inputs(w, 5, 31)]
    outs = cache.new_outputs()
    cache.graph_reserve(3)
    assert cache.read_rows() >= rows
    read = cache.read_layer(1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="relaxed"):
        cache.step(*x, outs)
        cache.read_layer(1, out=read)
    for _ in range(3):
        graph.replay()
        cache.graph_advance(1)
        c = read["cu_seqlens"].tolist()
        for b in range(3):
            p, k, v = rows_of_unit(cache.export_unit(b, 1), 128)
            s = slice(c[b], c[b + 1])
            np.testing.assert_array_equal(read["positions"][s].cpu().numpy(), p)
            assert torch.equal(read["k"][s].cpu(), torch.from_numpy(k).half())
            assert torch.equal(read["v"][s].cpu(), torch.from_numpy(v).half())
    assert cache.stats()["device_status"] == 0


def test_many_sequences():
    # more sequences than one length upload takes
    g = torch.Generator().manual_seed(8)
    lens = torch.randint(0, 30, (700,), generator=g).tolist()
    ks, vs = packed(lens, 1, 1, 64, F16, 8)
    cfg = config(lens, 1, 1, 1, 64, 8)
    a, b = ck.Cache(cfg), ck.Cache(cfg)
    by_layer(a, ks, vs, lens)
    b.prefill(padded(ks, lens), padded(vs, lens), lens)
    for s in range(0, 700, 37):
        same_unit(a.export_unit(s, 0), b.export_unit(s, 0))
    o = a.read_layer(0)
    assert o["cu_seqlens"].tolist() == [sum(lens[:i]) for i in range(701)]
    assert o["positions"].tolist() == [p for n in lens for p in range(n)]


def test_captured_read_follows_a_growing_cache():
    # captured when the INT8 region is empty, replayed when it is not
    w = Workload(name="grow", B=2, L=1, Hq=4, Hkv=2, d=64, V=1000, T0=10, steps=60, n_high=(200,), n_low=(200,), P=4,
                 W=16, q_dtype="f16")
    lens = [10, 4]
    ks, vs = packed(lens, 1, 2, 64, F16, 9)
    cache = ck.Cache(ck.config_from_workload(w, cap=256))
    by_layer(cache, ks, vs, lens)
    out = dict(k=torch.empty((200, 2, 64), dtype=F16, device="cuda"), positions=torch.empty(200, dtype=torch.int32, device="cuda"),
               cu_seqlens=torch.empty(3, dtype=torch.int32, device="cuda"))
    out["v"] = torch.empty_like(out["k"])
    cache.read_layer(0, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="relaxed"):
        cache.read_layer(0, out=out)
    for i in range(50):
        cache.step(*(x.cuda() for x in step_inputs(w, 3, i)))
    graph.replay()
    want = cache.read_layer(0)
    n = int(want["cu_seqlens"][2])
    assert n == 10 + 4 + 2 * 50
    assert torch.equal(out["cu_seqlens"], want["cu_seqlens"])
    for key in ("k", "v", "positions"):
        assert torch.equal(out[key][:n], want[key][:n])


def test_read_on_another_stream():
    lens = [300, 50]
    ks, vs = packed(lens, 1, 2, 128, F16, 10)
    cache = ck.Cache(config(lens, 1))
    by_layer(cache, ks, vs, lens)
    want = cache.read_layer(0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        got = cache.read_layer(0, stream=s)
    s.synchronize()
    for key in want:
        assert torch.equal(got[key], want[key])


def test_refusals_on_the_device():
    lens = [40]
    ks, vs = packed(lens, 1, 2, 128, F16, 11)
    cache = ck.Cache(config(lens, 1))
    with pytest.raises(ValueError):
        cache.prefill_begin([40, 1])
    with pytest.raises(ck.ConfkvError):
        cache.prefill_begin([-1])
    cache.prefill_begin(lens)
    k, v = ks[0], vs[0]
    for a, b in ((k[:39], v[:39]), (k, v.to(BF16)), (k[:, :1], v[:, :1]), (k.cpu(), v.cpu()), (k[:, :, :64], v[:, :, :64]),
                 (k.transpose(1, 2).contiguous().transpose(1, 2), v)):
        with pytest.raises(ValueError):
            cache.prefill_layer(0, a, b)
    with pytest.raises(ck.ConfkvError):                                  # heads that overlap
        cache.prefill_layer(0, k[:, :1].expand(-1, 2, -1), v)
    with pytest.raises(ck.ConfkvError):
        cache.prefill_layer(1, k, v)
    with pytest.raises(ck.ConfkvError):
        cache.prefill_layer(-1, k, v)
    cache.prefill_layer(0, k, v)
    o = cache.read_layer(0)
    for bad in (dict(o, positions=o["positions"].long()), dict(o, cu_seqlens=o["cu_seqlens"][:1]), dict(o, v=o["v"].to(BF16)),
                dict(o, k=o["k"][:39])):
        with pytest.raises(ValueError):
            cache.read_layer(0, out=bad)
    with pytest.raises(ck.ConfkvError):
        cache.read_layer(3)
    with pytest.raises(ValueError):
        cache.read_layer(0, dtype=torch.int32)
