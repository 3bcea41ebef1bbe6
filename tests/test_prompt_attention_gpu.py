"""Packed prompt attention against attention in float64 on the same inputs.

Tolerance per output element, with u = eps / 2 of the type (bf16 2^-8, fp16
2^-11), p the softmax weights and A = sum_j p_j |v_j|:
  - each weight rounded to the type for the product with v:      u A
  - the output rounded once:                                      u |out|
  - scores: d products summed in fp32 (taken as 2^-22 a step, for an adder
    that truncates) change a weight by the relative 2 d 2^-22 s with
    s = scale max|q| max|k| (norms, by Cauchy-Schwarz), numerator and
    denominator alike;                                            4 d 2^-22 s A
  - sums over n keys, the exponential (2^-22 each):               2 (n + 4) 2^-22 A
"""
import math
import os
import subprocess
import sys
import threading

import pytest
import torch

import confidence_gated_kv_gb300 as ck

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
F16, BF16 = torch.float16, torch.bfloat16


def cu(lens):
    t = [0]
    for n in lens:
        t.append(t[-1] + n)
    return torch.tensor(t, dtype=torch.int32, device="cuda")


def inputs(lq, lk, Hq, Hkv, d, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    mk = lambda n, h: torch.randn((n, h, d), generator=g, device="cuda").to(dtype)  # noqa: E731
    return mk(sum(lq), Hq), mk(sum(lk), Hkv), mk(sum(lk), Hkv)


def reference(q, k, v, lq, lk, causal, scale):
    """out, lse and the tolerances of both, in float64."""
    (nq, Hq, d), G = q.shape, q.shape[1] // k.shape[1]
    out = torch.zeros((nq, Hq, d), dtype=torch.float64, device="cuda")
    tol, lse = torch.zeros_like(out), torch.full((nq, Hq), -math.inf, dtype=torch.float64, device="cuda")
    ltol = torch.zeros_like(lse)
    u, q0, k0 = U[q.dtype], 0, 0
    for a, b in zip(lq, lk):
        if a and b:
            qq = q[q0:q0 + a].double().permute(1, 0, 2)
            kk, vv = (x[k0:k0 + b].double().permute(1, 0, 2).repeat_interleave(G, 0) for x in (k, v))
            s = qq @ kk.transpose(1, 2) * scale
            if causal:
                seen = torch.arange(b, device="cuda")[None] <= torch.arange(a, device="cuda")[:, None] + (b - a)
                s = torch.where(seen, s, -math.inf)
            z = torch.logsumexp(s, -1, keepdim=True)
            some = z > -math.inf
            p = torch.where(some, torch.exp(s - torch.where(some, z, 0.0)), 0.0)
            o, A = p @ vv, p @ vv.abs()
            smax = scale * float(qq.norm(dim=-1).max()) * float(kk.norm(dim=-1).max())
            rel = 4 * d * 2.0 ** -22 * smax + 2 * (b + 4) * 2.0 ** -22
            out[q0:q0 + a] = o.permute(1, 0, 2)
            tol[q0:q0 + a] = ((u * (A + o.abs()) + rel * A) * 1.01 + 2.0 ** -24).permute(1, 0, 2)
            lse[q0:q0 + a] = z[..., 0].T
            ltol[q0:q0 + a] = rel + 2.0 ** -22 * (1 + z[..., 0].T.abs())
        q0, k0 = q0 + a, k0 + b
    return out, tol, lse, ltol


def check(q, k, v, lq, lk, causal=True, scale=None, **kw):
    sc = 1.0 / math.sqrt(q.shape[2]) if scale is None else scale
    out, lse = ck.prompt_attention(q, k, v, cu(lq), cu(lk), causal=causal, scale=scale, return_lse=True, **kw)
    ref, tol, rl, ltol = reference(q, k, v, lq, lk, causal, sc)
    err = (out.double() - ref).abs()
    worst = float((err - tol).max()) if err.numel() else 0.0
    assert torch.isfinite(out).all()
    assert worst <= 0, "output off by %g above its tolerance" % worst
    assert torch.equal(lse == -math.inf, rl == -math.inf)
    fin = rl > -math.inf
    assert bool(((lse.double() - rl).abs()[fin] <= ltol[fin]).all())
    assert ck.prompt_status() == 0
    return out, lse


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq, Hkv", [(1, 1), (12, 12), (10, 2), (8, 1), (3, 1)])
def test_heads_and_types(Hq, Hkv, d, dtype):
    lens = [130, 1, 300]
    check(*inputs(lens, lens, Hq, Hkv, d, dtype), lens, lens)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 127, 128, 129, 255, 256, 257, 600, 1023, 2050])
@pytest.mark.parametrize("causal", [True, False])
def test_lengths(n, causal):
    check(*inputs([n], [n], 5, 1, 128, BF16, n), [n], [n], causal)


@pytest.mark.parametrize("lq, lk", [
    ([1] * 5, [1, 127, 128, 129, 1000]),            # single tokens against a history
    ([7, 100], [1500, 100]),                        # a chunk, a whole prompt
    ([50, 3, 400], [10, 3, 130]),                   # more queries than keys: rows without a key
    ([0, 5, 0, 9, 0], [7, 5, 0, 0, 300]),           # empty sequences, queries without keys
    ([3], [0]),
])
@pytest.mark.parametrize("causal", [True, False])
def test_chunks_and_empty_rows(lq, lk, causal):
    check(*inputs(lq, lk, 10, 2, 128, F16, 3), lq, lk, causal)
    check(*inputs(lq, lk, 4, 4, 64, BF16, 4), lq, lk, causal)


@pytest.mark.parametrize("G", [2, 4, 6, 7, 16, 48, 64, 100, 128])
def test_group_sizes(G):
    lens = [70, 9]
    check(*inputs(lens, lens, 2 * G, 2, 64, F16, G), lens, lens)


def test_many_short_sequences():
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 40, (300,), generator=g).tolist()
    check(*inputs(lens, lens, 8, 2, 64, BF16, 5), lens, lens)


def test_many_single_tokens():
    # a decode step of many sequences: several groups of 128 offsets
    g = torch.Generator().manual_seed(2)
    lk = torch.randint(1, 200, (515,), generator=g).tolist()
    check(*inputs([1] * 515, lk, 6, 2, 64, F16, 15), [1] * 515, lk)
    lq = [min(n, i % 3) for i, n in enumerate(lk)]
    check(*inputs(lq, lk, 4, 1, 64, BF16, 16), lq, lk)


def test_long_history():
    check(*inputs([1], [33000], 5, 1, 128, BF16, 6), [1], [33000])
    check(*inputs([200, 1], [5000, 9001], 5, 1, 128, F16, 7), [200, 1], [5000, 9001])


def test_growing_and_large_scores():
    # scores that grow along the keys move the reference of the exponentials
    # in every tile; a large scale makes the softmax nearly one-hot
    q, k, v = inputs([700], [700], 5, 1, 128, F16, 8)
    k = (k.float() * torch.linspace(0.1, 4.0, 700, device="cuda")[:, None, None]).half()
    check(q, k, v, [700], [700])
    check(q, k, v, [700], [700], scale=1.0)
    check(q, k.flip(0).contiguous(), v, [700], [700], scale=0.5)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_values_of_other_sequences_stay_out(bad):
    # three sequences; everything of the first and the last, and the rows
    # behind the last, is not finite: the middle one does not see it
    lens, tail = [150, 333, 90], 40
    n = sum(lens)
    q, k, v = inputs([n + tail], [n + tail], 10, 2, 128, BF16, 9)
    clean = ck.prompt_attention(q, k, v, cu(lens))[150:483]      # the same call on finite values
    for x in (q, k, v):
        x[:150] = bad
        x[483:] = bad
    out = torch.full_like(q, 7.0)
    lse = torch.full((n + tail, 10), 7.0, device="cuda")
    ck.prompt_attention(q, k, v, cu(lens), out=out, lse=lse)
    assert torch.equal(out[150:483], clean)
    assert bool((out[n:] == 7.0).all()) and bool((lse[n:] == 7.0).all())


def test_strided_views():
    # q, k, v as slices of one projection, the output into a wider buffer
    lens = [200, 77]
    n, Hq, Hkv, d = sum(lens), 10, 2, 128
    g = torch.Generator(device="cuda").manual_seed(10)
    x = torch.randn((n, Hq + 2 * Hkv, d), generator=g, device="cuda").to(BF16)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    want = ck.prompt_attention(q.contiguous(), k.contiguous(), v.contiguous(), cu(lens))
    big = torch.zeros((n, Hq + 3, d + 8), dtype=BF16, device="cuda")
    got = ck.prompt_attention(q, k, v, cu(lens), out=big[:, 1:Hq + 1, :d])
    assert torch.equal(got, want)
    assert float(big[:, 0].abs().max()) == 0 and float(big[:, Hq + 1:].abs().max()) == 0
    assert float(big[:, :, d:].abs().max()) == 0
    # heads outermost
    qh, kh, vh = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v))
    assert torch.equal(ck.prompt_attention(qh, kh, vh, cu(lens)), want)


def test_bad_offsets_stay_inside():
    # offsets that are not ascending or lie outside the tensors are clamped:
    # the call returns and writes only rows of its outputs
    q, k, v = inputs([100], [100], 4, 2, 64, F16, 11)
    for offsets in ([0, 5000], [-7, 60, 30, 100], [50, 20, 1 << 30], [90, 90, 90]):
        c = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        assert ck.prompt_attention(q, k, v, c).shape == q.shape
    torch.cuda.synchronize()
    assert ck.prompt_status() == 0


def test_same_result_every_time_on_streams_and_in_graphs():
    lens = [300, 1, 513]
    q, k, v = inputs(lens, lens, 10, 2, 128, BF16, 12)
    c = cu(lens)
    want = ck.prompt_attention(q, k, v, c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = ck.prompt_attention(q, k, v, c)
    b = ck.prompt_attention(q, k, v, c, stream=s)
    other = ck.prompt_attention(q, k, v, c)          # at the same time on another stream
    s.synchronize()
    for x in (a, b, other):
        assert torch.equal(x, want)
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ck.prompt_attention(q, k, v, c, out=out)
    for _ in range(2):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    # new data in the captured buffers, other lengths included
    q2, k2, v2 = inputs(lens, lens, 10, 2, 128, BF16, 13)
    want2 = ck.prompt_attention(q2, k2, v2, cu([800, 14]))
    q.copy_(q2), k.copy_(k2), v.copy_(v2), c.copy_(torch.tensor([0, 800, 814, 814], dtype=torch.int32))
    graph.replay()
    assert torch.equal(out, want2)


def test_split_keys_agree_with_whole_ones():
    # few rows against long keys are split over CTAs and warpgroups, many rows
    # are not: both within the tolerance of the same reference
    for lq, lk in (([2], [3000]), ([26], [1500]), ([51], [700]), ([1] * 12, [1 + 300 * i for i in range(12)])):
        check(*inputs(lq, lk, 40, 8, 128, BF16, 21), lq, lk)
        check(*inputs(lq, lk, 6, 2, 64, F16, 22), lq, lk)


def test_first_call_of_a_process_may_be_captured():
    code = (
        "import torch, confidence_gated_kv_gb300 as ck\n"
        "q = torch.randn(70, 4, 64, device='cuda').half()\n"
        "c = torch.tensor([0, 70], dtype=torch.int32, device='cuda')\n"
        "p = torch.arange(70, dtype=torch.int32, device='cuda')\n"
        "r, out, o2 = ck.Rotary(64), torch.zeros_like(q), torch.zeros_like(q)\n"
        "g = torch.cuda.CUDAGraph()\n"
        "with torch.cuda.graph(g):\n"
        "    ck.prompt_attention(q, q, q, c, out=out)\n"
        "    ck.qk_rotary(q, None, p, r, q_out=o2)\n"
        "g.replay()\n"
        "torch.cuda.synchronize()\n"
        "assert torch.equal(out, ck.prompt_attention(q, q, q, c))\n"
        "assert torch.equal(o2, ck.qk_rotary(q, None, p, r)[0])\n"
        "assert ck.prompt_status() == 0\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0, r.stderr[-2000:]


def test_calls_from_two_threads():
    lens = [400, 33]
    data = [inputs(lens, lens, 10, 2, 128, BF16, s) for s in (31, 32)]
    c = cu(lens)
    want = [ck.prompt_attention(*x, c) for x in data]
    torch.cuda.synchronize()
    got = [None, None]

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(50):
            got[i] = ck.prompt_attention(*data[i], c, stream=s)
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_inputs_that_require_gradients_are_refused():
    q, k, v = inputs([9], [9], 2, 1, 64, F16, 23)
    for x in (q, k, v):
        x.requires_grad_(True)
        with pytest.raises(ValueError):
            ck.prompt_attention(q, k, v, cu([9]))
        with torch.no_grad():
            ck.prompt_attention(q, k, v, cu([9]))
        x.requires_grad_(False)
    w = torch.ones(64, device="cuda", requires_grad=True)
    with pytest.raises(ValueError):
        ck.qk_rotary(q, k, None, None, w)


def test_refusals_on_the_device():
    q, k, v = inputs([20], [20], 4, 2, 64, F16, 24)
    c = cu([20])
    with pytest.raises(ck.ConfkvError):                                 # broadcast heads
        ck.prompt_attention(q, k[:, :1].expand(-1, 2, -1), v, c)
    with pytest.raises(ck.ConfkvError):                                 # rows off a 16-byte boundary
        ck.prompt_attention(torch.zeros(20, 4, 65, device="cuda", dtype=F16)[:, :, 1:], k, v, c)
    for bad in (dict(scale=0.0), dict(scale=float("nan"))):
        with pytest.raises(ck.ConfkvError):
            ck.prompt_attention(q, k, v, c, **bad)
    with pytest.raises(ck.ConfkvError):
        ck.prompt_attention(q.float(), k.float(), v.float(), c)
    for args in ((q, k[:19], v, c), (q, k, v.float(), c), (q, k, v, c.long()), (q, k, v, c.cpu()), (q, k.cpu(), v, c)):
        with pytest.raises(ValueError):
            ck.prompt_attention(*args)
    with pytest.raises(ValueError):
        ck.prompt_attention(q, k, v, c, out=torch.empty(20, 4, 64, device="cuda"))
    with pytest.raises(ValueError):
        ck.prompt_attention(q, k, v, c, lse=torch.empty(4, 20, device="cuda"))

