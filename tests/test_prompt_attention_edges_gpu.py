"""Packed prompt attention at its edges: weights of a row that lie far apart,
against attention in float64; waits that run out.

Tolerance: that of test_prompt_attention_gpu.py, and for fp16 the smallest
step of a weight.  A weight is held in fp16 relative to a reference that is at
most the row's largest score, 2^11 at the reference, so its error is at most
half a step, 2^-25 of 2^11 (and at most u of the weight itself): a row may be
off by 2^-36 p_max sum_j |v_j| more.
"""

import pytest
import torch

import confidence_gated_kv_gb300 as ck
from confidence_gated_kv_gb300 import binding, prompt

from test_prompt_attention_gpu import BF16, F16, cu, inputs, reference

pytestmark = pytest.mark.gpu


def sink_and_tail(n, Hkv, d, dtype, gap, spread, seed):
    """Keys and values of a sequence whose first key is `gap` nats above all
    others for the queries of sink_queries, and has a value of zero."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = torch.zeros((n, Hkv, d), device="cuda")
    k[:, :, 0] = spread * torch.rand((n, Hkv), generator=g, device="cuda")
    k[0, :, 0] = gap
    v = 1000.0 + 100.0 * torch.randn((n, Hkv, d), generator=g, device="cuda")
    v[0] = 0.0
    return k.to(dtype), v.to(dtype)


def sink_queries(rows, Hq, d, dtype):
    q = torch.zeros((rows, Hq, d), device="cuda")
    q[:, :, 0] = 4.0                           # times scale 1/4: the score is the key's first channel
    return q.to(dtype)


def check_rows(out, lse, q, k, v, rows):
    """The first `rows` rows of a call without the causal mask."""
    ref, tol, rl, ltol = reference(q[:rows], k, v, [rows], [len(k)], False, 0.25)
    if q.dtype == F16:
        s = torch.einsum("qhd,khd->qhk", q[:rows].double(),
                         k.double().repeat_interleave(q.shape[1] // k.shape[1], 1)) * 0.25
        p_max = torch.exp(s.amax(-1) - rl)
        total = v.double().abs().sum(0).repeat_interleave(q.shape[1] // k.shape[1], 0)
        tol = tol + 2.0 ** -36 * p_max[..., None] * total
    err = (out[:rows].double() - ref).abs()
    assert torch.isfinite(out).all()
    assert float((err - tol).max()) <= 0, "off by %.3g of %.3g" % (float(err.max()), float(ref.abs().max()))
    assert bool(((lse[:rows].double() - rl).abs() <= ltol).all())
    assert ck.prompt_status() == 0


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("spread", [0.0, 1.0])
@pytest.mark.parametrize("gap", [10.0, 14.0, 16.0, 17.5, 20.0])
@pytest.mark.parametrize("rows, Hq, Hkv, n", [
    (1, 2, 1, 16384),            # keys split over a cluster
    (4864, 8, 8, 4096),          # whole items
])
def test_a_dominating_key_without_value(rows, Hq, Hkv, n, gap, spread, d, dtype):
    k, v = sink_and_tail(n, Hkv, d, dtype, gap, spread, 1)
    q = sink_queries(rows, Hq, d, dtype)
    out, lse = ck.prompt_attention(q, k, v, cu([rows]), cu([n]), causal=False, scale=0.25, return_lse=True)
    check_rows(out, lse, q, k, v, min(rows, 64))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("step", [0.5, 2.7, 2.9, 6.0])
def test_a_reference_that_moves_after_the_tail(step, d):
    # the dominating key comes last, reached over keys that rise by `step`
    # nats a tile: below and above the distance at which the reference moves
    n = 4096
    for rows, Hq, Hkv in ((1, 2, 1), (4864, 8, 8)):
        k, v = sink_and_tail(n, Hkv, d, F16, 0.0, 0.0, 2)
        k[:, :, 0] = -15.0
        rise = min(10, int(15 / step))
        for i in range(rise):
            k[128 * (20 + i), :, 0] = -15.0 + step * (i + 1)
            v[128 * (20 + i)] = 0.0
        k[n - 1, :, 0], v[n - 1] = 1.0, 0.0
        q = sink_queries(rows, Hq, d, F16)
        out, lse = ck.prompt_attention(q, k, v, cu([rows]), cu([n]), causal=False, scale=0.25, return_lse=True)
        check_rows(out, lse, q, k, v, min(rows, 64))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lq, lk, Hq, Hkv", [
    ([256] * 80, [256] * 80, 8, 8),               # whole items: copies of an item and of the next one in flight
    ([1400] * 16, [1400] * 16, 8, 8),             # copies that wait for room
    ([1, 1, 1], [3000, 40, 900], 10, 2),          # keys split: the other CTAs of the cluster go on to the merge
    ([300, 2], [301, 2000], 4, 2),
])
def test_waits_that_run_out_are_reported(lq, lk, Hq, Hkv, d):
    # a CTA without its softmax: its other warps give up after half a
    # millisecond.  Rows are right, unwritten, or NaN where a part is missing.
    (q, k, v), n = inputs(lq, lk, Hq, Hkv, d, F16, 41), sum(lq)
    cq, ck_ = cu(lq), cu(lk)
    want = ck.prompt_attention(q, k, v, cq, ck_)
    assert ck.prompt_status() == 0
    big = torch.full((n + 16, Hq, d), 7.0, dtype=F16, device="cuda")
    out = big[8:8 + n]
    args = prompt._PROMPT.pack(len(lq), Hq, Hkv, d, 0, 1, n, sum(lk), d ** -0.5, q.data_ptr(), k.data_ptr(),
                               v.data_ptr(), out.data_ptr(), 0, cq.data_ptr(), ck_.data_ptr(), Hq * d, d, Hkv * d, d,
                               Hkv * d, d, Hq * d, d)
    assert ck.lib().confkv_selftest_prompt_timeout(args, torch.cuda.current_stream().cuda_stream) == 0
    assert ck.prompt_status() == binding.STATUS_TIMEOUT
    assert ck.prompt_status() == 0
    right = (out == want).all(-1)
    lost = (out == 7.0).all(-1) | out.isnan().all(-1)
    assert bool((right | lost).all()) and bool(lost.any()) and bool(right.any())
    assert bool((big[:8] == 7).all()) and bool((big[8 + n:] == 7).all())
    for _ in range(3):
        assert torch.equal(ck.prompt_attention(q, k, v, cq, ck_), want)
    assert ck.prompt_status() == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("Hq, Hkv, lq, lk, keys", [
    (4, 4, [900], [937], [0, 300, 511, 640, 936]),        # a token a row, queries off the tiles' start
    (10, 2, [900], [900], [255, 256, 899]),               # 25 tokens a tile
    (8, 8, [2600] * 8, [2600] * 8, [1283, 2500]),         # whole items
    (3, 1, [5, 40], [1000, 77], [960, 998]),              # keys split over a cluster
])
def test_reach_of_a_value_that_is_not_finite(Hq, Hkv, lq, lk, keys, bad):
    # a tile's rows share its keys, down to those that only its last token
    # sees: at most 126 + 128 / G keys behind a row's own last one
    G, d = Hq // Hkv, 64
    q, k, v = inputs(lq, lk, Hq, Hkv, d, BF16, 51)
    cq, ck_ = cu(lq), cu(lk)
    want = ck.prompt_attention(q, k, v, cq, ck_)
    seen = torch.arange(lq[0], device="cuda") + lk[0] - lq[0]              # last key of each row
    for key in keys:
        x = v.clone()
        x[key, 0, 7] = bad
        got = ck.prompt_attention(q, k, x, cq, ck_)
        touched = torch.zeros(q.shape, dtype=torch.bool, device="cuda")
        touched[:lq[0], :G, 7] = (seen + 126 + 128 // G >= key)[:, None]
        assert torch.equal(got[~touched], want[~touched])
        assert not bool(torch.isfinite(got[:lq[0], :G, 7][seen >= key]).any())


@pytest.mark.parametrize("Hq, Hkv", [(4, 2), (40, 8)])
@pytest.mark.parametrize("n", [100, 6000])
def test_bad_offsets_write_only_rows_of_sequences(n, Hq, Hkv):
    # offsets are clamped to [0, n] and a sequence whose end lies before its
    # start is empty: nothing but the rows of the rest is written, in the
    # tensors or around them.  100 rows: keys split; 6000: whole items.
    d, guard = 64, 40
    q, k, v = inputs([n], [n], Hq, Hkv, d, F16, 61)
    for offsets in ([0, n + 4900], [-7, n - 40, 30, n], [50, 20, 1 << 30], [90, 90, 90], [-(1 << 31), -5], [n, n + 9],
                    [0, 40, -3, -2]):
        out = torch.full((n + 2 * guard, Hq, d), 7.0, dtype=F16, device="cuda")
        lse = torch.full((n + 2 * guard, Hq), 7.0, device="cuda")
        c = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        ck.prompt_attention(q, k, v, c, out=out[guard:guard + n], lse=lse[guard:guard + n])
        written = torch.zeros(n + 2 * guard, dtype=torch.bool, device="cuda")
        for a, b in zip(offsets, offsets[1:]):
            a, b = min(max(a, 0), n), min(max(b, 0), n)
            written[guard + a:guard + max(a, b)] = True
        assert bool((out[~written] == 7).all()) and bool((lse[~written] == 7).all())
        if sorted(offsets) == offsets:                    # every row of a sequence
            assert not bool((out[written] == 7).all(-1).any()) and not bool((lse[written] == 7).any())
    assert ck.prompt_status() == 0
