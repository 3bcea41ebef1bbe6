"""Prompt operators on rows whose element offsets pass 32 bits: the same bits
as on contiguous copies."""
import pytest
import torch

import confidence_gated_kv_gb300 as ck

pytestmark = pytest.mark.gpu

N, STRIDE = 70000, 40960            # 70000 * 40960 elements: 5.7 GB of 16 bits
H, D = 2, 64


def test_offsets_past_32_bits():
    assert N * STRIDE > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn((N, h, D), generator=g, device="cuda").bfloat16() for h in (2 * H, H, H))
    x = torch.empty((N, STRIDE), dtype=torch.bfloat16, device="cuda")
    wq, wk, wv, wo = (x[:, c:c + h * D].unflatten(1, (h, D))
                      for c, h in ((0, 2 * H), (1000, H), (STRIDE - H * D, H), (2048, 2 * H)))
    wq.copy_(q), wk.copy_(k), wv.copy_(v)
    lens = [N - 4001, 1, 4000]
    cu = torch.tensor([0, lens[0], lens[0] + 1, N], dtype=torch.int32, device="cuda")
    want = ck.prompt_attention(q, k, v, cu)
    assert torch.equal(ck.prompt_attention(wq, wk, wv, cu, out=wo), want)
    # single tokens of the same histories: keys split
    last = cu[1:].long() - 1
    ones = torch.arange(4, dtype=torch.int32, device="cuda")
    assert torch.equal(ck.prompt_attention(q[last], wk, wv, ones, cu), ck.prompt_attention(q[last], k, v, ones, cu))

    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    for r in (ck.Rotary(64), ck.Rotary(24)):                       # rows of vectors, and of any size
        a, b = ck.qk_rotary(q, k, pos, r)
        ck.qk_rotary(wq, wk, pos, r, q_out=wo, k_out=wk)
        assert torch.equal(wo, a) and torch.equal(wk, b)
        wk.copy_(k)

    cfg = ck.make_config(L=1, Hq=H, Hkv=H, d=D, V=1000, B=3, cap=N, W=64, P=1, n_high=[N], n_low=[N])
    c = ck.Cache(cfg)
    c.prefill_begin(lens)
    c.prefill_layer(0, k, v)
    want = c.read_layer(0, dtype=torch.bfloat16)
    c.prefill_begin(lens)
    c.prefill_layer(0, wk, wv)
    wk.zero_(), wv.zero_()
    got = dict(k=wk, v=wv, positions=torch.empty_like(pos), cu_seqlens=torch.empty_like(cu))
    c.read_layer(0, out=got)
    for key in want:
        assert torch.equal(got[key], want[key]), key
    assert c.stats()["device_status"] == 0 and ck.prompt_status() == 0
