"""The operators of a prompt's path together, as a model would run them:
projections -> head norms and positions -> attention and cache, layer by
layer; decode steps from that cache; a further chunk of prompt tokens over
the entries that the evictions left."""
import math

import pytest
import torch

import confidence_gated_kv_gb300 as ck
from workload import Workload

from test_prompt_attention_gpu import cu, reference

pytestmark = pytest.mark.gpu


class Model:
    """Random projections of a few layers; tokens are vectors."""

    def __init__(self, L, Hq, Hkv, d, width, dtype, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.L, self.Hq, self.Hkv, self.d, self.dtype = L, Hq, Hkv, d, dtype
        rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.qkv = [(rand(width, (Hq + 2 * Hkv) * d) / math.sqrt(width)).to(dtype) for _ in range(L)]
        self.out = [(rand(Hq * d, width) / math.sqrt(Hq * d)).to(dtype) for _ in range(L)]
        self.w = [(1 + 0.1 * rand(d)).to(dtype) for _ in range(2 * L)]
        self.head = (rand(width, 1000) / math.sqrt(width)).to(dtype)
        self.rotary = ck.Rotary(d, 10000.0, "yarn", 4.0, original_length=256)

    def project(self, l, x):
        y = (x @ self.qkv[l]).view(-1, self.Hq + 2 * self.Hkv, self.d)
        return y[:, :self.Hq], y[:, self.Hq:self.Hq + self.Hkv], y[:, self.Hq + self.Hkv:]


def prompt(m, x, lens, cache, checked=False):
    """Runs packed prompt tokens and fills the cache; hidden states."""
    c = cu(lens)
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).cuda()
    cache.prefill_begin(lens)
    kept = []
    for l in range(m.L):
        q, k, v = m.project(l, x)
        q, k = ck.qk_rotary(q, k, pos, m.rotary, m.w[2 * l], m.w[2 * l + 1], q_out=q, k_out=k)   # in place
        a = ck.prompt_attention(q, k, v, c)
        cache.prefill_layer(l, k, v)
        if checked:
            ref, tol, _, _ = reference(q, k, v, lens, lens, True, 1 / math.sqrt(m.d))
            assert float(((a.double() - ref).abs() - tol).max()) <= 0
            kept.append((k.clone(), v.clone()))
        x = x + a.reshape(len(x), -1) @ m.out[l]
    return x, kept


def decode(m, x, pos, cache, d_in):
    """Inputs of one step: the queries and new K/V of every layer."""
    for l in range(m.L):
        q, k, v = m.project(l, x)
        ck.qk_rotary(q, k, pos, m.rotary, m.w[2 * l], m.w[2 * l + 1], q_out=d_in[0][l], k_out=d_in[1][l])
        d_in[2][l] = v
    return (*d_in, (x @ m.head).float())


@pytest.mark.parametrize("dtype, d", [(torch.bfloat16, 128), (torch.float16, 64)])
def test_prompt_decode_and_continue(dtype, d):
    L, Hq, Hkv, width, lens = 3, 10, 2, 256, [200, 57, 1, 333]
    B = len(lens)
    w = Workload(name="path", B=B, L=L, Hq=Hq, Hkv=Hkv, d=d, V=1000, T0=max(lens), steps=30, n_high=(96,) * L,
                 n_low=(160,) * L, P=8, W=32, q_dtype="bf16" if dtype == torch.bfloat16 else "f16")
    m = Model(L, Hq, Hkv, d, width, dtype)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((sum(lens), width), generator=g, device="cuda").to(dtype)
    cache, plain = ck.Cache(ck.config_from_workload(w)), ck.Cache(ck.config_from_workload(w))
    _, kept = prompt(m, x, lens, cache, checked=True)
    pk = torch.zeros((L, B, Hkv, max(lens), d), dtype=torch.float16, device="cuda")
    pv = torch.zeros_like(pk)
    for l, (k, v) in enumerate(kept):
        r = 0
        for b, n in enumerate(lens):
            pk[l, b, :, :n], pv[l, b, :, :n] = k[r:r + n].transpose(0, 1), v[r:r + n].transpose(0, 1)
            r += n
    plain.prefill(pk, pv, lens)

    # decode: the same steps from both caches, bit for bit
    pos = torch.tensor(lens, dtype=torch.int32, device="cuda")
    d_in = (torch.empty((L, B, Hq, d), dtype=dtype, device="cuda"),
            torch.empty((L, B, Hkv, d), dtype=torch.float16, device="cuda"),
            torch.empty((L, B, Hkv, d), dtype=torch.float16, device="cuda"))
    for step in range(12):
        x1 = torch.randn((B, width), generator=g, device="cuda").to(dtype)
        q, kn, vn, logits = decode(m, x1, pos, cache, d_in)
        # attention of the new token over what the cache holds, read back
        before = [cache.read_layer(l) for l in range(L)]
        o, want = cache.step(q, kn, vn, logits), plain.step(q, kn, vn, logits)
        for key in ("out", "budget", "confidence", "n_evicted"):
            assert torch.equal(o[key], want[key]), key
        for l, r in enumerate(before):
            c, k, v, lk = r["cu_seqlens"].tolist(), [], [], []
            for b in range(B):
                k += [r["k"][c[b]:c[b + 1]], kn[l, b:b + 1]]
                v += [r["v"][c[b]:c[b + 1]], vn[l, b:b + 1]]
                lk.append(c[b + 1] - c[b] + 1)
            qf = q[l].half()
            a = ck.prompt_attention(qf, torch.cat(k), torch.cat(v), cu([1] * B), cu(lk))
            _, tol, _, _ = reference(qf, torch.cat(k), torch.cat(v), [1] * B, lk, True, 1 / math.sqrt(d))
            # 2e-3: the step's own bound on its output
            assert float(((a.double() - o["out"][l].double()).abs() - tol).max()) <= 2e-3
        pos += 1

    # a further chunk of prompt over the entries left, with positions going on
    more = [5, 1, 40, 128]
    x2 = torch.randn((sum(more), width), generator=g, device="cuda").to(dtype)
    seq = torch.repeat_interleave(torch.arange(B), torch.tensor(more)).cuda()
    at = torch.cat([torch.arange(n) for n in more]).cuda()
    for l in range(L):
        q, k, v = m.project(l, x2)
        q, k = ck.qk_rotary(q, k, (pos[seq] + at).int(), m.rotary, m.w[2 * l], m.w[2 * l + 1])
        r = cache.read_layer(l, dtype=dtype)
        c, ks, vs, lk, r0 = r["cu_seqlens"].tolist(), [], [], [], 0
        for b in range(B):
            ks += [r["k"][c[b]:c[b + 1]], k[r0:r0 + more[b]]]
            vs += [r["v"][c[b]:c[b + 1]], v[r0:r0 + more[b]]]
            lk.append(c[b + 1] - c[b] + more[b])
            r0 += more[b]
        kk, vv = torch.cat(ks), torch.cat(vs)
        a = ck.prompt_attention(q, kk, vv, cu(more), cu(lk))
        ref, tol, _, _ = reference(q, kk, vv, more, lk, True, 1 / math.sqrt(d))
        assert float(((a.double() - ref).abs() - tol).max()) <= 0
    assert cache.stats()["device_status"] == 0 and ck.prompt_status() == 0
