"""Prompt operators have no derivatives: inputs that carry any are refused, in
both modes, instead of giving results that autograd takes for constants."""
import pytest
import torch
from torch.autograd import forward_ad

import confidence_gated_kv_gb300 as ck
from confidence_gated_kv_gb300 import binding


def test_the_check_itself():
    x = torch.zeros(3)
    g = torch.zeros(3, requires_grad=True)
    binding.no_gradients(x, None)
    with pytest.raises(ValueError):
        binding.no_gradients(None, x, g)
    with torch.no_grad():
        binding.no_gradients(x, g)
    with forward_ad.dual_level():
        binding.no_gradients(x, None)
        dual = forward_ad.make_dual(x, torch.ones(3))
        with pytest.raises(ValueError):
            binding.no_gradients(x, dual)
        with torch.no_grad(), pytest.raises(ValueError):
            binding.no_gradients(dual)
        binding.no_gradients(forward_ad.unpack_dual(dual).primal)
    binding.no_gradients(x)


@pytest.mark.gpu
def test_every_call():
    n = 20
    q, k, v = (torch.randn(n, h, 64, device="cuda").half() for h in (4, 2, 2))
    w, cu = torch.ones(64, device="cuda").half(), torch.tensor([0, n], dtype=torch.int32, device="cuda")
    cache = ck.Cache(ck.make_config(L=1, Hq=4, Hkv=2, d=64, V=1000, B=1, cap=32, W=16, P=1, n_high=[32], n_low=[32]))
    cache.prefill_begin([n])
    calls = [
        (lambda q, k, v: ck.prompt_attention(q, k, v, cu), (q, k, v)),
        (lambda q, k, w: ck.qk_rotary(q, k, None, None, w, w), (q, k, w)),
        (lambda k, v: cache.prefill_layer(0, k, v), (k, v)),
    ]
    for call, tensors in calls:
        for i, t in enumerate(tensors):
            before = [*tensors[:i]]
            t.requires_grad_(True)
            with pytest.raises(ValueError):
                call(*tensors)
            t.requires_grad_(False)
            with forward_ad.dual_level():
                dual = forward_ad.make_dual(t, torch.ones_like(t))
                with pytest.raises(ValueError):
                    call(*before, dual, *tensors[i + 1:])
                with torch.no_grad(), pytest.raises(ValueError):
                    call(*before, dual, *tensors[i + 1:])
    with pytest.raises(ck.ConfkvError):                 # the refused calls wrote no layer
        cache.read_layer(0)
    k.requires_grad_(True)
    with torch.no_grad():
        cache.prefill_layer(0, k, v)
    assert torch.equal(cache.read_layer(0)["positions"].cpu(), torch.arange(n, dtype=torch.int32))
