"""A context that was never prefilled and holds some imported units: the others
are empty, whatever the workspace held before.  Units that hold nothing yet
are not exported."""
import pytest
import torch

import confidence_gated_kv_gb300 as ck
from confidence_gated_kv_gb300 import binding

from test_layer_io_gpu import _over, config, packed, padded, same_unit

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("garbage", [0x7f, 0xff, 0x01])
@pytest.mark.parametrize("d", [64, 128])
def test_units_not_imported_are_empty(d, garbage):
    lens, L, Hkv = [150, 0], 2, 2
    cfg = config(lens, L, 2 * Hkv, Hkv, d, 32, cap=256)
    ks, vs = packed(lens, L, Hkv, d, torch.float16, 1)
    whole, part = ck.Cache(cfg), ck.Cache(cfg)
    whole.prefill(padded(ks, lens), padded(vs, lens), lens)
    part.workspace.fill_(garbage)
    workspace = part.workspace
    part.close()
    part = _over(cfg, workspace)
    if garbage == 1:
        part.set_clock(lens, 0)                         # the clock may come first
    part.import_unit(0, 0, whole.export_unit(0, 0))
    got, want = part.read_layer(0), whole.read_layer(0)
    assert got["cu_seqlens"].tolist() == [0, 150, 150] and part.read_layer(1)["cu_seqlens"].tolist() == [0, 0, 0]
    for key in ("k", "v", "positions"):
        assert torch.equal(got[key][:150], want[key][:150])
    # with the rest and the clock, steps as from the prefilled cache
    part.import_unit(0, 1, whole.export_unit(0, 1))
    if garbage != 1:
        part.set_clock(lens, 0)
    g = torch.Generator(device="cuda").manual_seed(2)
    for _ in range(20):
        x = [torch.randn((L, 2, h, d), generator=g, device="cuda").half() for h in (2 * Hkv, Hkv, Hkv)]
        x.append(torch.randn((2, 1000), generator=g, device="cuda"))
        a, b = part.step(*x), whole.step(*x)
        for key in ("out", "budget", "confidence", "n_evicted"):
            assert torch.equal(a[key], b[key]), key
    for l in range(L):
        for s in range(2):
            same_unit(part.export_unit(s, l), whole.export_unit(s, l))
    assert part.stats()["device_status"] == 0


def test_units_without_content_are_not_exported():
    lens = [40, 7]
    cfg = config(lens, 2, 4, 2, 64, 16)
    ks, vs = packed(lens, 2, 2, 64, torch.float16, 3)
    cache = ck.Cache(cfg)

    def refused(layer):
        with pytest.raises(ck.ConfkvError) as e:
            cache.export_unit(1, layer)
        return e.value.status == binding.ESTATE

    assert refused(0) and refused(1)
    cache.prefill_begin(lens)
    assert refused(0) and refused(1)
    cache.prefill_layer(1, ks[1], vs[1])
    first = cache.export_unit(1, 1)
    assert refused(0)
    cache.prefill_layer(0, ks[0], vs[0])
    same_unit(first, cache.export_unit(1, 1))
    cache.export_unit(1, 0)
    cache.prefill_begin(lens)
    assert refused(1)
