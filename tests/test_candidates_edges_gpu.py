"""Calls of tree attention and beam selection at the ends of their ranges, and
tree attention as it chooses its kernel by itself."""

import pytest
import torch

from confidence_gated_kv_gb300 import binding
from _candidates import BF16, F16, gen, make_cache
from test_tree_attention_gpu import check, drafts, tree

pytestmark = pytest.mark.gpu
MODES = [binding.TREE_AUTO, binding.TREE_ROWS, binding.TREE_TILES, binding.TREE_DEALT]
NAMES = ["auto", "rows", "tiles", "dealt"]
every_mode = pytest.mark.parametrize("mode", MODES, ids=NAMES)


# ------------------------------------------------- rows and scales next to zero

@every_mode
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T", [3, 40])
def test_rows_and_scales_next_to_zero(T, dtype, mode):
    # all scores are zero or next to it: the mean of what a row sees
    g = gen(T)
    cache = make_cache([70, 9, 1], 4, 2, 64, 16)
    cache.set_tree_mode(mode)
    q, k, v = drafts(g, 3, T, 4, 2, 64, dtype)
    q[:, 1] = 0
    q[1, 0, 2] = torch.finfo(dtype).tiny
    if dtype == BF16:
        q[:, 2] *= 2.0 ** -120
    parents = tree("random", 3, T, g)
    for scale in (2.0 ** -43, 2.0 ** -126, 2.0 ** -149):
        out, lse = check(cache, 0, q, k, v, parents, None, scale)
        assert not bool(out.isnan().any()) and not bool(lse.isnan().any())
    q[:] = 0
    for scale in (2.0 ** -149, 1.0, 2.0 ** 100, 3.4e38):
        check(cache, 0, q, k, v, parents, None, scale)


@every_mode
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T", [2, 30])
def test_scales_of_zero(T, dtype, mode):
    # an imported state may have them where all codes are zero
    g = gen(5)
    cache = make_cache([90], 4, 2, 64, 16)
    cache.set_tree_mode(mode)
    u = cache.export_unit(0, 0)
    u["k8"][:, 0], u["sK"][0], u["v8"][:, 0, 7], u["sV"][0, 7] = 0, 0.0, 0, 0.0
    u["k8"][:, 1, 3], u["sK"][1, 3] = 0, 0.0
    cache.import_unit(0, 0, u)
    q, k, v = drafts(g, 1, T, 4, 2, 64, dtype)
    check(cache, 0, 8 * q, k, v, tree("kary", 1, T, g))
    q[0, 0, 2:] *= 2.0 ** -12                                                # beside one that counts
    q[0, 0, 2:, 3] = 1000
    check(cache, 0, q, k, v, tree("kary", 1, T, g))
