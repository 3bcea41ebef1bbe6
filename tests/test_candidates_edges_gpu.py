"""Calls of tree attention and beam selection at the ends of their ranges, and
tree attention as it chooses its kernel by itself."""
import math

import pytest
import torch

import confidence_gated_kv_gb300 as ck
from confidence_gated_kv_gb300 import binding
from _candidates import BF16, F16, gen, make_cache, randn, tree_values
from test_beam_gpu import check as check_beams
from test_tree_attention_gpu import check, drafts, tree

pytestmark = pytest.mark.gpu
F32 = torch.float32
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


# ------------------------------------------------------- weights of few rows

@pytest.mark.parametrize("Hq,T,mode", [(Hq, T, mode) for Hq, T in [(2, 1), (8, 1), (16, 1), (2, 3), (4, 4)] for mode in MODES[:2]]
                         + [(2, 9, binding.TREE_ROWS), (16, 2, binding.TREE_ROWS), (6, 11, binding.TREE_ROWS)])
@pytest.mark.parametrize("d", [64, 128])
def test_weights_of_few_rows(d, Hq, T, mode):
    """The kernel of few rows, which up to eight rows take by default.  Rows that see two entries of equal values but unlike sign, with weights
    next to each other (and a draft of zeros): what is left is the weights' error.

    Held in two fp16 parts a weight is off by 2^-22 of itself, its exponential
    by 2^-21 and its score (below 0.01) by 2^-18 of 0.01; the products and the
    join are five fp32 operations on it.  In all less than 2^-19 of the sum of
    the magnitudes (below 1); one fp16 part alone is off by up to 2^-12."""
    B, Hkv = 40, 2
    g = gen(Hq + T)
    cache = make_cache([2] * B, Hq, Hkv, d, 16, seed=3)
    cache.set_tree_mode(mode)
    keys = 0.002 * torch.randn((B, Hkv, d), generator=g).half()
    for b in range(B):
        u = cache.export_unit(b, 0)
        u["k16"][0], u["k16"][1], u["v16"][0], u["v16"][1] = 0, keys[b].numpy(), 1, -1
        cache.import_unit(b, 0, u)
    q, k, v = drafts(g, B, T, Hq, Hkv, d, F16)
    k[:], v[:] = 0, 0
    out = cache.tree_attention(0, q, k, v, torch.full((T,), -1, dtype=torch.int32, device="cuda")).double().cpu()
    score = torch.einsum("bthgd,bhd->bthg", q.view(B, T, Hkv, Hq // Hkv, d).double().cpu(), keys.double()) * d ** -0.5
    assert 0.002 < float(score.abs().max()) < 0.012
    want = (-score.expm1() / (2 + score.exp())).reshape(B, T, Hq, 1)
    assert float(((out - want).abs() - 2.0 ** -11 * want.abs()).max()) <= 2.0 ** -19


@every_mode
@pytest.mark.parametrize("T", [1, 4, 7, 30])
def test_infinite_values_of_the_cache(T, mode):
    # as a step would leave them from values beyond fp16: they reach every row, in their channels
    g = gen(T)
    cache = make_cache([50], 4, 2, 64, 40)
    cache.set_tree_mode(mode)
    q, k, v = drafts(g, 1, T, 4, 2, 64, F16)
    clean, _ = check(cache, 0, 0.1 * q, k, v)
    u = cache.export_unit(0, 0)
    u["v16"][3, 0, 5], u["v16"][7, 0, 9], u["v16"][9, 1, 63], u["v16"][0, 1, 8] = math.inf, -math.inf, math.inf, math.nan
    cache.import_unit(0, 0, u)
    out = cache.tree_attention(0, 0.1 * q, k, v)[0]
    want = clean[0].clone()
    want[:, :2, 5], want[:, :2, 9], want[:, 2:, 63], want[:, 2:, 8] = math.inf, -math.inf, math.inf, math.nan
    assert torch.equal(out.isnan(), want.isnan())
    ends = want.isinf() | want.isnan()
    assert torch.equal(out[want.isinf()], want[want.isinf()])
    # a block of such values takes its weights in one part
    assert bool(((out - want).abs() <= 2.0 ** -10 * want.abs() + 2.0 ** -10)[~ends].all())


@every_mode
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d,Hq,T", [(64, 2, 1), (128, 8, 1), (64, 4, 4), (128, 4, 3), (64, 6, 5), (64, 4, 30)])
def test_keys_that_are_infinitely_far(d, Hq, T, dtype, mode):
    # a score of -inf (a key beyond fp16, in the cache or a draft) has no weight: as if the key were not there
    g = gen(T)
    cache = make_cache([30], Hq, 2, d, 40)
    cache.set_tree_mode(mode)
    u = cache.export_unit(0, 0)
    q, k, v = drafts(g, 1, T + 1, Hq, 2, d, dtype)
    q[..., 17] = q[..., 17].abs() + 0.5
    roots = torch.full((T + 1,), -1, dtype=torch.int32, device="cuda")
    below = torch.tensor([-1] + [0] * T, dtype=torch.int32, device="cuda")   # the others see draft 0
    few = {name: u[name][[i for i in range(30) if i != 4]] for name in ("posR", "emaR", "k16", "v16")}
    cache.import_unit(0, 0, {**u, **few})
    if T == 1 and Hq == 8:                                                   # one token alone, as a single draft
        q, k, v, roots, below = q[:, :1], k[:, :1], v[:, :1], roots[:1], roots[:1]
    want, wlse = check(cache, 0, q, k, v, roots)
    u["k16"][4, :, 17] = -math.inf
    cache.import_unit(0, 0, u)
    out, lse = cache.tree_attention(0, q, k, v, roots, return_lse=True)
    step = torch.finfo(dtype).eps
    near = lambda a, b: bool(((a - b).abs() <= 2 * step * b.abs() + 2.0 ** -11).all())  # noqa: E731
    assert near(out.double(), want.double()) and near(lse, wlse)
    if q.shape[1] > 1:
        k[0, 0, :, 17] = -1e38 if dtype == BF16 else -math.inf
        out, lse = cache.tree_attention(0, q, k, v, below, return_lse=True)
        assert near(out[:, 1:].double(), want[:, 1:].double()) and near(lse[:, 1:], wlse[:, 1:])


# ---------------------------------------- the kernel that a call takes by itself

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d,Hq,Hkv", [(128, 10, 2), (64, 3, 3), (128, 8, 1), (64, 6, 2)])
@pytest.mark.parametrize("T", [1, 2, 5, 9, 16, 27, 64, 128])
def test_default_mode_sizes(d, Hq, Hkv, T, dtype):
    g = gen(T)
    cache = make_cache([700, 0, 97], Hq, Hkv, d, 32, seed=T)
    check(cache, 0, *drafts(g, 3, T, Hq, Hkv, d, dtype), tree("random", 3, T, g),
          torch.tensor([T, T // 2, T], dtype=torch.int32).cuda())


@pytest.mark.parametrize("lens", [[0], [1], [64], [129], [3000], [0, 2500, 17], [800] * 9, [9, 0, 1500, 40] * 4])
@pytest.mark.parametrize("T", [1, 3, 12, 50])
def test_default_mode_lengths(lens, T):
    g = gen(len(lens))
    cache = make_cache(lens, 10, 2, 128, 100, seed=T)
    check(cache, 0, *drafts(g, len(lens), T, 10, 2, 128, BF16), tree("kary", len(lens), T, g))


def test_default_mode_as_the_cache_grows():
    # the host's bounds follow the steps, a captured call keeps the choice it was captured with, an import lifts them
    g = gen(6)
    cache = make_cache([40, 5], 10, 2, 64, 16, cap=4096)
    T = 12
    x = drafts(g, 2, T, 10, 2, 64, F16)
    lens = torch.tensor([T, T], dtype=torch.int32).cuda()
    out, _ = check(cache, 0, *x, None, lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.tree_attention(0, *x, None, lens, out=out)
    for _ in range(3):
        for _ in range(20):
            cache.step(randn(g, (1, 2, 10, 64), F16), randn(g, (1, 2, 2, 64), F16), randn(g, (1, 2, 2, 64), F16), randn(g, (2, 300)))
        check(cache, 0, *x, None, lens)
        graph.replay()
        torch.cuda.synchronize()
        want, _, tol, _ = tree_values(cache, 0, *x, None, lens, 64 ** -0.5)
        assert bool(((out.double().cpu() - want).abs() <= tol).all())
    long = make_cache([4000, 3000], 10, 2, 64, 16, cap=4096, seed=8)
    for b in range(2):
        cache.import_unit(b, 0, long.export_unit(b, 0))
    check(cache, 0, *x, None, lens)
    graph.replay()
    torch.cuda.synchronize()
    want, _, tol, _ = tree_values(cache, 0, *x, None, lens, 64 ** -0.5)
    assert bool(((out.double().cpu() - want).abs() <= tol).all())


@pytest.mark.parametrize("mode", [binding.TREE_AUTO, binding.TREE_DEALT], ids=["auto", "dealt"])
@pytest.mark.parametrize("B,Hkv,G,T", [(153, 2, 2, 6), (310, 1, 1, 9), (10, 8, 8, 64)])
def test_more_tiles_than_are_dealt(B, Hkv, G, T, mode):
    g = gen(B)
    lens = torch.randint(0, 300, (B,), generator=g).tolist()
    cache = make_cache(lens, Hkv * G, Hkv, 64, 32)
    cache.set_tree_mode(mode)
    assert B * Hkv * -(-T * G // 128) > 304 and cache._tree_workspace_bytes(T) == 0
    used = torch.randint(0, T + 1, (B,), generator=g).int().cuda()
    check(cache, 0, *drafts(g, B, T, Hkv * G, Hkv, 64, F16), tree("random", B, T, g), used)


# ------------------------------------------------------------------- beams

@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("V", [5, 3001, 9000])
def test_beams_whose_logits_are_all_the_lowest(V, dtype):
    # as a mask leaves them that rules everything out: all tokens are equally likely
    low = torch.finfo(dtype).min
    x = torch.full((2, 2, V), low, dtype=dtype, device="cuda")
    x[0, 1, 3] = 2.0                                                         # certain
    x[1, 1] = -low / 2
    got = ck.beam_select(x, torch.tensor([[-1.0, -2.0], [-3.0, -3.0]]).cuda(), 3)
    each = -math.log(V)
    want = [[(-2.0, 1, 3), (-1.0 + each, 0, 0), (-1.0 + each, 0, 1)], [(-3.0 + each, 0, i) for i in range(3)]]
    if V == 5:
        want[0] = sorted(want[0], reverse=True)
    for i in range(2):
        order = sorted(want[i], key=lambda w: (-w[0], w[1], w[2]))
        assert got[1][i].tolist() == [w[1] for w in order] and got[2][i].tolist() == [w[2] for w in order]
        assert all(abs(a - w[0]) <= 2.0 ** -18 + 2.0 ** -24 * abs(w[0]) for a, w in zip(got[0][i].tolist(), order))


@pytest.mark.parametrize("beams,V,n", [(16, 5000, 32), (32, 5000, 64), (4, 20000, 17), (64, 700, 64)])
@pytest.mark.parametrize("score", [-1000.0, -3000.0])
def test_long_running_scores(beams, V, n, score):
    g = gen(n)
    x = randn(g, (2, beams, V)) * 3
    check_beams(x, score + randn(g, (2, beams)), n)
    check_beams(x + score, score + randn(g, (2, beams)), n)                  # and logits far from zero
