"""Routing from logits with expert groups against a plain fp64 implementation.

Bars: ids equal (keys are defined in fp64, so two experts change places only where their keys differ in the last
bits of fp64; no test puts different logits that near); weights within 2^-20 relative: the scores may be summed in
fp32 (a softmax denominator of E <= 1024 terms in E/32 + 5 additions per partial sum, each 2^-24, and a few ulp of
the exponential), then one rounding to fp32.
"""
import numpy as np
import pytest
import torch

import oracle
import prefill_sigmoid_top_b200 as moe
from prefill_sigmoid_top_b200 import inputs
from tests._util import bf16_bits

pytestmark = pytest.mark.gpu
DEV = "cuda"
RTOL = 2.0 ** -20


def reference(z, bias, K, G, TG, group_score, scoring, renorm, scale):
    z = np.where(np.isnan(z), -np.inf, z.astype(np.float64))
    M, E = z.shape
    gs = E // G
    ids, w = np.zeros((M, K), np.int32), np.zeros((M, K))
    for t in range(M):
        with np.errstate(over="ignore", invalid="ignore"):
            if scoring == moe.SCORE_SIGMOID:
                p = 1.0 / (1.0 + np.exp(-z[t]))
            else:
                top = z[t].max()
                ex = (z[t] == np.inf) * 1.0 if top == np.inf else np.zeros(E) if top == -np.inf else np.exp(z[t] - top)
                p = ex / ex.sum() if ex.sum() > 0 else ex
            key = p + (0.0 if bias is None else bias.astype(np.float64))
            key = np.where(np.isnan(key), -np.inf, key)
            gr = np.sort(key.reshape(G, gs), axis=1)
            s = gr[:, -1] if group_score == moe.GROUP_MAX or gs == 1 else gr[:, -1] + gr[:, -2]
            s = np.where(np.isnan(s), -np.inf, s)
        keep = np.argsort(-s, kind="stable")[:TG]
        cand = [e for e in range(E) if e // gs in set(keep.tolist())]
        sel = sorted(cand, key=lambda e: (-key[e], e))[:K]
        ps = p[sel]
        if renorm:
            ps = ps / ps.sum() if ps.sum() > 0 else ps * 0
        ids[t], w[t] = sel, ps * scale
    return ids, w


def check(z, bias, K, G=1, TG=1, group_score=moe.GROUP_TOP2, scoring=moe.SCORE_SIGMOID, renorm=True, scale=1.0):
    """z: a CPU or CUDA tensor, fp32 or bf16, possibly strided."""
    zd = z.to(DEV) if not z.is_cuda else z
    bd = None if bias is None else bias.to(DEV)
    ids, w = moe.route_logits(zd, bd, K, G, TG, group_score, scoring, renorm, scale)
    ids_r, w_r = reference(zd.float().cpu().numpy(), None if bias is None else bias.numpy(), K, G, TG, group_score,
                           scoring, renorm, scale)
    assert np.array_equal(ids.cpu().numpy(), ids_r)
    w = w.cpu().numpy().astype(np.float64)
    assert (np.abs(w - w_r) <= RTOL * np.abs(w_r) + 2.0 ** -149).all()
    return ids, w


def rand(M, E, seed, dtype=torch.float32, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(M, E, generator=g) * spread).to(dtype), 0.05 * torch.randn(E, generator=g)


SHAPES = [  # M, groups, group size, groups kept, K
    (1, 8, 32, 4, 8), (37, 8, 32, 4, 8), (5, 1, 8, 1, 2), (9, 4, 64, 1, 16), (3, 16, 64, 16, 32), (17, 5, 7, 2, 6),
    (4, 32, 1, 32, 4), (6, 32, 32, 3, 32), (130, 2, 80, 1, 12), (7, 1, 1, 1, 1), (11, 3, 1, 2, 2), (2, 31, 33, 30, 32),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("M,G,gs,TG,K", SHAPES)
def test_shapes(M, G, gs, TG, K, dtype):
    z, b = rand(M, G * gs, M + gs, dtype)
    check(z, b, K, G, TG)
    check(z, None, K, G, TG, moe.GROUP_MAX, moe.SCORE_SOFTMAX, False, 2.5)


@pytest.mark.parametrize("scoring", [moe.SCORE_SIGMOID, moe.SCORE_SOFTMAX])
@pytest.mark.parametrize("group_score", [moe.GROUP_MAX, moe.GROUP_TOP2])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("with_bias", [True, False])
def test_variants(scoring, group_score, renorm, with_bias):
    z, b = rand(65, 256, 3)
    check(z, b if with_bias else None, 8, 8, 4, group_score, scoring, renorm, 2.5)


def test_no_groups_is_a_flat_top_k():
    z, b = rand(40, 256, 4)
    check(z, b, 16)


def test_equal_keys_take_the_lower_id():
    z = torch.zeros(3, 64)
    ids, _ = check(z, None, 6, 8, 2)
    assert ids[0].tolist() == [0, 1, 2, 3, 4, 5]
    # bf16 logits of few values: ties between experts and between groups everywhere
    g = torch.Generator().manual_seed(5)
    z = torch.randint(-2, 3, (200, 128), generator=g).to(torch.bfloat16)
    check(z, None, 8, 8, 3)
    check(z, torch.randint(0, 2, (128,), generator=g) * 0.25, 8, 8, 3, moe.GROUP_MAX)


def test_keys_that_fp32_cannot_tell_apart():
    """Scores and biases chosen so that the keys differ by less than one step of fp32, in both directions."""
    g = torch.Generator().manual_seed(6)
    E = 64
    z = 0.5 + torch.arange(E).float()[torch.randperm(E, generator=g)] * 2.0 ** -24
    z = torch.stack([z, z.flip(0)])
    check(z, None, 16, 4, 2)
    # sigmoid(z) + b with b cancelling all but about 2^-26 of the difference of the scores
    z2 = torch.randn(2, E, generator=g)
    p = 1.0 / (1.0 + torch.exp(-z2[:1].double()))
    check(z2[:1], (0.75 - p[0]).float(), 16, 4, 2)


@pytest.mark.parametrize("group_score", [moe.GROUP_MAX, moe.GROUP_TOP2])
@pytest.mark.parametrize("G,gs,TG", [(8, 32, 4), (4, 16, 1), (16, 16, 7), (2, 64, 1), (5, 24, 2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_groups_that_fp32_cannot_tell_apart(G, gs, TG, group_score, dtype):
    """Groups that are permutations of each other up to a few steps of fp32 (or exactly), with and without a bias; some
    with three or more nearly equal best experts."""
    g = torch.Generator().manual_seed(G * gs)
    M = 64
    one = torch.randn(M, gs, generator=g)
    one[16:32, :5] = one[16:32].amax(1, keepdim=True) + torch.arange(5) * 2.0 ** -22
    z = torch.stack([one[:, torch.randperm(gs, generator=g)] for _ in range(G)], 1)
    z += torch.randint(-3, 4, z.shape, generator=g) * 2.0 ** -24 * (torch.arange(M) % 4 > 0)[:, None, None]
    z = z.reshape(M, G * gs).to(dtype)
    b = torch.full((G * gs,), 0.125)
    b2 = b + torch.randint(-2, 3, (G * gs,), generator=g) * 2.0 ** -26
    for bias in (None, b, b2):
        check(z, bias, 6, G, TG, group_score)
        check(z, bias, 6, G, TG, group_score, moe.SCORE_SOFTMAX)


@pytest.mark.parametrize("scoring", [moe.SCORE_SIGMOID, moe.SCORE_SOFTMAX])
def test_infinities_and_nan(scoring):
    inf, nan = float("inf"), float("nan")
    z, b = rand(8, 64, 7)
    z[0, 3] = inf
    z[1, 5] = z[1, 40] = inf
    z[2, :] = -inf
    z[3, ::2] = nan
    z[4, :] = nan
    z[5, 8:16] = -inf
    z[6, 1] = 3e38
    z[7, 2] = -3e38
    for bias in (None, b):
        for renorm in (True, False):
            check(z, bias, 8, 8, 3, moe.GROUP_TOP2, scoring, renorm)
    bad = b.clone()
    bad[:50] = -inf                      # only 14 experts may be chosen; the rest of K = 20 by id
    check(z, bad, 20, 8, 4, moe.GROUP_TOP2, scoring)
    bad[51], bad[60], bad[61] = nan, inf, inf
    check(z, bad, 10, 4, 2, moe.GROUP_TOP2, scoring)


def test_far_logits():
    z = torch.tensor([[-100.0, -101.0, -102.0, -103.0] * 4, [100.0, 90.0, 80.0, 70.0] * 4, [-800.0] * 16])
    check(z, None, 4, 4, 2)
    check(z, None, 4, 4, 2, scoring=moe.SCORE_SOFTMAX)
    for K in (1, 2, 3, 5, 7):  # scores that are 1 (or 0) in fp64 whatever the logit: the lower id, with and without groups
        check(z, None, K)
        check(z, None, K, scoring=moe.SCORE_SOFTMAX)
        check(z, torch.zeros(16), K, 4, 2)
    z = torch.full((2, 64), 38.0)
    z[0, 40:50] = 45.0
    z[1, 5:] = -700.0
    z[1, 20:30] = -690.0
    for K in (1, 4, 9, 10, 11):
        check(z, None, K)
        check(z.to(torch.bfloat16), None, K)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("E,G,TG,K", [(64, 8, 3, 12), (256, 1, 1, 8), (1024, 4, 2, 32), (60, 5, 2, 7)])
@pytest.mark.parametrize("scoring", [moe.SCORE_SIGMOID, moe.SCORE_SOFTMAX])
def test_wide_narrow_and_shifted_logits(E, G, TG, K, dtype, scoring):
    """Logits far apart, nearly equal, far from zero, mostly at the type's lowest value, and quantised to few values;
    with and without a bias, which may be large against the scores."""
    g = torch.Generator().manual_seed(E + K)
    z = torch.randn(8, E, generator=g)
    z[1] *= 200.0
    z[2] = z[2] * 1e-3 + 0.25
    z[3] = z[3] * 2.0 - 300.0
    z[4, 5:] = torch.finfo(dtype).min
    z[5] = (z[5] * 2).round() / 2
    z[6] = z[6] * 8.0 + 1000.0
    z[7, ::3] -= 40.0
    b = torch.randn(E, generator=g)
    for bias in (None, b * 0.01, b * 30.0):
        check(z.to(dtype), bias, K, G, TG, moe.GROUP_TOP2, scoring, False)
        check(z.to(dtype), bias, K, G, TG, moe.GROUP_MAX, scoring)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("off,pad", [(0, 3), (1, 7), (3, 1), (4, 4)])
def test_strided_and_unaligned_rows(dtype, off, pad):
    z, b = rand(21, 256 + off + pad, 8, dtype)
    check(z.to(DEV)[:, off:off + 256], b[:256], 8, 8, 4)


def test_output_buffers_and_rows_beyond_are_kept():
    z, b = rand(6, 32, 9)
    ids = torch.full((8, 4), -7, dtype=torch.int32, device=DEV)
    w = torch.full((8, 4), -7.0, device=DEV)
    r = moe.route_logits(z.to(DEV), b.to(DEV), 4, 4, 2, topk_ids=ids[:6], topk_w=w[:6])
    assert r[0].data_ptr() == ids.data_ptr() and r[1].data_ptr() == w.data_ptr()
    assert (ids[6:] == -7).all() and (w[6:] == -7).all() and (ids[:6] >= 0).all()


@pytest.mark.parametrize("M", [1, 40, 300])
def test_route_group_from_x(M):
    """From x and w_router: the canonical logits of route (the oracle's) without a bias, then route_logits."""
    cfg = inputs.WORKLOADS[0].with_(M=M, H=512, E=64, K=6, bias="normal", seed=31)
    w_r, b, _, x = inputs.router_inputs(cfg)
    ids, w = moe.route_group(x.to(DEV), w_r.to(DEV), b.to(DEV), 6, 8, 3)
    z = oracle.router_logits(bf16_bits(x), bf16_bits(w_r), np.zeros(64, np.float32))
    ids_r, w_r_ = reference(z, b.numpy(), 6, 8, 3, moe.GROUP_TOP2, moe.SCORE_SIGMOID, True, 1.0)
    assert np.array_equal(ids.cpu().numpy(), ids_r)
    assert (np.abs(w.cpu().numpy() - w_r_) <= RTOL * w_r_).all()


def test_captured_replayed_and_on_another_stream():
    z, b = rand(33, 256, 10)
    zd, bd = z.to(DEV), b.to(DEV)
    want = moe.route_logits(zd, bd, 8, 8, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = moe.route_logits(zd, bd, 8, 8, 4)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = moe.route_logits(zd, bd, 8, 8, 4)
    z2, _ = rand(33, 256, 11)
    zd.copy_(z2)
    graph.replay()
    torch.cuda.synchronize()
    ids_r, _ = reference(z2.numpy(), b.numpy(), 8, 8, 4, moe.GROUP_TOP2, moe.SCORE_SIGMOID, True, 1.0)
    assert np.array_equal(out[0].cpu().numpy(), ids_r)


def test_refused_sizes_and_workspaces():
    z = torch.randn(5, 64, device=DEV)
    for K in (65, 2 ** 30):
        with pytest.raises(moe.MoEError) as e:
            moe.route_logits(z, None, K)
        assert e.value.status == 2
    x, w = torch.randn(5, 256, device=DEV).bfloat16(), torch.randn(64, 256, device=DEV).bfloat16()
    with pytest.raises(ValueError):  # one byte that claims to be many
        moe.route_group(x, w, None, 4, 8, 4, ws=torch.zeros(1, dtype=torch.uint8, device=DEV).expand(1 << 20))
    ws = torch.zeros((1 << 20) + 16, dtype=torch.uint8, device=DEV)
    with pytest.raises(moe.MoEError) as e:
        moe.route_group(x, w, None, 4, 8, 4, ws=ws[2:])
    assert e.value.status == 3
    a, b = moe.route_group(x, w, None, 4, 8, 4, ws=ws[16:]), moe.route_group(x, w, None, 4, 8, 4)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("scoring", [moe.SCORE_SIGMOID, moe.SCORE_SOFTMAX])
@pytest.mark.parametrize("far", [-6.0, -20.0, -60.0, -1e30, float(torch.finfo(torch.float32).min), -float("inf")])
@pytest.mark.parametrize("G,gs,TG,K", [(8, 32, 4, 4), (4, 16, 1, 1), (2, 4, 1, 1), (16, 64, 5, 5), (5, 7, 2, 2)])
def test_groups_with_one_expert_in_reach(G, gs, TG, K, far, scoring):
    """Groups of which one expert or a few are near the best and the others far below it, by their logits or by the
    bias: a sum of two keys has to see how far below."""
    g = torch.Generator().manual_seed(G * gs + 1)
    M = 96
    near = torch.rand(M, G, gs, generator=g) < 1.5 / gs
    near[:, :, 0] |= torch.rand(M, G, generator=g) < 0.5
    z = torch.randn(M, G, gs, generator=g) * 2.0
    hidden = torch.where(near, z, torch.full_like(z, far)).reshape(M, G * gs)
    check(hidden, None, K, G, TG, moe.GROUP_TOP2, scoring)
    check(hidden, None, K, G, TG, moe.GROUP_MAX, scoring)
    check(hidden, 0.05 * torch.randn(G * gs, generator=g), K, G, TG, moe.GROUP_TOP2, scoring)
    bias = torch.where(near[0], torch.zeros(G, gs), torch.full((G, gs), far))
    bias += torch.where(torch.arange(G)[:, None] % 2 == 1, -1.5 * (bias == 0), torch.zeros(G, gs))
    check(z.reshape(M, G * gs), bias.reshape(-1), K, G, TG, moe.GROUP_TOP2, scoring)
    check(z.reshape(M, G * gs), bias.reshape(-1), K, G, TG, moe.GROUP_MAX, scoring)


@pytest.mark.parametrize("scoring", [moe.SCORE_SIGMOID, moe.SCORE_SOFTMAX])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("part", [0.02, 0.5, 0.97])
@pytest.mark.parametrize("G,gs,TG,K", [(8, 32, 4, 8), (1, 64, 1, 4), (4, 16, 2, 10), (16, 64, 8, 16), (3, 5, 2, 3)])
def test_experts_masked_by_infinities(G, gs, TG, K, part, dtype, scoring):
    """A part of the experts masked by -inf in their logits, in the bias, or both; a few rows with +inf or NaN too."""
    g = torch.Generator().manual_seed(int(G * gs + 100 * part))
    z, b = rand(64, G * gs, G * gs + K, dtype)
    zm, bm = z.clone(), b.clone()
    zm[torch.rand(z.shape, generator=g) < part] = -float("inf")
    bm[torch.rand(b.shape, generator=g) < part] = -float("inf")
    zm[5, 2], zm[9, 1] = float("inf"), float("nan")
    for group_score in (moe.GROUP_MAX, moe.GROUP_TOP2):
        for logits, bias in ((zm, None), (zm, b), (z, bm), (zm, bm)):
            check(logits, bias, K, G, TG, group_score, scoring)
            check(logits, bias, K, G, TG, group_score, scoring, renorm=False)


@pytest.mark.parametrize("E,top", [(1024, 5.4), (1000, 5.0), (960, 6.0), (300, 4.2)])
def test_softmax_weights_with_a_wide_denominator(E, top):
    """One logit and E - 1 of about `top` below it, where the rounding of z - max in the denominator's exponentials counts
    most.  Units of 2^-24: numerator expf 4 and its correction 1; denominator expf 4, the rounding of differences in
    [4, 8) 4 (half a step), at most 11 levels of the sum; reciprocal 2, two products 2: 28."""
    g = torch.Generator().manual_seed(E)
    z = 3.7 - top + 0.1 * torch.rand(64, E, generator=g)
    z[torch.arange(64), torch.randint(0, E, (64,), generator=g)] = 3.7
    z -= torch.rand(64, 1, generator=g)
    for bias in (None, 0.001 * torch.randn(E, generator=g)):
        ids, w = moe.route_logits(z.to(DEV), None if bias is None else bias.to(DEV), 8, scoring=moe.SCORE_SOFTMAX,
                                  renormalize=False)
        ids_r, w_r = reference(z.numpy(), None if bias is None else bias.numpy(), 8, 1, 1, moe.GROUP_TOP2,
                               moe.SCORE_SOFTMAX, False, 1.0)
        assert np.array_equal(ids.cpu().numpy(), ids_r)
        assert (np.abs(w.cpu().numpy() - w_r) <= 28 * 2.0 ** -24 * w_r).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("G,gs,TG,K", [(8, 32, 4, 8), (1, 64, 1, 32), (4, 256, 2, 17), (1, 5, 1, 1), (17, 60, 9, 24), (5, 12, 2, 7)])
@pytest.mark.parametrize("spread", [0.01, 1.5, 12.0])
def test_weights_are_rounded_once(spread, G, gs, TG, K, dtype):
    """The weights of sigmoid scores and of a renormalised softmax are those of fp64 with one rounding to fp32: half a
    step, 2^-24, and 2^-5 of that for the arithmetic before it.  A softmax over all experts: 12 * 2^-24 (exponentials 4,
    their argument 1, at most 6 levels of an fp32 sum, the rounding 1)."""
    z, b = rand(500, G * gs, G + K, dtype, spread)
    for scoring, renorm, units in ((moe.SCORE_SIGMOID, True, 1 + 2.0 ** -5), (moe.SCORE_SIGMOID, False, 1 + 2.0 ** -5),
                                   (moe.SCORE_SOFTMAX, True, 1 + 2.0 ** -5), (moe.SCORE_SOFTMAX, False, 12)):
        for bias in (None, b):
            ids, w = moe.route_logits(z.to(DEV), None if bias is None else bias.to(DEV), K, G, TG, moe.GROUP_TOP2, scoring,
                                      renorm, 2.5)
            ids_r, w_r = reference(z.float().numpy(), None if bias is None else bias.numpy(), K, G, TG, moe.GROUP_TOP2,
                                   scoring, renorm, 2.5)
            assert np.array_equal(ids.cpu().numpy(), ids_r)
            w, normal = w.cpu().numpy().astype(np.float64), w_r >= 2.0 ** -126
            assert (np.abs(w - w_r)[normal] <= units * 2.0 ** -24 * w_r[normal]).all()


def test_weights_over_the_range_of_logits():
    """One expert's score itself, from e^-90 to 1, and pairs of which one is that far below the other.  Scores below
    2^-126 are subnormal numbers of fp32, 2^-149 apart: there half a step is 2^-150, whatever the value."""
    z = torch.cat([torch.linspace(-90.0, 40.0, 20011), torch.tensor([-80.0, -80.00001, 0.0, -0.0, 88.0, 100.0, 700.0, 3e38])])
    _, w = moe.route_logits(z[:, None].to(DEV), None, 1, renormalize=False)
    want = 1.0 / (1.0 + np.exp(-z.double().numpy()))
    bar = lambda v: (1 + 2.0 ** -5) * np.maximum(2.0 ** -24 * v, 2.0 ** -150)  # noqa: E731
    assert (np.abs(w.cpu().numpy()[:, 0] - want) <= bar(want)).all()
    pair = torch.stack([z[:20011], torch.zeros(20011)], 1)
    for scoring in (moe.SCORE_SIGMOID, moe.SCORE_SOFTMAX):
        ids, w = moe.route_logits(pair.to(DEV), None, 2, scoring=scoring)
        ids_r, w_r = reference(pair.numpy(), None, 2, 1, 1, moe.GROUP_TOP2, scoring, True, 1.0)
        assert np.array_equal(ids.cpu().numpy(), ids_r)
        assert (np.abs(w.cpu().numpy() - w_r) <= bar(w_r)).all()


@pytest.mark.parametrize("M", [2 ** 31 - 1, 2 ** 31 - 4])
def test_as_many_tokens_as_are_accepted(M):
    """One expert and one choice: M * top_k just below 2^31."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    z = torch.zeros(M, 1, dtype=torch.bfloat16, device=DEV)
    z[-1] = 1.0
    ids = torch.full((M, 1), -7, dtype=torch.int32, device=DEV)
    w = torch.full((M, 1), -7.0, device=DEV)
    moe.route_logits(z, None, 1, renormalize=False, topk_ids=ids, topk_w=w)
    assert not ids.any()
    assert float(w[-1]) == np.float32(1.0 / (1.0 + np.exp(-1.0)))
    assert not (w[:-1] != 0.5).any()
    del z, ids, w
    torch.cuda.empty_cache()
