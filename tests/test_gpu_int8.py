"""The int8 (W8A8) products against plain 64-bit implementations.

The codes are those of exact arithmetic (compared bit for bit) and the integer sums are exact, so what is left is
the fp32 scaling and the last rounding.  Bars, relative to the exact value v = sx sw sum:
  linear, down: sx (a / 127 rounded), sx sw, the sum as fp32 and the product are one rounding of at most 2^-24 each:
      5 * 2^-24 covers them and their products; a bf16 result adds its half step 2^-8.
  up: h = g sigma(g) u.  g and u carry 5 * 2^-24 each; silu's relative condition is at most 1 + |g|; the hardware
      exponential is off by 2 ulp plus |g| 2^-23 (its scaled argument), the fast division by 2 ulp:
      (16 + 16 |g|) 2^-24 covers all of it, plus the half step of bf16.
"""
import numpy as np
import pytest
import torch

import prefill_sigmoid_top_b200 as moe
from prefill_sigmoid_top_b200 import inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def quantize_ref(v):
    """Codes and scales of the rows of v (fp64, bf16 values): 127 v / a is exact up to one rounding of fp64, and a
    tie is representable, so rint decides as exact arithmetic does."""
    a = np.abs(v).max(axis=-1, keepdims=True)
    q = np.divide(127.0 * v, a, out=np.zeros_like(v), where=a > 0)
    return np.rint(q), a[..., 0] / 127.0


def codes_of(rows, cols, seed, pitch=None):
    g = gen(seed)
    c = torch.randint(-127, 128, (rows, pitch or cols), generator=g, dtype=torch.int64).to(torch.int8)
    return c[:, :cols], (torch.rand(rows, generator=g) + 0.5) * 0.01


def within(got, want, rel):
    got = got.detach().cpu().double().numpy()
    bad = ~(np.abs(got - want) <= rel * np.abs(want) + 1e-37)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


# ------------------------------------------------------------------ codes
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 5), (7, 127), (4, 128), (5, 1777), (2, 7168), (9, 256), (1, 131072)])
def test_quantize_codes_exact(rows, cols):
    w = torch.randn(rows, cols, generator=gen(cols)).to(torch.bfloat16)
    codes, scales = moe.quantize_int8(w.to(DEV))
    q, s = quantize_ref(w.double().numpy())
    assert np.array_equal(codes.cpu().numpy(), q)
    assert np.array_equal(scales.cpu().numpy(), s.astype(np.float32))
    assert codes.stride(0) % 16 == 0


def test_quantize_every_ratio_and_tie():
    """Every pair of bf16 significands at several exponent gaps: all quotients 127 v / a there are, ties included."""
    m = torch.arange(128, 256).double()
    rows = []
    for a in m:
        for gap in (0, 1, 2, 5, 7, 8):
            v = m * 2.0 ** -gap
            rows.append(torch.cat([a[None], torch.where(v <= a, v, -v / 2)]))
    w = torch.stack(rows)
    for scale in (1.0, 2.0 ** -130, 2.0 ** -60, 2.0 ** 120):
        b = (w * scale).to(torch.bfloat16)
        q, s = quantize_ref(b.double().numpy())
        codes, scales = moe.quantize_int8(b.to(DEV))
        assert np.array_equal(codes.cpu().numpy(), q)
        assert np.array_equal(scales.cpu().numpy(), s.astype(np.float32))


def test_quantize_special_rows():
    w = torch.randn(6, 40, generator=gen(1)).to(torch.bfloat16)
    w[0] = 0
    w[1, 7] = float("inf")
    w[2, 9] = float("nan")
    w[3, 0] = 3.3e38
    w[4] = 0
    w[4, 39] = -2.0 ** -133
    codes, scales = moe.quantize_int8(w.to(DEV))
    codes, scales = codes.cpu(), scales.cpu()
    assert scales[0] == 0 and (codes[0] == 0).all()
    assert scales[1:3].isnan().all() and (codes[1:3] == 0).all()
    assert codes[3, 0] == 127 and scales[3].isfinite() and (codes[3, 1:] == 0).all()
    assert codes[4, 39] == -127
    q, _ = quantize_ref(w[5:].double().numpy())
    assert np.array_equal(codes[5:].numpy(), q)


# ------------------------------------------------------------------ dense
def linear_case(M, N, K, out=torch.bfloat16, pad=0, off=0, seed=0):
    x = torch.randn(M, K + pad + off, generator=gen(seed)).to(torch.bfloat16)
    codes, scales = codes_of(N, K, seed + 1, (K + 15) // 16 * 16)
    xd = x.to(DEV)[:, off:off + K]
    cd = torch.empty(N, (K + 15) // 16 * 16, dtype=torch.int8, device=DEV).fill_(99)[:, :K]
    cd.copy_(codes)
    y = moe.linear_int8(xd, cd, scales.to(DEV), out_dtype=out)
    xq, sx = quantize_ref(x[:, off:off + K].double().numpy())
    want = (xq @ codes.double().numpy().T) * sx[:, None] * scales.double().numpy()
    assert y.dtype == out and tuple(y.shape) == (M, N)
    within(y, want, 5 * 2.0 ** -24 + STEP[out])


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 128, 128), (1, 2048, 7168), (2, 7168, 2048), (3, 131, 77), (16, 257, 129), (17, 640, 1000),
    (31, 129, 4097), (32, 512, 512), (33, 513, 511), (100, 300, 260), (128, 128, 128), (129, 1025, 2047),
    (255, 96, 33), (256, 1024, 640), (300, 1, 50), (40, 5, 1), (3, 200, 2), (4, 128, 131072), (513, 2049, 1777), (1000, 33, 7168), (1, 5, 131072),
])
def test_linear(M, N, K, out):
    linear_case(M, N, K, out, seed=M + N + K)


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("N,K", [(1, 128), (100, 15), (640, 1792), (5000, 256), (2048, 7168), (257, 8200), (40000, 96),
                                 (128, 14336), (3, 70000), (300, 9000)])
def test_linear_few_tokens(M, N, K):
    """A few tokens: one launch, one or several warps to a channel, odd lengths, too long for it; and the same bits
    as the two-launch form gives for these rows among others."""
    linear_case(M, N, K, torch.float32, pad=(K + M) % 3, seed=M + N)
    x = torch.randn(40, K, generator=gen(M)).to(torch.bfloat16).to(DEV)
    codes, scales = codes_of(N, K, M)
    wide = torch.zeros(N, (K + 15) // 16 * 16, dtype=torch.int8, device=DEV)[:, :K]
    wide.copy_(codes)
    scales = scales.to(DEV)
    assert torch.equal(moe.linear_int8(x[:M], wide, scales), moe.linear_int8(x, wide, scales)[:M])


@pytest.mark.parametrize("tile", ["0", "32", "96", "256"])
@pytest.mark.parametrize("M,N,K", [(20, 7, 40), (70, 1000, 300), (600, 2600, 128), (333, 513, 1777)])
def test_linear_tile_widths(M, N, K, tile, monkeypatch):
    monkeypatch.setenv("MOE_INT8_TILE", tile)
    for out in (torch.bfloat16, torch.float32):
        linear_case(M, N, K, out, seed=M)


def test_linear_pairs_many_tiles():
    """More tiles than pairs of SMs: the pairs take several, their accumulators in turn."""
    linear_case(2500, 6000, 130, torch.bfloat16, seed=1)
    linear_case(2500, 6001, 130, torch.bfloat16, seed=2)
    linear_case(1300, 6000, 400, torch.float32, seed=3)


@pytest.mark.parametrize("M", [1, 5, 40, 300])
@pytest.mark.parametrize("pad,off", [(3, 0), (1, 1), (8, 8), (0, 2)])
def test_linear_strided_rows(M, pad, off):
    linear_case(M, 200, 264, torch.float32, pad, off, seed=pad + off)


def test_linear_large_sums_are_exact():
    """K = 131072 with all codes at 127: the largest sum that is accepted, 131072 * 127^2 < 2^31."""
    K = 131072
    x = torch.ones(2, K, dtype=torch.bfloat16, device=DEV)
    x[1, ::2] = -1
    codes = torch.full((3, K), 127, dtype=torch.int8, device=DEV)
    codes[2] = -127
    y = moe.linear_int8(x, codes, torch.ones(3, device=DEV), out_dtype=torch.float32)
    want = np.array([[K * 127.0, K * 127.0, -K * 127.0], [0, 0, 0]])
    within(y, want, 5 * 2.0 ** -24)


def test_linear_special_values():
    x = torch.randn(5, 256, generator=gen(2)).to(torch.bfloat16)
    x[1] = 0
    x[2, 3] = float("inf")
    x[3, 255] = float("nan")
    codes, scales = codes_of(70, 256, 3)
    y = moe.linear_int8(x.to(DEV), codes.to(DEV), scales.to(DEV), out_dtype=torch.float32)
    assert (y[1] == 0).all() and y[2:4].isnan().all() and y[[0, 1, 4]].isfinite().all()


def test_linear_writes_its_rows_only():
    for M in (3, 40, 300):
        buf = torch.full((M + 2, 150), -5.0, device=DEV)
        codes, scales = codes_of(130, 64, 4)
        x = torch.randn(M, 64, generator=gen(5)).to(torch.bfloat16).to(DEV)
        out = buf[1:M + 1, 10:140]
        moe.linear_int8(x, codes.to(DEV), scales.to(DEV), out=out)
        inner = moe.linear_int8(x, codes.to(DEV), scales.to(DEV), out_dtype=torch.float32)
        assert torch.equal(out, inner)
        buf[1:M + 1, 10:140] = -5.0
        assert (buf == -5.0).all()


@pytest.mark.parametrize("M", [1, 24, 200, 1500])
def test_linear_same_bits_again_on_a_stream_and_replayed(M):
    codes, scales = (t.to(DEV) for t in codes_of(1500, 1024, 6))
    x = torch.randn(M, 1024, generator=gen(7)).to(torch.bfloat16).to(DEV)
    want = moe.linear_int8(x, codes, scales)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = moe.linear_int8(x, codes, scales)
    b = moe.linear_int8(x, codes, scales)  # both at once
    side.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = moe.linear_int8(x, codes, scales)
    x2 = torch.randn(M, 1024, generator=gen(8)).to(torch.bfloat16).to(DEV)
    want2 = moe.linear_int8(x2, codes, scales)
    x.copy_(x2)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want2)


# ------------------------------------------------------------------ experts
def random_ids(M, E, K, seed, skew=0.0):
    z = torch.randn(M, E, generator=gen(seed)) - skew * torch.arange(1, E + 1).log()
    return z.topk(K, dim=1).indices.int()


def experts_case(shape, seed=0, skew=0.0, ids=None):
    M, H, I, E, K = shape.M, shape.H, shape.I, shape.E, shape.top_k
    ids = random_ids(M, E, K, seed, skew) if ids is None else ids
    plan = moe.align_block_size(ids.to(DEV), E, shape.block_size)
    x = torch.randn(M, H, generator=gen(seed + 1)).to(torch.bfloat16)
    mats = {}
    for i, (n, r, c) in enumerate((("gate", I, H), ("up", I, H), ("down", H, I))):
        codes, scales = codes_of(E * r, c, seed + 2 + i)
        mats[n], mats[n + "_scales"] = codes.view(E, r, c), scales.view(E, r) * (1.0 / c ** 0.5)
    iw = moe.Int8Weights(**{k: v.to(DEV) for k, v in mats.items()})
    return x, ids, plan, mats, iw


def check_up(shape, x, plan, mats, iw):
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    cap = moe.align_capacity(shape)
    h = torch.full((cap, shape.I), -3.0, dtype=torch.bfloat16, device=DEV)
    moe.grouped_up_swiglu_int8(x.to(DEV), iw, plan, shape, h=h, err_flag=err)
    assert moe.get_device_error(err) == 0
    xq, sx = quantize_ref(x.double().numpy())
    counts, offs, sid = (plan[k].cpu().numpy() for k in ("expert_counts", "expert_offsets", "sorted_ids"))
    real = np.zeros(cap, bool)
    hc = h.cpu()
    for e in range(shape.E):
        rows = np.arange(offs[e], offs[e] + counts[e])
        if not len(rows):
            continue
        real[rows] = True
        t = sid[rows] // shape.top_k
        g, u = ((xq[t] @ mats[n][e].double().numpy().T) * sx[t][:, None] * mats[n + "_scales"][e].double().numpy()
                for n in ("gate", "up"))
        with np.errstate(over="ignore"):
            want = g / (1.0 + np.exp(-g)) * u
        within(hc[rows], want, 2.0 ** -8 + (16 + 16 * np.abs(g)) * 2.0 ** -24)
    assert (hc[~real] == -3.0).all()  # padding rows and rows behind the last block are left as they were
    return h


def check_down(shape, h, plan, mats, iw):
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = torch.full((shape.M * shape.top_k, shape.H), -3.0, dtype=torch.bfloat16, device=DEV)
    moe.grouped_down_int8(h, iw, plan, shape, y=y, err_flag=err)
    assert moe.get_device_error(err) == 0
    counts, offs, sid = (plan[k].cpu().numpy() for k in ("expert_counts", "expert_offsets", "sorted_ids"))
    hc, yc = h.double().cpu().numpy(), y.cpu()
    seen = 0
    for e in range(shape.E):
        rows = np.arange(offs[e], offs[e] + counts[e])
        if not len(rows):
            continue
        hq, sh = quantize_ref(hc[rows])
        want = (hq @ mats["down"][e].double().numpy().T) * sh[:, None] * mats["down_scales"][e].double().numpy()
        within(yc[sid[rows]], want, 2.0 ** -8 + 5 * 2.0 ** -24)
        seen += len(rows)
    assert seen == shape.M * shape.top_k


EXPERT_SHAPES = [  # M, H, I, E, K, B, skew
    (1, 256, 128, 1, 1, 16, 0), (1, 512, 256, 8, 2, 16, 0), (7, 256, 384, 8, 3, 16, 0), (16, 1024, 128, 4, 4, 32, 0),
    (40, 512, 256, 16, 2, 16, 1.0), (33, 256, 128, 1, 1, 64, 0), (130, 512, 384, 4, 2, 128, 0.5),
    (200, 768, 640, 3, 2, 256, 1.0), (513, 512, 512, 4, 2, 64, 1.0), (260, 256, 256, 1, 1, 16, 0),
    (96, 1280, 128, 64, 8, 16, 0.5), (700, 1024, 256, 2, 1, 16, 2.0),
]


@pytest.mark.parametrize("M,H,I,E,K,B,skew", EXPERT_SHAPES)
def test_experts(M, H, I, E, K, B, skew):
    shape = moe.Shape(M, H, I, E, K, B)
    x, ids, plan, mats, iw = experts_case(shape, seed=M + I, skew=skew)
    check_up(shape, x, plan, mats, iw)
    h = torch.randn(moe.align_capacity(shape), I, generator=gen(M)).to(torch.bfloat16).to(DEV)
    pad = torch.ones(h.shape[0], dtype=torch.bool)
    off, cnt = plan["expert_offsets"].cpu(), plan["expert_counts"].cpu()
    for e in range(E):
        pad[off[e]:off[e] + cnt[e]] = False
    h[pad.to(DEV)] = float("nan")  # what padding rows hold reaches no result
    check_down(shape, h, plan, mats, iw)


@pytest.mark.parametrize("M", [3, 150, 700])
@pytest.mark.parametrize("nmax,pair", [("32", "0"), ("128", "0"), ("128", "128"), ("128", "256")])
def test_experts_token_tile_widths(nmax, pair, M, monkeypatch):
    """Every kernel takes every shape: one tile per CTA of 32 or 128 tokens, pairs of 128 or 256."""
    monkeypatch.setenv("MOE_GEMM_NMAX", nmax)
    monkeypatch.setenv("MOE_GEMM_PAIR", pair)
    shape = moe.Shape(M, 512, 384, 5, 2, 16)
    x, ids, plan, mats, iw = experts_case(shape, seed=3, skew=1.0)
    check_up(shape, x, plan, mats, iw)
    check_down(shape, torch.randn(moe.align_capacity(shape), 384).to(torch.bfloat16).to(DEV), plan, mats, iw)


def test_experts_same_expert_twice_for_a_token():
    ids = torch.tensor([[2, 2, 0], [2, 2, 2]], dtype=torch.int32)
    shape = moe.Shape(2, 256, 128, 4, 3, 16)
    x, ids, plan, mats, iw = experts_case(shape, seed=6, ids=ids)
    check_up(shape, x, plan, mats, iw)
    check_down(shape, torch.randn(moe.align_capacity(shape), 128).to(torch.bfloat16).to(DEV), plan, mats, iw)


def test_experts_without_tokens_and_all_tokens_on_one():
    for ids in (torch.full((70, 1), 3, dtype=torch.int32), torch.tensor([[0], [9]], dtype=torch.int32)):
        shape = moe.Shape(ids.shape[0], 256, 128, 10, 1, 16)
        x, ids, plan, mats, iw = experts_case(shape, seed=4, ids=ids)
        check_up(shape, x, plan, mats, iw)
        check_down(shape, torch.randn(moe.align_capacity(shape), 128).to(torch.bfloat16).to(DEV), plan, mats, iw)


def test_experts_report_a_plan_with_bad_slots():
    """A slot id outside the plan's range is reported in the error word; the other rows keep their values."""
    for M in (8, 300):
        shape = moe.Shape(M, 256, 128, 4, 2, 16)
        x, ids, plan, mats, iw = experts_case(shape, seed=5)
        good = moe.grouped_up_swiglu_int8(x.to(DEV), iw, plan, shape)
        first = int(plan["expert_offsets"][:-1][plan["expert_counts"] > 0][0])
        bad = dict(plan, sorted_ids=plan["sorted_ids"].clone())
        for v in (-1, shape.M * shape.top_k + 5, 2 ** 31 - 1):
            bad["sorted_ids"][first] = v
            err = torch.zeros(1, dtype=torch.int32, device=DEV)
            h = torch.zeros_like(good)
            moe.grouped_up_swiglu_int8(x.to(DEV), iw, bad, shape, h=h, err_flag=err)
            assert moe.get_device_error(err) == 4
            assert torch.equal(h[first + 1], good[first + 1]) or int(plan["expert_counts"].max()) == 1
            err.zero_()
            moe.grouped_down_int8(good, iw, bad, shape, err_flag=err)
            assert moe.get_device_error(err) == 4


# ------------------------------------------------------------------ together
def layer_inputs(M, seed):
    cfg = inputs.WORKLOADS[0].with_(M=M, H=512, I=256, E=16, K=4, B=16, bias="normal", seed=seed)
    d = inputs.make_inputs(cfg, "cpu")
    return cfg, d, {k: v.to(DEV) for k, v in d.items()}


@pytest.mark.parametrize("M", [1, 8, 130, 600])
def test_layer_is_its_steps(M):
    cfg, _, d = layer_inputs(M, 21)
    iw = moe.int8_weights(d["w_gate"], d["w_up"], d["w_down"])
    shape = moe.Shape(M, cfg.H, cfg.I, cfg.E, cfg.K, cfg.B)
    ws = torch.empty(moe.layer_workspace_size(shape, moe.MOE_W_INT8), dtype=torch.uint8, device=DEV)
    ids = torch.empty(M, cfg.K, dtype=torch.int32, device=DEV)
    out = moe.layer_int8(d["x"], d["w_router"], d["bias"], iw, d["gamma"], cfg.eps, cfg.K, cfg.B, ws=ws, topk_ids=ids)
    assert moe.get_device_error(ws) == 0
    ids2, w = moe.route(d["x"], d["w_router"], d["bias"], cfg.K)
    plan = moe.align_block_size(ids2, cfg.E, cfg.B)
    h = moe.grouped_up_swiglu_int8(d["x"], iw, plan, shape)
    y = moe.grouped_down_int8(h, iw, plan, shape)
    want = moe.finalize_rmsnorm(d["x"], y.view(M, cfg.K, cfg.H), w, d["gamma"], cfg.eps)
    assert torch.equal(ids, ids2) and torch.equal(out, want)
    # every output, no bias, buffers of the caller
    res, w2 = torch.empty_like(out), torch.empty_like(w)
    out2 = torch.empty_like(out)
    moe.layer_int8(d["x"], d["w_router"], None, iw, d["gamma"], cfg.eps, cfg.K, cfg.B, out=out2, residual_out=res,
                   topk_ids=ids, topk_w=w2)
    ids3, w3 = moe.route(d["x"], d["w_router"], torch.zeros_like(d["bias"]), cfg.K)
    plan = moe.align_block_size(ids3, cfg.E, cfg.B)
    y = moe.grouped_down_int8(moe.grouped_up_swiglu_int8(d["x"], iw, plan, shape), iw, plan, shape)
    want, want_res = moe.finalize_rmsnorm(d["x"], y.view(M, cfg.K, cfg.H), w3, d["gamma"], cfg.eps, want_residual=True)
    assert torch.equal(ids, ids3) and torch.equal(w2, w3) and torch.equal(out2, want) and torch.equal(res, want_res)


@pytest.mark.parametrize("M", [6, 200])
def test_experts_on_two_streams_at_once(M):
    """Two projections at a time, each with its own workspace, give what each gives alone."""
    shape = moe.Shape(M, 1024, 512, 12, 3, 16)
    x, ids, plan, mats, iw = experts_case(shape, seed=31)
    x2 = torch.randn(M, 1024, generator=gen(32)).to(torch.bfloat16).to(DEV)
    x1 = x.to(DEV)
    want1, want2 = (moe.grouped_up_swiglu_int8(t, iw, plan, shape) for t in (x1, x2))
    real = torch.zeros(want1.shape[0], dtype=torch.bool, device=DEV)
    for e in range(12):
        o, c = int(plan["expert_offsets"][e]), int(plan["expert_counts"][e])
        real[o:o + c] = True
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(20):
        with torch.cuda.stream(side):
            a = moe.grouped_up_swiglu_int8(x2, iw, plan, shape)
        got.append((moe.grouped_up_swiglu_int8(x1, iw, plan, shape), a))
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a[real], want1[real]) and torch.equal(b[real], want2[real])


@pytest.mark.parametrize("M", [3, 300])
def test_experts_with_rows_that_are_not_numbers(M):
    """A token with an infinity or a NaN spoils its own rows only, a token of zeros gives zeros."""
    shape = moe.Shape(M, 512, 256, 6, 2, 16)
    x, ids, plan, mats, iw = experts_case(shape, seed=33)
    good = moe.grouped_up_swiglu_int8(x.to(DEV), iw, plan, shape)
    bad = x.clone()
    bad[0, 5], bad[1, 7], bad[2] = float("inf"), float("nan"), 0.0
    h = moe.grouped_up_swiglu_int8(bad.to(DEV), iw, plan, shape)
    y = moe.grouped_down_int8(h, iw, plan, shape).view(M, 2, 512)
    sid = plan["sorted_ids"].cpu()
    for e in range(6):
        o, c = int(plan["expert_offsets"][e]), int(plan["expert_counts"][e])
        for r in range(o, o + c):
            t = int(sid[r]) // 2
            if t < 2:
                assert h[r].isnan().all()
            elif t == 2:
                assert (h[r] == 0).all()
            else:
                assert torch.equal(h[r], good[r])
    assert y[:2].isnan().all() and (y[2] == 0).all() and y[3:].isfinite().all()


@pytest.mark.parametrize("M", [1, 37, 300])
def test_group_routed_layer_with_a_shared_expert(M):
    """As a user runs them together: group-limited routing, the plan, int8 experts, finalize, and a dense int8
    projection beside them, against a 64-bit layer that takes the stored codes and the same intermediate roundings."""
    cfg, c, d = layer_inputs(M, 22)
    iw = moe.int8_weights(d["w_gate"], d["w_up"], d["w_down"])
    shape = moe.Shape(M, cfg.H, cfg.I, cfg.E, cfg.K, cfg.B)
    ids, w = moe.route_group(d["x"], d["w_router"], d["bias"], cfg.K, 4, 2, routed_scale=2.5)
    plan = moe.align_block_size(ids, cfg.E, cfg.B)
    h = moe.grouped_up_swiglu_int8(d["x"], iw, plan, shape)
    y = moe.grouped_down_int8(h, iw, plan, shape)
    out, res = moe.finalize_rmsnorm(d["x"], y.view(M, cfg.K, cfg.H), w, d["gamma"], cfg.eps, want_residual=True)
    sc, ss = moe.quantize_int8(d["w_gate"][0])
    shared = moe.linear_int8(d["x"], sc, ss)
    # 64 bits
    mats = {n: getattr(iw, n).cpu().double().numpy() * getattr(iw, n + "_scales").cpu().double().numpy()[..., None]
            for n in ("gate", "up", "down")}
    xq, sx = quantize_ref(c["x"].double().numpy())
    xv = xq * sx[:, None]
    s = c["x"].double().numpy().copy()
    for t in range(M):
        for k in range(cfg.K):
            e = int(ids[t, k])
            g, u = mats["gate"][e] @ xv[t], mats["up"][e] @ xv[t]
            hv = torch.from_numpy(g / (1 + np.exp(-g)) * u).to(torch.bfloat16).double().numpy()
            hq, sh = quantize_ref(hv[None])
            yv = torch.from_numpy(mats["down"][e] @ (hq[0] * sh[0])).to(torch.bfloat16).double().numpy()
            s[t] += float(w[t, k]) * yv
    want = s / np.sqrt((s * s).mean(1, keepdims=True) + cfg.eps) * c["gamma"].double().numpy()
    # a bf16 rounding of h or y that falls the other way (fp32 against fp64 before it) moves a value by a step of
    # its own; the framework's bar for layer outputs covers it: 2e-2 of the RMS
    assert np.abs(out.cpu().double().numpy() - want).max() <= 2e-2 * np.sqrt((want * want).mean())
    assert np.abs(res.cpu().double().numpy() - s).max() <= 2e-2 * np.sqrt((s * s).mean())
    want = (xq @ sc.cpu().double().numpy().T) * sx[:, None] * ss.cpu().double().numpy()
    within(shared, want, 2.0 ** -8 + 5 * 2.0 ** -24)


def test_refusals_by_name():
    """What the binding refuses on CUDA tensors: types, shapes, strides, devices, missing matrices; and the statuses of
    the library as MoEError.  None of it launches anything."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    c, s = torch.zeros(8, 64, dtype=torch.int8, device=DEV), torch.zeros(8, device=DEV)
    z = torch.zeros(4, 8, device=DEV)
    shape = moe.Shape(4, 256, 128, 2, 1, 16)
    plan = moe.align_block_size(torch.zeros(4, 1, dtype=torch.int32, device=DEV), 2, 16)
    xe = torch.zeros(4, 256, dtype=torch.bfloat16, device=DEV)
    h = torch.zeros(moe.align_capacity(shape), 128, dtype=torch.bfloat16, device=DEV)
    iw = moe.int8_weights(*(torch.zeros(2, *d, dtype=torch.bfloat16, device=DEV) for d in ((128, 256), (128, 256), (256, 128))))
    for call in (lambda: moe.linear_int8(x.float(), c, s), lambda: moe.linear_int8(x, c.float(), s),
                 lambda: moe.linear_int8(x, c[:, :32], s), lambda: moe.linear_int8(x, c, s[:4]),
                 lambda: moe.linear_int8(x, c, s.double()), lambda: moe.linear_int8(x.t(), c, s),
                 lambda: moe.linear_int8(x, c, s, out_dtype=torch.float16), lambda: moe.linear_int8(x, c, s, out=z.t()),
                 lambda: moe.linear_int8(x, c, s, out=z.double()), lambda: moe.linear_int8(x, c, s.cpu()),
                 lambda: moe.linear_int8(x[0], c, s), lambda: moe.route_logits(z.half(), None, 2),
                 lambda: moe.route_logits(z, s[:4], 2), lambda: moe.route_logits(z, s.cpu(), 2),
                 lambda: moe.route_logits(z, None, 2, topk_ids=z), lambda: moe.route_logits(z[:, ::2], None, 2),
                 lambda: moe.grouped_up_swiglu_int8(xe, moe.Int8Weights(), plan, shape),
                 lambda: moe.grouped_up_swiglu_int8(xe[:3], iw, plan, shape),
                 lambda: moe.grouped_up_swiglu_int8(xe, iw, plan, shape, h=h[:3]),
                 lambda: moe.grouped_up_swiglu_int8(xe, iw, dict(plan, sorted_ids=z), shape),
                 lambda: moe.grouped_down_int8(h[:3], iw, plan, shape),
                 lambda: moe.grouped_down_int8(h, iw, plan, shape, y=xe[:2]),
                 lambda: moe.grouped_down_int8(h, moe.Int8Weights(down=iw.gate, down_scales=iw.gate_scales), plan, shape)):
        with pytest.raises(ValueError):
            call()
    for call, status in ((lambda: moe.route_logits(z, None, 9), 2), (lambda: moe.route_logits(z, None, 2, 3), 2),
                         (lambda: moe.route_logits(z, None, 2, routed_scale=0.0), 1),
                         (lambda: moe.linear_int8(x[:0], c, s), 2), (lambda: moe.linear_int8(x, c[:, :63], s), 0),
                         (lambda: moe.linear_int8(x[:, :40], c.flatten()[:8 * 40].view(8, 40), s), 1),
                         (lambda: moe.linear_int8(x.repeat(10, 1), c, s, ws=torch.zeros(16, dtype=torch.uint8, device=DEV)), 3)):
        if status == 0:
            with pytest.raises(ValueError):
                call()
            continue
        with pytest.raises(moe.MoEError) as e:
            call()
        assert e.value.status == status


def test_layer_against_bf16_layer():
    """8 bits instead of bf16: the layer's output moves by the quantisation error only (two roundings of at most
    half of 1/127 of a row's largest value in each product: a few percent of the RMS)."""
    cfg, _, d = layer_inputs(64, 23)
    iw = moe.int8_weights(d["w_gate"], d["w_up"], d["w_down"])
    a = moe.layer_int8(d["x"], d["w_router"], d["bias"], iw, d["gamma"], cfg.eps, cfg.K, cfg.B).double()
    b = moe.layer(d["x"], d["w_router"], d["bias"], d["w_gate"], d["w_up"], d["w_down"], d["gamma"], cfg.eps, cfg.K,
                  cfg.B).double()
    assert float((a - b).norm() / b.norm()) < 0.05


def test_layer_captured_and_replayed():
    cfg, _, d = layer_inputs(40, 24)
    iw = moe.int8_weights(d["w_gate"], d["w_up"], d["w_down"])
    run = lambda: moe.layer_int8(d["x"], d["w_router"], d["bias"], iw, d["gamma"], cfg.eps, cfg.K, cfg.B)  # noqa: E731
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    x2 = torch.randn(40, cfg.H, generator=gen(25)).to(torch.bfloat16)
    d["x"].copy_(x2)
    want = run()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("tile", ["32x1", "64x1", "128x1", "224x1", "256x1"])
@pytest.mark.parametrize("M,N,K", [(20, 7, 40), (70, 1000, 300), (600, 2600, 128), (333, 513, 1777), (2600, 5400, 200)])
def test_linear_tiles_of_256_channels(M, N, K, tile, monkeypatch):
    """One box of 128 channels per CTA: two accumulator sets, which tiles take in turn."""
    monkeypatch.setenv("MOE_INT8_TILE", tile)
    for out in (torch.bfloat16, torch.float32):
        linear_case(M, N, K, out, seed=M + 1)


PLAN = ("sorted_ids", "block_expert", "expert_counts", "expert_offsets", "num_tokens_post_padded")


@pytest.mark.parametrize("M,E,B", [(4, 2, 16), (60, 3, 64)])
def test_plans_of_another_shape_are_refused(M, E, B):
    """A plan array with fewer entries than the shape's plan has (one missing, none, that of fewer tokens, experts or a
    smaller block), and an error word without room, are refused before anything is launched."""
    shape = moe.Shape(M, 256, 128, E, 1, B)
    x, ids, plan, mats, iw = experts_case(shape, seed=41)
    xd = x.to(DEV)
    h = torch.zeros(moe.align_capacity(shape), 128, dtype=torch.bfloat16, device=DEV)
    need = dict(sorted_ids=moe.align_capacity(shape), block_expert=moe.align_capacity(shape) // B, expert_counts=E,
                expert_offsets=E + 1, num_tokens_post_padded=1)
    plans = [dict(plan, **{n: plan[n][:k]}) for n in PLAN for k in {0, need[n] - 1}]
    plans.append(moe.align_block_size(ids[:-1].to(DEV), E, B))
    plans.append(moe.align_block_size(torch.zeros_like(ids).to(DEV), E - 1, B))
    if B > 16:
        plans.append(moe.align_block_size(ids.to(DEV), E, B // 2))
    for p in plans:
        with pytest.raises(ValueError):
            moe.grouped_up_swiglu_int8(xd, iw, p, shape)
        with pytest.raises(ValueError):
            moe.grouped_down_int8(h, iw, p, shape)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    codes, scales = (t.to(DEV) for t in codes_of(8, 256, 1))
    for call in (lambda: moe.grouped_up_swiglu_int8(xd, iw, plan, shape, err_flag=none),
                 lambda: moe.grouped_down_int8(h, iw, plan, shape, err_flag=none),
                 lambda: moe.linear_int8(xd, codes, scales, err_flag=none)):
        with pytest.raises(ValueError):
            call()
    # exactly as many entries as the shape needs, and more, are taken
    want = moe.grouped_down_int8(h, iw, plan, shape)
    exact = {n: plan[n][:need[n]] for n in PLAN}
    more = {n: torch.cat([plan[n], plan[n].new_zeros(5)]) for n in PLAN}
    for p in (exact, more):
        assert torch.equal(moe.grouped_down_int8(h, iw, p, shape), want)


def set_widths(monkeypatch, nmax, pair):
    """The kernel for the expert projections: single CTAs (pair "0"), or pairs with tiles of this many tokens."""
    monkeypatch.setenv("MOE_GEMM_NMAX", nmax)
    monkeypatch.setenv("MOE_GEMM_PAIR", pair)


@pytest.mark.parametrize("nmax,pair", [("32", "0"), ("128", "128"), ("128", "256")])
def test_plans_that_reach_beyond_the_buffers(nmax, pair, monkeypatch):
    """Plans with enough entries whose contents belong to another shape (more tokens, a wider block, counts and offsets
    that are no such): rows behind the shape's capacity keep what they held, the error word says INVALID_INPUT, rows of
    experts that are in order keep their values."""
    set_widths(monkeypatch, nmax, pair)
    shape = moe.Shape(4, 256, 128, 2, 1, 16)
    cap = moe.align_capacity(shape)
    x, ids, plan, mats, iw = experts_case(shape, seed=42, ids=torch.tensor([[1], [1], [1], [0]], dtype=torch.int32))
    xd = x.to(DEV)
    good = moe.grouped_up_swiglu_int8(xd, iw, plan, shape, h=torch.zeros(cap, 128, dtype=torch.bfloat16, device=DEV))
    hin = torch.randn(cap, 128, generator=gen(43)).to(torch.bfloat16).to(DEV)

    def run(p, first_expert_intact):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        h = torch.full((cap + 300, 128), -3.0, dtype=torch.bfloat16, device=DEV)
        moe.grouped_up_swiglu_int8(xd, iw, p, shape, h=h, err_flag=err)
        assert moe.get_device_error(err) == 4
        assert (h[cap:] == -3.0).all()
        if first_expert_intact:
            assert torch.equal(h[0], good[0])
        err.zero_()
        y = moe.grouped_down_int8(hin, iw, p, shape, err_flag=err)
        assert moe.get_device_error(err) == 4 and tuple(y.shape) == (4, 256)

    more = torch.zeros(40, 1, dtype=torch.int32)
    more[:20] = 1
    run(moe.align_block_size(more.to(DEV), 2, 16), False)  # tokens 0 to 3 at rows 32 to 35 of 34
    wide = torch.tensor([[0], [1], [1], [1]], dtype=torch.int32)
    run(moe.align_block_size(wide.to(DEV), 2, 64), False)  # expert 1 from row 64 on
    for name, values in (("expert_counts", (-1, -2 ** 31, 5, 10 ** 6, 2 ** 31 - 1)),
                         ("expert_offsets", (-1, -40, cap, 2 ** 31 - 1, -2 ** 31))):
        for v in values:
            bad = plan[name].clone()
            bad[1] = v
            # the first expert's row 0 keeps its value unless it is one of the second's rows v .. v + 2 too
            run(dict(plan, **{name: bad}), not (name == "expert_offsets" and -3 < v <= 0))


# ------------------------------------------------------------------ scales whose product leaves fp32's normal range
def far_rows(M, cols):
    """Rows of one value each, so codes of 127 and scales of exactly 2^-117, 1, 2^90 and 0, in turn."""
    x = torch.tensor([127 * 2.0 ** -117, 127.0, 127 * 2.0 ** 90, 0.0]).repeat(M // 4 + 1)[:M]
    return x[:, None].expand(M, cols).to(torch.bfloat16).contiguous()


def far_weights(rows, cols, seed, scale):
    """Codes of 64 to 127, so sums of about 2^13.6 cols, and scales of `scale` times 1 to 2; every third channel has
    sums of 0 (halves of +1 and -1) and the scale 2^60."""
    g = gen(seed)
    c = torch.randint(64, 128, (rows, cols), generator=g).to(torch.int8)
    s = scale * (1.0 + torch.rand(rows, generator=g))
    c[::3, :cols // 2], c[::3, cols // 2:], s[::3] = 1, -1, 2.0 ** 60
    return c, s


def far_within(got, want, rel):
    """Relative where the exact value is a normal number of fp32; infinite above, one subnormal step of bf16 below."""
    got, top = got.detach().cpu().double().numpy(), float(torch.finfo(torch.bfloat16).max)
    normal = (np.abs(want) >= 2.0 ** -126) & (np.abs(want) <= top)
    assert normal.any() and (want == 0).any()
    assert (np.abs(got - want)[normal] <= rel * np.abs(want)[normal]).all()
    assert (got[np.abs(want) > 1.01 * top] == np.inf).all()
    assert (np.abs(got - want)[np.abs(want) < 2.0 ** -126] <= 2.0 ** -133).all()


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("M,N,tile", [(1, 40, None), (2, 40, None), (4, 300, None), (20, 136, None), (70, 136, "0"),
                                      (70, 136, "96"), (300, 520, "256"), (300, 520, "256x1"), (300, 515, "64")])
def test_linear_scales_far_apart(M, N, tile, out, monkeypatch):
    """Row scales from 2^-117 to 2^90 against channel scales of 2^-31 (their product has 2 bits left in fp32, the result
    is a normal number) and 2^60 (their product is infinite, the sum 0): the bars of the other tests hold."""
    if tile is not None:
        monkeypatch.setenv("MOE_INT8_TILE", tile)
    x = far_rows(M, 4096)
    codes, scales = far_weights(N, 4096, 51, 2.0 ** -31)
    y = moe.linear_int8(x.to(DEV), codes.to(DEV), scales.to(DEV), out_dtype=out)
    xq, sx = quantize_ref(x.double().numpy())
    want = (xq @ codes.double().numpy().T) * sx[:, None] * scales.double().numpy()
    far_within(y, want, 5 * 2.0 ** -24 + STEP[out])
    if M > 4:  # the same bits alone as among rows of other magnitudes
        for m in range(4):
            assert torch.equal(moe.linear_int8(x[m:m + 1].to(DEV), codes.to(DEV), scales.to(DEV), out_dtype=out)[0], y[m])


@pytest.mark.parametrize("nmax,pair", [("32", "0"), ("128", "128"), ("128", "256")])
@pytest.mark.parametrize("M", [3, 41, 300])
def test_experts_scales_far_apart(M, nmax, pair, monkeypatch):
    """The same in the projections: g is of order 1, u about 2^-122 out of scales of 2^-117 and 2^-31."""
    set_widths(monkeypatch, nmax, pair)
    shape = moe.Shape(M, 4096, 256, 2, 1, 16)
    ids = (torch.arange(M)[:, None] % 3 == 1).int()
    plan = moe.align_block_size(ids.to(DEV), 2, 16)
    x = torch.full((M, 4096), 127 * 2.0 ** -117).to(torch.bfloat16)
    gc, gs = far_weights(512, 4096, 52, 2.0 ** 91)
    uc, us = far_weights(512, 4096, 53, 2.0 ** -31)
    gs[::3] = 2.0 ** 91
    gc[::3] = gc[1]
    dc, ds = far_weights(8192, 256, 54, 2.0 ** -27)
    iw = moe.Int8Weights(gc.view(2, 256, 4096).to(DEV), uc.view(2, 256, 4096).to(DEV), dc.view(2, 4096, 256).to(DEV),
                         gs.view(2, 256).to(DEV), us.view(2, 256).to(DEV), ds.view(2, 4096).to(DEV))
    h = torch.zeros(moe.align_capacity(shape), 256, dtype=torch.bfloat16, device=DEV)
    moe.grouped_up_swiglu_int8(x.to(DEV), iw, plan, shape, h=h)
    hin = far_rows(h.shape[0], 256)
    y = moe.grouped_down_int8(hin.to(DEV), iw, plan, shape)
    xq, sx = quantize_ref(x.double().numpy())
    hq, sh = quantize_ref(hin.double().numpy())
    counts, offs, sid = (plan[k].cpu().numpy() for k in ("expert_counts", "expert_offsets", "sorted_ids"))
    g64 = lambda q, c, s, e, n, sc: (q @ c.view(2, n, -1)[e].double().numpy().T) * sc[:, None] * s.view(2, n)[e].double().numpy()  # noqa: E731
    yw = np.zeros((M, 4096))
    for e in range(2):
        rows = np.arange(offs[e], offs[e] + counts[e])
        t = sid[rows]
        g, u = g64(xq[t], gc, gs, e, 256, sx[t]), g64(xq[t], uc, us, e, 256, sx[t])
        far_within(h[rows], g / (1.0 + np.exp(-g)) * u, 2.0 ** -8 + (16 + 16 * np.abs(g).max()) * 2.0 ** -24)
        yw[t] = g64(hq[rows], dc, ds, e, 4096, sh[rows])
    far_within(y, yw, 2.0 ** -8 + 5 * 2.0 ** -24)


@pytest.mark.parametrize("M", [1, 2, 4, 20, 40])
@pytest.mark.parametrize("N,K", [(1, 1), (1, 15), (1, 17), (3, 33), (40, 1000), (5000, 47), (129, 8201), (2, 16400)])
def test_linear_last_weight_row_ends_at_its_last_code(M, N, K):
    """Weights whose storage ends with the last row's K codes: nothing behind them is asked for, and the last channel is
    that of a padded copy."""
    pitch = (K + 15) // 16 * 16
    x = torch.randn(M, K, generator=gen(61)).to(torch.bfloat16).to(DEV)
    codes, scales = (t.to(DEV) for t in codes_of(N, K, 62))
    tight = torch.zeros((N - 1) * pitch + K, dtype=torch.int8, device=DEV).as_strided((N, K), (pitch, 1))
    tight.copy_(codes)
    assert tight.untyped_storage().nbytes() == (N - 1) * pitch + K
    padded = torch.full((N + 1, pitch), 99, dtype=torch.int8, device=DEV)[:N, :K]
    padded.copy_(codes)
    y = moe.linear_int8(x, tight, scales, out_dtype=torch.float32)
    assert torch.equal(y, moe.linear_int8(x, padded, scales, out_dtype=torch.float32))
    xq, sx = quantize_ref(x.double().cpu().numpy())
    want = (xq @ codes.double().cpu().numpy().T) * sx[:, None] * scales.double().cpu().numpy()
    within(y, want, 5 * 2.0 ** -24)


@pytest.mark.parametrize("nmax,pair", [("32", "0"), ("128", "128"), ("128", "256")])
@pytest.mark.parametrize("M,E,K,skew", [(300, 1024, 2, 0.3), (90, 1000, 5, 1.0), (1, 1024, 32, 0.0), (700, 100, 1, 1.5)])
def test_experts_up_to_the_limit(M, E, K, skew, nmax, pair, monkeypatch):
    """As many experts as are accepted, and counts that are no multiple of 32: the counts and the tile list in shared
    memory, the search for a tile's expert, experts without a token, the last expert's tokens."""
    set_widths(monkeypatch, nmax, pair)
    shape = moe.Shape(M, 256, 128, E, K, 16)
    ids = random_ids(M, E, K, E + K, skew)
    ids[0, 0] = E - 1
    if K > 1:
        ids[0, 1] = 0
    x, ids, plan, mats, iw = experts_case(shape, seed=71, ids=ids)
    assert (plan["expert_counts"] == 0).any() and plan["expert_counts"][-1] > 0
    check_up(shape, x, plan, mats, iw)
    check_down(shape, torch.randn(moe.align_capacity(shape), 128, generator=gen(72)).to(torch.bfloat16).to(DEV), plan, mats, iw)
