"""Refusals of the int8 products and of the routing with groups: every call here fails its host checks before any
CUDA work, so nothing needs a GPU."""
import ctypes

import pytest
import torch

import prefill_sigmoid_top_b200 as moe
from prefill_sigmoid_top_b200 import _GroupOpts, _Plan, _Weights

FAKE = ctypes.c_void_p(0x10000)       # aligned non-null address, never dereferenced
FAKE_MIS = ctypes.c_void_p(0x10008)   # 8-byte aligned only
P = 0x10000
PLAN = ("sorted_ids", "block_expert", "expert_counts", "expert_offsets", "num_tokens_post_padded")
S = moe.Shape(M=16, H=256, I=128, E=8, top_k=2, block_size=16)


def route(logits=FAKE, dtype=0, ld=64, M=4, E=64, K=8, ids=FAKE, w=FAKE, o=(1, 1, 8, 4, 1, 1.0)):
    opts = None if o is None else ctypes.byref(_GroupOpts(*o))
    return moe.library().moe_route_logits(logits, dtype, ld, None, M, E, K, opts, ids, w, None)


def test_route_logits_refusals():
    inf, nan = float("inf"), float("nan")
    assert route(logits=None) == 1 and route(ids=None) == 1 and route(w=None) == 1 and route(o=None) == 1
    assert route(dtype=2) == 1 and route(dtype=-1) == 1 and route(ld=63) == 1
    assert route(logits=ctypes.c_void_p(P + 2)) == 1 and route(logits=ctypes.c_void_p(P + 1), dtype=1) == 1
    for o in [(2, 1, 8, 4, 1, 1.0), (1, 1, 8, 4, 2, 1.0), (1, 1, 8, 4, -1, 1.0), (1, 1, 8, 4, 1, 0.0),
              (1, 1, 8, 4, 1, inf), (1, 1, 8, 4, 1, nan), (1, 1, 8, 4, 1, -1.0)]:
        assert route(o=o) == 1
    for o in [(1, 1, 0, 1, 1, 1.0), (1, 1, 7, 4, 1, 1.0), (1, 1, 64, 4, 1, 1.0), (1, 1, 8, 0, 1, 1.0),
              (1, 1, 8, 9, 1, 1.0), (1, 1, 32, 3, 1, 1.0)]:
        assert route(o=o) == 2
    assert route(M=0) == 2 and route(E=0) == 2 and route(K=0) == 2 and route(K=33) == 2
    assert route(E=1032, ld=1032) == 2 and route(M=2 ** 28, K=8) == 2


def test_route_group_refusals():
    L, o = moe.library(), _GroupOpts(1, 1, 4, 2, 1, 1.0)
    call = lambda x=FAKE, s=S, o=ctypes.byref(o), ws=FAKE, n=1 << 20: L.moe_route_group(  # noqa: E731
        x, FAKE, None, s.c(), o, FAKE, FAKE, ws, n, None)
    assert call(x=None) == 1 and call(x=FAKE_MIS) == 1 and call(o=None) == 1
    assert call(ws=None) == 3 and call(n=4) == 3 and call(ws=FAKE_MIS) == 3
    assert call(o=ctypes.byref(_GroupOpts(1, 1, 3, 2, 1, 1.0))) == 2
    assert call(s=moe.Shape(16, 255, 128, 8, 2, 16)) == 2


def test_quantize_refusals():
    q = lambda src=FAKE, ld=64, rows=4, cols=64, codes=FAKE, pitch=64, sc=FAKE: moe.library().moe_quantize_int8(  # noqa: E731
        src, ld, rows, cols, codes, pitch, sc, None)
    assert q(src=None) == 1 and q(codes=None) == 1 and q(sc=None) == 1 and q(ld=63) == 1 and q(pitch=63) == 1
    assert q(rows=0) == 2 and q(cols=0) == 2 and q(rows=2 ** 31) == 2
    assert q(cols=131073, ld=131073, pitch=131073) == 2


def linear(x=FAKE, ldx=64, w=FAKE, ldw=64, sc=FAKE, M=40, N=8, K=64, out=FAKE, ldo=8, dt=1, ws=FAKE, n=1 << 20):
    return moe.library().moe_linear_int8(x, ldx, w, ldw, sc, M, N, K, out, ldo, dt, ws, n, None, None)


def test_linear_refusals():
    assert linear(x=None) == 1 and linear(w=None) == 1 and linear(sc=None) == 1 and linear(out=None) == 1
    assert linear(w=FAKE_MIS) == 1 and linear(ldx=63) == 1 and linear(ldw=72) == 1 and linear(ldw=48) == 1
    assert linear(ldo=7) == 1 and linear(dt=2) == 1
    assert linear(M=0) == 2 and linear(N=0) == 2 and linear(K=0) == 2 and linear(K=131073, ldx=1 << 20, ldw=1 << 20) == 2
    assert linear(M=2 ** 30 + 1) == 2 and linear(M=2 ** 30, N=2 ** 30, ldo=2 ** 30) == 2
    assert linear(ws=None) == 3 and linear(ws=FAKE_MIS) == 3 and linear(n=16) == 3
    assert moe.linear_int8_workspace_size(0, 1, 1) == 0
    assert moe.linear_int8_workspace_size(40, 8, 65) >= 40 * 80 + 160
    assert moe.linear_int8_workspace_size(1, 2048, 7168) == 0  # few tokens: one launch, nothing to keep
    assert moe.linear_int8_workspace_size(1, 2048, 131072) > 0


def test_expert_refusals():
    L, s = moe.library(), S.c()
    p = _Plan(P, P, P, P, P)
    up_ws, down_ws = moe.up_workspace_size(S, moe.MOE_W_INT8), moe.down_workspace_size(S, moe.MOE_W_INT8)
    assert up_ws >= 16 * 256 + 64 and down_ws >= moe.align_capacity(S) * (128 + 4)

    def up(w, plan=p, ws=FAKE, n=up_ws):
        return L.moe_grouped_up_swiglu(FAKE, ctypes.byref(w), ctypes.byref(plan), s, FAKE, ws, n, None, None)

    def down(w, plan=p, ws=FAKE, n=down_ws):
        return L.moe_grouped_down(FAKE, ctypes.byref(w), ctypes.byref(plan), s, FAKE, ws, n, None, None)

    w = _Weights(2, P, P, P, P, P, P)
    assert up(w, ws=None) == 3 and up(w, n=up_ws - 1) == 3 and up(w, ws=FAKE_MIS) == 3
    assert down(w, ws=None) == 3 and down(w, n=down_ws - 1) == 3
    for bad in (_Weights(2, P, P, P, None, P, P), _Weights(2, P, P, P, P, None, P), _Weights(2, P, None, P, P, P, P),
                _Weights(2, P + 8, P, P, P, P, P)):
        assert up(bad) == 1
    assert down(_Weights(2, P, P, P, P, P, None)) == 1 and down(_Weights(2, P, P, None, P, P, P)) == 1
    assert down(w, plan=_Plan(P, P, P, P, None)) == 1
    need = moe.layer_workspace_size(S, moe.MOE_W_INT8)
    layer = lambda w, n=need: L.moe_layer(FAKE, FAKE, None, ctypes.byref(w), FAKE, ctypes.c_float(1e-5), s, FAKE,  # noqa: E731
                                          None, None, None, FAKE, n, None)
    assert layer(w, need - 1) == 3 and layer(_Weights(2, P, P, P, P, P, None)) == 1
    assert moe.layer_kernel_count(S, moe.MOE_W_INT8) == 8
    assert moe.layer_kernel_count(moe.Shape(512, 7168, 2048, 256, 16, 64), moe.MOE_W_INT8) == 9  # screened routing
    assert moe.layer_kernel_count(moe.Shape(2048, 7168, 2048, 256, 16, 128), moe.MOE_W_INT8) == 9
    assert L.moe_layer_kernel_count(s, 3) == -1
    assert moe.layer_workspace_layout(S, moe.MOE_W_INT8)["total"] == need


def test_binding_refusals():
    """Wrong types, shapes and devices are refused by name before the library is called."""
    cpu = torch.zeros(4, 64)
    for call in (lambda: moe.route_logits(cpu, None, 2), lambda: moe.route_logits(cpu.double(), None, 2),
                 lambda: moe.route_logits(cpu.t(), None, 2), lambda: moe.route_logits(cpu[0], None, 2),
                 lambda: moe.linear_int8(cpu, cpu.to(torch.int8), cpu[:, 0]),
                 lambda: moe.linear_int8(cpu.to(torch.bfloat16), cpu, cpu[:, 0]),
                 lambda: moe.linear_int8(cpu.to(torch.bfloat16), cpu.to(torch.int8)[:, :32], cpu[:, 0]),
                 lambda: moe.linear_int8(cpu.to(torch.bfloat16), cpu.to(torch.int8), cpu[:, 0]),
                 lambda: moe.quantize_int8(cpu),
                 lambda: moe.grouped_up_swiglu_int8(cpu, moe.Int8Weights(), dict.fromkeys(PLAN, cpu), S),
                 lambda: moe.grouped_down_int8(cpu, moe.Int8Weights(), dict.fromkeys(PLAN, cpu), S),
                 lambda: moe.route_logits(None, None, 2), lambda: moe.route_logits("logits", None, 2),
                 lambda: moe.layer_int8(cpu, cpu, None, moe.Int8Weights(), cpu, 1e-5, 2, 16)):
        with pytest.raises(ValueError):
            call()
    iw = moe.Int8Weights(gate=torch.zeros(8, 128, 256, dtype=torch.int8), gate_scales=torch.zeros(8, 128))
    assert len(iw.check(S, "gate")) == 2
    with pytest.raises(ValueError):
        iw.check(S, "up")
    with pytest.raises(ValueError):
        moe.layer_int8(cpu, cpu, None, iw, cpu, 1e-5, 2, 16)
    iw.gate_scales = torch.zeros(8, 127)
    with pytest.raises(ValueError):
        iw.check(S, "gate")


def test_addresses_off_their_type_are_refused():
    """A pointer that is no multiple of its type's size would fault on the GPU: every argument that needs no more
    alignment than that is looked at (the others are tested above)."""
    L, odd, half = moe.library(), ctypes.c_void_p(P + 1), ctypes.c_void_p(P + 2)
    o = ctypes.byref(_GroupOpts(1, 1, 8, 4, 1, 1.0))
    logits = lambda bias=FAKE, ids=FAKE, w=FAKE: L.moe_route_logits(FAKE, 0, 64, bias, 4, 64, 8, o, ids, w, None)  # noqa: E731
    s64 = moe.Shape(4, 256, 128, 64, 8, 16).c()
    group = lambda bias=FAKE, ids=FAKE, w=FAKE: L.moe_route_group(  # noqa: E731
        FAKE, FAKE, bias, s64, o, ids, w, FAKE, 1 << 20, None)
    for call in (logits, group):
        for bad in (odd, half):
            assert call(bias=bad) == 1 and call(ids=bad) == 1 and call(w=bad) == 1
    quantize = lambda src=FAKE, sc=FAKE: L.moe_quantize_int8(src, 64, 4, 64, FAKE, 64, sc, None)  # noqa: E731
    assert quantize(src=odd) == 1 and quantize(sc=odd) == 1 and quantize(sc=half) == 1
    for M in (1, 40):
        dense = lambda x=FAKE, sc=FAKE, out=FAKE, dt=1, err=None: L.moe_linear_int8(  # noqa: E731
            x, 64, FAKE, 64, sc, M, 8, 64, out, 8, dt, FAKE, 1 << 20, err, None)
        assert dense(x=odd) == 1 and dense(sc=half) == 1 and dense(out=odd) == 1
        assert dense(out=half, dt=0) == 1 and dense(err=half) == 1
    s, n = S.c(), 1 << 22
    up = lambda w, p, err=None: L.moe_grouped_up_swiglu(FAKE, ctypes.byref(w), ctypes.byref(p), s, FAKE, FAKE, n, err, None)  # noqa: E731
    down = lambda w, p, err=None: L.moe_grouped_down(FAKE, ctypes.byref(w), ctypes.byref(p), s, FAKE, FAKE, n, err, None)  # noqa: E731
    w, p = _Weights(2, P, P, P, P, P, P), _Plan(P, P, P, P, P)
    assert up(_Weights(2, P, P, P, P + 2, P, P), p) == 1 and up(_Weights(2, P, P, P, P, P + 2, P), p) == 1
    assert down(_Weights(2, P, P, P, P, P, P + 2), p) == 1
    for bad in (_Plan(P, P, P + 2, P, P), _Plan(P, P, P, P + 2, P)):
        assert up(w, bad) == 1 and down(w, bad) == 1
    assert down(w, _Plan(P, P, P, P, P + 2)) == 1
    assert up(w, p, half) == 1 and down(w, p, half) == 1
    layer = lambda w: L.moe_layer(FAKE, FAKE, None, ctypes.byref(w), FAKE, ctypes.c_float(1e-5), s, FAKE, None, None,  # noqa: E731
                                  None, FAKE, 1 << 30, None)
    for i in range(3):
        assert layer(_Weights(2, P, P, P, *(P + 2 * (i == j) for j in range(3)))) == 1
