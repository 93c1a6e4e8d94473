"""Refusals of the feed-forward operators, on the CPU: the C entry points
check every argument before any HIP call, and the binding every tensor."""

import ctypes

import pytest
import torch

import mxfp4_block_scaled_quant_amd as mx

P, P_ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10001)
OK, NULL, SHAPE, ALIGN, WORK, DEVICE, ARG = 0, 1, 2, 3, 4, 5, 7
BIG = 1 << 50


@pytest.fixture(scope="module")
def lib():
    return mx.lib()


def test_route_entry(lib):
    def call(x=P, ld=64, dt=1, bias=P, T=3, E=64, k=6, sc=0, G=8, keep=4, gt=2, rn=1, scale=1.0, w=P, ldw=6, ids=P,
             ldi=6):
        return lib.moe_route(x, ld, dt, bias, T, E, k, sc, G, keep, gt, rn, scale, w, ldw, ids, ldi, None)

    assert call(dt=2) == ARG and call(sc=2) == ARG and call(gt=0) == ARG and call(gt=3) == ARG
    for bad in (dict(T=-1), dict(E=0), dict(E=1025, ld=1025), dict(k=0), dict(k=65), dict(E=4, k=5, G=1, keep=1),
                dict(G=0), dict(G=7), dict(G=65, E=130, ld=130), dict(keep=0), dict(keep=9), dict(keep=1, k=9, ldw=9, ldi=9),
                dict(ld=63), dict(ldw=5), dict(ldi=5)):
        assert call(**bad) == SHAPE, bad
    for name in ("x", "w", "ids"):
        assert call(**{name: None}) == NULL, name
        assert call(**{name: P_ODD}) == ALIGN, name
    assert call(bias=P_ODD) == ALIGN
    assert call(T=0, x=None, w=None, ids=None) == OK
    if not torch.cuda.is_available():
        assert call() == DEVICE and call(T=1, ld=0, ldw=0, ldi=0) == DEVICE and call(bias=None, G=1, keep=1) == DEVICE


def test_moe_entry(lib):
    def call(x=P, ldx=128, ids=P, ldi=2, w=P, ldw=2, up=P, ups=P, ub=P, dn=P, dns=P, db=P, r=P, ldr=128, out=P, ldo=128,
             T=3, k=2, E=4, H=128, I=64, act=1, gated=1, ws=P, wb=BIG):
        return lib.mxfp4_moe(x, ldx, ids, ldi, w, ldw, up, ups, ub, dn, dns, db, r, ldr, out, ldo, T, k, E, H, I, act,
                             gated, ws, wb, None)

    assert call(act=-1) == ARG and call(act=5) == ARG
    for bad in (dict(T=-1), dict(k=0), dict(k=65, ldi=65, ldw=65), dict(E=0), dict(E=1025), dict(H=96 + 16),
                dict(H=0), dict(I=0), dict(I=48), dict(I=(1 << 20) + 32), dict(T=(1 << 24), k=2), dict(ldx=120),
                dict(ldi=1), dict(ldw=1), dict(ldo=124), dict(ldr=124), dict(H=1 << 16, I=1 << 16, ldx=1 << 16, ldo=1 << 16, ldr=1 << 16)):
        assert call(**bad) == SHAPE, bad
    need = lib.mxfp4_moe_workspace_bytes(3, 2, 4, 128, 64)
    assert need > 0 and call(wb=need - 1) == WORK and call(ws=None, wb=need) == NULL
    for name in ("x", "ids", "w", "up", "ups", "dn", "dns", "out"):
        assert call(**{name: None}) == NULL, name
        assert call(**{name: P_ODD}) == ALIGN, name
    for name in ("ub", "db", "r", "ws"):
        assert call(**{name: P_ODD}) == ALIGN, name
    assert call(ldx=132) == ALIGN and call(ldo=130) == ALIGN and call(ldr=130) == ALIGN
    assert call(T=0, x=None, out=None, ws=None, wb=0) == OK
    if not torch.cuda.is_available():
        assert call() == DEVICE and call(ub=None, db=None, r=None, ldr=0) == DEVICE
        assert call(T=1, ldx=0, ldi=0, ldw=0, ldo=0, ldr=0) == DEVICE
    f = lib.mxfp4_moe_workspace_bytes
    assert f(0, 2, 4, 128, 64) == 0 and f(3, 0, 4, 128, 64) == 0 and f(3, 2, 4, 100, 64) == 0


def test_linear_act_entry(lib):
    def call(x=P, ldx=128, w=P, ws=P, bias=P, act=1, gated=1, r=P, ldr=64, out=P, ldo=64, dt=0, M=3, N=128, K=128,
             work=P, wb=BIG):
        return lib.mxfp4_linear_act(x, ldx, w, ws, bias, act, gated, r, ldr, out, ldo, dt, M, N, K, work, wb, None)

    assert call(act=5) == ARG and call(act=-1) == ARG and call(dt=2) == ARG
    for bad in (dict(M=-1), dict(N=0), dict(N=144), dict(K=0), dict(K=100), dict(ldx=96), dict(ldo=60), dict(ldr=60),
                dict(gated=0, ldr=128), dict(gated=0, ldo=128), dict(K=(1 << 20) + 32, ldx=1 << 21),
                dict(ldo=1 << 30)):
        assert call(**bad) == SHAPE, bad
    for name in ("x", "w", "ws", "out"):
        assert call(**{name: None}) == NULL, name
        assert call(**{name: P_ODD}) == ALIGN, name
    assert call(bias=P_ODD) == ALIGN and call(r=P_ODD) == ALIGN and call(ldx=132) == ALIGN
    need = lib.mxfp4_linear_act_workspace_bytes(300, 128, 128)
    assert need > 0 and call(M=300, wb=need - 1) == WORK and call(M=300, work=None, wb=need) == NULL
    assert call(M=300, work=P_ODD) == ALIGN
    assert call(M=0, x=None, out=None, work=None, wb=0) == OK
    if not torch.cuda.is_available():
        assert call() == DEVICE and call(gated=0, r=None, ldr=0, ldo=128, N=128) == DEVICE
        assert call(gated=0, r=None, ldo=144, N=144) == DEVICE


def _meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype)


def test_binding_refuses_host_tensors():
    with pytest.raises(ValueError, match="device"):
        mx.moe_route(_meta(3, 8, dtype=torch.float32), 2)
    w = mx.MXFP4Weight(_meta(8, dtype=torch.uint8), _meta(8, dtype=torch.uint8), 64, 64, 2)
    with pytest.raises(ValueError, match="device"):
        mx.mxfp4_moe(_meta(3, 64), _meta(3, 2, dtype=torch.int32), _meta(3, 2, dtype=torch.float32), w, w)
    with pytest.raises(ValueError, match="device"):
        mx.mxfp4_linear_act(_meta(3, 64), w.w_pre, w.ws_pre, 64)


@pytest.mark.gpu
def test_binding_refusals():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")

    def t(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    f32, i32 = torch.float32, torch.int32
    x = t(3, 16, dtype=f32)
    for bad in (dict(logits=t(3, 16, dtype=torch.float16)), dict(logits=t(16, dtype=f32)),
                dict(logits=t(16, 3, dtype=f32).t()), dict(bias=t(15, dtype=f32)), dict(bias=t(16)),
                dict(scoring="tanh"), dict(weights=t(3, 3, dtype=f32)), dict(ids=t(3, 2, dtype=torch.int64))):
        with pytest.raises(ValueError):
            mx.moe_route(**{"logits": x, "top_k": 2, **bad})
    with pytest.raises(mx.MXFP4Error):
        mx.moe_route(x, 17)
    with pytest.raises(mx.MXFP4Error):
        mx.moe_route(x, 9, groups=2, top_groups=1)

    up, down = mx.quantize_weight(t(2, 128, 96)), mx.quantize_weight(t(2, 96, 64))
    good = dict(x=t(3, 96), ids=t(3, 2, dtype=i32), weights=t(3, 2, dtype=f32), up=up, down=down)
    assert mx.mxfp4_moe(**good).shape == (3, 96)
    for bad in (dict(x=t(3, 64)), dict(x=t(3, 96, dtype=f32)), dict(x=t(96, 3).t()), dict(ids=t(2, 2, dtype=i32)),
                dict(ids=t(3, 2, dtype=torch.int64)), dict(weights=t(3, 3, dtype=f32)), dict(weights=t(3, 2)),
                dict(up=down), dict(gated=False), dict(activation="swish"), dict(up_bias=t(2, 64)),
                dict(up_bias=t(128)), dict(down_bias=t(2, 64)), dict(residual=t(2, 96)), dict(out=t(3, 96, dtype=f32)),
                dict(workspace=t(8, dtype=torch.uint8)), dict(up_bias=t(128, 2).t())):
        with pytest.raises(ValueError):
            mx.mxfp4_moe(**{**good, **bad})

    w = mx.quantize_weight(t(144, 96))
    good = dict(x=t(3, 96), w_pre=w.w_pre, ws_pre=w.ws_pre, N=144)
    assert mx.mxfp4_linear_act(**good).shape == (3, 144)
    for bad in (dict(gated=True), dict(x=t(3, 64, 2)), dict(N=1440), dict(bias=t(72)), dict(residual=t(3, 72)),
                dict(out_dtype=torch.float16), dict(out=t(3, 144, dtype=f32)), dict(activation="tanh")):
        with pytest.raises(ValueError):
            mx.mxfp4_linear_act(**{**good, **bad})
