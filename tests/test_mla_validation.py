"""Refusals of the latent-attention operators, on the CPU: the C entry points
check every argument before any HIP call, and the binding every tensor."""

import ctypes

import pytest
import torch

import mxfp4_block_scaled_quant_amd as mx
from mxfp4_block_scaled_quant_amd import mla

P, P_ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004)
OK, NULL, SHAPE, ALIGN, WORK, DEVICE, ARG = 0, 1, 2, 3, 4, 5, 7


@pytest.fixture(scope="module")
def lib():
    return mx.lib()


def _no_gpu():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: fake pointers must not reach a kernel")


def test_append_entry(lib):
    def call(kv=P, ldkv=576, w=P, eps=1e-6, cs=P, limit=100, pos=P, slots=P, inter=1, q=P, qt=1024, qh=64, o=P,
             ot=1024, oh=64, cache=P, pages=4, page=16, cp=16 * 576, cr=576, T=3, H=16):
        return lib.mla_cache_append(kv, ldkv, w, eps, cs, limit, pos, slots, inter, q, qt, qh, o, ot, oh, cache,
                                    pages, page, cp, cr, T, H, None)

    assert call(inter=2) == ARG and call(eps=-1.0) == ARG and call(eps=float("nan")) == ARG
    assert call(T=-1) == SHAPE and call(H=-1) == SHAPE and call(limit=-1) == SHAPE
    assert call(ldkv=568) == SHAPE
    assert call(page=0) == SHAPE and call(cr=568) == SHAPE and call(cp=15 * 576) == SHAPE
    assert call(oh=32) == SHAPE and call(ot=512) == SHAPE             # heads / tokens on top of each other
    assert call(q=None) == NULL and call(o=None) == NULL
    for name in ("kv", "w", "cs", "pos", "slots", "cache"):
        assert call(**{name: None}) == NULL, name
    for name in ("kv", "w", "cs", "pos", "slots", "cache", "q", "o"):
        assert call(**{name: P_ODD}) == ALIGN, name
    assert call(ldkv=580) == ALIGN and call(qt=1028) == ALIGN and call(cr=580, cp=16 * 580) == ALIGN
    assert call(T=0, kv=None, slots=None) == OK
    if not torch.cuda.is_available():
        assert call() == DEVICE and call(q=None, o=None, H=0) == DEVICE


def test_decode_entry(lib):
    big = 1 << 40

    def call(prefix=False, q=P, qb=16 * 576, qs=16 * 576, qh=576, cache=P, pages=9, page=16, cp=16 * 576, cr=576,
             pt=P, pp=4, pn=50, table=P, ldt=8, width=8, lens=P, B=2, S=1, H=16, scale=0.1, out=P, ob=16 * 512,
             os=16 * 512, oh=512, lse=P, ws=P, wb=big):
        pre = (pt, pp, pn) if prefix else ()
        f = lib.mla_decode_shared_prefix if prefix else lib.mla_decode
        return f(q, qb, qs, qh, cache, pages, page, cp, cr, *pre, table, ldt, width, lens, B, S, H, scale, out, ob,
                 os, oh, lse, ws, wb, None)

    for prefix in (False, True):
        c = lambda **kw: call(prefix, **kw)
        for bad in (0.0, -1.0, float("nan"), float("inf")):
            assert c(scale=bad) == ARG
        assert c(B=-1) == SHAPE and c(S=0) == SHAPE and c(H=0) == SHAPE and c(width=-1) == SHAPE
        assert c(B=1 << 23) == SHAPE and c(S=1 << 22) == SHAPE
        assert c(width=1 << 28, ldt=1 << 28) == SHAPE                  # more rows than 2^30
        assert c(ldt=7) == SHAPE and c(page=0) == SHAPE and c(cr=560) == SHAPE and c(cp=100) == SHAPE
        assert c(oh=256) == SHAPE and c(ob=512) == SHAPE and c(qh=-8) == SHAPE
        for name in ("q", "cache", "table", "lens", "out"):
            assert c(**{name: None}) == NULL, name
        for name in ("q", "cache", "out"):
            assert c(**{name: P_ODD}) == ALIGN, name
        assert c(table=ctypes.c_void_p(0x10002)) == ALIGN and c(qh=580) == ALIGN and c(oh=516, ob=16 * 516) == ALIGN
        need = lib.mla_decode_workspace_bytes(2, 1, 16, 128, 50 if prefix else 0)
        assert need > 0 and c(wb=need - 1) == WORK and c(ws=None) == NULL and c(ws=P_ODD) == ALIGN
        assert c(B=0, q=None, out=None) == OK
        if not torch.cuda.is_available():
            assert c(wb=need) == DEVICE and c(lse=None) == DEVICE and c(width=0, table=None) == DEVICE
    assert call(True, pn=-1) == SHAPE and call(True, pn=65) == SHAPE    # longer than its pages
    assert call(True, pt=None) == NULL and call(True, pt=ctypes.c_void_p(0x10002)) == ALIGN
    if not torch.cuda.is_available():
        assert call(True, pn=0, pp=0, pt=None) == DEVICE


def test_workspace_query(lib):
    f = mx.mla_decode_workspace_bytes
    assert f(0, 1, 16, 100) == 0 and f(1, 0, 16, 100) == 0 and f(1, 1, 16, -1) == 0
    # two parts of 16 query rows x (512 + 4) fp32 a workgroup, one workgroup per 128 keys up to 256
    assert f(1, 1, 16, 128) == 2 * 16 * 516 * 4
    assert f(128, 1, 16, 16384) == 256 * 2 * 16 * 516 * 4
    assert f(4, 1, 16, 4096, 1000) > f(4, 1, 16, 4096)


def test_rows_hook(lib):
    for bad in (-1, 8, 64, 256):
        assert lib.mla_testing_set_rows(bad) == ARG
    sizes = {}
    for rows in (16, 32, 128, 0):
        assert lib.mla_testing_set_rows(rows) == OK
        sizes[rows] = mx.mla_decode_workspace_bytes(1, 1, 128, 64000)
    assert sizes[16] < sizes[32] < sizes[128] == sizes[0]     # long, many rows: blocks of 128


def test_prefill_rows_hook(lib):
    for bad in (-1, 16, 64, 256):
        assert lib.mla_testing_set_prefill_rows(bad) == ARG
    for rows in (32, 128, 0):
        assert lib.mla_testing_set_prefill_rows(rows) == OK


def test_prefill_entry(lib):
    def call(q=P, qt=16 * 192, qh=192, k=P, kt=2048, kh=128, pe=P, pt=64, v=P, vt=2048, vh=128, cq=P, ck=P, B=1,
             H=16, Tq=5, Tk=5, dn=128, dv=128, causal=1, scale=0.1, out=P, ot=2048, oh=128, lse=None):
        return lib.mla_prefill(q, qt, qh, k, kt, kh, pe, pt, v, vt, vh, cq, ck, B, H, Tq, Tk, dn, dv, causal, scale,
                               out, ot, oh, lse, None)

    assert call(scale=0.0) == ARG and call(causal=2) == ARG
    assert call(dn=192) == SHAPE and call(dn=64) == SHAPE
    assert call(B=-1) == SHAPE and call(H=0) == SHAPE and call(Tq=-1) == SHAPE and call(Tk=-1) == SHAPE
    assert call(kt=1 << 25) == SHAPE and call(vt=1 << 25) == SHAPE and call(qt=-8) == SHAPE
    assert call(oh=64) == SHAPE and call(ot=128) == SHAPE
    for name in ("q", "k", "pe", "v", "cq", "ck", "out"):
        assert call(**{name: None}) == NULL, name
    for name in ("q", "k", "pe", "v", "out"):
        assert call(**{name: P_ODD}) == ALIGN, name
    assert call(qh=196) == ALIGN and call(pt=68) == ALIGN and call(cq=ctypes.c_void_p(0x10002)) == ALIGN
    assert call(Tq=0, q=None, out=None) == OK and call(B=0, q=None) == OK
    if not torch.cuda.is_available():
        assert call() == DEVICE and call(Tk=0, k=None, pe=None, v=None) == DEVICE


# ---- the binding, with meta tensors

META = torch.device("meta")


@pytest.fixture
def meta(monkeypatch):
    monkeypatch.setattr(mla, "_require_cuda", lambda t, name: None)


def t(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device=META)


def i32(*shape):
    return t(*shape, dtype=torch.int32)


def i64(*shape):
    return t(*shape, dtype=torch.int64)


def _raises(fn, *a, **kw):
    with pytest.raises(ValueError):
        fn(*a, **kw)


def test_host_tensors_are_refused():
    with pytest.raises(ValueError):
        mx.mla_decode(torch.empty(1, 1, 16, 576, dtype=torch.bfloat16), None, None, None, 0.1)


def test_decode_binding(meta):
    good = dict(q=t(2, 1, 16, 576), cache=t(9, 16, 576), block_table=i32(2, 8), lengths=i32(2), scale=0.1)

    def bad(**kw):
        _raises(mx.mla_decode, **{**good, **kw})

    bad(q=t(2, 1, 16, 512))
    bad(q=t(2, 1, 16, 576, dtype=torch.float16))
    bad(q=t(16, 576))
    bad(q=t(2, 1, 16, 1152)[..., ::2])
    bad(cache=t(9, 16, 512))
    bad(cache=t(9, 16, 576, dtype=torch.float32))
    bad(block_table=i64(2, 8))
    bad(block_table=i32(3, 8))
    bad(block_table=i32(2, 16)[:, ::2])
    bad(lengths=i32(3))
    bad(lengths=i32(4)[::2])
    bad(out=t(2, 1, 16, 576))
    bad(out=t(2, 1, 16, 512, dtype=torch.float32))
    bad(lse=t(2, 1, 16))
    bad(lse=t(2, 1, 32, dtype=torch.float32)[..., ::2])
    bad(workspace=t(16, dtype=torch.uint8))
    prefix = dict(good, prefix_table=i32(4), prefix_len=50)
    _raises(mx.mla_decode_shared_prefix, **{**prefix, "prefix_len": 65})
    _raises(mx.mla_decode_shared_prefix, **{**prefix, "prefix_len": -1})
    _raises(mx.mla_decode_shared_prefix, **{**prefix, "prefix_table": i64(4)})
    _raises(mx.mla_decode_shared_prefix, **{**prefix, "prefix_table": i32(8)[::2]})


def test_prefill_binding(meta):
    good = dict(q=t(5, 16, 192), k_nope=t(7, 16, 128), k_pe=t(7, 64), v=t(7, 16, 128), cu_q=i32(3), cu_k=i32(3),
                scale=0.1)

    def bad(**kw):
        _raises(mx.mla_prefill, **{**good, **kw})

    bad(q=t(5, 16, 256))
    bad(q=t(5, 8, 192))
    bad(k_nope=t(6, 16, 128))
    bad(k_pe=t(7, 32))
    bad(v=t(7, 16, 64))
    bad(v=t(7, 16, 256))
    bad(cu_q=i64(3))
    bad(cu_q=i32(0))
    bad(cu_k=i32(4))
    bad(cu_q=i32(6)[::2])
    bad(out=t(5, 16, 256))
    bad(lse=t(5, 8, dtype=torch.float32))


def test_append_binding(meta):
    good = dict(kv=t(5, 576), norm_weight=t(512), cache=t(4, 16, 576), slots=i64(5), positions=i64(5),
                cos_sin=t(100, 64, dtype=torch.float32), q_pe=t(5, 16, 64), q_out=t(5, 16, 64))

    def bad(**kw):
        _raises(mx.mla_cache_append, **{**good, **kw})

    bad(kv=t(5, 512))
    bad(norm_weight=t(512, dtype=torch.float32))
    bad(cache=t(4, 16, 512))
    bad(slots=i32(5))
    bad(slots=i64(4))
    bad(positions=i64(10)[::2])
    bad(cos_sin=t(100, 64))
    bad(cos_sin=t(100, 128, dtype=torch.float32)[:, :64])
    bad(q_pe=t(5, 16, 32))
    bad(q_out=t(5, 8, 64))
    bad(q_pe=None)
