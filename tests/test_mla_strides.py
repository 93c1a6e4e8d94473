"""Strides of the latent-attention operators' arguments, on the CPU: what
reaches the C entry points from the binding, and what those accept."""

import ctypes

import pytest
import torch

import mxfp4_block_scaled_quant_amd as mx
from mxfp4_block_scaled_quant_amd import mla

P = ctypes.c_void_p(0x10000)
OK, SHAPE, ALIGN, DEVICE = 0, 2, 3, 5
META = torch.device("meta")


def t(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device=META)


def i32(*shape):
    return t(*shape, dtype=torch.int32)


@pytest.fixture
def entry(monkeypatch):
    """The arguments of the last call into a recording library."""
    calls = {}

    class Recorder:
        def mla_decode_workspace_bytes(self, *args):
            return 64

        def __getattr__(self, name):
            def call(*args):
                calls[name] = args
                return OK
            return call

    monkeypatch.setattr(mla, "_require_cuda", lambda tensor, name: None)
    monkeypatch.setattr(mla, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(mla, "lib", Recorder)
    return calls


def decode(table, prefix):
    B = table.shape[0]
    args = (i32(4), 50) if prefix else ()
    fn = mx.mla_decode_shared_prefix if prefix else mx.mla_decode
    fn(t(B, 1, 16, 576), t(9, 16, 576), *args, table, i32(B), 0.1)


@pytest.mark.parametrize("prefix", [False, True])
def test_the_page_tables_row_stride_reaches_the_entry(entry, prefix):
    def stride_of(table):
        decode(table, prefix)
        args = entry["mla_decode_shared_prefix" if prefix else "mla_decode"]
        at = 13 if prefix else 10         # behind the table's address; its width follows
        assert args[at + 1] == table.shape[1]
        return args[at]

    assert stride_of(i32(3, 5)) == 5
    assert stride_of(i32(3, 9)[:, :5]) == 9
    assert stride_of(i32(1, 5).expand(4, -1)) == 0
    assert stride_of(i32(1, 5).expand(70, -1)) == 0
    assert stride_of(i32(5, 1).expand(5, 1)) == 1
    # one request's stride is never used
    assert stride_of(i32(20).as_strided((1, 5), (3, 1))) == 5


@pytest.mark.parametrize("prefix", [False, True])
def test_page_table_rows_that_overlap_in_part_are_refused(entry, prefix):
    with pytest.raises(ValueError, match="block_table"):
        decode(i32(14).as_strided((4, 5), (3, 1)), prefix)
    assert "mla_decode" not in entry and "mla_decode_shared_prefix" not in entry


def decode_entry(lib, prefix=False, qb=16 * 576, qs=16 * 576, qh=576, pages=9, page=16, cp=16 * 576, cr=576, ldt=8,
                 width=8, B=2, S=1, H=16, ob=16 * 512, os=16 * 512, oh=512):
    pre = (P, 4, 4 * page) if prefix else ()
    f = lib.mla_decode_shared_prefix if prefix else lib.mla_decode
    return f(P, qb, qs, qh, P, pages, page, cp, cr, *pre, P, ldt, width, P, B, S, H, 0.1, P, ob, os, oh, P, P, 1 << 40,
             None)


@pytest.fixture
def lib():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: fake pointers must not reach a kernel")
    return mx.lib()


@pytest.mark.parametrize("prefix", [False, True])
def test_entry_takes_one_table_row_for_all_requests(lib, prefix):
    assert decode_entry(lib, prefix, ldt=0) == DEVICE
    assert decode_entry(lib, prefix, ldt=0, width=0) == DEVICE
    assert decode_entry(lib, prefix, ldt=-1) == SHAPE and decode_entry(lib, prefix, ldt=3) == SHAPE
    assert decode_entry(lib, prefix, ldt=-1, width=0) == SHAPE


@pytest.mark.parametrize("prefix", [False, True])
def test_decode_entry_ignores_strides_of_single_elements(lib, prefix):
    # a dimension of one element: its stride may be anything a view has
    for stride in (1, 3, 580, 1 << 41):
        assert decode_entry(lib, prefix, B=1, qb=stride, ob=stride) == DEVICE
        assert decode_entry(lib, prefix, S=1, qs=stride, os=stride) == DEVICE
        assert decode_entry(lib, prefix, H=1, qh=stride, oh=stride) == DEVICE
        assert decode_entry(lib, prefix, B=1, ldt=stride) == DEVICE
        assert decode_entry(lib, prefix, pages=1, cp=stride) == DEVICE
        assert decode_entry(lib, prefix, page=1, cr=stride, cp=576) == DEVICE
    # and of two is still checked
    assert decode_entry(lib, prefix, B=2, qb=580) == ALIGN and decode_entry(lib, prefix, pages=2, cp=580) == SHAPE
    assert decode_entry(lib, prefix, S=2, qs=580, ob=2 * 16 * 512) == ALIGN and decode_entry(lib, prefix, cr=1) == SHAPE


def test_append_entry_ignores_strides_of_single_elements(lib):
    def call(ldkv=576, qt=1024, qh=64, ot=1024, oh=64, pages=4, page=16, cp=16 * 576, cr=576, T=3, H=16):
        return lib.mla_cache_append(P, ldkv, P, 1e-6, P, 100, P, P, 1, P, qt, qh, P, ot, oh, P, pages, page, cp, cr, T,
                                    H, None)

    for stride in (1, 3, 580, 1 << 41):
        assert call(T=1, ldkv=stride, qt=stride, ot=stride) == DEVICE
        assert call(H=1, qh=stride, oh=stride) == DEVICE
        assert call(pages=1, cp=stride) == DEVICE and call(page=1, cr=stride, cp=576) == DEVICE
    assert call(T=2, ldkv=580) == ALIGN and call(T=2, qt=1028) == ALIGN


def test_prefill_entry_ignores_strides_of_single_elements(lib):
    def call(qt=16 * 192, qh=192, kt=2048, kh=128, pt=64, vt=2048, vh=128, H=16, Tq=5, Tk=5, ot=2048, oh=128):
        return lib.mla_prefill(P, qt, qh, P, kt, kh, P, pt, P, vt, vh, P, P, 1, H, Tq, Tk, 128, 128, 1, 0.1, P, ot, oh,
                               None, None)

    for stride in (1, 3, 580, 1 << 41):
        assert call(Tq=1, qt=stride, ot=stride) == DEVICE
        assert call(Tk=1, kt=stride, pt=stride, vt=stride) == DEVICE
        assert call(H=1, qh=stride, kh=stride, vh=stride, oh=stride) == DEVICE
    assert call(Tq=2, qt=580) == ALIGN and call(Tk=2, vt=580) == ALIGN and call(H=2, kh=580) == ALIGN
