"""The feed-forward custom ops' fake implementations (no GPU)."""

import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from mxfp4_block_scaled_quant_amd import ops  # noqa: F401  (registers torch.ops.mxfp4)


def t(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda")


def test_route_shapes():
    with FakeTensorMode():
        for dtype in (torch.float32, torch.bfloat16):
            w, ids = torch.ops.mxfp4.moe_route(t(5, 64, dtype=dtype), 6, None, "sigmoid", 8, 3)
            assert w.shape == ids.shape == (5, 6)
            assert w.dtype == torch.float32 and ids.dtype == torch.int32


def test_moe_shapes():
    u8 = torch.uint8
    with FakeTensorMode():
        for T in (0, 7):
            out = torch.ops.mxfp4.moe(t(T, 256), t(T, 2, dtype=torch.int32), t(T, 2, dtype=torch.float32),
                                      t(4096, dtype=u8), t(64, dtype=u8), t(4096, dtype=u8), t(64, dtype=u8), 4, 128,
                                      residual=t(T, 256))
            assert out.shape == (T, 256) and out.dtype == torch.bfloat16


def test_linear_act_shapes():
    with FakeTensorMode():
        w, ws = t(4096, dtype=torch.uint8), t(64, dtype=torch.uint8)
        assert torch.ops.mxfp4.linear_act(t(3, 128), w, ws, 64, None, "silu", True).shape == (3, 32)
        out = torch.ops.mxfp4.linear_act(t(3, 128), w, ws, 64, None, "gelu", residual=t(3, 64),
                                         out_dtype=torch.float32)
        assert out.shape == (3, 64) and out.dtype == torch.float32


def test_symbolic_trace_of_the_layer():
    """The three operators traced with a symbolic number of tokens."""
    u8 = torch.uint8

    def layer(x, logits, up, ups, down, downs):
        w, ids = torch.ops.mxfp4.moe_route(logits, 2)
        y = torch.ops.mxfp4.moe(x, ids, w, up, ups, down, downs, 4, 128, residual=x)
        return torch.ops.mxfp4.linear_act(y, up, ups, 256, None, "silu", True)

    from torch.fx.experimental.proxy_tensor import make_fx
    args = (torch.empty(7, 256, dtype=torch.bfloat16), torch.empty(7, 4), torch.empty(4096, dtype=u8),
            torch.empty(64, dtype=u8), torch.empty(4096, dtype=u8), torch.empty(64, dtype=u8))
    graph = make_fx(layer, tracing_mode="symbolic")(*args)
    names = [str(n.target) for n in graph.graph.nodes if n.op == "call_function"]
    for op in ("moe_route", "moe", "linear_act"):
        assert any(n.startswith(f"mxfp4.{op}.") for n in names), names
