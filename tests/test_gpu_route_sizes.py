"""Routing of more tokens than one launch's work items hold."""

import pytest
import torch

import mxfp4_block_scaled_quant_amd as mx
from tests.helpers import need_gpu

pytestmark = pytest.mark.gpu


# 64 lanes a token: 2^32 work items at 2^26 tokens; the last slice one token
@pytest.mark.parametrize("T", [2 ** 26 + 4096, 2 ** 25 + 1])
def test_more_tokens_than_a_launch(T):
    need_gpu()
    E, k = 66, 2
    base = torch.randn(4096, E, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()
    x = base.repeat(T // 4096 + 1, 1)[:T]
    rw, rids = mx.moe_route(base, k, scoring="sigmoid")
    w, ids = mx.moe_route(x, k, scoring="sigmoid")
    n = T // 4096 * 4096
    assert (ids[:n].view(-1, 4096, k) == rids).all() and (w[:n].view(-1, 4096, k) == rw).all()
    assert torch.equal(ids[n:], rids[:T - n]) and torch.equal(w[n:], rw[:T - n])
