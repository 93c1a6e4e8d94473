"""The experts' products at the ends of their documented sizes."""

import pytest
import torch

import mxfp4_block_scaled_quant_amd as mx
from tests.helpers import need_gpu

pytestmark = pytest.mark.gpu


def test_columns_times_blocks_past_32_bits():
    """1024 experts of 2^20 inner columns: 32768 workgroups of columns for each of up to 2287 blocks, over 2^32 work
    items.  All values are powers of two and their sums integers below 256: exact in every type on the way."""
    need_gpu()
    T, k, E, H, I = 3150, 8, 1024, 32, 2 ** 20
    if torch.cuda.mem_get_info()[0] < 140 * 2 ** 30:
        pytest.skip("needs 140 GiB")
    dev = "cuda"
    one = 0x22                                                     # two codes of 1.0
    weights = []
    for N, K in ((I, H), (H, I)):
        w = torch.full((mx.weight_bytes(E, N, K),), one, dtype=torch.uint8, device=dev)
        s = torch.full((mx.weight_scale_bytes(E, N, K),), 127 if N == I else 107, dtype=torch.uint8, device=dev)
        weights.append(mx.MXFP4Weight(w, s, N, K, E))
    up, down = weights
    up.ws_pre.view(E, -1).add_((torch.arange(E, device=dev) % 3).to(torch.uint8)[:, None])   # expert e: times 2^(e % 3)
    t = torch.arange(T, device=dev)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device=dev)
    x[t, t % H] = (2.0 ** (t % 3)).bfloat16()
    ids = ((t[:, None] * k + torch.arange(k, device=dev)) % E).int()
    out = mx.mxfp4_moe(x, ids, torch.ones((T, k), device=dev), up, down, activation="none", gated=False)
    ref = 2.0 ** (t % 3) * (2.0 ** (ids % 3)).sum(1)
    assert torch.equal(out.float(), ref[:, None].expand(T, H).float())
