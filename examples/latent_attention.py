"""One latent-attention layer served with this library's operators.

A prompt is prefilled in the expanded form, its rows written to the paged
cache, and further tokens decoded in the absorbed form; then several samples
continue the prompt with its pages as a shared prefix.  Between the operators
stand the per-head MXFP4 products (a16wfp4_bmm): K-up and V-up once for the
expansion of a prompt's latents, and once absorbed into queries and outputs.

    python examples/latent_attention.py [--tokens 300] [--steps 8] [--samples 4]

prints the largest difference between each decoded token and the same token
prefilled, which are two orders of computing one formula.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mxfp4_block_scaled_quant_amd as mx  # noqa: E402

LATENT, ROPE = 512, 64


def angles(limit: int, device) -> torch.Tensor:
    """cos and sin of 32 angles per position, the table mla_cache_append reads."""
    freq = 10000.0 ** (-torch.arange(0, ROPE, 2, dtype=torch.float64, device=device) / ROPE)
    a = torch.arange(limit, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float()


class PagedLatents:
    """A page pool and the page tables of its sequences (bookkeeping on the host)."""

    def __init__(self, pages: int, page_size: int, device):
        self.rows = torch.zeros((pages, page_size, LATENT + ROPE), dtype=torch.bfloat16, device=device)
        self.page_size = page_size
        self.free = list(range(pages))[::-1]

    def grow(self, table: list, n: int) -> None:
        """Pages for n rows."""
        while len(table) * self.page_size < n:
            table.append(self.free.pop())

    def slots(self, table: list, start: int, n: int) -> torch.Tensor:
        at = torch.arange(start, start + n)
        return (torch.tensor(table)[at // self.page_size] * self.page_size + at % self.page_size).to(self.rows.device)

    def table(self, tables: list) -> torch.Tensor:
        width = max(1, max(len(t) for t in tables))
        return torch.tensor([t + [0] * (width - len(t)) for t in tables], dtype=torch.int32).to(self.rows.device)


class LatentAttention:
    """H heads of nope + 64 query values over one 512-value latent a token."""

    def __init__(self, w_uk: torch.Tensor, w_uv: torch.Tensor, norm: torch.Tensor, cos_sin: torch.Tensor):
        # w_uk [H, nope, 512]: key parts from the latent; w_uv [H, value, 512]: values from it
        self.heads, self.nope, _ = w_uk.shape
        self.value = w_uv.shape[1]
        self.expand_k = mx.quantize_weight(w_uk)                               # [H, nope, 512]
        self.absorb_k = mx.quantize_weight(w_uk.transpose(1, 2).contiguous())  # [H, 512, nope]
        self.expand_v = mx.quantize_weight(w_uv)                               # [H, value, 512]
        self.norm, self.cos_sin = norm, cos_sin
        self.scale = (self.nope + ROPE) ** -0.5

    def prefill(self, cache: PagedLatents, table: list, q: torch.Tensor, kv: torch.Tensor, start: int = 0):
        """A sequence's tokens [start, start + T): rows to the cache, then
        causal attention over the expanded keys of all start + T."""
        T, n = q.shape[0], start + q.shape[0]
        cache.grow(table, n)
        positions = torch.arange(start, n, device=q.device)
        q = q.clone()
        mx.mla_cache_append(kv, self.norm, cache.rows, cache.slots(table, start, T), positions, self.cos_sin,
                            q_pe=q[..., self.nope:], q_out=q[..., self.nope:])
        rows = cache.rows[torch.tensor(table, device=q.device)].reshape(-1, LATENT + ROPE)[:n]
        latents = rows[:, :LATENT].unsqueeze(0).expand(self.heads, -1, -1)
        k = mx.a16wfp4_bmm(latents, self.expand_k.w_pre, self.expand_k.ws_pre, self.nope, batch_major=True)
        v = mx.a16wfp4_bmm(latents, self.expand_v.w_pre, self.expand_v.ws_pre, self.value, batch_major=True)
        cu = lambda m: torch.tensor([0, m], dtype=torch.int32, device=q.device)
        return mx.mla_prefill(q, k, rows[:, LATENT:], v, cu(T), cu(n), self.scale)

    def _absorb(self, q: torch.Tensor) -> torch.Tensor:
        """[B, H, nope + 64] -> [B, H, 576], the rotated part still to be written."""
        a = torch.empty((q.shape[0], self.heads, LATENT + ROPE), dtype=torch.bfloat16, device=q.device)
        mx.a16wfp4_bmm(q[..., :self.nope].transpose(0, 1), self.absorb_k.w_pre, self.absorb_k.ws_pre, LATENT,
                       out=a[..., :LATENT].transpose(0, 1))
        return a

    def decode(self, cache: PagedLatents, tables: list, lengths: list, q: torch.Tensor, kv: torch.Tensor,
               prefix: tuple = ()):
        """One new token for each sequence (lengths count it); prefix: the
        page table and the number of rows that come before all of them."""
        dev = q.device
        before = prefix[1] if prefix else 0
        for t, n in zip(tables, lengths):
            cache.grow(t, n)
        slots = torch.cat([cache.slots(t, n - 1, 1) for t, n in zip(tables, lengths)])
        positions = torch.tensor([before + n - 1 for n in lengths], device=dev)
        a = self._absorb(q)
        mx.mla_cache_append(kv, self.norm, cache.rows, slots, positions, self.cos_sin, q_pe=q[..., self.nope:],
                            q_out=a[..., LATENT:])
        n = torch.tensor(lengths, dtype=torch.int32, device=dev)
        if prefix:
            table = torch.tensor(prefix[0], dtype=torch.int32, device=dev)
            o = mx.mla_decode_shared_prefix(a, cache.rows, table, before, cache.table(tables), n, self.scale)
        else:
            o = mx.mla_decode(a, cache.rows, cache.table(tables), n, self.scale)
        return mx.a16wfp4_bmm(o.transpose(0, 1), self.expand_v.w_pre, self.expand_v.ws_pre, self.value,
                              batch_major=True)


def demo(tokens: int = 300, steps: int = 8, samples: int = 4, heads: int = 16, nope: int = 192, value: int = 256,
         page_size: int = 64, device: str = "cuda"):
    """Runs the layer; returns the largest differences (decoded, sampled) and the largest output."""
    g = torch.Generator(device=device).manual_seed(1)
    randn = lambda *s: torch.randn(s, generator=g, device=device).to(torch.bfloat16)
    # weights on the FP4 grid, so that both orientations hold the same values
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0], device=device)
    pick = lambda *s: (grid[torch.randint(0, 6, s, generator=g, device=device)]
                       * (torch.randint(0, 2, s, generator=g, device=device) * 2 - 1) / 32).to(torch.bfloat16)
    total = tokens + steps
    layer = LatentAttention(pick(heads, nope, LATENT), pick(heads, value, LATENT), torch.ones_like(randn(LATENT)),
                            angles(total + 8, device))
    q, kv = randn(total, heads, nope + ROPE), randn(total, LATENT + ROPE)

    whole_cache, whole = PagedLatents(-(-total // page_size) + 1, page_size, device), []
    want = layer.prefill(whole_cache, whole, q, kv).float()

    cache = PagedLatents(-(-total // page_size) + 2 * samples + 2, page_size, device)
    table: list = []
    first = layer.prefill(cache, table, q[:tokens], kv[:tokens]).float()
    off = [(first - want[:tokens]).abs().max().item()]
    for i in range(tokens, total):
        o = layer.decode(cache, [table], [i + 1], q[i:i + 1], kv[i:i + 1]).float()
        off.append((o[0] - want[i]).abs().max().item())

    # samples that continue the same prompt: its pages are read once for all
    prompt, own = table[:-(-tokens // page_size)], [[] for _ in range(samples)]
    sampled = []
    for i in range(steps):
        qs = q[tokens + i:tokens + i + 1].expand(samples, -1, -1).contiguous()
        ks = kv[tokens + i:tokens + i + 1].expand(samples, -1).contiguous()
        o = layer.decode(cache, own, [i + 1] * samples, qs, ks, prefix=(prompt, tokens)).float()
        sampled.append((o - want[tokens + i]).abs().max().item())
    torch.cuda.synchronize()
    return max(off), max(sampled), want.abs().max().item()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=300)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--samples", type=int, default=4)
    args = ap.parse_args()
    decoded, sampled, top = demo(args.tokens, args.steps, args.samples)
    print(f"outputs up to {top:.3g}; decoded tokens off by {decoded:.3g}, sampled ones by {sampled:.3g} at most")
