"""GPU parity of the latent-attention operators against the fp64 oracle.

Tolerances, from what the kernels round.  Scores: products of bf16 values are
exact in fp32 and their sums are held to the library's accumulation bar,
2^-18 of sum |q k|; scaled, that is an error ez = 2^-18 E of a score, and a
relative error of 2 ez at most of a probability over its sum.  Probabilities
are rounded to bf16 once: 2^-8 each, so 2^-8 A of an output, A = sum p |v|.
The output is rounded to bf16 once: 2^-8 of its value.  The remaining fp32
steps (exp2, sums over keys, joins) stay below 2^-16 A.  The log-sum-exp
has only ez and fp32 rounding.
"""

import numpy as np
import pytest
import torch

import mxfp4_block_scaled_quant_amd as mx
from oracle import attention as A
from tests.helpers import host_bf16_bits, need_gpu

pytestmark = pytest.mark.gpu

BF = 2.0 ** -8


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def randn(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def bits(t):
    return host_bf16_bits(t.contiguous())


def check(got, lse, want):
    out, ref_lse, mag, top = want
    y = got.float().cpu().numpy().astype(np.float64)
    ez = 2.0 ** -18 * top[..., None]
    tol = (BF * 1.01 + 2.0 ** -16 + 2 * ez) * mag
    tol = tol + BF * (np.abs(out) + tol)
    assert np.isfinite(y).all(), "non-finite output"
    worst = np.max(np.abs(y - out) - tol)
    assert worst <= 0, f"output off by {worst:.3g} more than its tolerance"
    e = lse.cpu().numpy().astype(np.float64)
    empty = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(e), empty)
    off = np.abs(e[~empty] - ref_lse[~empty])
    assert np.all(off <= ez[..., 0][~empty] + 2.0 ** -20 * (1 + np.abs(ref_lse[~empty]))), f"lse off by {off.max():.3g}"
    assert np.all(y[empty] == 0)


def paged(seed, lens, page, spare=2, extra_width=0):
    """A shuffled page table over a cache with just enough pages."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    ids = rng.permutation(sum(need) + spare)
    width = max(1, max(need, default=1)) + extra_width
    table = np.zeros((len(lens), width), np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = ids[at:at + k]
        at += k
    return randn(seed, len(ids), page, 576), table


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


DECODE = [
    # B lengths, S, H, page
    ([1], 1, 16, 64),
    ([0], 1, 16, 16),
    ([777], 1, 16, 64),
    ([31, 32, 33, 0, 128, 129, 1], 1, 16, 16),
    ([5, 300, 64], 1, 1, 1),
    ([95, 257], 1, 5, 48),
    ([40, 130, 2], 2, 8, 64),
    ([2, 1, 3, 500], 3, 5, 16),           # a request shorter than its tokens
    ([70, 0, 260], 1, 32, 64),
    ([65, 129], 2, 16, 128),
    ([33, 200], 1, 20, 1),
    ([64, 65, 1], 1, 64, 64),
    ([190, 3], 4, 16, 16),
    ([150, 0, 321], 1, 128, 64),
    ([3, 97], 4, 20, 48),
    ([257], 4, 128, 16),
    ([1700], 3, 3, 7),
]


@pytest.mark.parametrize("lens,S,H,page", DECODE)
def test_decode(lens, S, H, page):
    B = len(lens)
    cache, table = paged(B * 7 + S + H, lens, page)
    q = randn(H, B, S, H, 576)
    out, lse = mx.mla_decode(q, cache, ints(table), ints(lens), 0.0625, return_lse=True)
    again = mx.mla_decode(q, cache, ints(table), ints(lens), 0.0625)
    torch.cuda.synchronize()
    check(out, lse, A.decode(bits(q), bits(cache), table, lens, 0.0625))
    assert torch.equal(out, again)


def _exact_on_gpu(q, rows, scale):
    """fp64 reference on the GPU for one request seen whole: (out, lse, A, E)."""
    k = rows.double()
    qq = q.double().reshape(-1, 576)
    z = torch.mm(qq, k.t().contiguous()) * scale
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    top = (torch.mm(qq.abs(), k.abs().t().contiguous()) * scale).amax(1)
    return [x.cpu().numpy() for x in (torch.mm(p, k[:, :512]), lse, torch.mm(p, k[:, :512].abs()), top)]


@pytest.mark.parametrize("B,H,n,page", [(1, 16, 40001, 64), (3, 16, 9000, 16), (2, 32, 20011, 64), (2, 64, 5003, 1),
                                        (1, 128, 12345, 64), (40, 16, 700, 48)])
def test_decode_long(B, H, n, page):
    lens = [n - 13 * i for i in range(B)]
    cache, table = paged(n, lens, page)
    q = randn(H + 1, B, 1, H, 576)
    t = ints(table)
    out, lse = mx.mla_decode(q, cache, t, ints(lens), 0.05, return_lse=True)
    for b in sorted({0, B // 2, B - 1}):
        rows = cache[t[b].long()].reshape(-1, 576)[:lens[b]]
        check(out[b, 0], lse[b, 0], _exact_on_gpu(q[b, 0], rows, 0.05))


def test_decode_peaked_scores():
    # scores far apart: the running maximum moves by more than its lag
    lens = [300, 1000]
    cache, table = paged(3, lens, 16)
    q = randn(5, 2, 1, 16, 576, scale=3.0)
    out, lse = mx.mla_decode(q, cache, ints(table), ints(lens), 1.0, return_lse=True)
    check(out, lse, A.decode(bits(q), bits(cache), table, lens, 1.0))


@pytest.mark.parametrize("H", [16, 32, 64, 128])
def test_decode_masked_slots_hold_anything(H):
    # unused slots of the last page and unused pages hold NaN and infinities;
    # page numbers outside the cache hide their rows
    lens = [37, 16, 75]
    cache, table = paged(11, lens, 16, extra_width=2)
    used = torch.zeros(cache.shape[:2], dtype=torch.bool)
    for b, n in enumerate(lens):
        for t in range(n):
            used[table[b, t // 16], t % 16] = True
    poison = torch.where(torch.arange(576, device="cuda") % 2 == 0, float("nan"), float("inf")).to(torch.bfloat16)
    cache[~used.cuda()] = poison
    table[:, -2:] = 2 ** 31 - 1
    table[2, 1] = -5
    table[1, 0] = cache.shape[0]          # all of request 1
    q = randn(2, 3, 2, H // 2, 576)
    out, lse = mx.mla_decode(q, cache, ints(table), ints(lens), 0.0625, return_lse=True)
    clean = cache.clone()
    clean[~used.cuda()] = 0
    check(out, lse, A.decode(bits(q), bits(clean), table, lens, 0.0625))


def test_decode_lengths_are_clamped():
    cache, table = paged(4, [64, 64], 16)
    q = randn(4, 2, 1, 16, 576)
    out, lse = mx.mla_decode(q, cache, ints(table), ints([1000, -3]), 0.0625, return_lse=True)
    check(out, lse, A.decode(bits(q), bits(cache), table, [64, 0], 0.0625))


def test_decode_strides_and_three_dimensional_query():
    lens = [70, 33]
    cache, table = paged(6, lens, 16)
    wide = torch.zeros((cache.shape[0], 20, 640), dtype=torch.bfloat16, device="cuda")
    wide[:, :16, :576] = cache
    q = randn(6, 8, 2, 600)[..., :576].transpose(0, 1)      # [2, 8, 576], heads outermost
    out = torch.zeros((8, 2, 520), dtype=torch.bfloat16, device="cuda")[..., :512].transpose(0, 1)
    t = torch.zeros((2, 31), dtype=torch.int32, device="cuda")[:, :table.shape[1]]
    t.copy_(ints(table))
    got, lse = mx.mla_decode(q, wide[:, :16, :576], t, ints(lens), 0.0625, return_lse=True, out=out)
    assert got.data_ptr() == out.data_ptr() and got.shape == (2, 8, 512) and lse.shape == (2, 8)
    want = A.decode(bits(q)[:, None], bits(cache), table, lens, 0.0625)
    check(got, lse, [w[:, 0] for w in want])


def test_decode_cache_past_32_bit_offsets():
    pages = 60000                                            # 64 * 1152 bytes each: 4.4 GB
    cache = torch.zeros((pages, 64, 576), dtype=torch.bfloat16, device="cuda")
    ids = [pages - 1, 3, pages - 2, pages // 2]
    cache[ids] = randn(8, 4, 64, 576)
    table = np.array([[0, 1, 2, 3]])
    q = randn(9, 1, 1, 16, 576)
    for H in (16, 5):
        out, lse = mx.mla_decode(q[:, :, :H], cache, ints([ids]), ints([250]), 0.0625, return_lse=True)
        check(out, lse, A.decode(bits(q[:, :, :H]), bits(cache[ids]), table, [250], 0.0625))


PREFIX = [
    # prefix, lengths, S, H, page
    (50, [3, 1], 1, 4, 16),
    (1, [1], 1, 1, 1),
    (129, [0, 40, 7], 1, 16, 16),         # a request without rows of its own
    (300, [33, 2, 64, 1, 9], 1, 16, 48),
    (257, [5, 70, 4], 2, 20, 64),
    (0, [5, 70], 1, 16, 64),
    (200, [2, 9], 3, 64, 16),
    (95, [1, 1], 2, 16, 7),               # a token that sees the prefix alone
]


@pytest.mark.parametrize("prefix,lens,S,H,page", PREFIX)
def test_decode_shared_prefix(prefix, lens, S, H, page):
    B = len(lens)
    cache, table = paged(prefix + H, list(lens) + [prefix], page)
    k = -(-prefix // page)
    ptab, table = table[-1, :max(k, 1)].copy(), table[:-1]
    q = randn(H, B, S, H, 576)
    out, lse = mx.mla_decode_shared_prefix(q, cache, ints(ptab), prefix, ints(table), ints(lens), 0.0625,
                                           return_lse=True)
    again = mx.mla_decode_shared_prefix(q, cache, ints(ptab), prefix, ints(table), ints(lens), 0.0625)
    # tokens past a request's own rows see the whole prefix and nothing else
    want = A.decode(bits(q), bits(cache), table, lens, 0.0625, ptab, prefix)
    check(out, lse, want)
    assert torch.equal(out, again)


def test_decode_shared_prefix_long():
    B, prefix = 24, 6001
    lens = [1 + 37 * i for i in range(B)]
    cache, table = paged(77, lens + [prefix], 64)
    ptab, t = ints(table[-1]), ints(table[:-1])
    q = randn(78, B, 1, 16, 576)
    out, lse = mx.mla_decode_shared_prefix(q, cache, ptab, prefix, t, ints(lens), 0.05, return_lse=True)
    shared = cache[ptab.long()].reshape(-1, 576)[:prefix]
    for b in (0, 11, 23):
        rows = torch.cat([shared, cache[t[b].long()].reshape(-1, 576)[:lens[b]]])
        check(out[b, 0], lse[b, 0], _exact_on_gpu(q[b, 0], rows, 0.05))


@pytest.mark.parametrize("prefix", [0, 2900])
def test_many_rows_whose_parts_single_waves_join(prefix):
    lens = [(53 * i) % 300 for i in range(149)]           # 149 requests of 17 heads: an odd number of rows
    lens[7], lens[40] = 30011, 0                          # one request spread over many workgroups, one empty
    cache, table = paged(55, lens + [prefix], 64)
    ptab, t = ints(table[-1, :max(-(-prefix // 64), 1)]), ints(table[:-1])
    q = randn(56, 149, 1, 17, 576)
    args = (ptab, prefix) if prefix else ()
    f = mx.mla_decode_shared_prefix if prefix else mx.mla_decode
    out, lse = f(q, cache, *args, t, ints(lens), 0.05, return_lse=True)
    assert torch.equal(out, f(q, cache, *args, t, ints(lens), 0.05))
    shared = cache[ptab.long()].reshape(-1, 576)[:prefix]
    for b in (0, 1, 7, 39, 41, 100, 147, 148):
        rows = torch.cat([shared, cache[t[b].long()].reshape(-1, 576)[:lens[b]]])
        if len(rows):
            check(out[b, 0], lse[b, 0], _exact_on_gpu(q[b, 0], rows, 0.05))
    if not prefix:
        assert not out[[0, 40]].any() and (lse[[0, 40]] == float("-inf")).all()
    else:
        check(out[40, 0], lse[40, 0], _exact_on_gpu(q[40, 0], shared, 0.05))


def cu(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


PREFILL = [
    # queries, keys, H, dn, dv, causal
    ([1], [1], 1, 128, 128, True),
    ([33], [33], 3, 128, 128, True),
    ([130], [130], 2, 192, 256, True),
    ([64, 0, 7, 129], [64, 5, 7, 129], 2, 192, 256, True),
    ([20, 31], [75, 160], 3, 128, 128, True),          # chunks over what came before
    ([1, 1, 1], [1, 32, 70], 16, 192, 256, True),
    ([40, 5], [33, 0], 2, 128, 128, True),             # more queries than keys: rows that see nothing
    ([40, 5], [33, 0], 2, 192, 256, False),
    ([100], [45], 5, 128, 128, False),
    ([260], [300], 1, 192, 256, True),
]


@pytest.fixture(params=[32, 128])
def prefill_rows(request):
    mx.set_mla_prefill_rows(request.param)
    yield request.param
    mx.set_mla_prefill_rows(0)


@pytest.mark.parametrize("nq,nk,H,dn,dv,causal", PREFILL)
def test_prefill(nq, nk, H, dn, dv, causal, prefill_rows):
    Tq, Tk = sum(nq), sum(nk)
    q, kn, kp, v = randn(1, Tq, H, dn + 64), randn(2, Tk, H, dn), randn(3, Tk, 64), randn(4, Tk, H, dv)
    out, lse = mx.mla_prefill(q, kn, kp, v, ints(cu(nq)), ints(cu(nk)), 0.09, causal=causal, return_lse=True)
    again = mx.mla_prefill(q, kn, kp, v, ints(cu(nq)), ints(cu(nk)), 0.09, causal=causal)
    check(out, lse, A.prefill(bits(q), bits(kn), bits(kp), bits(v), cu(nq), cu(nk), 0.09, causal))
    assert torch.equal(out, again)


def _prefill_on_gpu(q, kn, kp, v, scale, past):
    """fp64 on the GPU, one sequence: queries after `past` keys."""
    res = []
    n, H = q.shape[:2]
    for h in range(H):
        k = torch.cat([kn[:, h], kp], 1).double()
        z = torch.mm(q[:, h].double(), k.t().contiguous()) * scale
        top = torch.mm(q[:, h].double().abs(), k.abs().t().contiguous()) * scale
        hide = torch.ones_like(z).triu(past + 1).bool()
        z = z.masked_fill(hide, float("-inf"))
        lse = torch.logsumexp(z, 1)
        p = torch.exp(z - lse[:, None])
        vv = v[:, h].double()
        res.append((torch.mm(p, vv), lse, torch.mm(p, vv.abs()), top.masked_fill(hide, 0).amax(1)))
    return [torch.stack(x, 1).cpu().numpy() for x in zip(*res)]


@pytest.mark.parametrize("n,past,H,dn,dv", [(1000, 0, 3, 128, 128), (777, 1500, 2, 192, 256), (2049, 0, 9, 192, 256),
                                            (513, 3000, 16, 128, 128)])
def test_prefill_long(n, past, H, dn, dv, prefill_rows):
    q, kn, kp, v = randn(1, n, H, dn + 64), randn(2, n + past, H, dn), randn(3, n + past, 64), randn(4, n + past, H, dv)
    out, lse = mx.mla_prefill(q, kn, kp, v, ints([0, n]), ints([0, n + past]), 0.08, return_lse=True)
    check(out, lse, _prefill_on_gpu(q, kn, kp, v, 0.08, past))


def test_prefill_many_sequences(prefill_rows):
    nq = [(7 * i) % 50 for i in range(150)]              # more sequences than one scan step of the block search
    T, H = sum(nq), 2
    q, kn, kp, v = randn(1, T, H, 192), randn(2, T, H, 128), randn(3, T, 64), randn(4, T, H, 128)
    out, lse = mx.mla_prefill(q, kn, kp, v, ints(cu(nq)), ints(cu(nq)), 0.09, return_lse=True)
    check(out, lse, A.prefill(bits(q), bits(kn), bits(kp), bits(v), cu(nq), cu(nq), 0.09))


@pytest.mark.parametrize("dn,dv", [(128, 128), (192, 256)])
def test_prefill_strides_and_neighbours(dn, dv, prefill_rows):
    # projections' layouts: keys and values interleaved in one tensor, heads
    # outside tokens; what lies behind a sequence's keys must not matter
    n, nk, H = 45, 83, 3
    q = randn(1, H, n, dn + 64).transpose(0, 1)
    kvx = randn(2, nk + 40, H, dn + dv)
    kn, v = kvx[:, :, :dn], kvx[:, :, dn:]
    kp = randn(3, nk + 40, 576)[:, 512:]
    out = torch.zeros((H, n, dv), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    kvx[nk:] = float("nan")
    got, lse = mx.mla_prefill(q, kn, kp, v, ints([0, n]), ints([0, nk]), 0.09, return_lse=True, out=out)
    check(got, lse, A.prefill(bits(q), bits(kn[:nk]), bits(kp[:nk]), bits(v[:nk]), [0, n], [0, nk], 0.09))


def _angles(limit):
    f = 10000.0 ** (-np.arange(32) / 32)
    a = np.arange(limit)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def _check_append(got, want, parts):
    """One bf16 rounding of an fp32 result: the norm's 512-term sum and the
    two-term rotations stay within 2^-18 of their terms' magnitudes."""
    tol = BF * np.abs(want) * (1 + 2.0 ** -10) + 2.0 ** -18 * parts
    off = np.abs(got.float().cpu().numpy().astype(np.float64) - want) - tol
    assert np.max(off) <= 0, f"off by {np.max(off):.3g} more than its tolerance"


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("T,H,page", [(1, 16, 64), (5, 1, 1), (37, 5, 48), (300, 32, 16), (64, 0, 64), (9, 17, 7)])
def test_cache_append(T, H, page, interleaved):
    rng = np.random.default_rng(T + H)
    pages = -(-T // page) + 2
    cs = _angles(5000)
    pos = rng.integers(0, 5000, T)
    slots = rng.permutation(pages * page)[:T]
    pad = rng.random(T) < 0.2
    slots[pad] = np.where(rng.random(pad.sum()) < 0.5, -1, pages * page + 3)
    kv, w = randn(1, T, 600)[:, :576], randn(2, 512)
    cache = randn(3, pages, page, 576)
    before = bits(cache).copy()
    q = randn(4, T, max(H, 1), 256)[..., 192:]
    absorbed = randn(5, T, max(H, 1), 576)
    kept = bits(absorbed).copy()
    dev = lambda x: torch.tensor(x, device="cuda")
    args = dict(q_pe=q, q_out=absorbed[..., 512:]) if H else {}
    mx.mla_cache_append(kv, w, cache, dev(slots), dev(pos), dev(cs), eps=1e-5, interleaved=interleaved, **args)
    rows = A.cache_rows(bits(kv), bits(w), cs, pos, 1e-5, interleaved)
    k64 = A.f64(bits(kv))[:, 512:]
    parts = np.concatenate([np.abs(rows[:, :512]), np.abs(k64) + np.abs(A.rotate(k64, np.zeros((T, 32)), np.ones((T, 32)),
                                                                               interleaved))], 1)
    flat = cache.reshape(-1, 576)
    _check_append(flat[dev(slots[~pad])], rows[~pad], parts[~pad])
    rest = np.setdiff1d(np.arange(pages * page), slots[~pad])
    assert np.array_equal(bits(flat)[rest], before.reshape(-1, 576)[rest])
    if H:
        a = cs.astype(np.float64)[pos][:, None]
        q64 = A.f64(bits(q))
        want = A.rotate(q64, a[..., :32], a[..., 32:], interleaved)
        other = A.rotate(q64, np.zeros((1, 1, 32)), np.ones((1, 1, 32)), interleaved)
        _check_append(absorbed[..., 512:], want, np.abs(q64) + np.abs(other))
        assert np.array_equal(bits(absorbed)[..., :512], kept[..., :512])


def test_cache_append_position_outside_the_table_writes_nothing():
    cs = torch.tensor(_angles(10), device="cuda")
    kv, w, q = randn(1, 3, 576), randn(2, 512), randn(4, 3, 2, 64)
    cache = torch.zeros((1, 4, 576), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    i64 = lambda x: torch.tensor(x, device="cuda")
    mx.mla_cache_append(kv, w, cache, i64([0, 1, 2]), i64([-1, 3, 10]), cs, q_pe=q, q_out=out)
    assert not cache[0, [0, 2, 3]].any() and cache[0, 1].any()
    assert not out[[0, 2]].any() and out[1].any()


def test_cache_append_in_place_and_far_slots():
    cs = torch.tensor(_angles(100), device="cuda")
    pages = 60000
    cache = torch.zeros((pages, 64, 576), dtype=torch.bfloat16, device="cuda")
    kv, w, q = randn(1, 2, 576), randn(2, 512), randn(4, 2, 16, 64)
    i64 = lambda x: torch.tensor(x, device="cuda")
    slots, pos = i64([pages * 64 - 1, 5]), i64([99, 1])
    want = mx.mla_cache_append(kv, w, cache, slots, pos, cs, q_pe=q)
    got = mx.mla_cache_append(kv, w, cache, slots, pos, cs, q_pe=q, q_out=q)
    assert got is q and torch.equal(q, want)
    rows = A.cache_rows(bits(kv), bits(w), cs.cpu().numpy(), [99, 1], 1e-6, True)
    _check_append(torch.stack([cache[-1, -1], cache[0, 5]])[:, :512], rows[:, :512], np.abs(rows[:, :512]))


def test_streams_and_graph_follow_new_lengths():
    # one decode step captured, replayed for growing requests, against eager calls
    lens = [100, 37, 0, 64]
    cache, table = paged(21, [n + 40 for n in lens], 16)
    t, n = ints(table), ints(lens)
    q = randn(3, 4, 1, 16, 576)
    kv, w, cs = randn(5, 4, 576), randn(6, 512), torch.tensor(_angles(400), device="cuda")
    slots = torch.full((4,), -1, dtype=torch.int64, device="cuda")
    pos = torch.zeros(4, dtype=torch.int64, device="cuda")
    qr = randn(7, 4, 16, 64)

    def step():
        mx.mla_cache_append(kv, w, cache, slots, pos, cs, q_pe=qr, q_out=q[:, 0, :, 512:])
        return mx.mla_decode(q, cache, t, n, 0.0625, return_lse=True)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step()
    for i in range(4):
        now = [x + 9 * i + 1 for x in lens]
        n.copy_(ints(now))
        kv.copy_(randn(100 + i, 4, 576))
        pos.copy_(torch.tensor(now) - 1)
        slots.copy_(torch.tensor([int(table[b, (x - 1) // 16]) * 16 + (x - 1) % 16 for b, x in enumerate(now)]))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        want = step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        check(want[0], want[1], A.decode(bits(q), bits(cache), table, now, 0.0625))


@pytest.mark.parametrize("rows", [16, 32, 128])
def test_every_form_on_every_shape(rows):
    # the row block is chosen by size: here each form runs shapes it would not
    # be chosen for, with and without a prefix, its own lists and the joins
    cases = [([1, 0, 130, 33], 1, 16, 16, 0), ([700], 2, 9, 48, 0), ([95, 257], 1, 64, 64, 0),
             ([5, 70, 4], 2, 20, 64, 257), ([40, 3], 1, 128, 16, 130), ([1500], 3, 50, 64, 0)]
    try:
        mx.set_mla_rows(rows)
        for lens, S, H, page, prefix in cases:
            cache, table = paged(rows + H, list(lens) + [prefix], page)
            ptab, own = table[-1, :max(1, -(-prefix // page))].copy(), table[:-1]
            q = randn(H, len(lens), S, H, 576)
            out, lse = mx.mla_decode_shared_prefix(q, cache, ints(ptab), prefix, ints(own), ints(lens), 0.0625,
                                                   return_lse=True)
            check(out, lse, A.decode(bits(q), bits(cache), own, lens, 0.0625, ptab, prefix))
    finally:
        mx.set_mla_rows(0)


def test_decode_many_requests():
    # more requests than a wave's lanes: the shares are found by the whole workgroup
    lens = [(37 * i) % 211 for i in range(150)]
    cache, table = paged(5, lens, 16)
    q = randn(5, 150, 1, 4, 576)
    out, lse = mx.mla_decode(q, cache, ints(table), ints(lens), 0.0625, return_lse=True)
    check(out, lse, A.decode(bits(q), bits(cache), table, lens, 0.0625))


def test_decode_page_window_moves():
    # 128-row blocks keep a window of page numbers in LDS: pages of one row
    # outrun it several times
    n = 9000
    cache, table = paged(2, [n], 1)
    q = randn(3, 1, 1, 128, 576)
    try:
        mx.set_mla_rows(128)
        t = ints(table)
        out, lse = mx.mla_decode(q, cache, t, ints([n]), 0.05, return_lse=True)
        one = mx.mla_decode(q[:, :, :16], cache, t, ints([n]), 0.05)
    finally:
        mx.set_mla_rows(0)
    check(out[0, 0], lse[0, 0], _exact_on_gpu(q[0, 0], cache[t[0].long()].reshape(-1, 576)[:n], 0.05))
    assert torch.equal(one, out[:, :, :16])


def test_layer_example_decodes_what_it_prefills():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "latent_attention.py")
    spec = importlib.util.spec_from_file_location("latent_attention", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    # Both orders round K-up, V-up, probabilities and outputs to bf16 (2^-8
    # each) at different places: a dozen such roundings of the largest value.
    for dims in ((192, 256), (128, 128)):
        decoded, sampled, top = ex.demo(tokens=150, steps=3, samples=3, nope=dims[0], value=dims[1])
        assert decoded <= 12 * BF * top and sampled <= 12 * BF * top


def test_custom_ops_match_the_binding():
    from mxfp4_block_scaled_quant_amd import ops  # noqa: F401
    lens = [40, 7]
    cache, table = paged(9, lens + [30], 16)
    q = randn(1, 2, 1, 16, 576)
    t, n, pt = ints(table[:2]), ints(lens), ints(table[2])
    a, b = torch.ops.mxfp4.mla_decode(q, cache, t, n, 0.0625), mx.mla_decode(q, cache, t, n, 0.0625, return_lse=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a = torch.ops.mxfp4.mla_decode_shared_prefix(q, cache, pt, 30, t, n, 0.0625)
    b = mx.mla_decode_shared_prefix(q, cache, pt, 30, t, n, 0.0625, return_lse=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    x = [randn(2, 33, 2, 192), randn(3, 33, 2, 128), randn(4, 33, 64), randn(5, 33, 2, 128)]
    a = torch.ops.mxfp4.mla_prefill(*x, ints([0, 33]), ints([0, 33]), 0.09)
    b = mx.mla_prefill(*x, ints([0, 33]), ints([0, 33]), 0.09, return_lse=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    kv, w, cs = randn(5, 2, 576), randn(6, 512), torch.tensor(_angles(50), device="cuda")
    slots, pos = torch.tensor([3, 17], device="cuda"), torch.tensor([4, 9], device="cuda")
    one, two, qr = cache.clone(), cache.clone(), randn(7, 2, 16, 64)
    out = torch.empty_like(qr)
    torch.ops.mxfp4.mla_cache_append(kv, w, one, slots, pos, cs, qr, out)
    want = mx.mla_cache_append(kv, w, two, slots, pos, cs, qr)
    assert torch.equal(one, two) and torch.equal(out, want)


@pytest.mark.parametrize("rows", [16, 32, 128])
def test_one_key_is_its_value(rows):
    # a token that sees one key gives that key's value bit for bit, however
    # far its score lies from the running maximum's reference
    cache, table = paged(3, [1, 1, 1], 4)
    q = randn(2, 3, 1, 40, 576, scale=2.0)
    try:
        mx.set_mla_rows(rows)
        out = mx.mla_decode(q, cache, ints(table), ints([1, 1, 1]), 0.3)
    finally:
        mx.set_mla_rows(0)
    want = cache[ints(table)[:, 0].long(), 0, :512][:, None, None].expand_as(out)
    assert torch.equal(out, want)
    for dn, dv in ((128, 128), (192, 256)):
        v = randn(4, 9, 2, dv)
        got = mx.mla_prefill(randn(1, 9, 2, dn + 64), randn(2, 9, 2, dn), randn(3, 9, 64), v, ints([0, 9]),
                             ints([0, 9]), 0.09)
        assert torch.equal(got[0], v[0])
