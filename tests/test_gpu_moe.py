"""The experts' products against the fp64 oracle, within its derived bounds."""

import numpy as np
import pytest
import torch

import mxfp4_block_scaled_quant_amd as mx
from mxfp4_block_scaled_quant_amd import inputs
from oracle import feedforward as D
from oracle import formats as F
from oracle import quant as Q
from tests.helpers import dev_bf16, host_bf16_bits, need_gpu

pytestmark = pytest.mark.gpu


def problem(T, k, E, H, I, seed=0, gated=True, bias=False, residual=False, elsewhere=False, skew=False):
    r = np.random.default_rng([seed, T, k, E, H, I])
    N = 2 * I if gated else I
    up = Q.quant_1x32(inputs.weights(E * N, H, seed).reshape(E, N, H))
    down = Q.quant_1x32(inputs.weights(E * H, I, seed + 1).reshape(E, H, I))
    ids = np.stack([r.permutation(max(E, k))[:k] for _ in range(T)]) if T else np.zeros((0, k), np.int64)
    if skew and T:
        ids[:, 0] = E - 1                       # one expert that every token chose
    if elsewhere and T:
        ids = np.where(r.random(ids.shape) < 0.4, r.choice([-1, -7, E, E + 5, 2 ** 31 - 1, -2 ** 31], ids.shape), ids)
    p = {"x": inputs.activations(T, H, seed, outliers=True) if T else np.zeros((0, H), np.uint16),
         "ids": ids.astype(np.int32), "weights": r.random((T, k)).astype(np.float32), "up": up, "down": down,
         "up_bias": inputs.bias(E * N, seed).reshape(E, N) if bias else None,
         "down_bias": inputs.bias(E * H, seed + 1).reshape(E, H) if bias else None,
         "residual": inputs.activations(T, H, seed + 3) if residual and T else None}
    return p


def _weight(q, s):
    E, N, K2 = q.shape
    w, ws = mx.mxfp4_preshuffle_weight(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), N, 2 * K2, batch=E)
    return mx.MXFP4Weight(w, ws, N, 2 * K2, E)


def device(p):
    opt = lambda v: None if v is None else dev_bf16(v)  # noqa: E731
    return {"x": dev_bf16(p["x"]), "ids": torch.from_numpy(p["ids"]).cuda(),
            "weights": torch.from_numpy(p["weights"]).cuda(), "up": _weight(*p["up"]), "down": _weight(*p["down"]),
            "up_bias": opt(p["up_bias"]), "down_bias": opt(p["down_bias"]), "residual": opt(p["residual"])}


def check(p, out, act="silu", gated=True):
    ref, err = D.moe(p["x"], p["ids"], p["weights"].astype(np.float64), p["up"], p["down"], p["up_bias"],
                     p["down_bias"], act, gated, p["residual"],
                     # (experts of more than 24 rows on average: the tiled kernels)
                     half=p["ids"].size // p["up"][0].shape[0] > 24)
    got = F.bf16_to_f64(host_bf16_bits(out))
    assert np.isfinite(got).all()
    # the last rounding: half a step of bf16, of a value that may be err off
    bound = err + 2.0 ** -8 * (np.abs(ref) + err) + 1e-38
    worst = np.max(np.abs(got - ref) / bound) if got.size else 0.0
    assert worst <= 1.0, worst


@pytest.mark.parametrize("T,k,E,H,I", [
    (1, 1, 1, 32, 32), (1, 2, 8, 64, 96), (3, 2, 4, 160, 32), (7, 8, 8, 256, 160), (16, 4, 64, 512, 96),
    (33, 2, 4, 544, 288), (65, 6, 16, 128, 64), (200, 4, 8, 96, 128), (130, 2, 3, 1056, 544), (5, 3, 2, 64, 64)])
@pytest.mark.parametrize("opts", [dict(), dict(bias=True, residual=True), dict(elsewhere=True, bias=True),
                                  dict(skew=True, residual=True)])
def test_moe(T, k, E, H, I, opts):
    need_gpu()
    p = problem(T, k, E, H, I, **opts)
    check(p, mx.mxfp4_moe(**device(p)))


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T", [5, 150])
def test_activations(act, gated, T):
    need_gpu()
    p = problem(T, 2, 4, 256, 96, seed=3, gated=gated, bias=True)
    check(p, mx.mxfp4_moe(**device(p), activation=act, gated=gated), act, gated)


def test_no_token_and_no_expert_here():
    need_gpu()
    p = problem(0, 2, 4, 64, 32)
    assert mx.mxfp4_moe(**device(p)).shape == (0, 64)
    for residual in (True, False):
        p = problem(9, 2, 4, 64, 32, residual=residual)
        p["ids"][:] = -1
        out = host_bf16_bits(mx.mxfp4_moe(**device(p)))
        want = p["residual"] if residual else np.zeros_like(out)
        assert np.array_equal(F.bf16_to_f64(out), F.bf16_to_f64(want))


def test_the_same_expert_twice_and_weights_of_zero():
    need_gpu()
    p = problem(40, 4, 4, 128, 64, seed=5)
    p["ids"][:, 1] = p["ids"][:, 0]
    p["weights"][::3] = 0
    check(p, mx.mxfp4_moe(**device(p)))


def test_strides_views_and_in_place():
    need_gpu()
    p = problem(21, 2, 4, 96, 64, seed=7, residual=True)
    d = device(p)
    ref = mx.mxfp4_moe(**d)
    wide = {n: torch.full((21, 200), 3.0, dtype=torch.bfloat16, device="cuda") for n in ("x", "out", "residual")}
    for n in ("x", "residual"):
        wide[n][:, 8:104] = d[n]
    ids, w = torch.full((21, 9), -5, dtype=torch.int32, device="cuda"), torch.zeros((21, 5), device="cuda")
    ids[:, 3:5], w[:, 1:3] = d["ids"], d["weights"]
    e = {**d, "x": wide["x"][:, 8:104], "residual": wide["residual"][:, 8:104], "ids": ids[:, 3:5],
         "weights": w[:, 1:3]}
    assert torch.equal(mx.mxfp4_moe(**e, out=wide["out"][:, 8:104]), ref)
    assert (wide["out"][:, :8] == 3).all() and (wide["out"][:, 104:] == 3).all()
    assert torch.equal(mx.mxfp4_moe(**e, out=e["residual"]), ref)       # in place of its residual
    assert (wide["residual"][:, :8] == 3).all() and (wide["residual"][:, 104:] == 3).all()


def test_results_do_not_depend_on_the_run_or_the_workspace():
    need_gpu()
    p = problem(150, 6, 16, 256, 160, seed=8, residual=True)
    d = device(p)
    need = mx.mxfp4_moe_workspace_bytes(150, 6, 16, 256, 160)
    ref = mx.mxfp4_moe(**d)
    for fill in (0, 0xFF, 0x7F):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(mx.mxfp4_moe(**d, workspace=ws), ref)


def test_captured_with_changing_routes_and_on_another_stream():
    need_gpu()
    p = problem(24, 4, 8, 256, 128, seed=9, residual=True)
    d = device(p)
    out = torch.zeros((24, 256), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mx.mxfp4_moe(**d, out=out)
    torch.cuda.current_stream().wait_stream(s)
    ref = mx.mxfp4_moe(**d)
    assert torch.equal(out, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mx.mxfp4_moe(**d, out=out)
    r = np.random.default_rng(1)
    for n in range(4):
        ids = r.integers(-1, 9, (24, 4)).astype(np.int32)
        d["ids"].copy_(torch.from_numpy(ids).cuda())
        d["x"].copy_(dev_bf16(inputs.activations(24, 256, 50 + n)))
        g.replay()
        again = mx.mxfp4_moe(**d)
        torch.cuda.synchronize()
        assert torch.equal(out, again), n
    p["ids"], p["x"] = ids, inputs.activations(24, 256, 53)
    check(p, out)


def test_rows_between_the_products_are_the_library_s_quantisation():
    """The whole equals the framework's other operators one after the other, bit by bit, where one expert has all."""
    need_gpu()
    p = problem(40, 1, 1, 256, 128, seed=11, gated=False)
    p["weights"][:] = 1
    d = device(p)
    h = mx.mxfp4_linear_act(d["x"], d["up"].w_pre, d["up"].ws_pre, 128, activation="relu")
    y = mx.mxfp4_linear_act(h, d["down"].w_pre, d["down"].ws_pre, 256)
    out = mx.mxfp4_moe(**d, activation="relu", gated=False)
    # (sums of the same products in another order: an ulp of bf16 in a few places)
    same = (host_bf16_bits(out) == host_bf16_bits(y)).mean()
    assert same > 0.99


# On both sides of each change of form: pairs of one launch's sum (1024) and of
# the plan for itself (64 of 4 tokens), chunks of the plan, mean rows of one
# and of two row tiles, of the tiled kernels.
@pytest.mark.parametrize("T,k,E,H,I", [(4, 16, 20, 96, 64), (4, 17, 20, 96, 64), (128, 8, 128, 64, 64), (129, 8, 128, 64, 96),
                                       (1024, 1, 100, 64, 32), (1025, 1, 1024, 32, 32), (64, 16, 93, 96, 32),
                                       (96, 1, 4, 64, 64), (100, 1, 4, 64, 64), (2100, 1, 1, 64, 64)])
def test_borders_of_the_forms(T, k, E, H, I):
    need_gpu()
    p = problem(T, k, E, H, I, seed=21, residual=True, bias=True)
    check(p, mx.mxfp4_moe(**device(p)))


def test_rows_past_32_bits():
    """Rows between the products of more than 4 GiB: the last tokens as in a call of their own."""
    need_gpu()
    T, k, E, H, I = 33000, 8, 8, 8320, 32
    p = problem(400, k, E, H, I, seed=22, residual=True)
    d = device(p)
    few = mx.mxfp4_moe(**d)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand(T, k, generator=g, device="cuda")
    x[-400:], ids[-400:], w[-400:] = d["x"], d["ids"], d["weights"]
    out = torch.zeros_like(x)
    out[-400:] = d["residual"]
    mx.mxfp4_moe(x, ids, w, d["up"], d["down"], residual=out, out=out)
    assert torch.equal(out[-400:], few)


def test_two_calls_at_once():
    need_gpu()
    a, b = (device(problem(T, 4, 16, 512, 256, seed=23, residual=True)) for T in (150, 31))
    want = mx.mxfp4_moe(**a), mx.mxfp4_moe(**b)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for s, d in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                got.append(mx.mxfp4_moe(**d))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 2])


@pytest.mark.parametrize("T", [3, 40, 150])
def test_an_infinite_column_leaves_the_others(T):
    """A bias of +-inf or NaN in three columns: those are so, their neighbours are as without."""
    need_gpu()
    p = problem(T, 2, 4, 192, 64, seed=24, bias=True)
    d = device(p)
    at = [5, 70, 131]
    for n in at:
        p["down_bias"][:, n] = 0
    d["down_bias"][:, at] = torch.tensor([float("inf"), float("-inf"), float("nan")], dtype=torch.bfloat16, device="cuda")
    d["weights"].clamp_(min=0.125)
    p["weights"] = d["weights"].cpu().numpy()
    out = mx.mxfp4_moe(**d)
    assert (out[:, 5] == float("inf")).all() and (out[:, 70] == float("-inf")).all() and out[:, 131].isnan().all()
    out[:, at] = mx.mxfp4_moe(**{**d, "down_bias": dev_bf16(p["down_bias"])})[:, at]
    check(p, out)


@pytest.mark.parametrize("T,k,E", [(3, 2, 4), (40, 2, 16), (70, 4, 16), (150, 4, 16)])
def test_a_token_that_is_not_finite_and_weights_outside(T, k, E):
    """One token's infinities and NaN stay its own; the weight of an id outside is not read into the sum."""
    need_gpu()
    d = device(problem(T, k, E, 192, 64, seed=25, elsewhere=True))
    want = mx.mxfp4_moe(**d)
    outside = (d["ids"] < 0) | (d["ids"] >= E)
    d["weights"][outside] = float("nan")
    assert torch.equal(mx.mxfp4_moe(**d), want)
    d["x"][1, 3], d["x"][1, 40] = float("inf"), float("nan")
    out = mx.mxfp4_moe(**d)
    rest = [t for t in range(T) if t != 1]
    assert torch.equal(out[rest], want[rest])


def test_many_tiles_repeat_to_the_bit():
    """Thousands of tiles, each after another's epilogue: equal in every run, and the token of each row its own."""
    need_gpu()
    d = device(problem(400, 8, 8, 1024, 512, seed=26, residual=True))
    few = mx.mxfp4_moe(**d)
    wide = {n: d[n].repeat(20, 1) for n in ("x", "ids", "weights", "residual")}
    for _ in range(20):
        assert torch.equal(mx.mxfp4_moe(**{**d, **wide}), few.repeat(20, 1))
