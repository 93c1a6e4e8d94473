"""The attention oracle against brute force and exact identities (CPU)."""

import math

import numpy as np

from oracle import attention as A


def test_row_is_the_softmax_average():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=7), rng.normal(size=(5, 7)), rng.normal(size=(5, 3))
    out, lse, mag, top = A.attend_row(q, k, v, 0.3)
    e = [math.exp(0.3 * sum(a * b for a, b in zip(q, row))) for row in k]
    for j in range(3):
        assert math.isclose(out[j], sum(w * r[j] for w, r in zip(e, v)) / sum(e), rel_tol=1e-12)
        assert math.isclose(mag[j], sum(w * abs(r[j]) for w, r in zip(e, v)) / sum(e), rel_tol=1e-12)
    assert math.isclose(lse, math.log(sum(e)), rel_tol=1e-12)
    assert top >= max(abs(0.3 * float(q @ r)) for r in k) - 1e-12


def test_no_keys_and_one_key():
    out, lse, _, _ = A.attend_row(np.ones(4), np.zeros((0, 4)), np.zeros((0, 2)), 1.0)
    assert np.all(out == 0) and lse == -np.inf
    out, lse, _, _ = A.attend_row(np.ones(4), np.ones((1, 4)), np.array([[2.0, -3.0]]), 0.5)
    assert np.allclose(out, [2, -3]) and math.isclose(lse, 2.0)


def test_decode_joins_prefix_and_own_rows():
    rng = np.random.default_rng(1)
    cache = rng.normal(size=(9, 4, 576))
    q = rng.normal(size=(2, 2, 3, 576))
    prefix, own = np.array([5, 1]), np.array([[2, 7], [0, 8]])
    a = A.decode(q, cache, own, np.array([6, 3]), 0.05, prefix, 8)
    joined = np.array([[5, 1, 2, 7], [5, 1, 0, 8]])
    b = A.decode(q, cache, joined, np.array([14, 11]), 0.05)
    assert np.allclose(a[0], b[0]) and np.allclose(a[1], b[1])


def test_decode_last_token_is_a_one_token_call():
    rng = np.random.default_rng(2)
    cache, q = rng.normal(size=(4, 3, 576)), rng.normal(size=(1, 3, 2, 576))
    table = np.array([[3, 0, 2, 1]])
    a = A.decode(q, cache, table, np.array([8]), 0.04)
    for s in range(3):
        b = A.decode(q[:, s:s + 1], cache, table, np.array([6 + s]), 0.04)
        assert np.allclose(a[0][:, s], b[0][:, 0])
    # more tokens than rows: the first see nothing
    c = A.decode(q, cache, table, np.array([1]), 0.04)
    assert np.all(c[0][:, :2] == 0) and np.all(np.isneginf(c[1][:, :2]))


def test_prefill_last_rows_equal_a_chunk():
    rng = np.random.default_rng(3)
    q, kn, kp, v = (rng.normal(size=s) for s in ((10, 2, 192), (10, 2, 128), (10, 64), (10, 2, 128)))
    whole = A.prefill(q, kn, kp, v, [0, 10], [0, 10], 0.07)
    chunk = A.prefill(q[6:], kn, kp, v, [0, 4], [0, 10], 0.07)
    assert np.allclose(whole[0][6:], chunk[0]) and np.allclose(whole[1][6:], chunk[1])


def test_rotation_keeps_pair_lengths_and_relative_angle():
    rng = np.random.default_rng(4)
    x, y = rng.normal(size=64), rng.normal(size=64)
    f = 10000.0 ** (-np.arange(32) / 32)
    for inter in (True, False):
        rot = lambda z, p: A.rotate(z, np.cos(p * f), np.sin(p * f), inter)
        assert math.isclose(np.linalg.norm(rot(x, 5)), np.linalg.norm(x), rel_tol=1e-12)
        assert math.isclose(rot(x, 9) @ rot(y, 4), rot(x, 105) @ rot(y, 100), rel_tol=1e-9)
        assert np.allclose(rot(x, 0), x)
