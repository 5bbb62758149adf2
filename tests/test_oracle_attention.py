"""Pins of the attention block's oracle: hand-worked rotations and an exact
rational softmax, its limits, and the frequency tables of the binding's helper."""

import math

import numpy as np
import pytest

from oracle import attention as A


def test_rope_quarter_turn_and_layouts():
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    f = np.array([math.pi / 2, 0.0], np.float32)  # pair 0 turns a quarter per position, pair 1 not at all
    y, size = A.rope(x, [1], f)
    assert np.allclose(y[0, 0], [-3, 2, 1, 4, 5, 6, 7, 8], atol=1e-6)
    assert np.array_equal(size[0, 0], [4, 6, 4, 6, 0, 0, 0, 0])
    y, _ = A.rope(x, [1], f, interleaved=True)
    assert np.allclose(y[0, 0], [-2, 1, 3, 4, 5, 6, 7, 8], atol=1e-6)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_turns_back_and_keeps_lengths(interleaved):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 32))
    f = (10000.0 ** (-np.arange(8) / 8)).astype(np.float32)
    p = np.array([0, 1, 77, 131072, 999999])
    y, _ = A.rope(x, p, f, interleaved)
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
    back, _ = A.rope(y, -p, f, interleaved)
    assert np.allclose(back, x, atol=1e-12)
    # scores depend on the distance alone
    a, b = rng.standard_normal((1, 1, 32)), rng.standard_normal((1, 1, 32))
    d = [(A.rope(a, [s + 5], f, interleaved)[0] * A.rope(b, [s], f, interleaved)[0]).sum() for s in (0, 1000)]
    assert abs(d[0] - d[1]) < 1e-9


def test_attention_hand_worked():
    # one head of width 2, page of 2 tokens, three keys; scores 0, ln 2, ln 4 for the last token
    k = np.zeros((3, 2, 1, 2))
    v = np.zeros((3, 2, 1, 2))
    table = np.array([[2, 0]])
    k[2, 0, 0], k[2, 1, 0], k[0, 0, 0] = [0, 9], [math.log(2), 9], [math.log(4), 9]
    v[2, 0, 0], v[2, 1, 0], v[0, 0, 0] = [7, 0], [0, 7], [14, 14]
    k[0, 1], v[0, 1] = np.nan, np.nan  # behind the last key
    q = np.array([[[1.0, 0.0]], [[1.0, 0.0]]])
    r = A.paged_attention(q, k, v, table, [0, 2], [3], 1.0)
    assert np.allclose(r["out"][1, 0], [(7 + 4 * 14) / 7, (2 * 7 + 4 * 14) / 7])
    assert np.allclose(r["out"][0, 0], [7 / 3, 14 / 3])       # sees two keys
    assert np.allclose(r["lse"][:, 0], [math.log(3), math.log(7)])
    r = A.paged_attention(q, k, v, table, [0, 2], [3], 1.0, window=1)
    assert np.allclose(r["out"][:, 0], [[0, 7], [14, 14]])
    # more new tokens than keys: the first rows see nothing
    r = A.paged_attention(np.repeat(q, 2, 0), k, v, table, [0, 4], [3], 1.0)
    assert np.array_equal(r["out"][0, 0], [0, 0]) and r["lse"][0, 0] == -np.inf
    assert np.allclose(r["out"][3, 0], [9, 10])


def test_attention_against_a_plain_softmax():
    rng = np.random.default_rng(3)
    T, Hq, Hkv, D, m = 6, 4, 2, 8, 11
    k, v = rng.standard_normal((4, 4, Hkv, D)), rng.standard_normal((4, 4, Hkv, D))
    table = np.array([[3, 1, 0]])
    q = rng.standard_normal((T, Hq, D))
    r = A.paged_attention(q, k, v, table, [0, T], [m], 0.5)
    flat_k, flat_v = k[[3, 1, 0]].reshape(12, Hkv, D)[:m], v[[3, 1, 0]].reshape(12, Hkv, D)[:m]
    for t in range(T):
        for h in range(Hq):
            n = m - T + t + 1
            s = np.exp([0.5 * float(np.dot(q[t, h], flat_k[j, h // 2])) for j in range(n)])
            assert np.allclose(r["out"][t, h], (s[:, None] * flat_v[:n, h // 2]).sum(0) / s.sum())
            assert np.isclose(r["lse"][t, h], math.log(s.sum()))


def test_frequency_tables():
    f = pytest.importorskip("fp8_w8a8_linear_b200")
    base, amp = f.rope_frequencies(64)
    want = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    assert amp == 1.0 and np.array_equal(base.numpy(), want.astype(np.float32))
    lin, _ = f.rope_frequencies(64, scaling="linear", factor=4.0)
    assert np.array_equal(lin.numpy(), (want / 4).astype(np.float32))
    wl, amp = f.rope_frequencies(64, scaling="wavelength", factor=8.0, original_length=8192)
    turns = 8192 * want / (2 * np.pi)
    assert amp == 1.0
    assert np.array_equal(wl.numpy()[turns >= 4], want.astype(np.float32)[turns >= 4])
    assert np.array_equal(wl.numpy()[turns <= 1], (want / 8).astype(np.float32)[turns <= 1])
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and np.all(wl.numpy()[mid] < want[mid]) and np.all(wl.numpy()[mid] > want[mid] / 8)
    ya, amp = f.rope_frequencies(128, scaling="yarn", factor=8.0, original_length=4096, low=1.0, high=32.0)
    want = 10000.0 ** (-np.arange(0, 128, 2) / 128)
    assert math.isclose(amp, 0.1 * math.log(8) + 1)
    r = ya.numpy().astype(np.float64) / want
    assert np.all(np.diff(r) <= 1e-6) and math.isclose(r[0], 1, rel_tol=1e-6) and math.isclose(r[-1], 1 / 8, rel_tol=1e-6)
    for bad in (dict(rotary_dim=63), dict(rotary_dim=64, base=1.0), dict(rotary_dim=64, factor=0.0),
                dict(rotary_dim=64, scaling="other")):
        with pytest.raises(ValueError):
            f.rope_frequencies(**bad)
