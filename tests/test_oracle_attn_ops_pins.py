"""Pins of the oracle's attention-side operators against independent routes
(closed forms, complex arithmetic, central differences), on the CPU."""

import math

import numpy as np
import pytest

from oracle import attn_oracle as A


def test_rope_frequencies_closed_forms():
    w = A.rope_frequencies(8, 10000.0)
    assert np.allclose(w.astype(float), [1.0, 0.1, 0.01, 0.001], rtol=1e-12)
    assert np.allclose(A.rope_frequencies(8, 10000.0, "linear", 4.0).astype(float), w.astype(float) / 4)
    # the changed base divides the lowest frequency by the factor and keeps the highest
    b = A.rope_frequencies(8, 10000.0, "base", 4.0).astype(float)
    assert b[0] == 1.0 and np.isclose(b[-1], w[-1].astype(float) / 4)
    # bands: many turns kept, few turns divided, the middle between
    n = A.rope_frequencies(8, 10000.0, "bands", 8.0, original_len=2 * math.pi * 100, low=1.0,
                           high=4.0).astype(float)
    assert n[0] == 1.0 and np.isclose(n[1], 0.1) and np.isclose(n[2], 0.01 / 8) and np.isclose(n[3], 0.001 / 8)
    n = A.rope_frequencies(8, 10000.0, "bands", 8.0, original_len=2 * math.pi * 250, low=1.0,
                           high=4.0).astype(float)
    assert np.isclose(n[2], 0.01 * 0.5 + 0.01 / 8 * 0.5)          # 2.5 turns: half way
    # ramp over pair indices: index(n) = 8 log(len/2 pi n) / (2 log base)
    n = A.rope_frequencies(8, 10000.0, "ramp", 4.0, original_len=2 * math.pi * 1000, low=1.0,
                           high=1000.0).astype(float)
    assert np.allclose(n, [1.0, 0.1 * (2 / 3 + 1 / 12), 0.01 * (1 / 3 + 2 / 12), 0.001 / 4])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_is_a_complex_product(layout):
    rng = np.random.default_rng(0)
    x, pos, w = rng.standard_normal((5, 3, 12)), np.array([0, 1, -7, 1000, 2 ** 31 - 1]), \
        A.rope_frequencies(8, 100.0)
    y = A.rope_rotate(x, pos, w, layout, amplitude=1.5)
    a, b = (x[..., :4], x[..., 4:8]) if layout == "half" else (x[..., 0:8:2], x[..., 1:8:2])
    z = 1.5 * (a + 1j * b) * np.exp(1j * (pos[:, None].astype(np.longdouble) * w)[:, None, :])
    ya, yb = (y[..., :4], y[..., 4:8]) if layout == "half" else (y[..., 0:8:2], y[..., 1:8:2])
    assert np.allclose(ya, z.real, atol=1e-8) and np.allclose(yb, z.imag, atol=1e-8)
    assert np.array_equal(y[..., 8:], x[..., 8:])
    back = A.rope_rotate(y, pos, w, layout, amplitude=1 / 1.5, inverse=True)
    assert np.allclose(back, x, atol=1e-12)


def test_head_norm_gradient_against_differences():
    rng = np.random.default_rng(1)
    x, w, g, eps = rng.standard_normal((2, 2, 6)), rng.standard_normal(6), rng.standard_normal((2, 2, 6)), 1e-3
    assert np.allclose((A.head_norm(x, None, 1e-12) ** 2).mean(-1), 1.0)
    dx, dw = A.head_norm_backward(x, w, g, eps)
    h = 1e-6
    for idx in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[idx] = h
        num = ((A.head_norm(x + e, w, eps) - A.head_norm(x - e, w, eps)) * g).sum() / (2 * h)
        assert abs(num - dx[idx]) < 1e-8
    for i in range(6):
        e = np.zeros(6)
        e[i] = h
        num = ((A.head_norm(x, w + e, eps) - A.head_norm(x, w - e, eps)) * g).sum() / (2 * h)
        assert abs(num - dw[i]) < 1e-8


def test_visible_by_hand():
    s, inside = A.visible(6, True, [0, 2, 2, 5], [0, 9, 2])
    want = np.array([[1, 0, 0, 0, 0, 0], [1, 1, 0, 0, 0, 0], [0, 0, 1, 1, 0, 0], [0, 0, 1, 1, 0, 0],
                     [0, 0, 1, 1, 1, 0], [0, 0, 0, 0, 0, 0]], bool)
    assert np.array_equal(s, want) and list(inside) == [1, 1, 1, 1, 1, 0]
    assert A.visible(3, False)[0].all()


def test_scored_head_against_torch_and_closed_forms():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(2)
    q, k, v = (rng.standard_normal((9, 4)) for _ in range(3))
    seen, _ = A.visible(9, True)
    o, lse = A.scored_head(q, k, v, seen, 0.5)
    tt = [torch.from_numpy(x)[None, None] for x in (q, k, v)]
    want = torch.nn.functional.scaled_dot_product_attention(*tt, is_causal=True, scale=0.5)[0, 0].numpy()
    assert np.allclose(o, want, atol=1e-12)
    assert np.isclose(lse[0], 0.5 * q[0] @ k[0])
    # a large cap changes nothing, a tiny one makes all keys alike
    assert np.allclose(A.scored_head(q, k, v, seen, 0.5, cap=1e7)[0], o, atol=1e-9)
    flat = A.scored_head(q, k, v, np.ones((9, 9), bool), 0.5, cap=1e-9)[0]
    assert np.allclose(flat, v.mean(0))
    # a huge slope leaves the row itself
    assert np.allclose(A.scored_head(q, k, v, np.ones((9, 9), bool), 0.5, slope=1e4)[0], v)
    o, lse = A.scored_head(q, k, v, np.zeros((9, 9), bool), 0.5)
    assert not o.any() and np.all(lse == -np.inf)


@pytest.mark.parametrize("cap,slope", [(0.0, 0.0), (1.5, 0.0), (0.0, 0.3), (0.8, -0.2)])
def test_scored_gradients_against_differences(cap, slope):
    rng = np.random.default_rng(3)
    x = [rng.standard_normal((6, 3)) for _ in range(3)]
    do = rng.standard_normal((6, 3))
    seen, _ = A.visible(6, True, [0, 4, 5], [2, 0])
    grads = A.scored_head_backward(*x, do, seen, 0.7, cap, slope)
    h = 1e-6
    for n in range(3):
        for idx in np.ndindex(6, 3):
            y = [a.copy() for a in x]
            y[n][idx] += h
            up = (A.scored_head(*y, seen, 0.7, cap, slope)[0] * do).sum()
            y[n][idx] -= 2 * h
            down = (A.scored_head(*y, seen, 0.7, cap, slope)[0] * do).sum()
            assert abs((up - down) / (2 * h) - grads[n][idx]) < 1e-7


def test_scored_row_is_the_last_row_of_the_causal_head():
    rng = np.random.default_rng(5)
    q, k, v = (rng.standard_normal((7, 4)) for _ in range(3))
    seen, _ = A.visible(7, True)
    o, lse = A.scored_head(q, k, v, seen, 0.4, 2.0, 0.3)
    row, l1 = A.scored_row(q[6], k, v, 0.4, 2.0, 0.3)
    assert np.allclose(row, o[6], atol=1e-13) and abs(l1 - lse[6]) < 1e-12
    assert A.scored_row(q[0], k[:0], v[:0], 0.4)[1] == -np.inf
