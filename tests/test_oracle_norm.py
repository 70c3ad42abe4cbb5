"""Pins of the norm / 8-bit oracle: hand-worked values, gradients against differences, bf16 storage rounding."""
import numpy as np
import pytest

from oracle import norm as o


def test_store_is_round_to_nearest_even_bf16():
    # 1 + 2^-8 is half a step above 1 (even below), 1 + 3 * 2^-8 half a step below 1 + 2^-6 (even above)
    v = np.array([1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 1 + 2.0 ** -8 + 2.0 ** -30, -(1 + 2.0 ** -8), 0.0, 3.4e38, 1e-40])
    torch = pytest.importorskip("torch")
    ref = torch.tensor(v).to(torch.bfloat16).double().numpy()
    assert np.array_equal(o.store(v, "bf16")[:6], np.array([1.0, 1 + 2.0 ** -6, 1 + 2.0 ** -7, -1.0, 0.0, np.inf]))
    assert np.array_equal(o.store(v, "bf16")[[0, 1, 3, 4, 5, 6]], ref[[0, 1, 3, 4, 5, 6]])
    r = np.random.default_rng(0).standard_normal(4096).astype(np.float32)
    assert np.array_equal(o.store(r, "bf16"), torch.from_numpy(r).to(torch.bfloat16).double().numpy())


def test_norm_of_hand_worked_rows():
    # mean square of (3, 4) is 12.5; with eps 0 the norm would be 3 / sqrt(12.5)
    y = o.rms_norm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), 1e-30)
    assert np.allclose(y, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]], rtol=1e-15)
    assert np.array_equal(o.rms_norm(np.zeros((1, 4)), None, 1e-6), np.zeros((1, 4)))


def test_codes_of_halves_go_to_even_and_the_maximum_to_127():
    p = np.array([[127.0, -127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 0.0, 126.5]])
    q, m = o.codes(p)
    assert m[0, 0] == 127 and q.tolist() == [[127, -127, 0, 2, 2, 0, -2, 0, 126]]
    assert o.codes(np.zeros((2, 3)))[0].tolist() == [[0, 0, 0], [0, 0, 0]]


@pytest.mark.parametrize("with_w", [False, True])
@pytest.mark.parametrize("with_ds", [False, True])
def test_gradients_against_central_differences(with_w, with_ds):
    rng = np.random.default_rng(3)
    N, d, eps = 3, 5, 0.25                       # a large eps, so that its place in the formula matters
    s, dy = rng.standard_normal((N, d)), rng.standard_normal((N, d))
    w = rng.standard_normal(d) if with_w else None
    ds = rng.standard_normal((N, d)) if with_ds else None
    loss = lambda s_, w_: (o.rms_norm(s_, w_, eps) * dy).sum() + (0 if ds is None else (ds * s_).sum())  # noqa: E731
    dx, dw = o.rms_norm_backward(dy, s, w, eps, ds)
    h = 1e-6
    for i in range(N):
        for j in range(d):
            e = np.zeros((N, d))
            e[i, j] = h
            assert abs((loss(s + e, w) - loss(s - e, w)) / (2 * h) - dx[i, j]) < 1e-8
    ones = np.ones(d) if w is None else w
    for j in range(d):
        e = np.zeros(d)
        e[j] = h
        assert abs((loss(s, ones + e) - loss(s, ones - e)) / (2 * h) - dw[j]) < 1e-8


def test_bounds_see_a_planted_mistake():
    """The bounds are tight enough to tell a missing eps, a wrong mean and a dropped weight from roundings."""
    rng = np.random.default_rng(4)
    s, dy, w = rng.standard_normal((4, 64)), rng.standard_normal((4, 64)), 1 + 0.1 * rng.standard_normal(64)
    y = o.rms_norm(s, w, 1e-2)
    assert np.any(np.abs(o.rms_norm(s, w, 1e-6) - y) > o.rms_norm_bound(y, "f32"))
    assert np.any(np.abs(o.rms_norm(s, None, 1e-2) - y) > o.rms_norm_bound(y, "bf16"))
    dx, dw = o.rms_norm_backward(dy, s, w, 1e-2, None)
    bx, bw = o.backward_bounds(dy, s, w, 1e-2, None, "bf16")
    wrong = o.rms_norm_backward(dy, s, None, 1e-2, None)[0]
    assert np.any(np.abs(wrong - dx) > bx)
    assert np.any(np.abs(o.rms_norm_backward(dy[:3], s[:3], w, 1e-2, None)[1] - dw) > bw)


def test_product_of_hand_worked_operands():
    a, b = np.array([[1, -2, 3]]), np.array([[4, 5, 6], [-128, 127, 0]])
    out = o.matmul_i8(a, np.array([0.5]), b, np.array([2.0, 0.25]), np.array([1.0, 0.0]))
    assert out.tolist() == [[(4 - 10 + 18) * 1.0 + 1.0, (-128 - 254) * 0.125]]
