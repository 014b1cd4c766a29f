"""Pins of the attention-layer oracle (CPU): closed forms and brute force."""
import numpy as np
import pytest

from oracle import attention as A


def test_norm_of_a_constant_row_is_its_sign():
    x = np.full((1, 1, 16), -3.0)
    y, _ = A.norm_rope(x, None, np.zeros(1, np.int32), np.zeros(0), eps=0.0)
    assert np.allclose(y, -1.0, atol=1e-15)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product_and_keeps_relative_angles(interleaved):
    r = np.random.default_rng(1)
    f = 100.0 ** (-np.arange(8) / 8)
    q, k = r.normal(size=(2, 1, 1, 16))

    def dot(p0, p1):
        a, _ = A.norm_rope(q, None, [p0], f, interleaved)
        b, _ = A.norm_rope(k, None, [p1], f, interleaved)
        return (a * b).sum()

    assert abs(dot(5, 9) - dot(1005, 1009)) < 1e-11
    y, _ = A.norm_rope(q, None, [3], f, interleaved, eps=0.0)
    n = q[0, 0] / np.sqrt((q[0, 0] ** 2).mean())
    z = (n[0::2] + 1j * n[1::2] if interleaved else n[:8] + 1j * n[8:]) * np.exp(3j * f)
    got = y[0, 0, 0::2] + 1j * y[0, 0, 1::2] if interleaved else y[0, 0, :8] + 1j * y[0, 0, 8:]
    assert np.abs(got - z).max() < 1e-13


def test_quantised_row():
    codes, e = A.quantise([448.0, -1.0, 0.0, np.inf, np.nan, 1e-9])
    assert e == 127 and np.array_equal(codes[:3], [448.0, -1.0, 0.0]) and np.isnan(codes[3:5]).all()
    assert codes[5] == 0.0
    codes, e = A.quantise([449.0, 3.0])
    assert e == 128 and A.dequantise(codes, e)[1] == 3.0
    assert A.quantise(np.zeros(4))[1] == 127
    assert A.quantise([1e-38])[1] == 27 and A.quantise([3.39e38])[1] == 127 + 119


def test_attention_row_against_two_passes():
    r = np.random.default_rng(2)
    q, K, V = r.normal(size=8), r.normal(size=(9, 8)), r.normal(size=(9, 8))
    seen = A.seen_by(1, 5, 4, "tree", [0b1010])
    assert seen.tolist() == [True] * 5 + [False, True, False, True]
    K[5] = np.nan
    V[7] = np.inf
    out, lse, *_ = A.attend(q[None], K, V, seen[None], 0.3)
    e = np.exp(np.longdouble(0.3) * (K[seen].astype(np.longdouble) @ q))
    assert np.allclose(out[0], (e @ V[seen] / e.sum()).astype(float), atol=1e-14)
    assert abs(lse[0] - float(np.log(e.sum()))) < 1e-14
    out, *_ = A.attend(q[None], K, V, seen[None] | (np.arange(9) == 7), 0.3)
    assert np.isposinf(out).all()
    out, lse, *_ = A.attend(q[None], K, V, np.zeros((1, 9), bool), 0.3)
    assert not out.any() and lse[0] == -np.inf
    assert A.seen_by(2, 1, 4, "causal").tolist() == [True, True, True, True, False]
