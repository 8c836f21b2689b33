"""Pins of the fp64 oracle of the dense operators: hand-worked blocks, gradients against differences."""
import numpy as np
import pytest

from oracle import block as OB
from oracle import dense as OD
from oracle import formats as OF


def test_fp8_block_by_hand():
    x = np.zeros((2, 160), dtype=np.float32)
    x[0, :4] = [7.0, -3.5, 0.5, 7 * 17 / 448]  # scale 7/448 = 1/64: 448, -224, 32, 17
    x[0, 128:] = 1.0
    x[1, 3] = -896.0
    q, s = OD.fp8_quantize(x, 1)
    assert s.tolist() == [[1 / 64, np.float32(1) / np.float32(448)], [2.0, 0.0]]
    assert OF.e4m3fn_value(q[0, :5]).tolist() == [448, -224, 32, 16, 0]  # 17 lies half way between 16 and 18
    assert set(OF.e4m3fn_value(q[0, 128:]).tolist()) == {448.0}
    assert OF.e4m3fn_value(q[1, 3]) == -448 and not q[1, 128:].any()
    q, s = OD.fp8_quantize(x, 128)
    assert s.shape == (1, 2) and s[0, 0] == 2.0 and OF.e4m3fn_value(q[0, 0]) == 3.5


def test_fp8_blocks_that_are_not_finite():
    x = np.ones((3, 16), dtype=np.float32)
    x[0, 3], x[1, 5], x[2] = np.inf, np.nan, 1e-45
    q, s = OD.fp8_quantize(x, 1)
    assert np.isinf(s[0, 0]) and np.isnan(s[1, 0]) and s[2, 0] == 0
    assert q[0].tolist() == [0x7F if i == 3 else 0 for i in range(16)]
    assert (q[1] == 0x7F).all() and not q[2].any()


def test_fp8_values_of_two_matrices():
    r = np.random.default_rng(1)
    w = r.normal(size=(2 * 130, 144)).astype(np.float32)
    parts = [OD.fp8_quantize(h, 128) for h in (w[:130], w[130:])]
    q, s = np.concatenate([p[0] for p in parts]), np.concatenate([p[1] for p in parts])
    assert s.shape == (4, 2)
    v = OD.fp8_values(q, s, 128, gated=True)
    assert np.array_equal(v[:130], OD.fp8_values(*parts[0], 128)) and np.array_equal(v[130:], OD.fp8_values(*parts[1], 128))
    # e4m3 steps: 2^-4 of the value, or of the smallest normal 2^-6
    scale = np.concatenate([OD.spread(p[1], 128, 130, 144) for p in parts])
    unit = np.maximum(np.abs(w), 2.0**-6 * scale)
    assert (np.abs(v - w) <= unit * 2.0**-4 * (1 + 1e-6)).all()


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
def test_gradients_against_differences(act):
    r = np.random.default_rng(7)
    T, I, K, step = 5, 6, 8, 1e-6
    x, w, dh = r.normal(size=(T, K)), r.normal(size=(2 * I, K)), r.normal(size=(T, I))

    def loss(x, w):
        return float((OD.glu(x, w, act)[0] * dh).sum())

    dx, dw = OD.linear_grad(OD.glu_grad(dh, OD.glu(x, w, act)[1], act), x, w)
    for m, grad, of in ((x, dx, lambda m: loss(m, w)), (w, dw, lambda m: loss(x, m))):
        for i in np.ndindex(m.shape):
            hi, lo = m.copy(), m.copy()
            hi[i] += step
            lo[i] -= step
            # central differences: third derivatives of a few hundred times step^2 / 6, and 1e-16 / step of rounding
            assert abs((of(hi) - of(lo)) / (2 * step) - grad[i]) <= 1e-7 * (1 + abs(grad[i]))


def test_slopes_far_from_zero():
    g = np.array([-1e4, -800.0, -40.0, 40.0, 800.0, 1e4])
    for act in ("gelu", "silu"):
        with np.errstate(all="ignore"):
            np.testing.assert_allclose(OD.slope(g, act), [0, 0, 0, 1, 1, 1], atol=1e-15)
    assert OD.slope([0.0], "relu") == 0 and OD.slope([0.0], "silu") == 0.5 and OB.act([0.0], "silu") == 0
