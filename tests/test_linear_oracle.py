"""The float64 oracle of the calls for experts of one's own against closed
forms, brute force and differences (no GPU)."""
import numpy as np
import pytest

from oracle import linear_oracle as lo
from oracle.moe_oracle import e4m3_decode

ACTS = ("none", "relu", "gelu", "silu", "swiglu")


def test_grouping_by_hand():
    idx = np.array([[1, 0], [1, 2], [-1, 1], [0, 0]])
    offsets, row_token, slot_row = lo.group_rows(idx, 4)
    assert offsets.tolist() == [0, 3, 6, 7, 7]
    assert row_token.tolist() == [0, 3, 3, 0, 1, 2, 1]
    assert slot_row.tolist() == [[3, 0], [4, 6], [-1, 5], [1, 2]]
    offsets, row_token, slot_row = lo.group_rows(idx, 4, capacity=2)
    assert offsets.tolist() == [0, 2, 4, 5, 5]
    assert slot_row.tolist() == [[2, 0], [3, 4], [-1, -1], [1, -1]]


@pytest.mark.parametrize("act", ACTS)
def test_gradients_are_differences(act):
    """Central differences of L = sum(y dy), step 1e-6, float64: truncation
    ~1e-12 of third derivatives below 10, rounding ~1e-16 |L| / 1e-6."""
    rng = np.random.default_rng(3)
    offsets = np.array([0, 3, 3, 7])
    idx = np.array([1, 0, 2, 1, 1, 3, 0])
    F, zd, K = 64, 128 if act == "swiglu" else 64, 5
    x, w = rng.normal(size=(4, K)), rng.normal(size=(3, zd, K))
    bias, dy = rng.normal(size=(3, zd)), rng.normal(size=(7, F))

    def loss(x_, w_, b_):
        return float(np.sum(lo.grouped_linear(x_, offsets, w_, act, idx, b_)[0] * dy))

    _, z = lo.grouped_linear(x, offsets, w, act, idx, bias)
    dx, dw, db, _ = lo.grouped_linear_backward(x, offsets, w, dy, z, act, idx)
    per_token = np.zeros_like(x)
    np.add.at(per_token, idx, dx)
    h = 1e-6
    for grad, pick in ((per_token, 0), (dw, 1), (db, 2)):
        v = [np.zeros_like(x), np.zeros_like(w), np.zeros_like(bias)]
        v[pick] = rng.normal(size=v[pick].shape)
        up = loss(x + h * v[0], w + h * v[1], bias + h * v[2])
        dn = loss(x - h * v[0], w - h * v[1], bias - h * v[2])
        assert abs((up - dn) / (2 * h) - float(np.sum(grad * v[pick]))) < 1e-6


def test_gelu_keeps_its_lower_tail():
    """For z < 0 the normal CDF lies between its asymptotic series' partial
    sums phi/|z| (1 - 1/z^2) and phi/|z| (1 - 1/z^2 + 3/z^4)."""
    z = np.linspace(-30, -4, 105)[:, None]
    y = lo.activation("gelu", z)
    slope = lo.activation_backward("gelu", z, np.ones_like(z))
    phi = np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    low = phi / -z * (1 - z ** -2)
    high = low + phi / -z * 3 * z ** -4
    for cdf in (y / z, slope - z * phi):
        # the slope's difference cancels z^2 of its terms, each 2^-52 (z^2 / 2 + 4)
        assert np.all(cdf >= low - 2.0 ** -52 * (z * z + 8) * np.abs(z) * phi)
        assert np.all(cdf <= high + 2.0 ** -52 * (z * z + 8) * np.abs(z) * phi)


def test_checkpoint_codes_are_the_nearest():
    """Every code against all 127 magnitudes by brute force."""
    rng = np.random.default_rng(5)
    x = (rng.normal(size=(3, 128)) * np.exp(rng.normal(size=(3, 128)) * 4)).astype(np.float32)
    x[1, :64] = 0
    codes, scale = lo.checkpoint_pack(x)
    assert scale.shape == (3, 2) and scale[1, 0] == np.float32(1e-30) / np.float32(448)
    grid = e4m3_decode(np.arange(127, dtype=np.uint8))
    m = np.maximum(np.abs(x.reshape(3, 2, 64)).max(2), np.float32(1e-30))
    v = np.abs(x.reshape(3, 2, 64) * (np.float32(448) / m)[:, :, None]).astype(np.float64)
    got = np.abs(e4m3_decode(codes)).reshape(3, 2, 64)
    best = np.min(np.abs(v[..., None] - grid), axis=3)
    np.testing.assert_array_equal(np.abs(v - got), best)
    back = lo.checkpoint_unpack(codes, scale)
    # half a step: 2^-4 of a normal code, 2^-10 where the codes are 2^-9 apart
    worst = np.maximum(np.abs(x) / 16, np.repeat(m, 64, axis=1) / 448 * 2.0 ** -10)
    assert np.all(np.abs(back - x) <= worst * (1 + 1e-6))


def test_checkpoint_marks_what_is_not_finite():
    x = np.ones((1, 64), np.float32)
    x[0, 3], x[0, 4], x[0, 5] = np.nan, np.inf, -np.inf
    codes, scale = lo.checkpoint_pack(x)
    back = lo.checkpoint_unpack(codes, scale)
    assert np.isnan(back[0, 3:6]).all() and np.isfinite(back[0, 6:]).all()
    assert scale[0, 0] == np.float32(1) / np.float32(448)


def test_combine_gradients_are_differences():
    rng = np.random.default_rng(7)
    slot_row = np.array([[2, 0], [-1, 1], [3, -1]], np.int32)
    rows, gate = rng.normal(size=(5, 6)), rng.normal(size=(3, 2))
    dy = rng.normal(size=(3, 6))
    drows, dgate = lo.combine_rows_backward(rows, slot_row, gate, dy)
    assert np.isnan(drows[4]).all() and dgate[1, 0] == 0 and dgate[2, 1] == 0
    vr, vg = rng.normal(size=rows.shape), rng.normal(size=gate.shape)
    up = np.sum(lo.combine_rows(rows + 1e-6 * vr, slot_row, gate + 1e-6 * vg) * dy)
    dn = np.sum(lo.combine_rows(rows - 1e-6 * vr, slot_row, gate - 1e-6 * vg) * dy)
    want = np.nansum(drows * vr) + np.sum(dgate * vg)
    assert abs((up - dn) / 2e-6 - want) < 1e-7
