"""The oracle of the 8-bit calls and of the AdamW step against other ways to say
the same: torch's own cast, differences, and the step written in 64 bits."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as bo
from oracle.moe_oracle import e4m3_decode


def test_e4m3_encode_is_the_cast():
    every = torch.arange(-(1 << 15), 1 << 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    some = torch.randn(100000, generator=torch.Generator().manual_seed(0)) * 90
    for x in (every[every.abs() <= 448], some[some.abs() <= 448]):
        assert (x.to(torch.float8_e4m3fn).view(torch.uint8).numpy() == bo.e4m3_encode(x.numpy())).all()
    assert (bo.e4m3_encode([np.nan, np.inf, -np.inf]) & 0x7F == 0x7F).all()


def test_exponent_is_the_smallest():
    top = np.concatenate([np.exp2(np.random.RandomState(0).uniform(-130, 127, 10000)),
                          448 * np.exp2(np.arange(-100, 100.0)), np.nextafter(448, 500) * np.exp2(np.arange(-90, 90.0))])
    e = bo.exponent(top).astype(float)
    assert (top <= 448 * np.exp2(e)).all()
    assert ((top > 448 * np.exp2(e - 1)) | (e == -126)).all()
    assert bo.exponent(0) == -126


def test_packing_keeps_values():
    """Off by half a step: 2^-4 of the value or 2^(e - 10)."""
    x = np.random.RandomState(1).randn(20, 320) * np.exp(np.random.RandomState(2).randn(20, 1) * 3)
    codes, scale = bo.pack_rows(x)
    step = np.repeat(np.exp2(scale.T.astype(float) - 137), 128, axis=1)[:, :320]
    assert (np.abs(bo.unpack_rows(codes, scale) - x) <= np.maximum(2.0 ** -4 * np.abs(x), step)).all()
    codes, scale = bo.pack_weights(x)
    back = bo.unpack_weights(codes, scale)
    assert (np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x), np.exp2(scale.max() - 137.0))).all()


def test_turned_blocks_never_meet():
    rng = np.random.RandomState(3)
    for _ in range(200):
        n = rng.randint(1, 9)
        off = np.cumsum(np.concatenate([[rng.randint(0, 5)], rng.choice([0, 1, 3, 127, 128, 129, 400], n)]))
        rows = off[-1] + rng.randint(0, 3)
        seen = [b for b, _, _ in bo.turned_blocks(off)]
        assert len(set(seen)) == len(seen) and all(0 <= b < rows // 128 + n for b in seen)


@pytest.mark.parametrize("act", ["relu", "gelu", "silu", "swiglu"])
def test_gradient_against_differences(act):
    rng = np.random.RandomState(4)
    z, h = rng.randn(5, 128), 1e-6
    dy = rng.randn(5, 64 if act == "swiglu" else 128)
    got = bo.packed_values(act, z, dy)
    for i, j in [(0, 3), (2, 70), (4, 127)]:
        step = np.zeros_like(z)
        step[i, j] = h
        diff = ((bo.packed_values(act, z + step) - bo.packed_values(act, z - step)) * dy).sum() / (2 * h)
        assert abs(diff - got[i, j]) <= 1e-6 * (1 + abs(diff))


def test_product_gradients_against_differences():
    rng = np.random.RandomState(5)
    x, w, dz = rng.randn(9, 64), rng.randn(2, 128, 64), rng.randn(9, 128)
    off = np.array([1, 4, 9])
    dz[:1] = 0
    dw, _ = bo.weight_grad(x, dz, off)
    dx, _, _ = bo.block_linear(dz, np.swapaxes(w, 1, 2), off)
    f = lambda x, w: (bo.block_linear(x, w, off)[0] * dz).sum()  # noqa: E731
    for i, j in [(1, 0), (5, 63)]:
        s = np.zeros_like(x)
        s[i, j] = 1e-3
        assert abs((f(x + s, w) - f(x - s, w)) / 2e-3 - dx[i, j]) < 1e-8
    s = np.zeros_like(w)
    s[1, 7, 9] = 1e-3
    assert abs((f(x, w + s) - f(x, w - s)) / 2e-3 - dw[1, 7, 9]) < 1e-8


@pytest.mark.parametrize("eight", [False, True])
def test_adamw_against_64_bits(eight):
    """A few fp32 roundings (16 u of the terms) from the step in 64 bits; codes
    hold the two neighbours of the new state's place."""
    rng = np.random.RandomState(6)
    n, t, lr, b1, b2, eps, wd = 700, 5, 1e-2, 0.9, 0.95, 1e-8, 0.1
    p, g = rng.randn(n).astype(np.float32), (rng.randn(n) * 1e-3).astype(np.float32)
    kw = {}
    if eight:
        m, v = rng.randint(-127, 128, n).astype(np.int8), rng.randint(0, 256, n).astype(np.uint8)
        kw = dict(m_scale=rng.rand(3).astype(np.float32) * 1e-7, v_scale=rng.rand(3).astype(np.float32) * 1e-7)
        scale = lambda s: np.repeat(s.astype(float), 256)[:n]  # noqa: E731
        m0 = m.astype(float) * np.abs(m.astype(float)) * scale(kw["m_scale"])
        v0 = (v.astype(float) ** 2 * scale(kw["v_scale"])) ** 2
    else:
        m, v = (rng.randn(n) * 1e-3).astype(np.float32), (rng.randn(n) ** 2 * 1e-6).astype(np.float32)
        m0, v0 = m.astype(float), v.astype(float)
    out = bo.adamw(p, g, m, v, lr=lr, beta1=b1, beta2=b2, eps=eps, step=t, grad_scale=0.5,
                   weight_decay=wd, seed=3, index=1, **kw)
    gg = g.astype(float) * 0.5
    m1, v1 = b1 * m0 + (1 - b1) * gg, b2 * v0 + (1 - b2) * gg * gg
    step = lr / (1 - b1 ** t) * m1 / (np.sqrt(v1 / (1 - b2 ** t)) + eps)
    want = p.astype(float) * (1 - lr * wd) - step
    u = 2.0 ** -24
    # m may cancel: its error is that of its terms
    dm = 8 * u * (np.abs(b1 * m0) + np.abs((1 - b1) * gg))
    dstep = np.abs(step) * 16 * u + lr / (1 - b1 ** t) * dm / (np.sqrt(v1 / (1 - b2 ** t)) + eps)
    assert (np.abs(out[0] - want) <= 4 * u * np.abs(p) + dstep).all()
    if not eight:
        assert (np.abs(out[1] - m1) <= dm).all() and (np.abs(out[2] - v1) <= 16 * u * v1).all()
        return
    c, s = out[1].astype(float), scale(out[3])
    below, above = np.maximum(np.abs(c) - 1, 0) ** 2 * s, (np.abs(c) + 1) ** 2 * s
    assert (np.abs(m1) >= below * (1 - 1e-5) - dm).all() and (np.abs(m1) <= above * (1 + 1e-5) + dm).all()
    c, s = out[2].astype(float), scale(out[4])
    r = np.sqrt(v1)
    assert (r >= np.maximum(c - 1, 0) ** 2 * s * (1 - 1e-5)).all() and (r <= (c + 1) ** 2 * s * (1 + 1e-5)).all()


def test_adamw_codes_are_right_on_average():
    """Each code is drawn between two; over 4000 seeds the mean of v is within 5
    standard deviations (at most half the distance of the two over sqrt 4000)."""
    n, seeds = 8, 4000
    g = np.array([1, 0.9, 0.7, 0.5, 0.3, 0.1, 0.05, 0.01], dtype=np.float32)
    zero8, zero = np.zeros(n, dtype=np.int8), np.zeros(n, dtype=np.uint8)
    m, v = np.zeros(n), np.zeros(n)
    for s in range(seeds):
        out = bo.adamw(g, g, zero8, zero, lr=0.0, beta1=0.0, beta2=0.0, eps=1.0, step=1, seed=s,
                       m_scale=np.zeros(1, np.float32), v_scale=np.zeros(1, np.float32))
        c = out[1].astype(float)
        m += c * np.abs(c) * out[3][0]
        v += (out[2].astype(float) ** 2 * out[4][0]) ** 2
    k = np.floor(np.sqrt(g * 127.0 ** 2))
    assert (np.abs(m / seeds - g) <= 5 * 0.5 * (2 * k + 1) / 127 ** 2 / np.sqrt(seeds) + 1e-6).all()
    k = np.floor(np.sqrt(g * 255.0 ** 2))
    width = ((k + 1) ** 4 - k ** 4) / 255.0 ** 4
    assert (np.abs(v / seeds - g.astype(float) ** 2) <= 5 * 0.5 * width / np.sqrt(seeds) + 1e-6).all()
    assert e4m3_decode(np.array([0x38], dtype=np.uint8))[0] == 1
