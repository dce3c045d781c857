"""GPU tests of the calls for experts of one's own where values or sizes are
extreme: against float64, with bounds that count roundings (u = 2^-24)."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_router_amd as moe
from gpu_harness import say, to_np
from oracle import linear_oracle as lo
from oracle.moe_oracle import e4m3_decode
from test_gpu_linear import DEV, DT, U, V, Case, check, poison, workspace

pytestmark = pytest.mark.gpu


def test_fp32_gelu_keeps_its_lower_tail():
    """z in [-10, -4] by the bias alone, so exact.  Forward, relative: the
    argument z / sqrt 2 is off by 2 u, which moves erfc by 2 (z^2 + 1) u; erfcf
    is within 16 ulp (32 u); two products.  Slope Phi + z phi: the exponential's
    argument is rounded once, z^2 / 2 u, expf and products 10 u."""
    say("[linear] fp32 GELU tail")
    z = np.linspace(-10, -4, 64).astype(np.float32)
    c = Case([1], 64, 64, "gelu", "f32")
    c.x.zero_()
    c.w.zero_()
    c.bias = torch.tensor(z[None], device=DEV)
    y, _, _ = c.forward()
    torch.cuda.synchronize()
    zd = z.astype(np.float64)
    ref = lo.activation("gelu", zd)
    check("gelu", y[0], ref, np.abs(ref) * (2 * zd * zd + 64) * U)
    codes, scale = lo.checkpoint_pack(z[None])
    z = (e4m3_decode(codes).astype(np.float32) * scale)[0]
    zd = z.astype(np.float64)
    c.dy.fill_(1.0)
    db = poison((1, 64), torch.float32)
    moe.moe_grouped_linear_backward(
        c.cfg, None, c.offsets, None, c.dy, z_codes=torch.tensor(codes, device=DEV),
        z_scale=torch.tensor(scale, device=DEV), dbias=db,
        workspace=workspace(moe.alloc_linear_backward_workspace(c.cfg, DEV)))
    torch.cuda.synchronize()
    cdf = lo.activation("gelu", zd) / zd
    pdf = np.exp(-zd * zd / 2) / np.sqrt(2 * np.pi)
    ref = lo.activation_backward("gelu", zd, np.ones_like(zd))
    check("gelu slope", db[0], ref,
          (cdf * (2 * zd * zd + 64) + np.abs(zd) * pdf * (zd * zd + 64)) * U)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bias_gradient_of_many_rows(dtype):
    """A million equal values: every addition of a running fp32 sum would round
    the same way.  16 rows of a tile one after another (16 u), 8 tiles at a
    time (8 u), those in sums that keep what each addition rounds off (8 u)."""
    say(f"[linear] bias gradient of many rows {dtype}")
    sizes = [3, (1 << 20) + 5, 0, 40000]
    off = np.concatenate([[0], np.cumsum(sizes)])
    cfg = moe.make_linear_config(int(off[-1]), 4, 64, 64, dtype=DT[dtype])
    dy = torch.full((int(off[-1]), 64), 0.1, dtype=DT[dtype], device=DEV)
    dy[:, 1] = -0.7
    db = poison((4, 64), torch.float32)

    def run():
        moe.moe_grouped_linear_backward(
            cfg, None, torch.tensor(off, dtype=torch.int32, device=DEV), None, dy, dbias=db,
            workspace=workspace(moe.alloc_linear_backward_workspace(cfg, DEV)))
        torch.cuda.synchronize()

    run()
    ref = np.array(sizes)[:, None] * to_np(dy[0]).astype(np.float64)
    check("dbias", db, ref, 32 * U * np.abs(ref))
    # what is not finite stays what it is
    dy[5, 2], dy[6, 3], dy[6, 4], dy[70000, 4] = (float(v) for v in ("inf", "nan", "inf", "-inf"))
    before = db.clone()
    run()
    assert bool(torch.isposinf(db[1, 2])) and bool(torch.isnan(db[1, 3:5]).all())
    keep = torch.ones_like(db, dtype=torch.bool)
    keep[1, 2:5] = False
    assert torch.equal(db[keep], before[keep])


def test_fp8_weights_past_the_limit_of_a_gradient():
    """512 experts of 4096 -> 2 x 16448, 69 GB of codes, of which the first and
    the last have rows; their weights begin past 2^35 and end past 2^36."""
    say("[linear] 2^36 FP8 weights")
    G, K, F = 512, 4096, 16448
    cfg = moe.make_linear_config(3, G, K, F, activation="swiglu",
                                 weight_format=moe.MOE_WEIGHTS_FP8_E4M3)
    g = torch.Generator(device=DEV).manual_seed(4)
    w = torch.empty((G, 2 * F, K), dtype=torch.uint8, device=DEV)
    scale = torch.full((G, 2 * F), float("nan"), device=DEV)
    x = torch.randn((3, K), generator=g, device=DEV).bfloat16()
    offsets = torch.full((G + 1,), 1, dtype=torch.int32, device=DEV)
    offsets[0], offsets[G] = 0, 3
    y = poison((3, F), torch.bfloat16)
    for e in (0, G - 1):
        codes = torch.randint(0, 120, (2 * F, K), generator=g, device=DEV, dtype=torch.uint8)
        w[e] = codes ^ (torch.randint(0, 2, (2 * F, K), generator=g, device=DEV,
                                      dtype=torch.uint8) << 7)
        scale[e] = 1e-4 * (1 + torch.rand(2 * F, generator=g, device=DEV))
    moe.moe_grouped_linear(cfg, x, offsets, w, y, w_scale=scale,
                           workspace=workspace(moe.alloc_linear_workspace(cfg, DEV)))
    torch.cuda.synchronize()
    for e, r in ((0, slice(0, 1)), (G - 1, slice(1, 3))):
        we = w[e].view(torch.float8_e4m3fn).float().double() * scale[e].double()[:, None]
        z = (x[r].double() @ we.t()).cpu().numpy()
        dz = (K + 8) * U * (x[r].double().abs() @ we.abs().t()).cpu().numpy()
        a, b = np.split(z, 2, axis=1)
        da, db = np.split(dz, 2, axis=1)
        ref = lo.activation("swiglu", z)
        err = 1.1 * da * np.abs(b) + np.abs(lo.activation("silu", a)) * db + da * db
        err = err + 2.0 ** -17 * np.abs(a) * np.abs(b)
        check(f"expert {e}", y[r], ref, (1 + V) * err + V * np.abs(ref))


@pytest.mark.parametrize("sizes,K,F,act", [
    ([3, 2], 64, 64, "none"), ([1, 3], 1024, 192, "swiglu"), ([90, 40], 2112, 320, "silu"),
    ([200, 130], 192, 192, "swiglu"), ([300, 270, 513], 256, 8192, "none"),
    ([300, 270, 513], 128, 4160, "swiglu")])
@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
def test_checkpoint_of_a_forward_that_is_not_finite(sizes, K, F, act, dtype):
    """Infinities and NaN in z, by its bias: the NaN code, and no part in the
    scale of their blocks, whose other values keep their bounds."""
    say(f"[linear] not finite {sizes} {K}x{F} {act} {dtype}")
    c = Case(sizes, K, F, act, "f32" if dtype == "f32" else "bf16", fp8=dtype == "fp8", bias=True)
    _, good_codes, good_scale = c.forward(True)
    for e in range(len(sizes)):
        for i, v in enumerate(("inf", "nan", "-inf")):
            c.bias[e, (17 * e + 21 * i) % c.zd] = float(v)
    c.bias[0, c.zd - 64:] = float("-inf")  # a block without a finite value
    y, codes, scale = c.forward(True)
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):  # -inf * 0
        ref, z = lo.grouped_linear(c.hx, c.off, c.hw, act, None, to_np(c.bias))
    n = c.rows
    ok = np.isfinite(z)
    assert np.array_equal(np.isfinite(to_np(y)), np.isfinite(ref))
    hc = to_np(codes)
    assert np.array_equal((hc & 0x7F) == 0x7F, ~ok)
    dz = np.where(ok, (K + 8) * U * c.z_bound(), 0.0)
    zf = np.where(ok, z, 0.0)
    m = np.maximum(np.abs(zf).reshape(n, -1, 64).max(2), 1e-30)
    dm = dz.reshape(n, -1, 64).max(2)
    check("scale", scale, m / 448, (dm + 4 * U * m) / 448)
    back = np.where(ok, lo.checkpoint_unpack(hc, to_np(scale)), 0.0)
    step = np.repeat((m + dm) / 448 * 2.0 ** -10, 64, axis=1)
    check("checkpoint", torch.tensor(back), zf,
          dz + np.maximum((np.abs(zf) + dz) / 16, step) * (1 + 8 * U))
    whole = ok.reshape(n, -1, 64).all(2)
    assert np.array_equal(to_np(scale)[whole], to_np(good_scale)[whole])
    assert np.array_equal(hc.reshape(n, -1, 64)[whole],
                          to_np(good_codes).reshape(n, -1, 64)[whole])


def test_rows_gathered_from_four_gigabytes():
    """x of more than 2^32 bytes read through row_index, its last rows among
    those read; the rows that are not read hold NaN."""
    say("[linear] gather from 4 GiB")
    sizes, K, F, n_x = [600, 0, 300], 1024, 8192, (1 << 21) + 5
    rows = sum(sizes)
    off = np.concatenate([[0], np.cumsum(sizes)])
    g = torch.Generator(device=DEV).manual_seed(6)
    index = torch.randint(0, n_x, (rows,), generator=g, device=DEV, dtype=torch.int32)
    index[::7] = n_x - 1
    index[1::7] = torch.arange(n_x - 130, n_x - 1, device=DEV, dtype=torch.int32)[:len(index[1::7])]
    x = poison((n_x, K), torch.bfloat16)
    x[index.long()] = torch.randn((rows, K), generator=g, device=DEV).bfloat16()
    w = (torch.randn((3, F, K), generator=g, device=DEV) / 32).bfloat16()
    dy = torch.randn((rows, F), generator=g, device=DEV).bfloat16()
    offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
    cfg = moe.make_linear_config(rows, 3, K, F, x_rows=n_x)
    y, dw = poison((rows, F), torch.bfloat16), poison((3, F, K), torch.bfloat16)
    moe.moe_grouped_linear(cfg, x, offsets, w, y, row_index=index,
                           workspace=workspace(moe.alloc_linear_workspace(cfg, DEV)))
    moe.moe_grouped_linear_backward(
        cfg, x, offsets, None, dy, row_index=index, dw=dw,
        workspace=workspace(moe.alloc_linear_backward_workspace(cfg, DEV)))
    torch.cuda.synchronize()
    for e, n in enumerate(sizes):
        r = slice(int(off[e]), int(off[e + 1]))
        xe, we, de = x[index[r].long()].double(), w[e].double(), dy[r].double()
        for name, got, ref, terms, k in (
                ("y", y[r], xe @ we.t(), xe.abs() @ we.abs().t(), K),
                ("dw", dw[e], de.t() @ xe, de.abs().t() @ xe.abs(), n)):
            tol = (1 + V) * (k + 8) * U * terms + V * ref.abs()
            check(f"{name}[{e}]", got, ref.cpu().numpy(), tol.cpu().numpy())


def test_combine_of_the_widest_rows():
    """d = 2^31 - 64: columns up to the last that 31 bits can count."""
    say("[combine] widest rows")
    d = (1 << 31) - 64
    rows = torch.empty((2, d), dtype=torch.bfloat16, device=DEV)
    rows[0].fill_(float("nan"))
    rows[1].view(-1, 64).copy_(torch.arange(64, device=DEV, dtype=torch.bfloat16))
    rows[1, -1] = 77
    guard = poison((d + 8192,), torch.bfloat16)
    y, tail = guard[:d].view(1, d), guard[d:]
    slot = torch.tensor([[1]], dtype=torch.int32, device=DEV)
    moe.moe_combine(rows, slot, y)
    torch.cuda.synchronize()
    assert torch.equal(y[0].view(torch.int16), rows[1].view(torch.int16))
    assert bool(torch.isnan(tail).all())
    drows = poison((2, d), torch.bfloat16)
    moe.moe_combine_backward(rows, slot, None, y, drows, None)
    torch.cuda.synchronize()
    assert bool(torch.isnan(drows[0]).all())
    assert torch.equal(drows[1].view(torch.int16), rows[1].view(torch.int16))


@pytest.mark.parametrize("last", [-(1 << 31), -(1 << 31) + 5, -1, (1 << 31) - 1])
def test_gathered_rows_stay_inside_whatever_the_offsets(last):
    """dW of rows read through row_index, on the large tiles, with a last
    offset far outside [0, rows]: nothing past the workspace is written."""
    say(f"[linear] gather with last offset {last}")
    rows, K, F = 37, 2048, 2048
    cfg = moe.make_linear_config(rows, 2, K, F, x_rows=11)
    n = moe.moe_linear_backward_workspace_size(cfg)
    space = torch.full((n + (1 << 20),), 0xA5, dtype=torch.uint8, device=DEV)
    x, dy = (torch.randn((r, c), device=DEV).bfloat16() for r, c in ((11, K), (rows, F)))
    index = (torch.arange(rows, device=DEV) % 11).int()
    dw = poison((2, F, K), torch.bfloat16)
    moe.moe_grouped_linear_backward(
        cfg, x, torch.tensor([0, 20, last], dtype=torch.int32, device=DEV), None, dy,
        row_index=index, dw=dw, workspace=space[:n])
    torch.cuda.synchronize()
    assert bool((space[n:] == 0xA5).all())
    if last > 0:
        for e, r in ((0, slice(0, 20)), (1, slice(20, rows))):
            de, xe = dy[r].double(), x[index[r].long()].double()
            ref = (de.t() @ xe).cpu().numpy()
            terms = (de.abs().t() @ xe.abs()).cpu().numpy()
            check(f"dw[{e}]", dw[e], ref, (1 + V) * 45 * U * terms + V * np.abs(ref))
    else:
        assert bool((dw[1] == 0).all())  # the second group has no rows
