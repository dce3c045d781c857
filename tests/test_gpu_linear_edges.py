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
