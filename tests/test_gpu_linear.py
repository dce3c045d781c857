"""GPU parity of the calls for experts of one's own against the float64 oracle
(oracle/linear_oracle.py), element by element.

Tolerances count roundings.  u = 2^-24 (fp32), v = 2^-8 (bf16, half a step).
  z    sum of K products in fp32: (K + 8) u S with S = sum |x w| + |b|, the
       terms of the sum; FP8 weights are exact in bf16 and one multiplication
       by the scale adds u.
  act  slopes are below 1.13 (GELU 1.129, SiLU 1.0998), so an error dz in z
       gives 1.13 dz; SwiGLU 1.1 da |b| + |SiLU(a)| db + da db.  Evaluating
       the function: fp32 16 u |z| (erff, expf, a division and products, each
       a few u), bf16 2^-17 |z| (the hardware's exponential and reciprocal);
       SwiGLU times |b|.
  y    one rounding to its type, of the exact value and of the error: v or u.
  dz   slope evaluation 16 u (1 + |z|) or 2^-16 (1 + |z|) on |dy| (|u| for
       SwiGLU), then a rounding to the type; z itself is code * scale, one
       fp32 rounding, within 4 u |z| |dy| (second derivatives are below 1.1).
  dx, dw   sum |dz w| times (the relative error of dz + (K + 8) u), and the
       rounding of the result.
Groups, rows behind the last one, NaN in every place that a call must not
read, and outputs that start as NaN are part of every case.
"""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_router_amd as moe
from gpu_harness import say, to_np
from oracle import linear_oracle as lo
from oracle.moe_oracle import e4m3_decode
from workloads import to_e4m3

pytestmark = pytest.mark.gpu

U, V = 2.0 ** -24, 2.0 ** -8
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"


def poison(shape, dtype):
    if dtype in (torch.int32, torch.uint8):
        return torch.full(shape, 0x7F if dtype == torch.uint8 else -7, dtype=dtype, device=DEV)
    return torch.full(shape, float("nan"), dtype=dtype, device=DEV)


def workspace(t):
    return t.fill_(0xFF)


def check(label, got, ref, tol):
    got = to_np(got).astype(np.float64)
    diff = np.abs(got - ref)
    bad = ~(diff <= tol)
    worst = float(np.max(diff / np.maximum(tol, 1e-300))) if diff.size else 0.0
    say(f"[linear] {label}: worst {worst:.3f} of its bound")
    assert not bad.any(), (f"{label}: {int(bad.sum())} of {bad.size} off, first at "
                           f"{np.argwhere(bad)[0]}: {got[bad][0]} for {ref[bad][0]}, bound "
                           f"{np.broadcast_to(tol, bad.shape)[bad][0]}")


class Case:
    """One random problem: groups of the given sizes, `spare` rows behind the
    last one, x read through row_index (from x_rows rows, some of them never)
    or directly."""

    def __init__(self, sizes, K, F, act, dtype="bf16", gather=False, bias=False, residual=False,
                 fp8=False, spare=0, seed=0):
        self.act, self.dtype, self.fp8, self.K, self.F = act, dtype, fp8, K, F
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        dt = self.dt = DT[dtype]
        G, self.used = len(sizes), sum(sizes)
        self.rows = self.used + spare
        self.zd = F * (2 if act == "swiglu" else 1)
        self.off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        self.offsets = torch.tensor(self.off, device=DEV)
        randn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
        self.x_rows = (self.rows * 2 // 3 + 3) if gather else 0
        n_x = self.x_rows or self.rows
        self.x = randn(n_x, K).to(dt)
        self.index = None
        if gather:  # the same row several times, some rows never (NaN), garbage behind the last
            self.index = torch.randint(0, n_x - 2, (self.rows,), generator=g, device=DEV,
                                       dtype=torch.int32)
            self.index[self.used:] = 1 << 29
            unused = torch.ones(n_x, dtype=torch.bool, device=DEV)
            unused[self.index[:self.used].long()] = False
            self.x[unused] = float("nan")
        else:
            self.x[self.used:] = float("nan")
        self.w = (randn(G, self.zd, K) * K ** -0.5).to(dt)
        self.w_scale = None
        if fp8:
            self.w, self.w_scale = to_e4m3(self.w)
        self.bias = randn(G, self.zd) * 0.3 if bias else None
        self.residual = None
        if residual:
            self.residual = randn(self.rows, F).to(dt)
        self.dy = randn(self.rows, F).to(dt)
        self.dy[self.used:] = float("nan")
        self.cfg = moe.make_linear_config(
            self.rows, G, K, F, dtype=dt, activation=act, x_rows=self.x_rows,
            weight_format=moe.MOE_WEIGHTS_FP8_E4M3 if fp8 else moe.MOE_WEIGHTS_DTYPE)
        # host copies for the oracle
        self.hx = to_np(self.x).astype(np.float64)
        self.hi = None if self.index is None else to_np(self.index)
        w = e4m3_decode(to_np(self.w)) * to_np(self.w_scale)[..., None] if fp8 else to_np(self.w)
        self.hw = w.astype(np.float64)

    def forward(self, save=False, stream=None, inplace=False):
        y = poison((self.rows, self.F), self.dt)
        if inplace:
            y = self.residual.clone()
        codes = poison((self.rows, self.zd), torch.uint8) if save else None
        scale = poison((self.rows, self.zd // 64), torch.float32) if save else None
        moe.moe_grouped_linear(self.cfg, self.x, self.offsets, self.w, y, row_index=self.index,
                               w_scale=self.w_scale, bias=self.bias,
                               residual=y if inplace else self.residual, z_codes=codes,
                               z_scale=scale, workspace=workspace(
                                   moe.alloc_linear_workspace(self.cfg, DEV)), stream=stream)
        return y, codes, scale

    def z_bound(self):
        """sum |x w| + |b| of every z."""
        z = np.zeros((self.used, self.zd))
        for e in range(len(self.off) - 1):
            a, b = self.off[e], self.off[e + 1]
            if b > a:
                src = self.hx[self.hi[a:b]] if self.hi is not None else self.hx[a:b]
                z[a:b] = np.abs(src) @ np.abs(self.hw[e]).T
                if self.bias is not None:
                    z[a:b] += np.abs(to_np(self.bias[e]))
        return z

    def check_forward(self, label, save=False, inplace=False):
        y, codes, scale = self.forward(save, inplace=inplace)
        torch.cuda.synchronize()
        n = self.used
        res = None if self.residual is None else to_np(self.residual)[:n]
        ref, z = lo.grouped_linear(self.hx, self.off, self.hw, self.act, self.hi,
                                   None if self.bias is None else to_np(self.bias), res)
        dz = (self.K + 8) * U * self.z_bound()
        f = 16 * U if self.dtype == "f32" else 2.0 ** -17
        r = U if self.dtype == "f32" else V
        if self.act == "swiglu":
            a, b = np.split(z, 2, axis=1)
            da, db = np.split(dz, 2, axis=1)
            err = 1.1 * da * np.abs(b) + np.abs(lo.activation("silu", a)) * db + da * db
            err = err + f * np.abs(a) * np.abs(b)
        elif self.act == "none":
            err = dz
        else:
            err = 1.13 * dz + f * np.abs(z)
        err = err + (0 if res is None else 2 * U * np.abs(res))
        check(f"{label} y", y[:n], ref, (1 + r) * err + r * np.abs(ref) + 1e-37)
        tail = self.residual[n:] if inplace else poison((self.rows - n, self.F), self.dt)
        assert torch.equal(y[n:].view(torch.uint8), tail.view(torch.uint8)), "rows behind the last"
        if save:
            m = np.maximum(np.abs(z).reshape(n, self.zd // 64, 64).max(2), 1e-30)
            dm = dz.reshape(n, self.zd // 64, 64).max(2)
            check(f"{label} scale", scale[:n], m / 448, (dm + 4 * U * m) / 448)
            back = lo.checkpoint_unpack(to_np(codes)[:n], to_np(scale)[:n])
            step = np.repeat((m + dm) / 448 * 2.0 ** -10, 64, axis=1)
            tol = dz + np.maximum((np.abs(z) + dz) / 16, step) * (1 + 8 * U)
            check(f"{label} checkpoint", torch.tensor(back), z, tol)
            assert bool((codes[n:] == 0x7F).all()) and bool(torch.isnan(scale[n:]).all())
        return y, codes, scale

    def check_backward(self, label, codes=None, scale=None, want=("dx", "dw", "dbias")):
        n, G = self.used, len(self.off) - 1
        if self.act != "none" and codes is None:
            z = torch.randn((self.rows, self.zd), device=DEV,
                            generator=torch.Generator(device=DEV).manual_seed(99)) * 1.5
            c, s = lo.checkpoint_pack(z.cpu().numpy())
            codes, scale = torch.tensor(c, device=DEV), torch.tensor(s, device=DEV)
            codes[n:], scale[n:] = 0x7F, float("nan")
        out = {"dx": poison((self.rows, self.K), self.dt) if "dx" in want else None,
               "dw": poison((G, self.zd, self.K), self.dt) if "dw" in want else None,
               "dbias": poison((G, self.zd), torch.float32) if "dbias" in want else None}
        moe.moe_grouped_linear_backward(
            self.cfg, self.x if "dw" in want else None, self.offsets,
            self.w if "dx" in want else None, self.dy,
            row_index=self.index if "dw" in want else None, z_codes=codes, z_scale=scale,
            workspace=workspace(moe.alloc_linear_backward_workspace(self.cfg, DEV)), **out)
        torch.cuda.synchronize()
        dy = to_np(self.dy).astype(np.float64)
        z = None
        if self.act != "none":
            z = lo.checkpoint_unpack(to_np(codes), to_np(scale))
        dx, dw, db, dz = lo.grouped_linear_backward(self.hx, self.off, self.hw, dy, z, self.act,
                                                    self.hi)
        r = U if self.dtype == "f32" else V
        e = np.zeros_like(dz)  # error of dz before it is rounded to its type
        if self.act != "none":
            f = 16 * U if self.dtype == "f32" else 2.0 ** -16
            if self.act == "swiglu":
                a, b = np.split(z, 2, axis=1)
                da = np.abs(dy) * np.abs(b) * ((f + 4 * U) * (1 + np.abs(a)))
                db_ = np.abs(dy) * (f + 8 * U) * (1 + np.abs(a))
                e = np.concatenate([da, db_], axis=1)
            else:
                e = np.abs(dy) * (f + 4 * U) * (1 + np.abs(z))
        eb = e + r * (np.abs(dz) + e) if self.act != "none" else e  # and after
        aw = np.abs(self.hw)
        for g in range(G):
            a, b = self.off[g], self.off[g + 1]
            src = np.abs(self.hx[self.hi[a:b]] if self.hi is not None else self.hx[a:b])
            t = np.abs(dz[a:b])
            if out["dx"] is not None and b > a:
                err = eb[a:b] @ aw[g] + (self.zd + 8) * U * ((t + eb[a:b]) @ aw[g])
                check(f"{label} dx[{g}]", out["dx"][a:b], dx[a:b],
                      (1 + r) * err + r * np.abs(dx[a:b]) + 1e-37)
            if out["dw"] is not None:
                err = eb[a:b].T @ src + (b - a + 8) * U * ((t + eb[a:b]).T @ src)
                check(f"{label} dw[{g}]", out["dw"][g], dw[g],
                      (1 + r) * err + r * np.abs(dw[g]) + 1e-37)
            if out["dbias"] is not None:
                err = e[a:b].sum(0) + (b - a + 8) * U * (t + e[a:b]).sum(0)
                check(f"{label} dbias[{g}]", out["dbias"][g], db[g], err + U * np.abs(db[g]))
        if out["dx"] is not None:
            assert bool(torch.isnan(out["dx"][n:]).all()), "rows behind the last"
        return out


RAGGED = [130, 257, 0, 64, 300, 1, 0, 31, 16, 17, 33, 512]
FORWARD = [
    # sizes, K, F, act, options
    ([1], 64, 64, "none", {}),
    ([3, 0, 5, 1], 128, 64, "gelu", dict(bias=True)),
    ([33, 31, 0, 32, 65], 192, 128, "silu", dict(gather=True, spare=3)),
    ([0, 0, 0], 64, 64, "relu", dict(spare=5)),
    ([17, 2], 448, 320, "swiglu", dict(gather=True, bias=True)),
    ([1] * 70, 64, 128, "swiglu", dict(residual=True)),
    ([130, 257, 0, 64], 256, 192, "relu", dict(residual=True, bias=True, spare=40)),
    ([700], 320, 576, "none", dict(bias=True, residual=True)),
    ([511, 1, 300], 512, 448, "swiglu", dict(gather=True, bias=True, spare=9)),
    ([260, 513], 1024, 256, "gelu", dict()),
    ([2, 300, 0, 1], 640, 320, "silu", dict(bias=True, gather=True)),
    # few workgroups and a long K: split over K, joined by a second launch
    ([1, 0, 3], 1024, 192, "gelu", dict(bias=True, residual=True)),
    ([2, 5, 0, 1], 1152, 128, "swiglu", dict(gather=True, bias=True, spare=3)),
    ([0, 30, 17], 2112, 64, "none", dict(spare=70)),
    ([1], 4096, 64, "silu", dict(bias=True)),
    # the same with more rows, on 64 x 64 tiles
    ([200, 0, 77], 4160, 192, "swiglu", dict(gather=True, bias=True, spare=5)),
    ([90], 2112, 320, "silu", dict(bias=True, residual=True)),
    ([60, 0, 0, 61, 0, 200], 2304, 64, "none", dict(residual=True, spare=70)),
    # enough 256 x 256 tiles (more than a quarter of the compute units) for the
    # large-tile kernel in dX and dW, groups of all fillings
    (RAGGED, 1088, 1088, "silu", dict(gather=True, bias=True)),
    (RAGGED, 1024, 576, "swiglu", dict(gather=True, bias=True, spare=9)),
    (RAGGED, 640, 832, "none", dict(bias=True, residual=True, spare=1)),
    (RAGGED, 1152, 1088, "gelu", dict(residual=True)),
    ([0] * 20 + [160] + [0] * 9 + [96] * 2, 512, 320, "relu", dict()),
    # and in the forward (by the rows, or with few rows a group by the groups)
    (RAGGED, 320, 3264, "silu", dict(gather=True, bias=True)),
    (RAGGED, 384, 1664, "swiglu", dict(gather=True, bias=True, spare=9)),
    (RAGGED, 256, 3264, "none", dict(bias=True, residual=True, spare=1)),
    (RAGGED[:6] + [20] * 34, 384, 1664, "gelu", dict(residual=True)),
    # full rounds of 128 x 128 tiles in fp32: forward and dW, dX
    ([1000], 1024, 8192, "relu", dict(bias=True)),
    ([1010], 8192, 64, "silu", dict(spare=5)),
]
IDS = [f"{len(s)}g{sum(s)}r_{K}x{F}_{a}" for s, K, F, a, _ in FORWARD]


@pytest.mark.parametrize("save", [False, True], ids=["plain", "saved"])
@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("sizes,K,F,act,opt", FORWARD, ids=IDS)
def test_forward(sizes, K, F, act, opt, dtype, save):
    say(f"[linear] forward {sizes} {K}x{F} {act} {opt} {dtype} save={save}")
    c = Case(sizes, K, F, act, "f32" if dtype == "f32" else "bf16", fp8=dtype == "fp8", **opt)
    c.check_forward(f"{act} {dtype}", save)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sizes,K,F,act,opt", FORWARD, ids=IDS)
def test_backward(sizes, K, F, act, opt, dtype):
    say(f"[linear] backward {sizes} {K}x{F} {act} {opt} {dtype}")
    opt = {k: v for k, v in opt.items() if k != "residual"}
    Case(sizes, K, F, act, dtype, **opt).check_backward(f"{act} {dtype}")


@pytest.mark.parametrize("want", [("dx",), ("dw",), ("dbias",), ("dw", "dbias")], ids="-".join)
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_backward_of_some(act, want):
    say(f"[linear] backward of {want} {act}")
    Case([5, 0, 300], 128, 192, act, gather=True, spare=2).check_backward(act, want=want)


def test_residual_in_place():
    say("[linear] y is the residual")
    for sizes, F in (([9, 4], 192), ([300, 270], 192), (RAGGED, 1088),
                     (RAGGED, 3264)):
        Case(sizes, 128, F, "gelu", residual=True, spare=3).check_forward("in place", inplace=True)


@pytest.mark.parametrize("groups,K,F", [(3, 128, 192), (40, 512, 448), (40, 448, 1664)],
                         ids=["small", "large", "wide"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_neighbours_stay_apart(dtype, groups, K, F):
    """One group's NaN and infinities reach none of the others' outputs,
    whatever tiles they share."""
    say(f"[linear] neighbours {dtype}")
    c = Case([37, 70, 5] + [9] * (groups - 3), K, F, "silu", dtype)
    a, b = int(c.off[1]), int(c.off[2])
    ref = c.check_backward("before")
    y0, codes, scale = c.forward(True)
    ref = c.check_backward("saved", codes, scale)
    c.x[a:b], c.dy[a:b] = float("inf"), float("nan")
    c.w[1] = float("nan")
    y, _, _ = c.forward()
    out = {"dx": poison((c.rows, c.K), c.dt), "dw": poison((groups, c.zd, c.K), c.dt),
           "dbias": poison((groups, c.zd), torch.float32)}
    moe.moe_grouped_linear_backward(c.cfg, c.x, c.offsets, c.w, c.dy, z_codes=codes,
                                    z_scale=scale, workspace=workspace(
                                        moe.alloc_linear_backward_workspace(c.cfg, DEV)), **out)
    torch.cuda.synchronize()
    for r in (slice(0, a), slice(b, c.rows)):
        assert torch.equal(y[r], y0[r]) and torch.equal(out["dx"][r], ref["dx"][r])
    for e in [0] + list(range(2, groups)):
        assert torch.equal(out["dw"][e], ref["dw"][e])
        assert torch.equal(out["dbias"][e], ref["dbias"][e])


@pytest.mark.parametrize("rows,groups", [(40, 4), (700, 3)])
def test_offsets_are_clamped(rows, groups):
    """Offsets outside [0, rows] or decreasing are clamped: rows of a group
    that they still describe are right, and nothing outside is written."""
    say(f"[linear] clamped offsets {rows} {groups}")
    c = Case([rows // groups] * groups, 64, 128, "none")
    good, _, _ = c.forward()
    guard = poison((c.rows + 64, c.F), c.dt)
    y = guard[32:32 + c.rows]
    n = rows // groups
    off = [0, n, 1 << 30, 5] if groups == 3 else [-9, n, 2 * n, 1 << 30, -1]
    moe.moe_grouped_linear(c.cfg, c.x, torch.tensor(off, dtype=torch.int32, device=DEV), c.w, y,
                           workspace=moe.alloc_linear_workspace(c.cfg, DEV))
    torch.cuda.synchronize()
    assert torch.equal(y[:n], good[:n])
    if groups == 4:
        assert torch.equal(y[n:2 * n], good[n:2 * n])
    assert bool(torch.isnan(guard[:32]).all()) and bool(torch.isnan(guard[32 + c.rows:]).all())
    # the backward writes nothing outside either, and every group's dw and dbias
    gx = poison((c.rows + 64, c.K), c.dt)
    gw = poison((groups + 2, c.zd, c.K), c.dt)
    gb = poison((groups + 2, c.zd), torch.float32)
    moe.moe_grouped_linear_backward(
        c.cfg, c.x, torch.tensor(off, dtype=torch.int32, device=DEV), c.w, c.dy,
        dx=gx[32:32 + c.rows], dw=gw[1:1 + groups], dbias=gb[1:1 + groups],
        workspace=workspace(moe.alloc_linear_backward_workspace(c.cfg, DEV)))
    torch.cuda.synchronize()
    assert bool(torch.isnan(gx[:32]).all()) and bool(torch.isnan(gx[32 + c.rows:]).all())
    for t in (gw, gb):
        assert bool(torch.isnan(t[0]).all()) and bool(torch.isnan(t[-1]).all())
        assert not bool(torch.isnan(t[1]).any())


def test_results_repeat_and_streams_do_not_matter():
    say("[linear] repeat, another stream")
    for sizes, F in (([3, 17, 0, 9], 192), ([300, 40, 600], 192), (RAGGED, 576), ([2, 1], 128)):
        c = Case(sizes, {192: 256, 576: 1024, 128: 2048}[F], F, "swiglu", gather=True, bias=True)
        y0, codes, scale = c.forward(True)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        y1, codes1, scale1 = c.forward(True, stream=side)
        with torch.cuda.stream(side):
            y2, _, _ = c.forward(False)
        torch.cuda.synchronize()
        for a, b in ((y0, y1), (y0, y2), (codes, codes1), (scale, scale1)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        g0 = c.check_backward("first", codes, scale)
        g1 = c.check_backward("second", codes, scale)
        for n in g0:
            assert torch.equal(g0[n].view(torch.uint8), g1[n].view(torch.uint8))


@pytest.mark.parametrize("sizes,K,F", [([3, 4, 2, 6, 1], 64, 64), (RAGGED, 832, 1088)],
                         ids=["few", "many"])
def test_a_range_of_experts(sizes, K, F):
    """A call on some of the experts: offsets that start past row 0 and end
    before the last row.  The other rows are left as they were."""
    say(f"[linear] experts 1 .. {len(sizes) - 2} of {len(sizes)}")
    c = Case(sizes, K, F, "gelu", gather=True, bias=True)
    y0, codes0, scale0 = c.forward(True)
    g0 = c.check_backward("all", codes0, scale0)
    G = len(sizes) - 2
    a, b = int(c.off[1]), int(c.off[G + 1])
    cfg = moe.make_linear_config(c.rows, G, K, F, activation="gelu", x_rows=c.x_rows)
    off, w, bias = c.offsets[1:G + 2], c.w[1:G + 1], c.bias[1:G + 1]
    y, codes = poison((c.rows, F), c.dt), poison((c.rows, c.zd), torch.uint8)
    scale = poison((c.rows, c.zd // 64), torch.float32)
    moe.moe_grouped_linear(cfg, c.x, off, w, y, row_index=c.index, bias=bias, z_codes=codes,
                           z_scale=scale, workspace=workspace(moe.alloc_linear_workspace(cfg)))
    out = {"dx": poison((c.rows, K), c.dt), "dw": poison((G, c.zd, K), c.dt),
           "dbias": poison((G, c.zd), torch.float32)}
    moe.moe_grouped_linear_backward(
        cfg, c.x, off, w, c.dy, row_index=c.index, z_codes=codes, z_scale=scale,
        workspace=workspace(moe.alloc_linear_backward_workspace(cfg)), **out)
    torch.cuda.synchronize()
    r = to_np(y[a:b]).astype(np.float64) - to_np(y0[a:b])  # another kernel may take fewer experts
    assert np.abs(r).max(initial=0) <= 2 * V * np.abs(to_np(y0[a:b])).max(initial=0)
    assert bool(torch.isnan(y[:a]).all()) and bool(torch.isnan(y[b:]).all())
    assert bool((codes[:a] == 0x7F).all()) and bool((codes[b:] == 0x7F).all())
    assert bool(torch.isnan(out["dx"][:a]).all()) and bool(torch.isnan(out["dx"][b:]).all())
    for n, part in (("dx", slice(a, b)), ("dw", slice(1, G + 1)), ("dbias", slice(1, G + 1))):
        got = out[n][part] if n == "dx" else out[n]
        ref = to_np(g0[n][part]).astype(np.float64)
        assert np.linalg.norm(to_np(got) - ref) <= 2 ** -6 * np.linalg.norm(ref), n


@pytest.mark.parametrize("groups", [64, 65, 128, 511, 512])
def test_many_groups(groups):
    """As many groups as lanes, one more, and the most there may be, a third
    of them without rows."""
    say(f"[linear] {groups} groups")
    sizes = [(7 * e) % 9 if e % 3 else 0 for e in range(groups)]
    sizes[-1] = 5
    c = Case(sizes, 128, 64, "silu", gather=True, spare=2)
    y, codes, scale = c.check_forward(f"{groups} groups", True)
    c.check_backward(f"{groups} groups", codes, scale)
    Case(sizes, 64, 64, "none", "f32").check_backward(f"{groups} groups f32")


def test_offsets_past_32_bits():
    """Arrays of more than 2^31 elements and 4 GiB: the last rows of every
    output, and the sums over all rows, against fp32 products on the GPU (sums
    of 64 products; over 70000 rows (70000 / 64 + 64) u of the terms)."""
    say("[linear] past 32 bits")
    R, K, F = 70000, 64, 32768
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn((R, K), generator=g, device=DEV).bfloat16()
    w = (torch.randn((1, F, K), generator=g, device=DEV) * 0.125).bfloat16()
    off = torch.tensor([0, R], dtype=torch.int32, device=DEV)
    cfg = moe.make_linear_config(R, 1, K, F, activation="silu")
    y = poison((R, F), torch.bfloat16)
    codes, scale = poison((R, F), torch.uint8), poison((R, F // 64), torch.float32)
    moe.moe_grouped_linear(cfg, x, off, w, y, z_codes=codes, z_scale=scale,
                           workspace=moe.alloc_linear_workspace(cfg))
    tail = slice(R - 300, R)
    z = x[tail].float() @ w[0].float().t()
    h = z * torch.sigmoid(z)
    assert bool(((y[tail].float() - h).abs() <= 1.01 * V * h.abs() + 1e-4).all())
    back = poison((R, F), torch.bfloat16)
    moe.moe_checkpoint_unpack(codes, scale, back)
    m = z.abs().reshape(300, -1, 64).amax(2, keepdim=True).expand(-1, -1, 64).reshape(300, F)
    assert bool(((back[tail].float() - z).abs() <= z.abs() * (1 / 16 + 2 * V) + m / 448 / 512).all())
    again, ascale = poison((R, F), torch.uint8), poison((R, F // 64), torch.float32)
    moe.moe_checkpoint_pack(back, again, ascale)
    e4m3 = torch.float8_e4m3fn
    zq = again[tail].view(e4m3).float()
    zq = (zq.reshape(300, -1, 64) * ascale[tail][:, :, None]).reshape(300, F)
    assert bool(((zq - back[tail].float()).abs() <= back[tail].float().abs() / 8 + m / 448 / 256).all())
    del again, ascale
    dy = back  # any values: |dy| of ordinary size
    dx, dw = poison((R, K), torch.bfloat16), poison((1, F, K), torch.bfloat16)
    moe.moe_grouped_linear_backward(cfg, x, off, w, dy, z_codes=codes, z_scale=scale, dx=dx, dw=dw,
                                    workspace=moe.alloc_linear_backward_workspace(cfg))
    acc, terms = torch.zeros((F, K), device=DEV), torch.zeros((F, K), device=DEV)
    for i in range(0, R, 1000):
        r = slice(i, i + 1000)
        zz = (codes[r].view(e4m3).float().reshape(1000, -1, 64) * scale[r][:, :, None]).reshape(-1, F)
        p = torch.sigmoid(zz)
        dz = dy[r].float() * (p + zz * p * (1 - p))
        acc += dz.t() @ x[r].float()
        terms += dz.abs().t() @ x[r].float().abs()
    bound = V * acc.abs() + terms * (2 * V)
    assert bool(((dw[0].float() - acc).abs() <= bound).all())
    ref = dz[-300:] @ w[0].float()
    tx = dz[-300:].abs() @ w[0].float().abs()
    assert bool(((dx[tail].float() - ref).abs() <= V * ref.abs() + tx * 2 * V).all())
    # combine: the same rows, two a token
    slot = torch.arange(R, device=DEV, dtype=torch.int32).reshape(-1, 2)
    o = poison((R // 2, F), torch.bfloat16)
    moe.moe_combine(y, slot, o)
    want = y[tail].float().reshape(150, 2, F).sum(1)
    assert bool(((o[-150:].float() - want).abs() <= V * want.abs() + 1e-6).all())
    drows = poison((R, F), torch.bfloat16)
    moe.moe_combine_backward(y, slot, None, o, drows, None)
    torch.cuda.synchronize()
    assert torch.equal(drows[tail], o[-150:].repeat_interleave(2, dim=0))


def test_small_and_large_values():
    """Activations where the exponential over- or underflows."""
    say("[linear] extremes")
    for dtype in ("bf16", "f32"):
        for act in ("silu", "gelu", "swiglu", "relu"):
            c = Case([2], 64, 64, act, dtype)
            c.x.zero_()
            c.w.zero_()
            vals = torch.tensor([-200., -100., -88., -20., -1e-3, 0., 1e-30, 1e-3, 20., 88., 100.,
                                 200., -3., 3., -0.5, 0.5]).repeat(4)
            c.bias = vals.repeat(c.zd // 64).expand(1, c.zd).contiguous().to(DEV)
            c.hx[:], c.hw[:] = 0, 0
            c.check_forward(f"extremes {act} {dtype}")


def test_two_streams_at_once():
    """Two calls in flight together, each with a workspace of its own."""
    say("[linear] two streams")
    for sizes, K, F in (([1, 2], 4096, 128), (RAGGED, 1024, 576)):
        cases = [Case(sizes, K, F, "swiglu", gather=True, bias=True, seed=s) for s in (1, 2)]
        want = [c.forward(True) for c in cases]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in cases]
        args = []
        for c in cases:
            args.append((poison((c.rows, F), c.dt), poison((c.rows, c.zd), torch.uint8),
                         poison((c.rows, c.zd // 64), torch.float32),
                         workspace(moe.alloc_linear_workspace(c.cfg, DEV))))
        torch.cuda.synchronize()
        for _ in range(5):
            for c, s, (y, codes, scale, ws) in zip(cases, streams, args):
                moe.moe_grouped_linear(c.cfg, c.x, c.offsets, c.w, y, row_index=c.index,
                                       bias=c.bias, z_codes=codes, z_scale=scale, workspace=ws,
                                       stream=s)
        torch.cuda.synchronize()
        for w, a in zip(want, args):
            for p, q in zip(w, a):
                assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))


def test_binding_refuses_what_the_c_side_cannot_see():
    say("[linear] refusals")
    c = Case([3, 2], 64, 64, "gelu")
    ws = moe.alloc_linear_workspace(c.cfg, DEV)
    y = poison((5, 64), c.dt)
    good = dict(x=c.x, offsets=c.offsets, w=c.w, y=y, workspace=ws)
    bad = [dict(x=c.x.float()), dict(x=c.x[:4]), dict(offsets=c.offsets.long()),
           dict(offsets=c.offsets[:2]), dict(w=c.w[:1]), dict(w=c.w.transpose(1, 2)),
           dict(y=poison((5, 128), c.dt)[:, :64]), dict(y=y.cpu()), dict(workspace=ws.cpu()),
           dict(bias=poison((2, 64), c.dt)), dict(residual=poison((4, 64), c.dt)),
           dict(z_codes=poison((5, 64), torch.uint8), z_scale=poison((5, 2), torch.float32)),
           dict(row_index=torch.zeros(4, dtype=torch.int32, device=DEV))]
    for over in bad:
        a = {**good, **over}
        with pytest.raises(ValueError):
            moe.moe_grouped_linear(c.cfg, a.pop("x"), a.pop("offsets"), a.pop("w"), a.pop("y"), **a)
    with pytest.raises(moe.MoEError):  # a checkpoint is needed to differentiate GELU
        moe.moe_grouped_linear_backward(c.cfg, c.x, c.offsets, c.w, c.dy, dx=poison((5, 64), c.dt),
                                        workspace=moe.alloc_linear_backward_workspace(c.cfg, DEV))
    with pytest.raises(moe.MoEError):  # 8 of 16-byte aligned
        flat = torch.zeros(5 * 64 + 4, dtype=c.dt, device=DEV)
        moe.moe_grouped_linear(c.cfg, c.x, c.offsets, c.w, flat[4:].view(5, 64), workspace=ws)
    with pytest.raises(ValueError):
        moe.moe_checkpoint_pack(c.x.half(), poison((5, 64), torch.uint8),
                                poison((5, 1), torch.float32))
    with pytest.raises(ValueError):
        moe.moe_combine(c.x, torch.zeros((2, 2), dtype=torch.int64, device=DEV),
                        poison((2, 64), c.dt))
    assert bool(torch.isnan(y).all())


# ---------------------------------------------------------------- checkpoints
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 64), (3, 192), (37, 1024), (300, 4032)])
def test_pack_and_unpack(rows, cols, dtype):
    """Codes and scales are exactly the definition's; unpack is one fp32
    product rounded to the type."""
    say(f"[checkpoint] {rows}x{cols} {dtype}")
    g = torch.Generator(device=DEV).manual_seed(rows)
    x = torch.randn((rows, cols), generator=g, device=DEV)
    x *= torch.exp(4 * torch.randn((rows, cols), generator=g, device=DEV))
    x[0, :64] = 0
    if cols >= 192:
        x[-1, 64:128] *= 1e-36   # the block's maximum below 1e-30
        x[rows // 2, 128:192] *= 1e34
        x[0, 70], x[0, 71], x[0, 72] = float("nan"), float("inf"), float("-inf")
    x = x.to(DT[dtype])
    codes, scale = poison((rows, cols), torch.uint8), poison((rows, cols // 64), torch.float32)
    moe.moe_checkpoint_pack(x, codes, scale)
    back = poison((rows, cols), x.dtype)
    moe.moe_checkpoint_unpack(codes, scale, back)
    torch.cuda.synchronize()
    c, s = lo.checkpoint_pack(x.float().cpu().numpy())
    got = to_np(codes)
    nan = (c & 0x7F) == 0x7F
    assert np.array_equal(got[~nan], c[~nan]) and np.all((got[nan] & 0x7F) == 0x7F)
    assert np.array_equal(to_np(scale), s)
    ref = torch.tensor((e4m3_decode(got).astype(np.float32).reshape(rows, -1, 64)
                        * s[:, :, None]).reshape(rows, cols)).to(x.dtype)
    assert torch.equal(torch.nan_to_num(back.cpu(), 7.0), torch.nan_to_num(ref, 7.0))


def test_every_code_decodes():
    say("[checkpoint] 256 codes")
    codes = torch.arange(256, dtype=torch.uint8, device=DEV).reshape(4, 64)
    scale = torch.tensor([[1.0], [0.5], [3.0], [2.0 ** -100]], device=DEV)
    x = poison((4, 64), torch.float32)
    moe.moe_checkpoint_unpack(codes, scale, x)
    ref = lo.checkpoint_unpack(to_np(codes), to_np(scale))
    np.testing.assert_array_equal(to_np(x), ref.astype(np.float32))


# ---------------------------------------------------------------- grouping
def group(idx, N, capacity=0, guard=3):
    T, k = idx.shape
    out = (poison((N + 1,), torch.int32), poison((T * k,), torch.int32),
           poison((T, k), torch.int32))
    moe.moe_group_rows(idx, N, *out, capacity=capacity,
                       workspace=workspace(moe.alloc_group_workspace(T, N, k, DEV)))
    return out


@pytest.mark.parametrize("T,N,k,capacity,skew", [
    (0, 4, 2, 0, 0), (1, 1, 1, 0, 0), (1, 512, 16, 0, 0), (7, 3, 2, 1, 0), (255, 8, 2, 0, 0),
    (2048, 8, 2, 0, 2), (2049, 8, 2, 300, 2), (513, 512, 8, 0, 0), (3001, 128, 8, 40, 1.2),
    (40000, 511, 8, 0, 1.2), (70000, 2, 1, 0, 0)])
def test_group_rows(T, N, k, capacity, skew):
    say(f"[group] T={T} N={N} k={k} capacity={capacity}")
    g = torch.Generator().manual_seed(T)
    if k <= N:
        score = torch.randn((T, N), generator=g) - skew * torch.log(torch.arange(1., N + 1))
        idx = torch.topk(score, k, dim=1).indices.int()
    if T > 4:  # padding, indices that are no expert, the same expert twice in a token
        idx[3] = -1
        idx[4, 0] = N
        idx[T // 2] = 0
        idx[T - 1, k - 1] = 1 << 30
    off, tok, slot = (to_np(t) for t in group(idx.to(DEV), N, capacity))
    ro, rt, rs = lo.group_rows(idx.numpy(), N, capacity)
    assert np.array_equal(off, ro)
    assert np.array_equal(tok[:len(rt)], rt) and np.all(tok[len(rt):] == -7)
    assert np.array_equal(slot, rs)


def test_group_rows_agrees_with_the_layer():
    """The layer's own router: the counts it reports and the rows' order."""
    say("[group] from moe_route")
    from workloads import MoEShape, make_inputs
    shape = MoEShape("route", T=333, d=128, N=16, k=4, F=64)
    inp = make_inputs(shape, 3, DEV)
    cfg = moe.make_config(333, 128, 16, 4, 64)
    idx, gate = poison((333, 4), torch.int32), poison((333, 4), torch.float32)
    counts = poison((16,), torch.int32)
    moe.moe_route(cfg, inp["x"], inp, topk_idx=idx, topk_gate=gate, counts=counts,
                  workspace=moe.alloc_workspace(cfg, DEV))
    off, _, _ = group(idx, 16)
    assert torch.equal(off[1:] - off[:-1], counts)


# ---------------------------------------------------------------- combine
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,d,gated", [(1, 1, 64, True), (5, 2, 192, False), (70, 9, 2112, True),
                                         (33, 16, 320, True), (300, 3, 4160, False)])
def test_combine(T, k, d, gated, dtype):
    say(f"[combine] T={T} k={k} d={d} gated={gated} {dtype}")
    g = torch.Generator(device=DEV).manual_seed(T)
    n_rows = T * k + 3
    rows = torch.randn((n_rows, d), generator=g, device=DEV).to(DT[dtype])
    slot = torch.randperm(n_rows, generator=g, device=DEV)[:T * k].int().reshape(T, k)
    if T > 4:
        slot[1] = -1                 # a token without rows
        slot[2, 0], slot[3, k - 1] = n_rows, -5
    used = torch.zeros(n_rows, dtype=torch.bool, device=DEV)
    used[slot[(slot >= 0) & (slot < n_rows)].long()] = True
    rows[~used] = float("nan")
    gate = torch.rand((T, k), generator=g, device=DEV) if gated else None
    dy = torch.randn((T, d), generator=g, device=DEV).to(DT[dtype])
    y = poison((T, d), rows.dtype)
    moe.moe_combine(rows, slot, y, gate=gate)
    drows, dgate = poison((n_rows, d), rows.dtype), poison((T, k), torch.float32)
    moe.moe_combine_backward(rows, slot, gate, dy, drows, dgate)
    only = poison((n_rows, d), rows.dtype)
    moe.moe_combine_backward(rows, slot, gate, dy, only, None)
    torch.cuda.synchronize()
    hr, hs, hd = to_np(rows), to_np(slot), to_np(dy)
    hg = None if gate is None else to_np(gate)
    ref = lo.combine_rows(hr, hs, hg)
    terms = lo.combine_rows(np.abs(hr), hs, hg)
    r = U if dtype == "f32" else V
    check("y", y, ref, r * np.abs(ref) + (1 + r) * (k + 2) * U * terms)
    rr, rg = lo.combine_rows_backward(hr, hs, hg, hd)
    tg = lo.combine_rows_backward(np.abs(hr), hs, hg, np.abs(hd))[1]
    keep = to_np(used)
    check("drows", drows[used], rr[keep], r * np.abs(rr[keep]) * (1 + U) + U * np.abs(rr[keep]))
    check("dgate", dgate, rg, (d + 8) * U * tg)
    assert bool(torch.isnan(drows[~used]).all())
    assert torch.equal(only[used], drows[used])


# ---------------------------------------------------------------- together
class Mlp:
    """Router indices to output and back through every call, as a training
    step of GELU experts with biases uses them: grouping, up projection (its
    input read through row_token, its pre-activation saved in 8 bits), down
    projection, combine; and their gradients."""

    def __init__(self, T, N, k, d, F, act="gelu", dtype="bf16", seed=0, capacity=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        dt = self.dt = DT[dtype]
        self.T, self.N, self.k, self.d, self.F, self.act = T, N, k, d, F, act
        self.capacity = capacity
        zd = F * (2 if act == "swiglu" else 1)
        randn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
        self.x, self.dy = randn(T, d).to(dt), randn(T, d).to(dt)
        self.idx = torch.topk(randn(T, N), k, dim=1).indices.int().contiguous()
        gate = torch.rand((T, k), generator=g, device=DEV) + 0.1
        self.gate = gate / gate.sum(1, keepdim=True)
        self.w1 = (randn(N, zd, d) * d ** -0.5).to(dt)
        self.w2 = (randn(N, d, F) * F ** -0.5).to(dt)
        self.b1, self.b2 = randn(N, zd) * 0.2, randn(N, d) * 0.2
        R = T * k
        e = lambda *s, t=dt: torch.zeros(s, dtype=t, device=DEV)  # noqa: E731
        i32, f32 = torch.int32, torch.float32
        self.off, self.tok, self.slot = e(N + 1, t=i32), e(R, t=i32), e(T, k, t=i32)
        self.h, self.o, self.y = e(R, F), e(R, d), e(T, d)
        self.codes, self.scale = e(R, zd, t=torch.uint8), e(R, zd // 64, t=f32)
        self.do, self.dgate, self.dh = e(R, d), e(T, k, t=f32), e(R, F)
        self.dw1, self.dw2 = e(N, zd, d), e(N, d, F)
        self.db1, self.db2 = e(N, zd, t=f32), e(N, d, t=f32)
        self.dxr, self.dx = e(R, d), e(T, d)
        self.up = moe.make_linear_config(R, N, d, F, dtype=dt, activation=act, x_rows=T)
        self.down = moe.make_linear_config(R, N, F, d, dtype=dt)
        self.ws = [moe.alloc_group_workspace(T, N, k, DEV),
                   moe.alloc_linear_workspace(self.up, DEV),
                   moe.alloc_linear_workspace(self.down, DEV),
                   moe.alloc_linear_backward_workspace(self.up, DEV),
                   moe.alloc_linear_backward_workspace(self.down, DEV)]
        for w in self.ws:
            w.fill_(0xFF)

    def step(self):
        moe.moe_group_rows(self.idx, self.N, self.off, self.tok, self.slot, workspace=self.ws[0],
                           capacity=self.capacity)
        moe.moe_grouped_linear(self.up, self.x, self.off, self.w1, self.h, row_index=self.tok,
                               bias=self.b1, z_codes=self.codes, z_scale=self.scale,
                               workspace=self.ws[1])
        moe.moe_grouped_linear(self.down, self.h, self.off, self.w2, self.o, bias=self.b2,
                               workspace=self.ws[2])
        moe.moe_combine(self.o, self.slot, self.y, gate=self.gate)
        moe.moe_combine_backward(self.o, self.slot, self.gate, self.dy, self.do, self.dgate)
        moe.moe_grouped_linear_backward(self.down, self.h, self.off, self.w2, self.do, dx=self.dh,
                                        dw=self.dw2, dbias=self.db2, workspace=self.ws[4])
        moe.moe_grouped_linear_backward(self.up, self.x, self.off, self.w1, self.dh,
                                        row_index=self.tok, z_codes=self.codes,
                                        z_scale=self.scale, dx=self.dxr, dw=self.dw1,
                                        dbias=self.db1, workspace=self.ws[3])
        moe.moe_combine(self.dxr, self.slot, self.dx)

    OUT = ("y", "codes", "scale", "dgate", "dw1", "dw2", "db1", "db2", "dx")

    def outputs(self):
        return {n: getattr(self, n).clone() for n in self.OUT}


@pytest.mark.parametrize("T,N,k,d,F,act,dtype,capacity", [
    (5, 8, 2, 128, 192, "gelu", "bf16", 0), (300, 4, 2, 256, 320, "swiglu", "bf16", 0),
    (64, 4, 2, 128, 256, "silu", "f32", 0), (900, 3, 2, 192, 256, "relu", "bf16", 500),
    (700, 16, 2, 832, 640, "swiglu", "bf16", 0), (3, 4, 2, 1088, 1024, "gelu", "bf16", 0)])
def test_a_training_step(T, N, k, d, F, act, dtype, capacity):
    """Every output of the chain against float64, the saved activations being
    the only 8-bit values: the 2-norms differ by at most 2^-6 (bf16: six
    tensors of the chain rounded to bf16, 2^-8 of the norm each at most, and
    2^-7 of the products' terms; the codes themselves enter both sides) or
    2^-16 (fp32: sums of up to 900 terms, (900 + 8) u < 2^-14 of the terms in
    the worst case, its square root in the norm of random signs)."""
    say(f"[step] T={T} N={N} k={k} d={d} F={F} {act} {dtype}")
    m = Mlp(T, N, k, d, F, act, dtype, capacity=capacity)
    m.step()
    torch.cuda.synchronize()
    H = lambda t: to_np(t).astype(np.float64)  # noqa: E731
    off, tok, slot = lo.group_rows(to_np(m.idx), N, capacity)
    n = int(off[-1])
    assert np.array_equal(to_np(m.off), off) and np.array_equal(to_np(m.slot), slot)
    h, z = lo.grouped_linear(H(m.x), off, H(m.w1), act, tok, H(m.b1))
    o, _ = lo.grouped_linear(h, off, H(m.w2), "none", None, H(m.b2))
    zq = lo.checkpoint_unpack(to_np(m.codes)[:n], to_np(m.scale)[:n])
    assert np.linalg.norm(zq - z) <= np.linalg.norm(z) * (2.0 ** -4 + 2.0 ** -8)
    y = lo.combine_rows(o, slot, H(m.gate))
    do, dgate = lo.combine_rows_backward(o, slot, H(m.gate), H(m.dy))
    dh, dw2, db2, _ = lo.grouped_linear_backward(h, off, H(m.w2), do, None)
    dxr, dw1, db1, _ = lo.grouped_linear_backward(H(m.x), off, H(m.w1), dh, zq, act, tok)
    dx = lo.combine_rows(dxr, slot)
    bound = 2.0 ** -6 if dtype == "bf16" else 2.0 ** -16
    for name, ref in (("y", y), ("dgate", dgate), ("dw2", dw2), ("db2", db2), ("dw1", dw1),
                      ("db1", db1), ("dx", dx)):
        off_by = np.linalg.norm(H(getattr(m, name)) - ref) / np.linalg.norm(ref)
        say(f"[step] {name}: {off_by:.2e} of its norm")
        assert off_by <= bound, name


def test_gradients_are_differences():
    """fp32 ReLU experts: the loss is piecewise linear in x, and 8 bits keep a
    pre-activation's sign, so a central difference that crosses no kink is the
    gradient up to fp32: the loss's terms times 2^-20 over the step, and sums
    of the gradient's products (2^-10 of its terms leaves room)."""
    say("[step] differences")
    m = Mlp(6, 4, 2, 128, 192, "relu", "f32", seed=5)
    v = torch.randn(m.x.shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    x0, h = m.x.clone(), 2.0 ** -12
    z = {}

    def loss(sign):
        m.x.copy_(x0 + sign * h * v)
        m.step()
        z[sign] = lo.checkpoint_unpack(to_np(m.codes), to_np(m.scale)) > 0
        return float((m.y.double() * m.dy.double()).sum())

    up, dn = loss(1), loss(-1)
    loss(0)
    crossed = (z[1] != z[-1]).sum()
    got = float((m.dx.double() * v.double()).sum())
    diff = (up - dn) / (2 * h)
    terms = float((m.y.double() * m.dy.double()).abs().sum())
    # each kink crossed moves the difference by at most half its slope's share
    say(f"[step] difference {diff:.6f} gradient {got:.6f}, {crossed} kinks")
    scale = float((m.dx.double() * v.double()).abs().sum())
    assert abs(diff - got) <= terms * 2.0 ** -20 / h + scale * 2.0 ** -10 + crossed * scale * 2.0 ** -6


def test_a_step_replays_from_a_graph():
    """Captured once, replayed with other inputs between eager work; two
    graphs with workspaces of their own; every replay equals the eager step."""
    say("[step] graph")
    for shape in ((6, 8, 2, 128, 192), (400, 4, 2, 256, 320), (500, 16, 2, 832, 640),
                  (3, 4, 2, 1024, 1152)):
        a, b = Mlp(*shape, act="swiglu", seed=1), Mlp(*shape, act="gelu", seed=2)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            a.step()
            b.step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graphs = []
        for m in (a, b):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                m.step()
            graphs.append(g)
        for rep in range(4):
            for m in (a, b):
                gen = torch.Generator(device=DEV).manual_seed(10 + rep)
                m.x.copy_(torch.randn(m.x.shape, generator=gen, device=DEV))
                m.idx.copy_(torch.topk(torch.randn((m.T, m.N), generator=gen, device=DEV), m.k,
                                       dim=1).indices)
                m.step()
            want = [a.outputs(), b.outputs()]
            for m in (a, b):
                for n in m.OUT:
                    getattr(m, n).zero_()
            torch.cuda.synchronize()
            graphs[0].replay()
            graphs[1].replay()
            torch.cuda.synchronize()
            for m, w in zip((a, b), want):
                for n in m.OUT:
                    assert torch.equal(getattr(m, n).view(torch.uint8), w[n].view(torch.uint8)), n
