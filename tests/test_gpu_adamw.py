"""The AdamW step on the GPU against the float32 oracle (oracle/block_oracle.py).

Every operation on the states is one correctly rounded fp32 operation, in the
oracle's order: fp32 states, codes and scales have to match bit for bit.  The
parameter's update may fuse or refine: it is off by at most 8 u of the update
and u of the parameter (u = 2^-24), to which a rounding to bf16 adds a step,
for one drawn or nearest rounding may fall to the other side of a border.
"""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_router_amd as moe
from gpu_harness import say, to_np
from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8)


def tensor(n, dtype, grad, master, eight, seed, shift=0):
    """One tensor's buffers, `shift` elements into larger ones."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    randn = lambda k: torch.randn(k, generator=g, device=DEV)  # noqa: E731
    at = lambda t: torch.cat([torch.zeros(shift, device=DEV).to(t.dtype), t])[shift:]  # noqa: E731
    p = randn(n) * 0.02
    t = dict(param=at(p.to(DT[dtype])), grad=at((randn(n) * 1e-3).to(DT[grad])), weight_decay=0.1 * (seed % 2))
    if master:
        t["master"] = at(p)
    m, v = randn(n) * 3e-4, (randn(n) * 1e-3).square()
    if eight:
        blocks = -(-n // 256)
        t["m"] = at(torch.randint(-127, 128, (n,), generator=g, device=DEV).to(torch.int8))
        t["v"] = at(torch.randint(0, 256, (n,), generator=g, device=DEV).to(torch.uint8))
        t["m_scale"] = torch.rand(blocks, generator=g, device=DEV) * 1e-7
        t["v_scale"] = torch.rand(blocks, generator=g, device=DEV) * 1e-7
    else:
        t["m"], t["v"] = at(m), at(v)
    return t


def names(t):
    return [n for n in ("param", "master", "m", "v", "m_scale", "v_scale") if t.get(n) is not None]


def step_and_check(ts, step=3, seed=11, grad_scale=0.5, label="", **kw):
    host = [{k: (to_np(x) if isinstance(x, torch.Tensor) else x) for k, x in t.items()} for t in ts]
    handle = moe.make_adamw_tensors(ts)
    moe.moe_adamw_step(handle, step=step, seed=seed, grad_scale=grad_scale, **HYPER, **kw)
    torch.cuda.synchronize()
    worst = 0.0
    for i, (t, h) in enumerate(zip(ts, host)):
        n = t["param"].numel()
        if n == 0:
            continue
        narrow = t["param"].dtype == torch.bfloat16 and t.get("master") is None
        p0 = h["master"] if t.get("master") is not None else h["param"]
        ref = bo.adamw(p0.reshape(-1), h["grad"].reshape(-1), h["m"].reshape(-1), h["v"].reshape(-1), step=step, seed=seed, index=i,
                       grad_scale=grad_scale, weight_decay=t["weight_decay"], m_scale=h.get("m_scale"),
                       v_scale=h.get("v_scale"), narrow=narrow, **HYPER)
        for name, r in zip(("m", "v", "m_scale", "v_scale"), ref[1:]):
            got = to_np(t[name]).reshape(-1)
            assert np.array_equal(got, r), f"{label} tensor {i} {name}: {np.argwhere(got != r)[:3].ravel()}"
        exact = bo.adamw(p0.reshape(-1), h["grad"].reshape(-1), h["m"].reshape(-1), h["v"].reshape(-1), step=step, seed=seed, index=i,
                         grad_scale=grad_scale, weight_decay=t["weight_decay"], m_scale=h.get("m_scale"),
                         v_scale=h.get("v_scale"), **HYPER)[0].astype(np.float64)
        tol = 8 * U * np.abs(exact - p0.reshape(-1)) + 2 * U * np.abs(p0.reshape(-1))
        if t.get("master") is not None:
            d = np.abs(to_np(t["master"]).reshape(-1) - exact)
            worst = max(worst, float(np.max(d / tol)))
            assert (d <= tol).all(), f"{label} tensor {i} master"
            assert torch.equal(t["param"].view(-1), t["master"].view(-1).to(torch.bfloat16)), label
            continue
        if narrow:
            tol = tol + 2.0 ** -7 * np.abs(exact)
            # drawn from the same words: the same result but for values at a border
            assert np.mean(to_np(t["param"]).reshape(-1) != ref[0]) <= 1e-3 + 1.0 / n, label
        d = np.abs(to_np(t["param"]).reshape(-1) - exact)
        worst = max(worst, float(np.max(d / tol)))
        assert (d <= tol).all(), f"{label} tensor {i} param"
    say(f"[adamw] {label}: worst {worst:.3f} of its bound")


SIZES = [1, 7, 8, 255, 256, 257, 2047, 2048, 2049, 10000]


@pytest.mark.parametrize("eight", [False, True], ids=["f32", "8bit"])
@pytest.mark.parametrize("dtype,grad,master", [
    ("f32", "f32", False), ("f32", "bf16", False), ("bf16", "bf16", True), ("bf16", "f32", True),
    ("bf16", "bf16", False), ("bf16", "f32", False)])
def test_step(dtype, grad, master, eight):
    ts = [tensor(n, dtype, grad, master, eight, i) for i, n in enumerate(SIZES)]
    step_and_check(ts, label=f"{dtype} {grad} master={master} 8bit={eight}")
    step_and_check(ts, step=4, seed=12, label="again")


@pytest.mark.parametrize("eight", [False, True], ids=["f32", "8bit"])
@pytest.mark.parametrize("shift", [1, 3, 4])
def test_unaligned(shift, eight):
    ts = [tensor(n, "bf16", "bf16", shift == 3, eight, i, shift) for i, n in enumerate(SIZES)]
    step_and_check(ts, label=f"shift {shift}")


def test_many_tensors_and_empty_ones():
    ts = [tensor((i * 37) % 700, "bf16", "f32", True, True, i) for i in range(131)]
    step_and_check(ts, label="131 tensors")


def test_shapes_are_free():
    t = tensor(24 * 50, "f32", "f32", False, True, 3)
    for n in ("param", "grad", "m", "v"):
        t[n] = t[n].view(24, 50)
    step_and_check([t], label="matrix")


def test_from_nothing():
    """The first step of states that are zero, and gradients that are zero."""
    for eight in (False, True):
        t = tensor(700, "f32", "f32", False, eight, 0)
        for n in ("m", "v", "m_scale", "v_scale"):
            if t.get(n) is not None:
                t[n].zero_()
        t["grad"][256:512] = 0
        step_and_check([t], step=1, label="first")
        if eight:
            assert float(t["m_scale"][1]) == 0 and not t["m"][256:512].any()


def test_values_near_the_ends_of_the_range():
    """Gradients and states from 1e-25 to 1e18 in neighbouring blocks, zeros among
    them, beside ordinary ones: the short forms and the long ones."""
    for grad in ("f32", "bf16"):
        t = tensor(256 * 40, "f32", grad, False, True, 5)
        size = 10.0 ** torch.linspace(-25, 18, 40, device=DEV).repeat_interleave(256)
        t["grad"] = (t["grad"].float() * 1e3 * size).to(DT[grad])
        t["grad"][::7] = 0
        for n in ("m_scale", "v_scale"):
            t[n] *= size[::256] * 1e3
            t[n][::5] = 0
        t["param"] *= 1e3
        step_and_check([t], label="ends of the range")
    t = tensor(2048 * 8, "bf16", "bf16", False, True, 6)
    t["grad"][::2] = 0
    t["v_scale"][::2] = 0
    step_and_check([t], label="no root")


def test_scale_zero_leaves_everything():
    t = tensor(3000, "bf16", "bf16", True, True, 1)
    t["grad"][5] = float("nan")
    before = {n: t[n].clone() for n in names(t)}
    handle = moe.make_adamw_tensors([t])
    moe.moe_adamw_step(handle, step=2, grad_scale=0.0)
    moe.moe_adamw_step(handle, scalars=torch.tensor([1e-3, 0.1, 0.1, 0.0, 0.0], device=DEV))
    assert all(torch.equal(before[n], t[n]) for n in names(t))


def test_not_finite_gradients_spoil_their_element_or_block():
    for eight in (False, True):
        t = tensor(1024, "f32", "f32", False, eight, 2)
        t["grad"][300], t["grad"][900] = float("nan"), float("inf")
        moe.moe_adamw_step(moe.make_adamw_tensors([t]), step=5, **HYPER)
        p = to_np(t["param"])
        assert not np.isfinite(p[[300, 900]]).any()
        keep = np.ones(1024, dtype=bool)
        keep[[300, 900]] = False
        assert np.isfinite(p[keep]).all()
        if eight:
            assert (np.isfinite(to_np(t["m_scale"])) == [True, False, True, False]).all()


def test_scalars_stand_for_the_arguments():
    a, b = (tensor(5000, "bf16", "bf16", False, True, 4) for _ in range(2))
    moe.moe_adamw_step(moe.make_adamw_tensors([a]), step=9, seed=1 << 31, grad_scale=0.25, **HYPER)
    words = torch.tensor([1e-2, 1 - 0.9 ** 9, 1 - 0.95 ** 9, 0.25, 0.0], device=DEV)
    words.view(torch.int32)[4] = -(1 << 31)
    moe.moe_adamw_step(moe.make_adamw_tensors([b]), scalars=words, **HYPER)
    assert all(torch.equal(a[n], b[n]) for n in names(a))


def test_rounding_keeps_the_states_on_average():
    """With one gradient throughout, a drawn code is right on average.  v moves by
    1 in 2000 a step here, a code near 200 is 4 / 200 wide in v: to nearest it
    would never move.  2048 equal elements (in blocks whose first element pins
    the scale), 200 steps: the mean of v follows the fp32 states within 2 % (a
    step's drawn rounding has an r.m.s. of half a code, 2 % of v at code 200; 200
    independent steps of 2040 elements bring the mean's to 2 % sqrt(200 / 2040),
    0.6 %, of which this is three)."""
    n, steps = 2048, 200
    grad = torch.full((n,), 0.6, device=DEV)
    grad[::256] = 1.0
    z = lambda dt, k=n: torch.zeros(k, dtype=dt, device=DEV)  # noqa: E731
    v0 = torch.full((n,), 0.7 ** 2, device=DEV)
    v0[::256] = 1.0
    t = dict(param=z(torch.float32), grad=grad, m=z(torch.int8), m_scale=z(torch.float32, 8),
             v=torch.round(torch.sqrt(v0.sqrt() * 65025.0)).to(torch.uint8),
             v_scale=torch.full((8,), 1 / 65025.0, device=DEV))
    code = t["v"].float()
    start = ((code * code) / 65025.0) ** 2
    r = dict(param=z(torch.float32), grad=grad, m=z(torch.float32), v=start.clone())
    a, b = moe.make_adamw_tensors([t]), moe.make_adamw_tensors([r])
    for i in range(steps):
        for h in (a, b):
            moe.moe_adamw_step(h, step=i + 1, lr=0.0, beta1=0.9, beta2=0.9995)
    c = t["v"].float()
    got = ((c * c) * t["v_scale"].repeat_interleave(256)) ** 2
    inner = torch.ones(n, dtype=torch.bool, device=DEV)
    inner[::256] = False
    have, want, was = (float(x[inner].mean()) for x in (got, r["v"], start))
    say(f"[adamw] mean of v: {have:.5f}, in fp32 {want:.5f}, at the start {was:.5f}")
    assert abs(have - want) <= 0.02 * want and abs(want - was) > 0.02 * want
    c = t["m"].float()
    m = (c * c.abs() * t["m_scale"].repeat_interleave(256))[inner].mean()
    assert abs(float(m) - 0.6) <= 0.02 * 0.6


def test_learns():
    """Runs with a training loop's usual calls; every parameter moves."""
    t = tensor(4096, "bf16", "bf16", False, True, 6)
    before = t["param"].clone()
    h = moe.make_adamw_tensors([t])
    for i in range(3):
        t["grad"].normal_()
        moe.moe_adamw_step(h, step=i + 1, lr=0.05)
    assert (before != t["param"]).float().mean() > 0.99
    assert torch.isfinite(t["param"]).all()


def test_binding_refuses():
    t = tensor(64, "f32", "f32", False, True, 0)
    for bad in (dict(t, m_scale=None), dict(t, grad=t["grad"][:60]), dict(t, v=t["v"].to(torch.int8)),
                dict(t, master=t["param"].cpu())):
        with pytest.raises(ValueError):
            moe.make_adamw_tensors([bad])
    with pytest.raises(moe.MoEError):  # fp32 parameters have no copy
        moe.moe_adamw_step(moe.make_adamw_tensors([dict(t, master=t["param"].clone())]), step=1)
    with pytest.raises(moe.MoEError):
        moe.moe_adamw_step(moe.make_adamw_tensors([t]), step=0)
    with pytest.raises(ValueError):
        make = moe.make_adamw_tensors([t])
        moe.moe_adamw_step(make, scalars=torch.zeros(4, device=DEV))
