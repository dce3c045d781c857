"""The calls for experts of one's own without a GPU: their structs mirror the
header, sizes are answered, and bad arguments are refused on the host before
anything is launched."""
import ctypes
import os
import re

import pytest
import torch

import sparse_mixture_experts_router_amd as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe.h")

pytestmark = pytest.mark.skipif(not os.path.exists(moe.LIB_PATH),
                                reason="libmoe.so not built (run __graft_entry__.build())")

FAKE = 1 << 20  # a 256-byte aligned non-null address; never dereferenced on these paths
BIG = 1 << 40
INVALID, UNSUPPORTED, WORKSPACE = (moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED,
                                   moe.MOE_ERR_WORKSPACE)


def _body(name):
    with open(HEADER) as fh:
        text = re.sub(r"/\*.*?\*/", "", fh.read(), flags=re.S)
    return re.search(r"typedef struct \{([^}]*)\} " + name + ";", text).group(1)


@pytest.mark.parametrize("name,struct", [("moe_linear_config", moe.MoELinearConfig),
                                         ("moe_linear_args", moe.MoELinearArgs),
                                         ("moe_linear_grad_args", moe.MoELinearGradArgs)])
def test_structs_match_the_header(name, struct):
    assert re.findall(r"(\w+);", _body(name)) == [f for f, _ in struct._fields_]


def test_activation_codes_match_the_header():
    with open(HEADER) as fh:
        codes = dict(re.findall(r"MOE_ACT_(\w+) = (\d+)", fh.read()))
    assert [codes[a.upper()] for a in moe.ACTIVATIONS] == [str(i) for i in range(5)]


def cfg(**over):
    c = moe.make_linear_config(100, 4, 128, 192, activation="gelu")
    for k, v in over.items():
        setattr(c, k, v)
    return c


BAD_CONFIGS = [
    (dict(rows=-1), INVALID), (dict(x_rows=-1), INVALID), (dict(groups=0), INVALID),
    (dict(in_dim=0), INVALID), (dict(out_dim=-64), INVALID), (dict(dtype=2), INVALID),
    (dict(weight_format=2), INVALID), (dict(activation=5), INVALID), (dict(activation=-1), INVALID),
    (dict(groups=513), UNSUPPORTED), (dict(in_dim=96), UNSUPPORTED), (dict(out_dim=100), UNSUPPORTED),
    (dict(in_dim=(1 << 20) + 64), UNSUPPORTED), (dict(rows=1 << 27), UNSUPPORTED),
    (dict(x_rows=1 << 30), UNSUPPORTED),
    (dict(dtype=moe.MOE_F32, weight_format=moe.MOE_WEIGHTS_FP8_E4M3), UNSUPPORTED),
    (dict(rows=(1 << 27) - 1, out_dim=1 << 20), UNSUPPORTED),          # too many tiles
    (dict(groups=512, in_dim=1 << 20, out_dim=1 << 20), UNSUPPORTED),  # too many tiles of dw
]


def forward(c, a, ws=FAKE, nbytes=BIG):
    return moe.lib().moe_grouped_linear(None if c is None else ctypes.byref(c),
                                        None if a is None else ctypes.byref(a), ws, nbytes, None)


def backward(c, a, ws=FAKE, nbytes=BIG):
    return moe.lib().moe_grouped_linear_backward(None if c is None else ctypes.byref(c),
                                                 None if a is None else ctypes.byref(a), ws,
                                                 nbytes, None)


def args(**over):
    a = dict(x=FAKE, offsets=FAKE, w=FAKE, y=FAKE)
    a.update(over)
    return moe.MoELinearArgs(**a)


def grads(**over):
    a = dict(x=FAKE, offsets=FAKE, w=FAKE, dy=FAKE, z_codes=FAKE, z_scale=FAKE, dx=FAKE, dw=FAKE,
             dbias=FAKE)
    a.update(over)
    return moe.MoELinearGradArgs(**a)


@pytest.mark.parametrize("over,status", BAD_CONFIGS, ids=[str(o) for o, _ in BAD_CONFIGS])
def test_bad_configurations(over, status):
    c = cfg(**over)
    assert forward(c, args()) == status and moe.lib().moe_last_error()
    assert moe.moe_linear_workspace_size(c) == 0
    assert moe.moe_linear_backward_workspace_size(c) == 0
    assert backward(c, grads()) == status


def test_workspace_sizes():
    c = cfg()
    assert moe.moe_linear_workspace_size(c) % 256 == 0
    n = moe.moe_linear_backward_workspace_size(c)
    assert n % 256 == 0 and n >= 100 * 192 * 2
    assert moe.moe_linear_backward_workspace_size(cfg(rows=0)) > 0
    assert moe.moe_group_workspace_size(0, 8, 2) > 0
    assert moe.moe_group_workspace_size(1 << 20, 512, 16) >= 512 * 4
    for bad in ((-1, 8, 2), (4, 0, 2), (4, 8, 0), (4, 513, 2), (4, 32, 17), (1 << 27, 32, 16)):
        assert moe.moe_group_workspace_size(*bad) == 0


@pytest.mark.parametrize("over,status", [
    (dict(x=None), INVALID), (dict(offsets=None), INVALID), (dict(w=None), INVALID),
    (dict(y=None), INVALID), (dict(y=FAKE + 8), INVALID), (dict(x=FAKE + 2), INVALID),
    (dict(bias=FAKE + 4), INVALID), (dict(residual=FAKE + 8), INVALID),
    (dict(w_scale=FAKE), INVALID),            # weights are not FP8
    (dict(z_codes=FAKE), INVALID), (dict(z_scale=FAKE), INVALID),
    (dict(row_index=FAKE), INVALID),          # x_rows is 0
])
def test_forward_refusals(over, status):
    assert forward(cfg(), args(**over)) == status
    assert moe.lib().moe_last_error()


def test_forward_refusals_by_configuration():
    assert forward(None, args()) == INVALID
    assert forward(cfg(), None) == INVALID
    assert forward(cfg(x_rows=7), args()) == INVALID  # no row_index
    assert forward(cfg(weight_format=moe.MOE_WEIGHTS_FP8_E4M3), args()) == INVALID  # no scales
    assert forward(cfg(), args(), ws=None) == WORKSPACE
    assert forward(cfg(), args(), ws=FAKE + 64) == WORKSPACE
    assert forward(cfg(), args(), nbytes=0) == WORKSPACE
    assert forward(cfg(rows=0), args(x=None, y=None)) == moe.MOE_OK


@pytest.mark.parametrize("over,status", [
    (dict(dx=None, dw=None, dbias=None), INVALID), (dict(offsets=None), INVALID),
    (dict(dy=None), INVALID), (dict(w=None), INVALID), (dict(x=None), INVALID),
    (dict(z_codes=None), INVALID), (dict(z_scale=None), INVALID), (dict(row_index=FAKE), INVALID),
    (dict(dx=FAKE + 8), INVALID), (dict(dw=FAKE + 2), INVALID), (dict(dbias=FAKE + 4), INVALID),
])
def test_backward_refusals(over, status):
    assert backward(cfg(), grads(**over)) == status
    assert moe.lib().moe_last_error()


def test_backward_refusals_by_configuration():
    assert backward(None, grads()) == INVALID
    assert backward(cfg(), None) == INVALID
    assert backward(cfg(weight_format=moe.MOE_WEIGHTS_FP8_E4M3), grads()) == UNSUPPORTED
    assert backward(cfg(x_rows=5), grads()) == INVALID
    need = moe.moe_linear_backward_workspace_size(cfg())
    assert backward(cfg(), grads(), nbytes=need - 1) == WORKSPACE
    assert backward(cfg(), grads(), ws=None) == WORKSPACE
    assert backward(cfg(rows=0), grads(dw=None, dbias=None, dx=None)) == moe.MOE_OK


# the last configuration inside each limit of the header, and the first outside it
LIMITS = [
    (dict(groups=512), dict(groups=513)),
    (dict(in_dim=1 << 20, groups=1), dict(in_dim=(1 << 20) + 64, groups=1)),
    (dict(out_dim=1 << 20, groups=1), dict(out_dim=(1 << 20) + 64, groups=1)),
    (dict(rows=(1 << 27) - 1), dict(rows=1 << 27)),
    (dict(x_rows=(1 << 30) - 1), dict(x_rows=1 << 30)),
    (dict(rows=128 * 508 + 127, in_dim=1 << 20), dict(rows=128 * 509, in_dim=1 << 20)),
    (dict(groups=512, in_dim=1 << 15, out_dim=1 << 15), dict(groups=512, in_dim=1 << 15, out_dim=(1 << 15) + 64)),
    # FP8 experts of 8192 -> 2 x 14336, 120 GB of codes
    (dict(groups=512, in_dim=8192, out_dim=14336, activation=4, weight_format=1),
     dict(groups=512, in_dim=1 << 17, out_dim=14336, activation=4, weight_format=1)),
]


@pytest.mark.parametrize("inside,outside", LIMITS, ids=[str(o) for _, o in LIMITS])
def test_limits_are_the_headers(inside, outside):
    """Inside a limit only the missing x is refused, outside it the size."""
    assert moe.moe_linear_workspace_size(cfg(**inside)) > 0
    assert moe.moe_linear_backward_workspace_size(cfg(**inside)) > 0
    a = args(x=None, w_scale=FAKE if inside.get("weight_format") else None)
    assert forward(cfg(**inside), a) == INVALID
    assert forward(cfg(**outside), a) == UNSUPPORTED
    assert moe.moe_linear_workspace_size(cfg(**outside)) == 0
    if not inside.get("weight_format"):
        assert backward(cfg(**inside), grads(dw=None, dy=None)) == INVALID
        assert backward(cfg(**outside), grads(dw=None, dy=None)) == UNSUPPORTED


def test_limit_of_dw():
    """2^36 weights have a forward and a dx, but no dw."""
    c = cfg(groups=512, in_dim=1 << 14, out_dim=1 << 13)
    assert backward(c, grads(dw=None, dy=None)) == INVALID
    assert backward(c, grads(dy=None)) == UNSUPPORTED
    c.out_dim -= 64
    assert backward(c, grads(dy=None)) == INVALID


def test_group_refusals():
    lib = moe.lib()

    def call(T=8, N=4, k=2, cap=0, idx=FAKE, off=FAKE, tok=FAKE, slot=FAKE, ws=FAKE, n=BIG):
        return lib.moe_group_rows(T, N, k, cap, idx, off, tok, slot, ws, n, None)

    assert call(T=-1) == INVALID and call(N=0) == INVALID and call(k=0) == INVALID
    assert call(cap=-1) == INVALID and call(N=513) == UNSUPPORTED and call(k=17) == UNSUPPORTED
    assert call(T=1 << 29) == UNSUPPORTED
    for name in ("idx", "off", "tok", "slot"):
        assert call(**{name: None}) == INVALID
    assert call(ws=None) == WORKSPACE and call(ws=FAKE + 4) == WORKSPACE
    assert call(n=8) == WORKSPACE


def test_checkpoint_refusals():
    lib = moe.lib()
    for fn in (lib.moe_checkpoint_pack, lib.moe_checkpoint_unpack):
        assert fn(-1, 64, 1, FAKE, FAKE, FAKE, None) == INVALID
        assert fn(4, 0, 1, FAKE, FAKE, FAKE, None) == INVALID
        assert fn(4, 100, 1, FAKE, FAKE, FAKE, None) == UNSUPPORTED
        assert fn(1 << 40, 64, 1, FAKE, FAKE, FAKE, None) == UNSUPPORTED
        assert fn(4, 64, 3, FAKE, FAKE, FAKE, None) == INVALID
        for i in range(3):
            p = [FAKE] * 3
            p[i] = None
            assert fn(4, 64, 1, *p, None) == INVALID
        assert fn(0, 64, 1, None, None, None, None) == moe.MOE_OK
    assert lib.moe_checkpoint_pack(4, 64, 1, FAKE + 8, FAKE, FAKE, None) == INVALID
    assert lib.moe_checkpoint_unpack(4, 64, 1, FAKE + 8, FAKE, FAKE, None) == INVALID


def test_combine_refusals():
    lib = moe.lib()

    def fwd(T=4, k=2, n=8, d=64, dt=1, rows=FAKE, slot=FAKE, gate=FAKE, y=FAKE):
        return lib.moe_combine(T, k, n, d, dt, rows, slot, gate, y, None)

    def bwd(T=4, k=2, n=8, d=64, dt=1, rows=FAKE, slot=FAKE, gate=FAKE, dy=FAKE, dr=FAKE, dg=FAKE):
        return lib.moe_combine_backward(T, k, n, d, dt, rows, slot, gate, dy, dr, dg, None)

    for call in (fwd, bwd):
        assert call(T=-1) == INVALID and call(k=0) == INVALID and call(n=-1) == INVALID
        assert call(d=0) == INVALID and call(dt=4) == INVALID
        assert call(d=96) == UNSUPPORTED and call(k=17) == UNSUPPORTED
        assert call(T=1 << 23) == UNSUPPORTED
        assert call(rows=None) == INVALID and call(slot=None) == INVALID
        assert call(rows=FAKE + 8) == INVALID
        assert call(T=0) == moe.MOE_OK
    assert fwd(y=None) == INVALID and fwd(y=FAKE + 4) == INVALID
    assert bwd(dy=None) == INVALID and bwd(dr=None, dg=None) == INVALID
    assert bwd(dr=FAKE + 8) == INVALID


def test_binding_refuses_tensors():
    """What the C ABI cannot see: placement, type, shape and layout."""
    c = moe.make_linear_config(8, 2, 64, 64)
    t = dict(x=torch.zeros(8, 64, dtype=torch.bfloat16), offsets=torch.zeros(3, dtype=torch.int32),
             w=torch.zeros(2, 64, 64, dtype=torch.bfloat16),
             y=torch.zeros(8, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_grouped_linear(c, t["x"], t["offsets"], t["w"], t["y"],
                               workspace=torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_checkpoint_pack(t["x"], torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 1))
    with pytest.raises(ValueError):
        moe.make_linear_config(8, 2, 64, 64, activation="tanh")
    with pytest.raises(ValueError):
        moe.make_linear_config(8, 2, 64, 64, dtype=torch.float16)
    with pytest.raises(moe.MoEError):
        moe.alloc_linear_workspace(moe.make_linear_config(8, 2, 60, 64), "cpu")
    with pytest.raises(moe.MoEError):
        moe.alloc_group_workspace(8, 1000, 2, "cpu")


def test_sizes_past_32_bits_are_refused():
    """2^32 + n is not n, in shapes (of tensors that take no memory) or numbers."""
    def wide(*shape, dtype=torch.bfloat16):
        return torch.zeros(1, dtype=dtype).expand(*shape)

    big, i32 = (1 << 32) + 64, torch.int32
    ws = torch.zeros(256, dtype=torch.uint8)
    calls = [
        lambda: moe.moe_combine(wide(1, big), wide(1, 1, dtype=i32), wide(1, big)),
        lambda: moe.moe_combine(wide(big, 64), wide(1, 1, dtype=i32), wide(1, 64)),
        lambda: moe.moe_combine(wide(1, 64), wide(big, 1, dtype=i32), wide(big, 64)),
        lambda: moe.moe_combine_backward(wide(1, big), wide(1, 1, dtype=i32), None, wide(1, big),
                                         wide(1, big), None),
        lambda: moe.moe_checkpoint_pack(wide(1, big), wide(1, big, dtype=torch.uint8),
                                        wide(1, big // 64, dtype=torch.float32)),
        lambda: moe.moe_checkpoint_unpack(wide(1, big, dtype=torch.uint8),
                                          wide(1, big // 64, dtype=torch.float32), wide(1, big)),
        lambda: moe.moe_group_rows(wide(big, 1, dtype=i32), 8, wide(9, dtype=i32),
                                   wide(big, dtype=i32), wide(big, 1, dtype=i32), workspace=ws),
        lambda: moe.moe_group_rows(wide(4, 1, dtype=i32), 8, wide(9, dtype=i32),
                                   wide(4, dtype=i32), wide(4, 1, dtype=i32), workspace=ws,
                                   capacity=(1 << 32) + 1),
        lambda: moe.alloc_group_workspace(big, 8, 2, "cpu"),
        lambda: moe.make_linear_config(big, 1, 64, 64),
        lambda: moe.make_linear_config(8, 1, 64, big),
    ]
    for call in calls:
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_limit_of_a_checkpoint():
    """Up to 2^35 elements only the alignment is refused."""
    for fn in (moe.lib().moe_checkpoint_pack, moe.lib().moe_checkpoint_unpack):
        for cols in (64, 192, 1 << 30):
            rows = (1 << 35) // cols
            assert fn(rows, cols, 1, FAKE + 8, FAKE, FAKE, None) == INVALID
            assert fn(rows + 1, cols, 1, FAKE + 8, FAKE, FAKE, None) == UNSUPPORTED
