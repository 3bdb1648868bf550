"""The operators around the recurrence on the host: what their entry points refuse before anything
is enqueued, empty batches, workspace sizes, and the 64-bit reference forms against autograd."""
import ctypes
import math

import pytest
import torch

import bit_recurrent_state_gdn_b200 as gdn
import layer_ref as ref
from bit_recurrent_state_gdn_b200 import _abi, build

BAD, LACK = _abi.GDN_ERR_INVALID_ARG, _abi.GDN_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _abi.load()


def tok(ptr=4096, sb=1 << 20, sl=64, sh=16):
    return ctypes.byref(_abi.gdn_tokens(ptr, sb, sl, sh))


def scan_call(lib, cfg, L=4, x=None, g=None, o=None, lens=None):
    return lib.gdn_gated_scan(ctypes.byref(cfg), L, x or tok(4096), g or tok(8192), o or tok(12288),
                              None, None, None, lens, None, 0, None)


def norm_call(lib, cfg, L=4, x=None, y=None, w=4096, z=None):
    return lib.gdn_group_norm(ctypes.byref(cfg), L, x or tok(4096), w, None, z, y or tok(12288),
                              None, None)


def conv_call(lib, cfg, L=4, x=None, y=None, w=4096):
    return lib.gdn_short_conv(ctypes.byref(cfg), L, x or tok(4096), w, None, None, y or tok(12288),
                              None, None, None)


MAKE = {
    "scan": (lambda **k: gdn.make_scan_config(**{**dict(B=2, H=4, D=16), **k}), scan_call),
    "norm": (lambda **k: gdn.make_norm_config(**{**dict(B=2, H=4, D=16), **k}), norm_call),
    "conv": (lambda **k: gdn.make_conv_config(**{**dict(B=2, H=4, D=16), **k}), conv_call),
}


@pytest.mark.parametrize("op", list(MAKE))
@pytest.mark.parametrize("field,value", [("B", -1), ("H", -1), ("D", 0), ("act_dtype", 2)])
def test_bad_sizes_are_refused(lib, op, field, value):
    make, call = MAKE[op]
    cfg = make()
    setattr(cfg, field, value)
    assert call(lib, cfg) == BAD and lib.gdn_last_error() != b""


@pytest.mark.parametrize("op", list(MAKE))
def test_sizes_beyond_the_limits_are_refused(lib, op):
    make, call = MAKE[op]
    assert call(lib, make(H=1 << 20, D=2048)) == BAD       # H D > 2^30
    assert call(lib, make(B=1 << 20, H=1 << 20)) == BAD    # B H >= 2^31
    assert call(lib, make(B=1 << 20, H=1 << 10, D=128)) == BAD  # B H D > 2^36
    assert call(lib, make(), L=-1) == BAD
    assert call(lib, make(), L=(1 << 30) + 1) == BAD
    assert lib.gdn_gated_scan(None, 1, *[None] * 8, 0, None) == BAD
    assert lib.gdn_group_norm(None, 1, *[None] * 7) == BAD
    assert lib.gdn_short_conv(None, 1, *[None] * 8) == BAD


@pytest.mark.parametrize("op", list(MAKE))
def test_bad_token_arrays_are_refused(lib, op):
    make, call = MAKE[op]
    cfg, f32 = make(), make(act="f32")
    out = "o" if op == "scan" else "y"
    assert call(lib, cfg, x=tok(0)) == BAD
    assert call(lib, cfg, x=tok(4097)) == BAD                  # not on an element
    assert call(lib, f32, x=tok(4098)) == BAD
    assert call(lib, cfg, x=tok(sl=-64)) == BAD
    assert call(lib, cfg, x=tok(sb=1 << 62)) == BAD            # offsets overflow
    assert call(lib, cfg, x=tok(sb=1 << 40, sl=(1 << 27) + 1)) == LACK
    assert call(lib, cfg, **{out: tok(12288, sl=0)}) == BAD    # written elements share memory
    assert call(lib, cfg, **{out: tok(12288, sh=15)}) == BAD
    assert call(lib, cfg, **{out: tok(12288, sl=63)}) == BAD
    assert call(lib, cfg, **{out: tok(12288, sb=100)}) == BAD
    assert call(lib, cfg, x=tok(4096), **{out: tok(4096)}) == BAD


@pytest.mark.parametrize("op", list(MAKE))
def test_empty_batches_are_valid(lib, op):
    make, call = MAKE[op]
    assert call(lib, make(B=0)) == _abi.GDN_OK
    assert call(lib, make(H=0)) == _abi.GDN_OK


def test_bad_options_are_refused(lib):
    cfg = MAKE["scan"][0]()
    cfg.scale = 3
    assert scan_call(lib, cfg) == BAD
    assert scan_call(lib, MAKE["scan"][0](), lens=4098) == BAD
    for field, value, want in (("center", 2, BAD), ("activation", 3, BAD), ("weight", 2, BAD),
                               ("eps", 0.0, BAD), ("eps", -1.0, BAD), ("eps", math.nan, BAD),
                               ("eps", math.inf, BAD), ("D", 8193, LACK)):
        cfg = MAKE["norm"][0]()
        setattr(cfg, field, value)
        assert norm_call(lib, cfg, y=tok(12288, 1 << 26, 1 << 20, 1 << 14)) == want, field
    assert norm_call(lib, MAKE["norm"][0](), w=None) == BAD
    for field, value, want in (("activation", 2, BAD), ("K", 0, BAD), ("K", 1, LACK),
                               ("K", 5, LACK)):
        cfg = MAKE["conv"][0]()
        setattr(cfg, field, value)
        assert conv_call(lib, cfg) == want, field
    assert conv_call(lib, MAKE["conv"][0](), w=None) == BAD
    for bad in (lambda: gdn.make_scan_config(1, 1, 8, scale="half"),
                lambda: gdn.make_norm_config(1, 1, 8, activation="relu"),
                lambda: gdn.make_norm_config(1, 1, 8, weight="row"),
                lambda: gdn.make_conv_config(1, 1, 8, act="fp16")):
        with pytest.raises(KeyError):
            bad()


def test_backward_refusals(lib):
    c = ctypes.byref
    sc, nc, cc = (MAKE[op][0]() for op in ("scan", "norm", "conv"))

    def scan(hist=4096, dx=None, dg=None):
        return lib.gdn_gated_scan_backward(c(sc), 4, tok(4096), tok(8192), hist, tok(16384), None,
                                           dx or tok(20480), dg or tok(24576), None, None, None, 0, None)

    assert scan(hist=None) == BAD
    assert scan(dx=tok(4096)) == BAD and scan(dg=tok(8192)) == BAD
    assert scan(dg=tok(24576, sl=8)) == BAD

    def norm(bias=None, db=None, z=None, dz=None, ws=4096, n=1 << 30, dw=4096, dx=None):
        return lib.gdn_group_norm_backward(c(nc), 4, tok(4096), 4096, bias, z, tok(8192),
                                           dx or tok(12288), dz, dw, db, None, ws, n, None)

    assert norm(bias=4096) == BAD and norm(db=4096) == BAD
    assert norm(z=tok(16384)) == BAD and norm(dz=tok(16384)) == BAD
    assert norm(dw=None) == BAD and norm(ws=None) == BAD and norm(ws=4104) == BAD
    need = gdn.gdn_group_norm_backward_workspace_bytes(nc, 4)
    assert need > 0 and norm(n=need - 1) == BAD
    assert norm(dx=tok(8192)) == BAD
    assert norm(z=tok(16384), dz=tok(12288)) == BAD            # grad_z is grad_x

    def conv(bias=None, db=None, ws=4096, n=1 << 30, si=None, dso=None, dsi=None):
        return lib.gdn_short_conv_backward(c(cc), 4, tok(4096), 4096, bias, si, tok(8192), dso,
                                           tok(12288), 4096, db, dsi, None, ws, n, None)

    assert conv(bias=4096) == BAD and conv(db=8192) == BAD and conv(ws=None) == BAD
    need = gdn.gdn_short_conv_backward_workspace_bytes(cc, 4)
    assert need > 0 and conv(n=need - 1) == BAD
    assert conv(si=4096, dsi=4096) == BAD and conv(dso=4096, dsi=4096) == BAD


def test_scan_workspace(lib):
    """Only few and long sequences are split; a call that needs the workspace refuses to go without."""
    long = MAKE["scan"][0](B=1, H=2)
    need = gdn.gdn_gated_scan_workspace_bytes(long, 5000)
    assert need > 0 and gdn.gdn_gated_scan_workspace_bytes(long, 4095) == 0
    assert gdn.gdn_gated_scan_workspace_bytes(MAKE["scan"][0](B=40), 5000) == 0
    assert gdn.gdn_gated_scan_workspace_bytes(gdn.make_scan_config(0, 2, 16), 5000) == 0
    assert scan_call(lib, long, L=5000) == BAD and b"workspace" in lib.gdn_last_error()


def test_workspaces_of_what_is_refused_are_empty(lib):
    assert gdn.gdn_group_norm_backward_workspace_bytes(gdn.make_norm_config(1, 1, 9000), 4) == 0
    assert gdn.gdn_short_conv_backward_workspace_bytes(gdn.make_conv_config(1, 1, 8, 7), 4) == 0
    assert gdn.gdn_group_norm_backward_workspace_bytes(gdn.make_norm_config(0, 1, 8), 4) == 0


def test_wrapper_refusals(lib):
    """What the C entry points cannot see, refused before they are reached."""
    cfg = gdn.make_scan_config(2, 3, 8, act="f32")
    x = torch.zeros((2, 5, 3, 8))
    with pytest.raises(ValueError, match="CUDA device"):
        gdn.gdn_gated_scan(cfg, x, x, x)
    with pytest.raises(ValueError, match="dimensions"):
        gdn.gdn_gated_scan(cfg, x[0], x, x)
    with pytest.raises(ValueError, match="g has shape"):
        gdn.gdn_gated_scan(cfg, x, x[:, :4], x)
    with pytest.raises(ValueError, match="x has dtype"):
        gdn.gdn_gated_scan(cfg, x.bfloat16(), x, x)
    with pytest.raises(ValueError, match="contiguous channels"):
        gdn.gdn_gated_scan(cfg, torch.zeros((2, 5, 3, 16))[..., ::2], x, x)
    with pytest.raises(ValueError, match="h0 has"):
        gdn.gdn_gated_scan(cfg, x, x, x, h0=torch.zeros((2, 3, 7)))
    with pytest.raises(ValueError, match="lens has dtype"):
        gdn.gdn_gated_scan(cfg, x, x, x, lens=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="hT must be contiguous"):
        gdn.gdn_gated_scan(cfg, x, x, x, hT=torch.zeros((3, 2, 8)).transpose(0, 1))
    with pytest.raises(ValueError, match="expected cpu"):
        gdn.gdn_gated_scan(cfg, x, x.to("meta"), x)
    nc = gdn.make_norm_config(2, 3, 8, weight="channel", act="f32")
    with pytest.raises(ValueError, match="w has"):
        gdn.gdn_group_norm(nc, x, torch.zeros(8), x)
    cc = gdn.make_conv_config(2, 3, 8, 4, act="f32")
    with pytest.raises(ValueError, match="state_in has"):
        gdn.gdn_short_conv(cc, x, torch.zeros((24, 4)), x, state_in=torch.zeros((2, 4, 24)))


# ---- the reference forms ----------------------------------------------------------------------


def grads(f, args):
    args = [a.double().requires_grad_(True) for a in args]
    out, weight = f(*args)
    return torch.autograd.grad((out * weight).sum(), args)


@pytest.mark.parametrize("scale", ["none", "complement", "sqrt"])
def test_reference_scan_gradients(scale):
    r = torch.Generator().manual_seed(1)
    x, R = (torch.randn((2, 9, 1, 3), generator=r).double() for _ in range(2))
    g = -torch.rand((2, 9, 1, 3), generator=r).double() - 0.1
    h0, RT = (torch.randn((2, 1, 3), generator=r).double() for _ in range(2))

    def f(x, g, h0):
        h, outs = h0, []
        for t in range(9):
            h = g[:, t].exp() * h + ref.scan_factor(g[:, t], scale) * x[:, t]
            outs.append(h)
        return torch.cat([torch.stack(outs, 1), h[:, None]], 1), torch.cat([R, RT[:, None]], 1)

    want = grads(f, [x, g, h0])
    got = ref.scan_backward(x, g, h0, R, RT, scale)
    for a, b in zip(want, got):
        assert torch.allclose(a, b, rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("activation", ["none", "silu", "sigmoid"])
def test_reference_norm_gradients(center, gate, activation):
    r = torch.Generator().manual_seed(2)
    x, z, R = (torch.randn((2, 3, 2, 5), generator=r).double() for _ in range(3))
    w, b = (torch.randn((2, 5), generator=r).double() for _ in range(2))
    z = z if gate else None

    def f(x, w, b, *zz):
        m = x.mean(-1, keepdim=True) if center else 0.0
        u = (x - m) / torch.sqrt(((x - m) ** 2).mean(-1, keepdim=True) + 1e-5) * w + b
        fn = {"none": lambda v: v, "silu": torch.nn.functional.silu,
              "sigmoid": torch.sigmoid}[activation]
        return (u * fn(zz[0]) if zz else fn(u)), R

    want = grads(f, [x, w, b] + ([z] if gate else []))
    dx, _, dz, _, tw, tb = ref.norm_backward(x, w, b, z, R, activation, center, 1e-5)
    got = [dx, tw[0].sum((0, 1)), tb[0].sum((0, 1))] + ([dz] if gate else [])
    for a, c in zip(want, got):
        assert torch.allclose(a, c, rtol=1e-9, atol=1e-12)


@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("activation", ["none", "silu"])
def test_reference_conv_gradients(K, activation):
    r = torch.Generator().manual_seed(3)
    x, R = (torch.randn((2, 7, 4), generator=r).double() for _ in range(2))
    w, b = torch.randn((4, K), generator=r).double(), torch.randn((4,), generator=r).double()
    s, RS = (torch.randn((2, K - 1, 4), generator=r).double() for _ in range(2))

    def f(x, w, b, s):
        rows = torch.cat([s, x], 1)
        p = torch.nn.functional.conv1d(rows.transpose(1, 2), w[:, None], b, groups=4).transpose(1, 2)
        y = torch.nn.functional.silu(p) if activation == "silu" else p
        return torch.cat([y, rows[:, 7:]], 1), torch.cat([R, RS], 1)

    want = grads(f, [x, w, b, s])
    got = ref.conv_backward(x, w, b, s, R, RS, activation)
    for a, c in zip(want, (got[0], got[1], got[2], got[3])):
        assert torch.allclose(a, c[0], rtol=1e-9, atol=1e-12)
