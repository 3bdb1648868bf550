"""Outputs of the operators around the recurrence that share memory with another array of the call are
refused before anything is enqueued, wherever the arrays begin."""
import ctypes

import pytest

import bit_recurrent_state_gdn_b200 as gdn
from bit_recurrent_state_gdn_b200 import _abi, build

BAD = _abi.GDN_ERR_INVALID_ARG
B, L, H, D, K = 2, 8, 3, 16, 4
C = H * D
E = B * L * C  # elements of a token array
M = 1 << 20    # arrays of a call lie so far apart


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _abi.load()


def tok(ptr, sb=L * C, sl=C, sh=D):
    return ctypes.byref(_abi.gdn_tokens(ptr, sb, sl, sh))


def refused(lib, status, *names):
    assert status == BAD
    said = lib.gdn_last_error().decode()
    assert "overlaps" in said and all(n in said for n in names), said


def scan(lib, x=M, g=2 * M, o=3 * M, h0=4 * M, hT=5 * M, hist=6 * M, lens=7 * M, **strides):
    cfg = gdn.make_scan_config(B, H, D, act="f32")
    return lib.gdn_gated_scan(ctypes.byref(cfg), L, tok(x), tok(g), tok(o, **strides), h0, hT, hist,
                              lens, None, 0, None)


@pytest.mark.parametrize("where,names", [
    (dict(o=M), "ox"), (dict(o=M + 4 * (E - 1)), "ox"), (dict(o=M - 4 * (E - 1)), "ox"),
    (dict(o=2 * M + 4 * C), "og"), (dict(h0=3 * M + 4 * (E - 1)), ("o", "h0")),
    (dict(hT=3 * M), ("o", "hT")), (dict(hT=4 * M + 4), ("hT", "h0")),
    (dict(hT=4 * M + 4 * (B * C - 1)), ("hT", "h0")), (dict(hist=5 * M + 4), ("hist", "hT")),
    (dict(hist=4 * M), ("hist", "h0")), (dict(hist=M + 64), ("hist", "x")),
    (dict(lens=5 * M + 8), ("hT", "lens")), (dict(lens=3 * M), ("o", "lens")),
    # rows of twice the length: the gaps between them hold no element, the rows do
    (dict(o=M - 4 * 2 * C, sl=2 * C, sb=2 * L * C), "ox"),
    (dict(x=3 * M + 4 * C, sl=2 * C, sb=2 * L * C), "ox"),
])
def test_scan(lib, where, names):
    refused(lib, scan(lib, **where), *names)


@pytest.mark.parametrize("where,names", [
    (dict(dx=M + 4), ("grad_x", "x")), (dict(dg=2 * M + 4), ("grad_g", "g")),
    (dict(dx=3 * M + 4 * C), ("grad_x", "grad_o")), (dict(dg=4 * M + 4), ("grad_g", "grad_x")),
    (dict(dh0=6 * M + 4), ("grad_h0", "grad_hT")), (dict(dh0=8 * M), ("grad_h0", "hist")),
    (dict(dh0=4 * M), ("grad_h0", "grad_x")), (dict(lens=7 * M), ("grad_h0", "lens")),
])
def test_scan_backward(lib, where, names):
    at = dict(x=M, g=2 * M, do=3 * M, dx=4 * M, dg=5 * M, dhT=6 * M, dh0=7 * M, hist=8 * M, lens=9 * M)
    at.update(where)
    cfg = gdn.make_scan_config(B, H, D, act="f32")
    t = {n: tok(at[n]) for n in ("x", "g", "do", "dx", "dg")}
    refused(lib, lib.gdn_gated_scan_backward(
        ctypes.byref(cfg), L, t["x"], t["g"], at["hist"], t["do"], at["dhT"], t["dx"], t["dg"],
        at["dh0"], at["lens"], None, 0, None), *names)


def test_scan_workspace(lib):
    """The workspace of split sequences is written too."""
    cfg = gdn.make_scan_config(1, 1, 64, act="f32")
    n, G = 8192, 1 << 24
    need = gdn.gdn_gated_scan_workspace_bytes(cfg, n)
    t = {k: tok(v, n * 64, 64, 64) for k, v in dict(x=G, g=2 * G, o=3 * G).items()}

    def call(ws, hT):
        return lib.gdn_gated_scan(ctypes.byref(cfg), n, t["x"], t["g"], t["o"], None, hT, None, None,
                                  ws, need, None)

    refused(lib, call(G + 16, None), "workspace", "x")
    refused(lib, call(4 * G, 4 * G + need - 4), "workspace", "hT")


@pytest.mark.parametrize("where,names", [
    (dict(y=M + 4), "yx"), (dict(y=2 * M - 4), "yz"), (dict(y=4 * M - 4 * C), "yw"),
    (dict(y=5 * M - 4), ("y", "bias")), (dict(y=6 * M), ("y", "lens")),
])
def test_norm(lib, where, names):
    at = dict(x=M, z=2 * M, y=3 * M, w=4 * M, b=5 * M, lens=6 * M)
    at.update(where)
    cfg = gdn.make_norm_config(B, H, D, weight="channel", act="f32")
    refused(lib, lib.gdn_group_norm(ctypes.byref(cfg), L, tok(at["x"]), at["w"], at["b"], tok(at["z"]),
                                    tok(at["y"]), at["lens"], None), *names)


@pytest.mark.parametrize("where,names", [
    (dict(dw=6 * M), ("grad_w", "w")), (dict(db=7 * M), ("grad_bias", "bias")),
    (dict(db=8 * M + 4), ("grad_bias", "grad_w")), (dict(dw=7 * M - 4), ("grad_w", "bias")),
    (dict(dz=2 * M), ("grad_z", "z")), (dict(dz=4 * M + 8), ("grad_z", "grad_x")),
    (dict(dx=3 * M + 4 * C), ("grad_x", "grad_y")), (dict(ws=4 * M), ("workspace", "grad_x")),
    (dict(ws=M + 16), ("workspace", "x")),
])
def test_norm_backward(lib, where, names):
    at = dict(x=M, z=2 * M, dy=3 * M, dx=4 * M, dz=5 * M, w=6 * M, b=7 * M, dw=8 * M, db=9 * M,
              ws=16 * M)
    at.update(where)
    cfg = gdn.make_norm_config(B, H, D, act="f32")
    t = {n: tok(at[n]) for n in ("x", "z", "dy", "dx", "dz")}
    refused(lib, lib.gdn_group_norm_backward(
        ctypes.byref(cfg), L, t["x"], at["w"], at["b"], t["z"], t["dy"], t["dx"], t["dz"], at["dw"],
        at["db"], None, at["ws"], 1 << 30, None), *names)


@pytest.mark.parametrize("where,names", [
    (dict(y=M + 4), "yx"), (dict(y=3 * M), "yw"), (dict(y=4 * M - 4), ("y", "bias")),
    (dict(so=5 * M + 4), ("state_out", "state_in")), (dict(so=2 * M), ("state_out", "y")),
    (dict(so=M), ("state_out", "x")),
])
def test_conv(lib, where, names):
    at = dict(x=M, y=2 * M, w=3 * M, b=4 * M, si=5 * M, so=6 * M)
    at.update(where)
    cfg = gdn.make_conv_config(B, H, D, K, act="f32")
    refused(lib, lib.gdn_short_conv(ctypes.byref(cfg), L, tok(at["x"]), at["w"], at["b"], at["si"],
                                    tok(at["y"]), at["so"], None, None), *names)


@pytest.mark.parametrize("where,names", [
    (dict(dw=4 * M), ("grad_w", "w")), (dict(db=5 * M), ("grad_bias", "bias")),
    (dict(db=6 * M + 4), ("grad_bias", "grad_w")), (dict(dx=2 * M + 4), ("grad_x", "grad_y")),
    (dict(dsi=8 * M), ("grad_state_in", "state_in")), (dict(dsi=9 * M + 4), ("grad_state_in", "grad_state_out")),
    (dict(dsi=3 * M), ("grad_state_in", "grad_x")), (dict(ws=2 * M), ("workspace", "grad_y")),
])
def test_conv_backward(lib, where, names):
    at = dict(x=M, dy=2 * M, dx=3 * M, w=4 * M, b=5 * M, dw=6 * M, db=7 * M, si=8 * M, dso=9 * M,
              dsi=10 * M, ws=16 * M)
    at.update(where)
    cfg = gdn.make_conv_config(B, H, D, K, act="f32")
    refused(lib, lib.gdn_short_conv_backward(
        ctypes.byref(cfg), L, tok(at["x"]), at["w"], at["b"], at["si"], tok(at["dy"]), at["dso"],
        tok(at["dx"]), at["dw"], at["db"], at["dsi"], None, at["ws"], 1 << 30, None), *names)
