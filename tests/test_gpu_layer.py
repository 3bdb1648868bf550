"""The operators around the recurrence (include/gdnq_layer.h) against their plain 64-bit forms
(layer_ref), element by element within bounds on fp32's roundings: sizes around the kernels' tiles,
odd ones, one token and none, every placement of the token arrays, padded batches with garbage
behind the sequences, both types; gradients also against differences of the forward pass; one
layer run end to end."""
import math

import pytest
import torch

import bit_recurrent_state_gdn_b200 as gdn
import layer_ref as ref
from layer_ref import close

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
MARK = 777.0  # what outputs hold before a call


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def place(t, how):
    """A CUDA copy of [B][L][H][D] laid out in one of the ways that callers have."""
    B, L, H, D = t.shape
    t = t.cuda()
    if how == "tokens":
        return t.contiguous()
    if how == "heads":
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if how == "wide":
        buf = torch.full((B, L, 2 * H * D), float("nan"), dtype=t.dtype, device="cuda")
        out = buf[..., H * D:].unflatten(-1, (H, D))
    elif how == "odd":  # one element off any alignment, rows of odd length
        buf = torch.full((B * L * (H * D + 1) + 1,), float("nan"), dtype=t.dtype, device="cuda")
        out = buf[1:].view(B, L, H * D + 1)[..., :H * D].unflatten(-1, (H, D))
    else:
        raise KeyError(how)
    out.copy_(t)
    return out


def blank(shape, dtype, how):
    return place(torch.full(shape, MARK, dtype=dtype), how)


def check_rows(got, want, bound, lens, dtype, where):
    """Live tokens within the bound, the others as they were."""
    B, L = want.shape[:2]
    live = ref.live_mask(lens, B, L)
    got = got.cpu()
    close(got[live], want[live], bound[live], dtype, where)
    assert bool((got[~live] == MARK).all()), where


def poison(t, lens):
    """NaN behind every sequence's end."""
    if lens is None:
        return t
    t = t.clone()
    t[~ref.live_mask(lens, *t.shape[:2])] = float("nan")
    return t


# ---- gated scan ---------------------------------------------------------------------------

SCAN = [
    # B, L, H, D, dtype, scale, place, lens
    (2, 1, 3, 16, "bf16", "none", "tokens", None),
    (3, 1, 2, 5, "f32", "sqrt", "odd", [1, 0, 1]),
    (1, 2, 1, 1, "f32", "complement", "tokens", None),
    (2, 7, 2, 64, "bf16", "sqrt", "heads", None),
    (2, 8, 1, 64, "f32", "sqrt", "wide", None),
    (2, 9, 4, 32, "bf16", "complement", "tokens", [9, 4]),
    (1, 63, 2, 33, "f32", "none", "odd", None),
    (2, 64, 2, 66, "bf16", "sqrt", "odd", None),
    (3, 65, 1, 130, "bf16", "none", "heads", [65, 64, 1]),
    (2, 128, 3, 50, "f32", "complement", "heads", [127, 500]),
    (4, 129, 2, 64, "bf16", "sqrt", "wide", [-3, 129, 0, 63]),
    (1, 200, 5, 7, "f32", "sqrt", "tokens", None),
    (2, 513, 1, 128, "bf16", "complement", "tokens", [511, 300]),
    (1, 1100, 2, 64, "f32", "sqrt", "heads", None),
    (1, 2049, 1, 48, "bf16", "none", "tokens", None),
    (150, 70, 4, 64, "bf16", "sqrt", "tokens", None),
    (37, 190, 16, 128, "f32", "complement", "tokens", None),
    # every way of sharing the work out: four warps, one warp, clusters of four and two
    (10, 190, 32, 64, "bf16", "sqrt", "tokens", [190, 0, 1, 64, 65, 128, 129, 189, 16, 17]),
    (10, 140, 32, 64, "f32", "none", "heads", None),
    (10, 77, 32, 65, "bf16", "sqrt", "odd", None),
    (64, 100, 32, 64, "bf16", "complement", "tokens", [100, 3] * 32),
    (15, 1100, 4, 64, "bf16", "sqrt", "tokens", [1100, 0, 513] * 5),
    (20, 300, 4, 64, "f32", "sqrt", "wide", [300, 128, 129, 1] * 5),
    # sequences of one run, many of them
    (52, 1, 5, 43, "bf16", "complement", "wide", [1, 0, 1, 1] * 13),
    (33, 8, 2, 64, "bf16", "sqrt", "heads", None),
    (33, 5, 3, 33, "f32", "sqrt", "odd", [5, 0, 3] * 11),
    # sequences split into spans
    (1, 4096, 1, 16, "bf16", "sqrt", "tokens", None),
    (3, 4500, 1, 70, "f32", "complement", "heads", [4500, 1, 4097]),
    (2, 5001, 1, 33, "bf16", "none", "odd", [0, 4999]),
    (5, 4200, 2, 64, "bf16", "sqrt", "wide", [4200, 129, 128, 2000, 4199]),
]


def scan_inputs(B, L, H, D, dtype, lens, seed=0):
    r = gen(seed)
    x = torch.randn((B, L, H, D), generator=r).to(DT[dtype])
    rate = torch.exp(torch.rand((H, D), generator=r) * math.log(700.0)) * 1e-3
    g = -2.0 * rate * torch.sigmoid(torch.randn((B, L, H, D), generator=r))
    k = torch.rand((B, L, H, D), generator=r)
    g = torch.where(k < 0.02, -math.inf, torch.where(k > 0.99, 0.0, g))
    g = torch.where((k > 0.02) & (k < 0.03), -90.0, g)  # e^g is subnormal or zero
    h0 = torch.randn((B, H, D), generator=r)
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    return x, g.float(), h0, n


def cuda(t):
    return None if t is None else t.cuda()


@pytest.mark.parametrize("case", SCAN, ids=[f"{c[:7]}{'r' if c[7] else ''}" for c in SCAN])
@pytest.mark.parametrize("given", [True, False])
def test_scan(case, given):
    B, L, H, D, dtype, scale, how, lens = case
    x, g, h0, n = scan_inputs(B, L, H, D, dtype, lens)
    h0 = h0 if given else torch.zeros_like(h0)
    cfg = gdn.make_scan_config(B, H, D, scale=scale, act=dtype)
    o = blank(x.shape, DT[dtype], how)
    hT = torch.full((B, H, D), MARK, device="cuda")
    hist = torch.full(gdn.gdn_scan_hist_shape(cfg, L), MARK, device="cuda")
    gdn.gdn_gated_scan(cfg, place(poison(x, n), how), place(poison(g, n), how), o,
                       h0=cuda(h0) if given else None, hT=hT, hist=hist if given else None,
                       lens=cuda(n))
    want, end, before, err, err_before, err_end = ref.scan(x, g, h0, scale, n)
    check_rows(o, want, err, n, DT[dtype], "o")
    close(hT, end, err_end, torch.float32, "hT")
    if given:
        for b, e in enumerate(ref.lens_of(n, B, L)):
            kept = -(-e // 64)
            close(hist[b, :kept], before[b, 0:e:64], err_before[b, 0:e:64], torch.float32, "hist")
            assert bool((hist[b, kept:] == MARK).all())


@pytest.mark.parametrize("case", SCAN, ids=[f"{c[:7]}{'r' if c[7] else ''}" for c in SCAN])
@pytest.mark.parametrize("given", [True, False])
def test_scan_backward(case, given):
    B, L, H, D, dtype, scale, how, lens = case
    x, g, h0, n = scan_inputs(B, L, H, D, dtype, lens, seed=1)
    r = gen(2)
    do = torch.randn(x.shape, generator=r).to(DT[dtype])
    dhT = torch.randn((B, H, D), generator=r) if given else torch.zeros((B, H, D))
    cfg = gdn.make_scan_config(B, H, D, scale=scale, act=dtype)
    xs, gs = place(poison(x, n), how), place(poison(g, n), "tokens")
    hist = torch.full(gdn.gdn_scan_hist_shape(cfg, L), float("nan"), device="cuda")
    gdn.gdn_gated_scan(cfg, xs, gs, blank(x.shape, DT[dtype], how), h0=cuda(h0), hist=hist,
                       lens=cuda(n))
    dx, dg = blank(x.shape, DT[dtype], how), blank(x.shape, torch.float32, "tokens")
    dh0 = torch.full((B, H, D), MARK, device="cuda") if given else None
    gdn.gdn_gated_scan_backward(cfg, xs, gs, hist, place(poison(do, n), how), dx, dg,
                                dhT=cuda(dhT) if given else None, dh0=dh0, lens=cuda(n))
    wx, wg, w0, ex, eg, e0 = ref.scan_backward(x, g, h0, do, dhT, scale, n)
    check_rows(dx, wx, ex, n, DT[dtype], "dx")
    check_rows(dg, wg, eg, n, torch.float32, "dg")
    if given:
        close(dh0, w0, e0, torch.float32, "dh0")


def test_scan_state_in_place_and_split_over_calls():
    """Decode: calls of 100, 1 and 60 tokens with one state array give the states of one call."""
    B, L, H, D = 3, 161, 2, 64
    x, g, h0, _ = scan_inputs(B, L, H, D, "f32", None, seed=3)
    cfg = gdn.make_scan_config(B, H, D, scale="complement", act="f32")
    xs, gs, h = x.cuda(), g.cuda(), h0.cuda()
    o = torch.zeros_like(xs)
    for lo, hi in ((0, 100), (100, 101), (101, 161)):
        gdn.gdn_gated_scan(cfg, xs[:, lo:hi], gs[:, lo:hi], o[:, lo:hi], h0=h, hT=h)
    want, end, _, err, _, err_end = ref.scan(x, g, h0, "complement")
    close(o, want, err, torch.float32)
    close(h, end, err_end, torch.float32)


def test_scan_state_in_place_of_split_sequences():
    """Long sequences are split over CTAs that all need the first state, which the last one replaces."""
    B, L, H, D = 2, 9000, 1, 96
    x, g, h0, _ = scan_inputs(B, L, H, D, "f32", None, seed=6)
    cfg = gdn.make_scan_config(B, H, D, scale="sqrt", act="f32")
    assert gdn.gdn_gated_scan_workspace_bytes(cfg, L) > 0
    h, o = h0.cuda(), torch.zeros_like(x, device="cuda")
    gdn.gdn_gated_scan(cfg, x.cuda(), g.cuda(), o, h0=h, hT=h)
    want, end, _, err, _, err_end = ref.scan(x, g, h0, "sqrt")
    close(o, want, err, torch.float32)
    close(h, end, err_end, torch.float32)


@pytest.mark.parametrize("back", [False, True])
def test_scan_of_no_tokens(back):
    cfg = gdn.make_scan_config(2, 3, 8, act="f32")
    e = torch.zeros((2, 0, 3, 8), device="cuda")
    h = torch.randn((2, 3, 8), device="cuda")
    out = torch.full_like(h, MARK)
    if back:
        gdn.gdn_gated_scan_backward(cfg, e, e, torch.zeros((2, 0, 3, 8), device="cuda"), e, e, e,
                                    dhT=h, dh0=out)
    else:
        gdn.gdn_gated_scan(cfg, e, e, e, h0=h, hT=out)
    assert torch.equal(out, h)


def test_scan_reads_a_broadcast_gate():
    """One gate per head, seen as [B][L][H][D] with stride 0 over the batch."""
    x, g, h0, _ = scan_inputs(3, 40, 2, 32, "f32", None, seed=4)
    g = g[:1].expand(3, 40, 2, 32)
    cfg = gdn.make_scan_config(3, 2, 32, act="f32")
    o = torch.zeros_like(x, device="cuda")
    gdn.gdn_gated_scan(cfg, x.cuda(), g[:1].cuda().expand(3, 40, 2, 32), o, h0=h0.cuda())
    want, _, _, err, _, _ = ref.scan(x, g, h0, "none")
    close(o, want, err, torch.float32)


def test_scan_forgets_what_is_not_finite():
    """A channel's inf or NaN stays in it, and a gate of -inf ends an inf's reach only by the
    definition (0 x inf is NaN): other channels never see either."""
    x, g, h0, _ = scan_inputs(2, 150, 2, 64, "bf16", None, seed=5)
    want, _, _, err, _, _ = ref.scan(x, g, h0, "none")
    x[0, 3, 0, 7], x[1, 20, 1, 9] = float("inf"), float("nan")
    cfg = gdn.make_scan_config(2, 2, 64)
    o = torch.zeros_like(x, device="cuda")
    gdn.gdn_gated_scan(cfg, x.cuda(), g.cuda(), o, h0=h0.cuda())
    o = o.cpu()
    assert not torch.isfinite(o[0, 3, 0, 7]) and torch.isnan(o[1, 20, 1, 9])
    keep = torch.ones_like(x, dtype=torch.bool)
    keep[0, 3:, 0, 7] = keep[1, 20:, 1, 9] = False
    close(o[keep], want[keep], err[keep], torch.bfloat16)


# ---- group norm ---------------------------------------------------------------------------

NORM = [
    # B, L, H, D, dtype, center, bias, gate, act, weight, place, lens
    (2, 1, 2, 128, "bf16", False, False, True, "silu", "head", "tokens", None),
    (1, 1, 1, 1, "f32", True, True, False, "silu", "channel", "tokens", None),
    (2, 5, 3, 4, "f32", True, True, True, "sigmoid", "channel", "odd", None),
    (2, 9, 4, 16, "bf16", True, False, False, "none", "head", "heads", [9, 2]),
    (3, 17, 2, 31, "bf16", False, True, True, "none", "channel", "odd", [0, 17, 99]),
    (2, 33, 3, 64, "bf16", False, False, True, "silu", "channel", "wide", None),
    (1, 40, 5, 100, "f32", True, True, False, "silu", "channel", "tokens", None),
    (2, 77, 2, 128, "bf16", False, False, True, "sigmoid", "head", "heads", [77, 40]),
    (2, 70, 3, 128, "f32", False, True, False, "sigmoid", "head", "wide", None),
    (2, 21, 2, 129, "bf16", True, True, True, "silu", "head", "tokens", None),
    (1, 13, 3, 256, "bf16", True, True, True, "silu", "channel", "heads", None),
    (1, 11, 2, 512, "f32", False, True, True, "silu", "head", "tokens", None),
    (2, 6, 1, 1000, "bf16", True, False, True, "sigmoid", "channel", "tokens", [3, 6]),
    (1, 5, 2, 1025, "f32", True, True, False, "none", "head", "odd", None),
    (1, 4, 1, 2048, "bf16", False, False, True, "silu", "head", "tokens", None),
    (1, 3, 1, 8192, "bf16", True, True, False, "silu", "channel", "tokens", None),
    (60, 31, 8, 64, "bf16", False, False, True, "silu", "head", "heads", None),
    (3, 700, 6, 32, "f32", True, True, False, "silu", "channel", "tokens", [700, 1, 350]),
    # pieces of 8 and 4 bytes, single elements, few lanes, more than a warp's
    (2, 9, 5, 36, "bf16", True, True, True, "silu", "channel", "wide", None),
    (2, 30, 3, 122, "bf16", False, True, True, "sigmoid", "channel", "heads", [30, 11]),
    (1, 12, 3, 250, "bf16", True, False, True, "silu", "head", "tokens", None),
    (1, 12, 3, 250, "f32", True, True, False, "silu", "channel", "heads", None),
    (2, 50, 6, 7, "bf16", True, True, True, "silu", "channel", "tokens", [50, 20]),
    (2, 50, 33, 8, "bf16", False, False, True, "silu", "head", "tokens", None),
    (2, 20, 9, 2, "f32", True, True, False, "sigmoid", "channel", "heads", None),
    (1, 9, 2, 333, "bf16", False, True, True, "silu", "head", "odd", None),
    (1, 9, 2, 501, "f32", True, True, True, "silu", "channel", "odd", None),
    (1, 7, 2, 600, "bf16", True, True, True, "silu", "head", "tokens", None),
    (1, 7, 2, 999, "bf16", True, False, True, "none", "channel", "odd", [5]),
    (1, 7, 1, 1024, "f32", False, True, True, "sigmoid", "head", "tokens", None),
]


def norm_inputs(case, seed):
    B, L, H, D, dtype, center, bias, gate, activation, weight, how, lens = case
    r = gen(seed)
    x = (torch.randn((B, L, H, D), generator=r) + 0.5).to(DT[dtype])
    n = (D,) if weight == "head" else (H, D)
    w = 1.0 + 0.3 * torch.randn(n, generator=r)
    b = 0.3 * torch.randn(n, generator=r) if bias else None
    z = (2.0 * torch.randn((B, L, H, D), generator=r)).to(DT[dtype]) if gate else None
    dy = torch.randn((B, L, H, D), generator=r).to(DT[dtype])
    return x, w, b, z, dy, None if lens is None else torch.tensor(lens, dtype=torch.int32)


def norm_cfg(case):
    B, L, H, D, dtype, center, bias, gate, activation, weight, how, lens = case
    return gdn.make_norm_config(B, H, D, eps=1e-5, center=center, activation=activation,
                                weight=weight, act=dtype)


@pytest.mark.parametrize("case", NORM, ids=[str(c[:11]) for c in NORM])
def test_norm(case):
    dtype, center, activation, how = case[4], case[5], case[8], case[10]
    x, w, b, z, _, n = norm_inputs(case, 10)
    y = blank(x.shape, DT[dtype], "tokens")
    gdn.gdn_group_norm(norm_cfg(case), place(poison(x, n), how), w.cuda(), y, b=cuda(b),
                       z=None if z is None else place(poison(z, n), "wide"), lens=cuda(n))
    want, err = ref.norm(x, w, b, z, activation, center, 1e-5)
    check_rows(y, want, err, n, DT[dtype], "y")


@pytest.mark.parametrize("case", NORM, ids=[str(c[:11]) for c in NORM])
def test_norm_backward(case):
    B, L, H, D, dtype, center, bias, gate, activation, weight, how, lens = case
    x, w, b, z, dy, n = norm_inputs(case, 11)
    dx = blank(x.shape, DT[dtype], how)
    dz = blank(x.shape, DT[dtype], "tokens") if gate else None
    dw = torch.full(w.shape, MARK, device="cuda")
    db = torch.full(w.shape, MARK, device="cuda") if bias else None
    gdn.gdn_group_norm_backward(norm_cfg(case), place(poison(x, n), how), w.cuda(),
                                place(poison(dy, n), "tokens"), dx, dw, b=cuda(b),
                                z=None if z is None else place(poison(z, n), "wide"), dz=dz, db=db,
                                lens=cuda(n))
    live = ref.live_mask(n, B, L)
    wx, ex, wz, ez, tw, tb = ref.norm_backward(x, w, b, z, dy, activation, center, 1e-5)
    check_rows(dx, wx, ex, n, DT[dtype], "dx")
    if gate:
        check_rows(dz, wz, ez, n, DT[dtype], "dz")
    dims, rows = ((0, 1), H) if weight == "head" else ((0,), 1)
    want, err = ref.summed(tw[0][live], tw[1][live], dims, int(live.sum()) * rows)
    close(dw, want, err, torch.float32, "dw")
    if bias:
        want, err = ref.summed(tb[0][live], tb[1][live], dims, int(live.sum()) * rows)
        close(db, want, err, torch.float32, "db")


@pytest.mark.parametrize("center", [False, True])
def test_norm_of_rows_without_spread(center):
    """Rows of zeros, and with the mean taken off rows of one value: n is 0."""
    cfg = gdn.make_norm_config(1, 2, 64, eps=1e-6, center=center, act="f32")
    x = torch.zeros((1, 3, 2, 64), device="cuda")
    if center:
        x[:, 1] = 3.0
    w, b = torch.ones(64, device="cuda"), torch.full((64,), 0.25, device="cuda")
    y = torch.full_like(x, MARK)
    gdn.gdn_group_norm(cfg, x, w, y, b=b)
    assert torch.equal(y, torch.full_like(y, 0.25))
    dx, dw, db = torch.full_like(x, MARK), torch.empty_like(w), torch.empty_like(b)
    dy = torch.ones_like(x)
    gdn.gdn_group_norm_backward(cfg, x, w, dy, dx, dw, b=b, db=db)
    # n = 0: dx = rstd (dy - [center] mean(dy)), dw = 0
    assert float(dw.abs().max()) == 0.0 and torch.equal(db, torch.full_like(db, 6.0))
    want = torch.zeros_like(dx) if center else torch.full_like(dx, 1e3)
    assert torch.allclose(dx, want, rtol=1e-5, atol=0.0)


def test_norm_of_no_tokens_has_no_parameter_gradient():
    cfg = gdn.make_norm_config(2, 3, 8, weight="channel", act="f32")
    e, w = torch.zeros((2, 0, 3, 8), device="cuda"), torch.ones((3, 8), device="cuda")
    dw, db = torch.full_like(w, MARK), torch.full_like(w, MARK)
    gdn.gdn_group_norm_backward(cfg, e, w, e, e, dw, b=w, db=db)
    assert float(dw.abs().max()) == 0.0 and float(db.abs().max()) == 0.0
    gdn.gdn_group_norm(cfg, e, w, e)


def test_norm_row_with_nan_stays_alone():
    x = torch.randn((1, 9, 4, 16), generator=gen(12))
    cfg = gdn.make_norm_config(1, 4, 16, act="f32")
    w = torch.ones(16, device="cuda")
    clean, y = torch.empty_like(x, device="cuda"), torch.empty_like(x, device="cuda")
    gdn.gdn_group_norm(cfg, x.cuda(), w, clean)
    x[0, 4, 2, 3] = float("nan")
    gdn.gdn_group_norm(cfg, x.cuda(), w, y)
    assert bool(torch.isnan(y[0, 4, 2]).all())
    y[0, 4, 2] = clean[0, 4, 2]
    assert torch.equal(y, clean)


# ---- short convolution ----------------------------------------------------------------------

CONV = [
    # B, L, H, D, dtype, K, bias, act, place, lens
    (2, 1, 2, 64, "bf16", 4, False, "silu", "tokens", None),
    (3, 1, 1, 5, "f32", 3, True, "silu", "odd", [1, 0, 1]),
    (2, 2, 2, 16, "bf16", 4, True, "none", "heads", None),
    (2, 3, 1, 33, "f32", 2, False, "silu", "wide", [1, 3]),
    (2, 15, 3, 40, "bf16", 3, True, "silu", "odd", None),
    (4, 16, 2, 32, "bf16", 4, False, "silu", "tokens", [2, 16, 0, 9]),
    (2, 31, 1, 128, "f32", 4, True, "silu", "heads", None),
    (2, 32, 2, 64, "bf16", 2, True, "none", "wide", None),
    (3, 33, 1, 48, "bf16", 4, True, "silu", "tokens", [33, 32, -1]),
    (2, 64, 2, 17, "f32", 3, False, "none", "tokens", None),
    (1, 65, 3, 128, "bf16", 4, False, "silu", "heads", None),
    (2, 130, 1, 256, "bf16", 4, True, "silu", "wide", [129, 700]),
    (1, 500, 2, 72, "f32", 4, True, "silu", "tokens", None),
    (40, 70, 4, 128, "bf16", 4, True, "silu", "tokens", None),
    (300, 1, 8, 128, "bf16", 4, False, "silu", "tokens", None),
    # channels in pairs and fours, several sequences a thread, long sequences in many runs
    (3, 70, 3, 50, "bf16", 4, True, "silu", "heads", [70, 3, 69]),
    (2, 33, 1, 50, "f32", 3, True, "silu", "tokens", None),
    (2, 90, 3, 20, "bf16", 4, False, "none", "heads", None),
    (2100, 1, 16, 128, "bf16", 4, True, "silu", "tokens", [1, 1, 0] * 700),
    (2100, 1, 3, 50, "f32", 2, False, "silu", "tokens", None),
    (1, 5000, 1, 64, "bf16", 4, True, "silu", "tokens", None),
    # few channels
    (5, 300, 1, 32, "bf16", 3, True, "silu", "wide", [300, 299, 0, 1, 40]),
    (3, 200, 2, 7, "bf16", 4, True, "silu", "heads", None),
    (2, 200, 1, 26, "f32", 4, True, "none", "tokens", None),
]


def conv_inputs(case, seed):
    B, L, H, D, dtype, K, bias, activation, how, lens = case
    r, dt = gen(seed), DT[dtype]
    C = H * D
    x = torch.randn((B, L, H, D), generator=r).to(dt)
    w = torch.randn((C, K), generator=r) / math.sqrt(K)
    b = 0.3 * torch.randn((C,), generator=r) if bias else None
    state = torch.randn((B, K - 1, C), generator=r).to(dt)
    dy = torch.randn((B, L, H, D), generator=r).to(dt)
    dso = torch.randn((B, K - 1, C), generator=r).to(dt)
    return x, w, b, state, dy, dso, None if lens is None else torch.tensor(lens, dtype=torch.int32)


@pytest.mark.parametrize("case", CONV, ids=[str(c[:9]) for c in CONV])
@pytest.mark.parametrize("given", [True, False])
def test_conv(case, given):
    B, L, H, D, dtype, K, bias, activation, how, lens = case
    x, w, b, state, _, _, n = conv_inputs(case, 20)
    state = state if given else torch.zeros_like(state)
    cfg = gdn.make_conv_config(B, H, D, K, activation=activation, act=dtype)
    y = blank(x.shape, DT[dtype], "heads" if how == "wide" else how)
    out = cuda(state) if given else torch.full(state.shape, MARK, dtype=DT[dtype], device="cuda")
    gdn.gdn_short_conv(cfg, place(poison(x, n), how), w.cuda(), y, bias=cuda(b),
                       state_in=out if given else None, state_out=out, lens=cuda(n))
    want, end, err = ref.conv(x.view(B, L, -1), w, b, state, activation, n)
    check_rows(y, want.view(x.shape), err.view(x.shape), n, DT[dtype], "y")
    assert torch.equal(out.cpu().double(), end)


@pytest.mark.parametrize("case", CONV, ids=[str(c[:9]) for c in CONV])
@pytest.mark.parametrize("given", [True, False])
def test_conv_backward(case, given):
    B, L, H, D, dtype, K, bias, activation, how, lens = case
    x, w, b, state, dy, dso, n = conv_inputs(case, 21)
    if not given:
        state, dso = torch.zeros_like(state), torch.zeros_like(dso)
    cfg = gdn.make_conv_config(B, H, D, K, activation=activation, act=dtype)
    dx = blank(x.shape, DT[dtype], how)
    dw = torch.full(w.shape, MARK, device="cuda")
    db = torch.full((H * D,), MARK, device="cuda") if bias else None
    dsi = torch.full(state.shape, MARK, dtype=DT[dtype], device="cuda") if given else None
    gdn.gdn_short_conv_backward(cfg, place(poison(x, n), how), w.cuda(), place(poison(dy, n), how),
                                dx, dw, bias=cuda(b), db=db, state_in=cuda(state) if given else None,
                                dstate_out=cuda(dso) if given else None, dstate_in=dsi,
                                lens=cuda(n))
    rx, rw, rb, rs = ref.conv_backward(x.view(B, L, -1), w, b, state, dy.view(B, L, -1), dso,
                                       activation, n)
    check_rows(dx, rx[0].view(x.shape), rx[1].view(x.shape), n, DT[dtype], "dx")
    close(dw, *rw, torch.float32, "dw")
    if bias:
        close(db, *rb, torch.float32, "db")
    if given:
        close(dsi, *rs, DT[dtype], "dstate_in")


def test_conv_of_no_tokens():
    cfg = gdn.make_conv_config(2, 1, 8, 3, act="f32")
    e, w = torch.zeros((2, 0, 1, 8), device="cuda"), torch.randn((8, 3), device="cuda")
    s, out = torch.randn((2, 2, 8), device="cuda"), torch.full((2, 2, 8), MARK, device="cuda")
    gdn.gdn_short_conv(cfg, e, w, e, state_in=s, state_out=out)
    assert torch.equal(out, s)
    dw, dsi = torch.full_like(w, MARK), torch.full_like(s, MARK)
    gdn.gdn_short_conv_backward(cfg, e, w, e, e, dw, state_in=s, dstate_out=s, dstate_in=dsi)
    assert float(dw.abs().max()) == 0.0 and torch.equal(dsi, s)


def test_conv_split_over_calls_carries_the_state():
    case = (2, 50, 2, 64, "bf16", 4, True, "silu", "tokens", None)
    x, w, b, state, _, _, _ = conv_inputs(case, 22)
    cfg = gdn.make_conv_config(2, 2, 64, 4)
    xs, y, s = x.cuda(), torch.zeros_like(x, device="cuda"), state.cuda()
    for lo, hi in ((0, 1), (1, 3), (3, 44), (44, 50)):
        gdn.gdn_short_conv(cfg, xs[:, lo:hi], w.cuda(), y[:, lo:hi], bias=b.cuda(), state_in=s,
                           state_out=s)
    want, end, err = ref.conv(x.view(2, 50, -1), w, b, state, "silu")
    close(y.view(2, 50, -1), want, err, torch.bfloat16)
    assert torch.equal(s.cpu().double(), end)


# ---- gradients against differences, streams and graphs, together --------------------------------


def difference(f, args, grads, i, seed):
    """<grad, v> against the central difference of sum(f R) along v, in fp32: the difference's
    own error is its step squared and the outputs' rounding over its step."""
    r = torch.Generator(device="cuda")
    r.manual_seed(seed)
    v = torch.randn(args[i].shape, generator=r, device="cuda")
    v /= v.norm()
    eps = 1e-2
    hi, lo = list(args), list(args)
    hi[i], lo[i] = args[i] + eps * v, args[i] - eps * v
    num = (f(*hi) - f(*lo)) / (2 * eps)
    ana = float((grads[i].double() * v.double()).sum())
    # third derivatives of order one along a unit vector: eps^2; sums of about 1e3 terms of order
    # one, each rounded at 2^-24, over 2 eps: about 1e3 2^-24 / 1e-2
    scale = float(grads[i].double().norm())
    assert abs(num - ana) <= 2e-3 * max(scale, 1.0), (i, num, ana, scale)


@pytest.mark.parametrize("scale", ["none", "complement", "sqrt"])
def test_scan_gradients_against_differences(scale):
    B, L, H, D = 2, 70, 1, 8
    r = torch.Generator(device="cuda")
    r.manual_seed(30)
    x = torch.randn((B, L, H, D), generator=r, device="cuda")
    g = -0.3 - torch.rand((B, L, H, D), generator=r, device="cuda")
    h0 = torch.randn((B, H, D), generator=r, device="cuda")
    R, RT = torch.randn_like(x), torch.randn_like(h0)
    cfg = gdn.make_scan_config(B, H, D, scale=scale, act="f32")
    hist = torch.empty(gdn.gdn_scan_hist_shape(cfg, L), device="cuda")

    def f(x, g, h0):
        o, hT = torch.empty_like(x), torch.empty_like(h0)
        gdn.gdn_gated_scan(cfg, x, g, o, h0=h0, hT=hT, hist=hist)
        return float((o.double() * R).sum() + (hT.double() * RT).sum())

    f(x, g, h0)
    dx, dg, dh0 = torch.empty_like(x), torch.empty_like(g), torch.empty_like(h0)
    gdn.gdn_gated_scan_backward(cfg, x, g, hist, R, dx, dg, dhT=RT, dh0=dh0)
    for i in range(3):
        difference(f, [x, g, h0], [dx, dg, dh0], i, 31 + i)


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("center", [False, True])
def test_norm_gradients_against_differences(gate, center):
    B, L, H, D = 2, 9, 2, 24
    r = torch.Generator(device="cuda")
    r.manual_seed(40)
    x = torch.randn((B, L, H, D), generator=r, device="cuda")
    w = 1 + 0.3 * torch.randn((H, D), generator=r, device="cuda")
    b = 0.3 * torch.randn((H, D), generator=r, device="cuda")
    z = torch.randn((B, L, H, D), generator=r, device="cuda")
    R = torch.randn_like(x)
    cfg = gdn.make_norm_config(B, H, D, center=center, activation="silu", weight="channel",
                               act="f32")

    def f(x, w, b, z):
        y = torch.empty_like(x)
        gdn.gdn_group_norm(cfg, x, w, y, b=b, z=z if gate else None)
        return float((y.double() * R).sum())

    dx, dz, dw, db = torch.empty_like(x), torch.empty_like(z), torch.empty_like(w), torch.empty_like(b)
    gdn.gdn_group_norm_backward(cfg, x, w, R, dx, dw, b=b, z=z if gate else None,
                                dz=dz if gate else None, db=db)
    for i in range(4 if gate else 3):
        difference(f, [x, w, b, z], [dx, dw, db, dz], i, 41 + i)


def test_conv_gradients_against_differences():
    B, L, H, D, K = 2, 40, 1, 12, 4
    r = torch.Generator(device="cuda")
    r.manual_seed(50)
    x = torch.randn((B, L, H, D), generator=r, device="cuda")
    w = 0.5 * torch.randn((D, K), generator=r, device="cuda")
    b = 0.3 * torch.randn((D,), generator=r, device="cuda")
    s = torch.randn((B, K - 1, D), generator=r, device="cuda")
    R, RS = torch.randn_like(x), torch.randn_like(s)
    cfg = gdn.make_conv_config(B, H, D, K, act="f32")

    def f(x, w, b, s):
        y, out = torch.empty_like(x), torch.empty_like(s)
        gdn.gdn_short_conv(cfg, x, w, y, bias=b, state_in=s, state_out=out)
        return float((y.double() * R).sum() + (out.double() * RS).sum())

    dx, dw, db, ds = (torch.empty_like(t) for t in (x, w, b, s))
    gdn.gdn_short_conv_backward(cfg, x, w, R, dx, dw, bias=b, db=db, state_in=s, dstate_out=RS,
                                dstate_in=ds)
    for i in range(4):
        difference(f, [x, w, b, s], [dx, dw, db, ds], i, 51 + i)


@pytest.mark.parametrize("dims,strides", [
    ((2, 20, 2, 64), (2 ** 31 + 64, 128, 64)),      # sequences further apart than 2^31 elements
    ((1, 20, 2, 64), (0, 2 ** 27, 64)),             # tokens as far apart as they may be
])
def test_arrays_far_apart(dims, strides):
    """Offsets beyond 32 bits, read and written, in all three operators."""
    B, L, H, D = dims
    n = sum((d - 1) * s for d, s in zip(dims, strides)) + D
    free = torch.cuda.mem_get_info()[0]
    if free < 4 * n + (2 << 30):
        pytest.skip("needs two arrays of that size")

    def far(t):
        out = torch.empty(n, dtype=torch.bfloat16, device="cuda").as_strided(dims, (*strides, 1))
        return out.copy_(t)

    x, g, h0, _ = scan_inputs(B, L, H, D, "bf16", None, seed=80)
    xs, out = far(x), far(torch.full_like(x, MARK))
    gdn.gdn_gated_scan(gdn.make_scan_config(B, H, D), xs, g.cuda(), out, h0=h0.cuda())
    want, _, _, err, _, _ = ref.scan(x, g, h0, "none")
    close(out, want, err, torch.bfloat16, "scan")
    w = torch.ones(D)
    gdn.gdn_group_norm(gdn.make_norm_config(B, H, D), xs, w.cuda(), out)
    close(out, *ref.norm(x, w, None, None, "none", False, 1e-6), torch.bfloat16, "norm")
    w = torch.randn((H * D, 4), generator=gen(81))
    gdn.gdn_short_conv(gdn.make_conv_config(B, H, D, 4), xs, w.cuda(), out)
    want, _, err = ref.conv(x.view(B, L, -1), w, None, torch.zeros((B, 3, H * D)), "silu")
    close(out, want.view(x.shape), err.view(x.shape), torch.bfloat16, "conv")


def test_two_layers_at_once():
    """The same layer on two streams side by side, each with arrays and workspaces of its own."""
    sides = [torch.cuda.Stream() for _ in range(2)]
    sets = [layer_state(90 + i, B=3, L=700, H=4) for i in range(2)]
    want = []
    for t, bufs in sets:
        run_layer(t, bufs)
        torch.cuda.synchronize()
        want.append({n: v.clone() for n, v in bufs.items()})
        for v in bufs.values():
            v.fill_(MARK)
    torch.cuda.synchronize()
    for _ in range(3):
        for side, (t, bufs) in zip(sides, sets):
            run_layer(t, bufs, stream=side)
    torch.cuda.synchronize()
    for (t, bufs), w in zip(sets, want):
        for n in w:
            assert torch.equal(bufs[n], w[n]), n


def layer(x, w_conv, g, w_norm, z, h0, bufs, stream=None):
    """conv -> scan -> gated norm, as a layer calls them."""
    B, L, H, D = x.shape
    gdn.gdn_short_conv(gdn.make_conv_config(B, H, D, 4), x, w_conv, bufs["u"], stream=stream)
    gdn.gdn_gated_scan(gdn.make_scan_config(B, H, D, scale="sqrt"), bufs["u"], g, bufs["o"],
                       h0=h0, hT=bufs["hT"], hist=bufs["hist"], stream=stream)
    gdn.gdn_group_norm(gdn.make_norm_config(B, H, D, activation="silu"), bufs["o"], w_norm,
                       bufs["y"], z=z, stream=stream)


def layer_backward(x, w_conv, g, w_norm, z, dy, bufs, stream=None):
    B, L, H, D = x.shape
    gdn.gdn_group_norm_backward(gdn.make_norm_config(B, H, D, activation="silu"), bufs["o"], w_norm,
                                dy, bufs["do"], bufs["dw_norm"], z=z, dz=bufs["dz"], stream=stream)
    gdn.gdn_gated_scan_backward(gdn.make_scan_config(B, H, D, scale="sqrt"), bufs["u"], g,
                                bufs["hist"], bufs["do"], bufs["du"], bufs["dg"], stream=stream)
    gdn.gdn_short_conv_backward(gdn.make_conv_config(B, H, D, 4), x, w_conv, bufs["du"], bufs["dx"],
                                bufs["dw_conv"], stream=stream)


def layer_state(seed, B=2, L=150, H=2, D=64):
    r = torch.Generator(device="cuda")
    r.manual_seed(seed)

    def randn(*s):
        return torch.randn(s, generator=r, device="cuda")

    t = dict(x=randn(B, L, H, D).bfloat16(), w_conv=0.5 * randn(H * D, 4),
             g=-torch.nn.functional.softplus(randn(B, L, H, D)), w_norm=1 + 0.2 * randn(D),
             z=randn(B, L, H, D).bfloat16(), h0=randn(B, H, D), dy=randn(B, L, H, D).bfloat16())
    bufs = {n: torch.zeros_like(t["x"]) for n in ("u", "o", "y", "do", "du", "dx", "dz")}
    bufs.update(hT=torch.zeros_like(t["h0"]), dg=torch.zeros_like(t["g"]),
                hist=torch.zeros((B, -(-L // 64), H, D), device="cuda"),
                dw_norm=torch.zeros_like(t["w_norm"]), dw_conv=torch.zeros_like(t["w_conv"]))
    return t, bufs


def run_layer(t, bufs, stream=None):
    layer(t["x"], t["w_conv"], t["g"], t["w_norm"], t["z"], t["h0"], bufs, stream)
    layer_backward(t["x"], t["w_conv"], t["g"], t["w_norm"], t["z"], t["dy"], bufs, stream)


def test_a_layer_end_to_end():
    """conv -> scan -> gated norm and back, each stage against its 64-bit form on what the stage
    before it left."""
    t, bufs = layer_state(60)
    run_layer(t, bufs)
    c = {n: v.cpu() for n, v in {**t, **bufs}.items()}
    B, L, H, D = c["x"].shape
    zero = torch.zeros((B, 3, H * D))
    v, _, err = ref.conv(c["x"].view(B, L, -1), c["w_conv"], None, zero, "silu")
    close(c["u"].view(B, L, -1), v, err, torch.bfloat16, "u")
    o, hT, _, err, _, e_end = ref.scan(c["u"], c["g"], c["h0"], "sqrt")
    close(c["o"], o, err, torch.bfloat16, "o")
    close(c["hT"], hT, e_end, torch.float32, "hT")
    y, err = ref.norm(c["o"], c["w_norm"], None, c["z"], "silu", False, 1e-6)
    close(c["y"], y, err, torch.bfloat16, "y")
    dx, ex, dz, ez, tw, _ = ref.norm_backward(c["o"], c["w_norm"], None, c["z"], c["dy"], "silu",
                                              False, 1e-6)
    close(c["do"], dx, ex, torch.bfloat16, "do")
    close(c["dz"], dz, ez, torch.bfloat16, "dz")
    close(c["dw_norm"], *ref.summed(*tw, (0, 1, 2), B * L * H), torch.float32, "dw_norm")
    dx, dg, _, ex, eg, _ = ref.scan_backward(c["u"], c["g"], c["h0"], c["do"],
                                             torch.zeros((B, H, D)), "sqrt")
    close(c["du"], dx, ex, torch.bfloat16, "du")
    close(c["dg"], dg, eg, torch.float32, "dg")
    rx, rw, _, _ = ref.conv_backward(c["x"].view(B, L, -1), c["w_conv"], None, zero,
                                     c["du"].view(B, L, -1), zero, "silu")
    close(c["dx"].view(B, L, -1), *rx, torch.bfloat16, "dx")
    close(c["dw_conv"], *rw, torch.float32, "dw_conv")


def test_a_layer_is_the_same_on_another_stream_and_in_a_graph():
    """Eager, on a stream of its own (handed over and made current), captured and replayed twice:
    bit for bit the same."""
    t, want = layer_state(61)
    run_layer(t, want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for handed in (True, False):
        _, got = layer_state(61)
        torch.cuda.synchronize()
        if handed:
            run_layer(t, got, stream=side)
        else:
            with torch.cuda.stream(side):
                run_layer(t, got)
        side.synchronize()
        for n in want:
            assert torch.equal(got[n], want[n]), (handed, n)
    _, got = layer_state(61)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_layer(t, got)
    for _ in range(2):
        for n in got:
            got[n].fill_(MARK)
        graph.replay()
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(got[n], want[n]), n


def test_conv_norm_prefill_and_gated_norm():
    """The path of a GDN layer: q, k, v from slices of one projection through the convolution into
    the prefill's head-major arrays, unit queries and keys by the norm, the prefill, the gated norm
    of its head-major output; the recurrence against the oracle on what it was given."""
    import numpy as np

    import oracle
    from gdn_harness import O_TOL, rel_l2, round_act

    B, L, H, D = 2, 96, 2, 128
    r = torch.Generator(device="cuda")
    r.manual_seed(70)
    proj = torch.randn((B, L, 4, H, D), generator=r, device="cuda").bfloat16()
    cc = gdn.make_conv_config(B, H, D, 4)
    unit = gdn.make_norm_config(B, H, D, eps=1e-6 / D)
    heads = {}
    for i, n in enumerate("qkv"):
        w = 0.5 * torch.randn((H * D, 4), generator=r, device="cuda")
        out = torch.zeros((B, H, L, D), dtype=torch.bfloat16, device="cuda")
        gdn.gdn_short_conv(cc, proj[:, :, i], w, out.transpose(1, 2))
        if n != "v":
            normed = torch.zeros_like(out)
            gdn.gdn_group_norm(unit, out.transpose(1, 2), torch.full((D,), D ** -0.5, device="cuda"),
                               normed.transpose(1, 2))
            out = normed
        heads[n] = out
    assert float((heads["k"].float().norm(dim=-1) - 1).abs().max()) < 0.02
    g = -torch.nn.functional.softplus(torch.randn((B, H, L), generator=r, device="cuda"))
    beta = torch.sigmoid(torch.randn((B, H, L), generator=r, device="cuda"))
    o = torch.zeros_like(heads["q"])
    S = torch.zeros((B, H, D, D), device="cuda")
    gdn.gdn_prefill(gdn.make_config(B, H, D), heads["q"], heads["k"], heads["v"], g, beta, o, S)
    y = torch.zeros((B, L, H, D), dtype=torch.bfloat16, device="cuda")
    w = 1 + 0.2 * torch.randn((D,), generator=r, device="cuda")
    gdn.gdn_group_norm(gdn.make_norm_config(B, H, D, activation="silu"), o.transpose(1, 2), w, y,
                       z=proj[:, :, 3])

    def np64(t):  # [B][H][L](D) -> [L][B*H](D)
        return t.reshape(B * H, L, *t.shape[3:]).transpose(0, 1).double().cpu().numpy()

    o_ref, _ = oracle.plain_run(*(np64(t) for t in (heads["q"], heads["k"], heads["v"], g, beta)),
                                S0=np.zeros((B * H, D, D)))
    assert rel_l2(np64(o), round_act(o_ref, "bf16")) <= O_TOL
    want, err = ref.norm(o.transpose(1, 2).cpu(), w.cpu(), None, proj[:, :, 3].cpu(), "silu", False,
                         1e-6)
    close(y, want, err, torch.bfloat16)
