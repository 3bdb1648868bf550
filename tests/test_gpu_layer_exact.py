"""The operators around the recurrence on whole numbers, where sums are exact: a token, row or partial
sum that is left out or counted twice changes the result, however many there are."""
import math

import pytest
import torch

import bit_recurrent_state_gdn_b200 as gdn
import layer_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def whole(r, shape, most, dtype=torch.float32):
    return torch.randint(-most, most + 1, shape, generator=r, device="cuda").to(dtype)


def rng(seed):
    r = torch.Generator(device="cuda")
    r.manual_seed(seed)
    return r


def lens_for(B, L, kind):
    if kind is None:
        return None
    full = [(L, L - 1, L // 2, 0, 1, L // 3 + 1)[i % 6] for i in range(B)]
    return torch.tensor([max(0, v) for v in full], dtype=torch.int32, device="cuda")


def live(n, B, L):
    t = torch.arange(L, device="cuda")
    return (t < (torch.full((B,), L, device="cuda") if n is None else n)[:, None])[:, :, None, None]


SCAN = [
    (3, 1, 2, 20, "f32"), (5, 8, 1, 70, "bf16"), (40, 100, 16, 33, "f32"), (10, 200, 32, 64, "bf16"),
    (64, 100, 32, 64, "f32"), (15, 1100, 4, 64, "bf16"), (6, 700, 1, 96, "f32"), (1, 4095, 1, 64, "f32"),
    (2, 4097, 1, 72, "f32"), (1, 9001, 3, 17, "f32"), (7, 20000, 2, 64, "bf16"), (18, 140000, 1, 64, "f32"),
]


@pytest.mark.parametrize("ragged", [None, True])
@pytest.mark.parametrize("case", SCAN, ids=str)
def test_scan_sums(case, ragged):
    """Gates of 1, and of 0 at some tokens: the states are sums since the last of these."""
    B, L, H, D, dtype = case
    r, dt, n = rng(L), DT[dtype], lens_for(B, L, ragged)
    m = live(n, B, L)
    x, do = (torch.where(m, whole(r, (B, L, H, D), 1), 0.0) for _ in range(2))
    reset = torch.rand((B, L, 1, 1), generator=r, device="cuda") < 1 / 400
    g = torch.where(reset, -math.inf, 0.0).expand(B, L, H, D).contiguous()
    h0, dhT = (whole(r, (B, H, D), 5) for _ in range(2))
    cfg = gdn.make_scan_config(B, H, D, act=dtype)
    xs, o = x.to(dt), torch.zeros((B, L, H, D), dtype=dt, device="cuda")
    hT, hist = torch.zeros_like(h0), torch.zeros(gdn.gdn_scan_hist_shape(cfg, L), device="cuda")
    gdn.gdn_gated_scan(cfg, xs, g, o, h0=h0, hT=hT, hist=hist, lens=n)

    def sums(v, first, cut):  # s_t = sum of v since the last t' <= t with cut (and first before any)
        c = torch.cumsum(torch.cat([first[:, None], v], 1).double(), 1)
        at = torch.cummax(torch.where(cut, torch.arange(1, L + 1, device="cuda").view(1, L, 1, 1), 0), 1).values
        base = torch.cat([torch.zeros_like(c[:, :1]), c], 1)  # base[t] = sum before entry t
        return c[:, 1:] - torch.gather(base, 1, at.expand(B, L, H, D))

    cut = reset & m
    h = sums(x, h0, cut)
    keep = m.expand_as(h)
    assert torch.equal(o[keep], h.to(dt)[keep])
    end = h[:, -1] if L else h0.double()
    assert torch.equal(hT.double(), end)
    before = torch.cat([h0.double()[:, None], h[:, :-1]], 1)
    kept = before[:, ::64]
    there = live(n, B, L)[:, ::64].expand_as(kept)
    assert torch.equal(hist.double()[there], kept[there])

    dx, dg, dh0 = torch.zeros_like(o), torch.zeros_like(g), torch.zeros_like(h0)
    gdn.gdn_gated_scan_backward(cfg, xs, g, hist, do.to(dt), dx, dg, dhT=dhT, dh0=dh0, lens=n)
    # backward a token with a gate of 0 takes what is behind it, and hands nothing on: the cut is at the
    # token before it
    after = torch.cat([cut[:, 1:], torch.zeros_like(cut[:, :1])], 1)
    dh = sums(do.flip(1), dhT, after.flip(1)).flip(1)
    assert torch.equal(dx[keep], dh.to(dt)[keep])
    want = torch.where(cut, 0.0, before * dh)
    assert float(want.abs().max()) < 2 ** 24
    assert torch.equal(dg.double()[keep], want[keep])
    assert torch.equal(dh0.double(), torch.where(cut[:, 0], 0.0, dh[:, 0]))


NORM = [
    # B, L, H, D, dtype: every number of lanes, pieces and heads of a CTA, a CTA a row
    (4, 500, 3, 16, "bf16"), (60, 31, 8, 64, "bf16"), (3, 700, 6, 32, "f32"), (2, 900, 33, 8, "bf16"),
    (5, 203, 1, 128, "bf16"), (2, 129, 40, 512, "bf16"), (2, 300, 36, 256, "f32"), (1, 90, 7, 1024, "f32"),
    (3, 111, 2, 2048, "bf16"), (1, 8000, 1, 4, "f32"), (8, 1000, 1, 2, "bf16"), (1, 41, 300, 128, "bf16"),
]


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("weight", ["head", "channel"])
@pytest.mark.parametrize("ragged", [None, True])
@pytest.mark.parametrize("case", NORM, ids=str)
def test_norm_parameter_sums(case, ragged, weight, gate):
    """Rows of +-1, whose n is themselves, and whole gradients: grad_bias is exact, grad_w but for
    what 1 / sqrt(1 + eps) is off."""
    B, L, H, D, dtype = case
    r, dt, n = rng(D + L), DT[dtype], lens_for(B, L, ragged)
    s, p = (B, L, H, D), (D,) if weight == "head" else (H, D)
    m = live(n, B, L)
    x = torch.where(torch.rand(s, generator=r, device="cuda") < 0.5, -1.0, 1.0)
    k = torch.randint(1, 3, s, generator=r, device="cuda").float()
    z = torch.randint(1, 4, s, generator=r, device="cuda").float() if gate else None
    dy = x * k  # du n is then positive everywhere, so that nothing cancels
    cfg = gdn.make_norm_config(B, H, D, eps=1e-12, weight=weight, act=dtype)
    w, b = torch.ones(p, device="cuda"), torch.zeros(p, device="cuda")
    dw, db = torch.full_like(w, 777.0), torch.full_like(w, 777.0)
    dx = torch.zeros(s, dtype=dt, device="cuda")
    gdn.gdn_group_norm_backward(cfg, x.to(dt), w, dy.to(dt), dx, dw, b=b, db=db, lens=n,
                                z=z.to(dt) if gate else None, dz=torch.zeros_like(dx) if gate else None)
    du = torch.where(m, dy * (z if gate else 1.0), 0.0).double()
    dims = (0, 1, 2) if weight == "head" else (0, 1)
    assert torch.equal(db.double(), du.sum(dims))
    want = (du * x).sum(dims)
    # n is +-(1 + c), c up to 4 half steps from the root and 4 from the mean square: every term is off
    # by that. Where c is not 0 sums round too: a term goes through at most 30 additions in its lane
    # (8000 tokens on 296 CTAs), 128 over the rows of its CTA, 64 over the parts.
    bound = (8 + 30 + 128 + 64) * 2.0 ** -24 * want
    assert bool(((dw.double() - want).abs() <= bound).all())


CONV = [
    (2, 1, 2, 64, "bf16", 4), (300, 1, 3, 50, "f32", 3), (5, 2, 1, 33, "bf16", 4), (4, 33, 2, 7, "bf16", 2),
    (40, 70, 4, 128, "bf16", 4), (6, 301, 1, 26, "f32", 4), (1, 5000, 1, 64, "bf16", 3),
    (12, 900, 5, 24, "f32", 2), (2, 4097, 3, 20, "bf16", 4), (7, 260, 32, 64, "f32", 4),
]


@pytest.mark.parametrize("ragged", [None, True])
@pytest.mark.parametrize("case", CONV, ids=str)
def test_conv_sums(case, ragged):
    B, L, H, D, dtype, K = case
    r, dt, n, C = rng(L + K), DT[dtype], lens_for(B, L, ragged), H * D
    x, dy = (whole(r, (B, L, H, D), 3) for _ in range(2))
    w, b = whole(r, (C, K), 2), whole(r, (C,), 2)
    si, dso = (whole(r, (B, K - 1, C), 3) for _ in range(2))
    cfg = gdn.make_conv_config(B, H, D, K, activation="none", act=dtype)
    y, dx = (torch.zeros((B, L, H, D), dtype=dt, device="cuda") for _ in range(2))
    so, dsi = (torch.zeros((B, K - 1, C), dtype=dt, device="cuda") for _ in range(2))
    dw, db = torch.zeros_like(w), torch.zeros_like(b)
    gdn.gdn_short_conv(cfg, x.to(dt), w, y, bias=b, state_in=si.to(dt), state_out=so, lens=n)
    gdn.gdn_short_conv_backward(cfg, x.to(dt), w, dy.to(dt), dx, dw, bias=b, db=db, state_in=si.to(dt),
                                dstate_out=dso.to(dt), dstate_in=dsi, lens=n)
    c = [None if t is None else t.cpu() for t in (x.view(B, L, C), w, b, si, dy.view(B, L, C), dso, n)]
    m = live(n, B, L).expand(B, L, H, D).cpu()
    want, end, _ = ref.conv(*c[:4], "none", c[6])
    assert torch.equal(y.cpu()[m].double(), want.view(B, L, H, D)[m])  # whole numbers below 256
    assert torch.equal(so.cpu().double(), end)
    rx, rw, rb, rs = ref.conv_backward(*c[:6], "none", c[6])
    assert torch.equal(dx.cpu()[m].double(), rx[0].view(B, L, H, D)[m])
    assert torch.equal(dw.cpu().double(), rw[0]) and torch.equal(db.cpu().double(), rb[0])
    assert torch.equal(dsi.cpu().double(), rs[0])


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (33, "f32"), (50, "bf16")])
@pytest.mark.parametrize("L,lens", [(3, None), (70, None), (70, [70, 37]), (5000, None)])
def test_conv_gradient_of_what_is_not_finite(L, lens, D, dtype):
    """An infinite input meets the taps that it has in its own sequence, no others: the last token of a
    sequence only the last tap, at any place in the middle every tap."""
    B, K, dt = 2, 4, DT[dtype]
    r = rng(L)
    x, dy = (torch.randint(1, 4, (B, L, 1, D), generator=r, device="cuda").to(dt) for _ in range(2))
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    w = whole(r, (D, K), 2)
    cfg = gdn.make_conv_config(B, 1, D, K, activation="none", act=dtype)
    ends = [L] * B if lens is None else lens
    want = torch.zeros((D, K), dtype=torch.float64, device="cuda")
    x[0, ends[0] - 1, 0, 1] = x[1, ends[1] - 1, 0, 2] = math.inf
    if L > 64:
        for t in range(28, 37):  # around the ends of runs
            x[0, t, 0, t - 20] = math.inf
    for b, e in enumerate(ends):
        xs, ds = x[b, :e, 0].double(), dy[b, :e, 0].double()
        for j in range(K):
            want[:, j] += (xs[:e - (K - 1 - j)] * ds[K - 1 - j:]).sum(0) if e > K - 1 - j else 0.0
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    gdn.gdn_short_conv_backward(cfg, x, w, dy, dx, dw, lens=n)
    assert torch.equal(dw.double(), want)
