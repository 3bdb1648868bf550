"""The gated scan with gates above 1, on sequences that are split into spans and on ones that are
not: what the entry points take as long as the gates of no stretch of up to 1024 tokens sum to 88 or
more, however much all of a sequence's gates together grow."""
import pytest
import torch

import bit_recurrent_state_gdn_b200 as gdn
import layer_ref as ref
from layer_ref import close

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
GROWTH = 0.08  # 1024 tokens sum to 82
WINDOW = 300


def windows_of(n):
    """First tokens of the stretches of a sequence of n that hold anything: its beginning, its end,
    and some in between that lie over borders of every kind."""
    at = [0, n // 3, n // 2 + 77, n - WINDOW]
    return [p for i, p in enumerate(at) if i == 0 or p >= at[i - 1] + WINDOW + 1]


def grown(B, L, H, D, dtype, lens, seed):
    """Inputs that are zero outside of windows, each of which begins (but for the first) and ends
    with a gate of -inf; between windows every gate is above 1, so that states and gradients are
    zero there and the product of the gates is beyond any number."""
    r = torch.Generator()
    r.manual_seed(seed)
    x = torch.zeros((B, L, H, D), dtype=DT[dtype], device="cuda")
    do = torch.zeros_like(x)
    g = torch.full((B, L, H, D), GROWTH, device="cuda")
    parts = []
    for b, n in enumerate(ref.lens_of(lens, B, L)):
        for p in windows_of(n) if n > 2 * WINDOW else ([0] if n else []):
            q = min(p + WINDOW, n)
            s = (1, q - p, H, D)
            wx, wdo = (torch.randn(s, generator=r).to(DT[dtype]) for _ in range(2))
            wg = torch.rand(s, generator=r) * 0.6 - 0.5
            if p:
                wg[:, 0] = -torch.inf
            x[b, p:q], do[b, p:q], g[b, p:q] = wx[0].cuda(), wdo[0].cuda(), wg[0].cuda()
            if q < n:
                g[b, q] = -torch.inf
            parts.append((b, p, q, q == n, wx, wg, wdo))
        x[b, n:] = do[b, n:] = g[b, n:] = torch.nan
    h0, dhT = (torch.randn((B, H, D), generator=r) for _ in range(2))
    return x, g, do, h0, dhT, parts


CASES = [
    # B, L, H, D, dtype, scale, lens
    (1, 4000, 1, 64, "bf16", "none", None),                  # not split: clusters
    (1, 6000, 1, 64, "bf16", "none", None),                  # spans of 128 tokens
    (2, 20000, 1, 70, "f32", "complement", [20000, 9001]),
    (3, 20000, 1, 33, "bf16", "none", [0, 299, 19997]),      # single channels
    (18, 40000, 1, 64, "bf16", "complement", None),          # spans of 2560 tokens
    (17, 70001, 1, 64, "bf16", "none", [70001, 33000, 1] + [70000] * 14),
    (18, 140000, 1, 64, "bf16", "none", None),               # a warp takes more than 1024 tokens
]


def check_windows(got, wants, parts, n, dtype, where):
    """The windows within their bounds, zero everywhere else before a sequence's end."""
    for b, p, q, want, bound in wants:
        close(got[b:b + 1, p:q], want, bound, dtype, (where, b, p))
        got[b, p:q] = 0
    for b, end in enumerate(n):
        bad = got[b, :end] != 0
        assert not bool(bad.any()), (where, b, int(bad.sum()), int(bad.flatten(1).any(1).nonzero()[0]))


@pytest.mark.parametrize("case", CASES, ids=[str(c[:6]) for c in CASES])
def test_growth_over_nothing(case):
    B, L, H, D, dtype, scale, lens = case
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    ends = ref.lens_of(n, B, L)
    x, g, do, h0, dhT, parts = grown(B, L, H, D, dtype, n, 100 + L)
    cfg = gdn.make_scan_config(B, H, D, scale=scale, act=dtype)
    dev = None if n is None else n.cuda()
    o, hT = torch.zeros_like(x), torch.zeros((B, H, D), device="cuda")
    hist = torch.zeros(gdn.gdn_scan_hist_shape(cfg, L), device="cuda")
    gdn.gdn_gated_scan(cfg, x, g, o, h0=h0.cuda(), hT=hT, hist=hist, lens=dev)
    wants, last = [], {}
    for b, p, q, end, wx, wg, _ in parts:
        want, at, _, err, _, e_at = ref.scan(wx, wg, h0[b:b + 1] if p == 0 else torch.zeros((1, H, D)), scale)
        wants.append((b, p, q, want, err))
        if end:
            last[b] = (at, e_at)
    check_windows(o, wants, parts, ends, DT[dtype], "o")
    for b in range(B):
        at, e_at = last.get(b, (h0[b:b + 1].double(), torch.zeros((1, H, D))))
        close(hT[b:b + 1], at, e_at, torch.float32, ("hT", b))

    dx, dg = torch.zeros_like(x), torch.zeros_like(g)
    dh0 = torch.zeros((B, H, D), device="cuda")
    gdn.gdn_gated_scan_backward(cfg, x, g, hist, do, dx, dg, dhT=dhT.cuda(), dh0=dh0, lens=dev)
    in_x, in_g, first = [], [], {}
    for b, p, q, end, wx, wg, wdo in parts:
        w = ref.scan_backward(wx, wg, h0[b:b + 1] if p == 0 else torch.zeros((1, H, D)), wdo,
                              dhT[b:b + 1] if end else torch.zeros((1, H, D)), scale)
        in_x.append((b, p, q, w[0], w[3].abs()))  # the factor 1 - a is negative for a > 1
        in_g.append((b, p, q, w[1], w[4]))
        if p == 0:
            first[b] = (w[2], w[5])
    check_windows(dx, in_x, parts, ends, DT[dtype], "dx")
    check_windows(dg, in_g, parts, ends, torch.float32, "dg")
    for b in range(B):
        at, e_at = first.get(b, (dhT[b:b + 1].double(), torch.zeros((1, H, D))))
        close(dh0[b:b + 1], at, e_at, torch.float32, ("dh0", b))


@pytest.mark.parametrize("L", [4000, 5000])
@pytest.mark.parametrize("scale", ["none", "complement"])
def test_growth_and_decay_in_turn(L, scale):
    """Stretches of 500 tokens that grow by e^10 and fade by e^10, on both sides of the split."""
    B, H, D = 2, 1, 48
    r = torch.Generator()
    r.manual_seed(7)
    x, do = (torch.randn((B, L, H, D), generator=r) for _ in range(2))
    sign = 1.0 - 2.0 * (torch.arange(L) // 500 % 2)
    g = (sign.view(1, L, 1, 1) * 0.02 + 0.01 * torch.randn((B, L, H, D), generator=r)).float()
    h0, dhT = (torch.randn((B, H, D), generator=r) for _ in range(2))
    cfg = gdn.make_scan_config(B, H, D, scale=scale, act="f32")
    o, hT = torch.zeros_like(x, device="cuda"), torch.zeros((B, H, D), device="cuda")
    hist = torch.zeros(gdn.gdn_scan_hist_shape(cfg, L), device="cuda")
    gdn.gdn_gated_scan(cfg, x.cuda(), g.cuda(), o, h0=h0.cuda(), hT=hT, hist=hist)
    dx, dg, dh0 = torch.zeros_like(o), torch.zeros_like(o), torch.zeros_like(hT)
    gdn.gdn_gated_scan_backward(cfg, x.cuda(), g.cuda(), hist, do.cuda(), dx, dg, dhT=dhT.cuda(),
                                dh0=dh0)

    want, end, _, err, _, e_end = ref.scan(x, g, h0, scale)
    close(o, want, err, torch.float32, "o")
    close(hT, end, e_end, torch.float32, "hT")
    wx, wg, w0, ex, eg, e0 = ref.scan_backward(x, g, h0, do, dhT, scale)
    close(dx, wx, ex.abs(), torch.float32, "dx")
    close(dg, wg, eg, torch.float32, "dg")
    close(dh0, w0, e0, torch.float32, "dh0")
