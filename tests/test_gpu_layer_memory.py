"""What the operators around the recurrence read and write: states in place, arrays in one
buffer, nothing outside of an output or of a workspace of the size that is asked for."""
import pytest
import torch

import bit_recurrent_state_gdn_b200 as gdn
import layer_ref as ref
from layer_ref import close

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.mark.parametrize("B,L,D,lens", [
    (40, 8, 70, None),                 # one warp a sequence
    (200, 130, 128, None),             # one CTA a unit
    (3, 1500, 100, [1500, 0, 640]),    # clusters
    (2, 9000, 96, [9000, 4097]),       # spans
    (3, 20000, 33, [0, 20000, 1]),
])
def test_scan_state_gradient_in_place(B, L, D, lens):
    """grad_h0 may be grad_hT, however the sequences are shared out."""
    r = torch.Generator(device="cuda")
    r.manual_seed(L)

    def randn(*s):
        return torch.randn(s, generator=r, device="cuda")

    cfg = gdn.make_scan_config(B, 1, D, scale="sqrt", act="f32")
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    x, do, g = randn(B, L, 1, D), randn(B, L, 1, D), -0.001 * torch.rand((B, L, 1, D), generator=r, device="cuda")
    dhT = randn(B, 1, D)
    hist = torch.zeros(gdn.gdn_scan_hist_shape(cfg, L), device="cuda")
    gdn.gdn_gated_scan(cfg, x, g, torch.zeros_like(x), hist=hist, lens=n)
    runs = []
    for dh0 in (torch.zeros_like(dhT), dhT.clone()):
        dx, dg = torch.zeros_like(x), torch.zeros_like(g)
        gdn.gdn_gated_scan_backward(cfg, x, g, hist, do, dx, dg, lens=n, dh0=dh0,
                                    dhT=dhT if len(runs) == 0 else dh0)
        runs.append((dx, dg, dh0))
    for apart, same in zip(*runs):
        assert torch.equal(apart, same)
    for b in range(B):
        if lens and lens[b] == 0:
            assert torch.equal(runs[1][2][b], dhT[b])


def test_inputs_and_outputs_in_one_buffer():
    """Slices of one buffer's rows, states and parameters side by side: nothing is shared, so nothing
    is refused, and the results are those of arrays of their own."""
    B, L, H, D, K = 2, 70, 2, 64, 4
    C = H * D
    r = torch.Generator(device="cuda")
    r.manual_seed(5)
    rows = torch.randn((B, L, 6, H, D), generator=r, device="cuda").bfloat16()
    apart = rows.clone()
    flat = torch.randn((8 * C + 2 * B * C,), generator=r, device="cuda")
    w_conv, bias = flat[:4 * C].view(C, K), flat[4 * C:5 * C]
    w_norm, dw = flat[5 * C:5 * C + D], flat[5 * C + D:5 * C + 2 * D]
    h0, hT = flat[8 * C:8 * C + B * C].view(B, H, D), flat[8 * C + B * C:].view(B, H, D)
    g = -torch.rand((B, L, H, D), generator=r, device="cuda")
    conv, scan = gdn.make_conv_config(B, H, D, K), gdn.make_scan_config(B, H, D, scale="sqrt")
    norm = gdn.make_norm_config(B, H, D, activation="silu")

    def run(x, u, o, z, y, dx):
        gdn.gdn_short_conv(conv, x, w_conv, u, bias=bias)
        gdn.gdn_gated_scan(scan, u, g, o, h0=h0, hT=hT)
        gdn.gdn_group_norm(norm, o, w_norm, y, z=z)
        gdn.gdn_group_norm_backward(norm, o, w_norm, y, dx, dw, z=z, dz=torch.empty_like(z))
        return [t.clone() for t in (u, o, y, dx, hT, dw)]

    want = run(apart[:, :, 0].clone(), *(torch.empty_like(g, dtype=torch.bfloat16) for _ in range(2)),
               apart[:, :, 3].clone(), *(torch.empty_like(g, dtype=torch.bfloat16) for _ in range(2)))
    for a, b in zip(run(*(rows[:, :, i] for i in range(6))), want):
        assert torch.equal(a, b)
    assert torch.equal(rows[:, :, 0], apart[:, :, 0]) and torch.equal(rows[:, :, 3], apart[:, :, 3])


@pytest.mark.parametrize("B,L,H", [(2, 5, 0), (0, 5, 3), (2, 0, 3)])
def test_norm_gradients_of_an_empty_batch(B, L, H):
    """Weights that the heads share have a gradient of zero where there is no head, as where there is no
    sequence or token."""
    cfg = gdn.make_norm_config(B, H, 8, act="f32")
    e, w = torch.zeros((B, L, H, 8), device="cuda"), torch.ones(8, device="cuda")
    dw, db = torch.full_like(w, 777.0), torch.full_like(w, 777.0)
    gdn.gdn_group_norm_backward(cfg, e, w, e.clone(), e.clone(), dw, b=w.clone(), db=db)
    assert float(dw.abs().max()) == 0.0 and float(db.abs().max()) == 0.0
    per_channel = gdn.make_norm_config(B, H, 8, weight="channel", act="f32")
    w, dw = (torch.full((H, 8), 777.0, device="cuda") for _ in range(2))
    gdn.gdn_group_norm_backward(per_channel, e, w, e.clone(), e.clone(), dw)
    assert float(dw.abs().sum()) == 0.0


MARK = 777.0


class Guarded:
    """A token array or a dense one inside a larger buffer of marks; clean() says whether everything
    outside of it still holds them."""

    def __init__(self, shape, dtype, how="dense"):
        n = 1
        for s in shape:
            n *= s
        pad = 1024  # 16 bytes of any type divide it
        if how == "dense" or how == "tokens":
            self.buf = torch.full((n + 2 * pad,), MARK, dtype=dtype, device="cuda")
            self.view = self.buf[pad:pad + n].view(shape)
        else:
            B, L, H, D = shape
            if how == "heads":
                self.buf = torch.full((n + 2 * pad,), MARK, dtype=dtype, device="cuda")
                self.view = self.buf[pad:pad + n].view(B, H, L, D).transpose(1, 2)
            elif how == "wide":
                self.buf = torch.full((2 * n + 2 * pad,), MARK, dtype=dtype, device="cuda")
                self.view = self.buf[pad:pad + 2 * n].view(B, L, 2 * H * D)[..., H * D:].unflatten(-1, (H, D))
            else:  # "odd"
                m = B * L * (H * D + 1)
                self.buf = torch.full((m + 2 * pad + 1,), MARK, dtype=dtype, device="cuda")
                self.view = self.buf[pad + 1:pad + 1 + m].view(B, L, H * D + 1)[..., :H * D].unflatten(-1, (H, D))

    def clean(self):
        kept = self.view.clone()
        self.view.fill_(MARK)
        ok = bool((self.buf == MARK).all())
        self.view.copy_(kept)
        return ok


class GuardedBytes:
    """A workspace of exactly n bytes with marked ones behind it."""

    def __init__(self, n):
        self.n, self.buf = n, torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")

    def get(self):
        return self.buf[:self.n] if self.n else None

    def clean(self):
        return bool((self.buf[self.n:] == 0xA5).all())


def clean(**arrays):
    torch.cuda.synchronize()
    for name, a in arrays.items():
        assert a is None or a.clean(), name


def lens_for(B, L, ragged):
    return torch.tensor([(L, L // 2, 0, 1)[i % 4] for i in range(B)], dtype=torch.int32,
                        device="cuda") if ragged else None


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("how", ["tokens", "heads", "wide", "odd"])
@pytest.mark.parametrize("B,L,H,D,dtype", [
    (3, 1, 2, 20, "bf16"), (5, 8, 1, 64, "f32"), (40, 100, 16, 33, "bf16"), (10, 200, 32, 64, "bf16"),
    (2, 1030, 2, 40, "f32"), (4, 700, 1, 96, "bf16"), (2, 4100, 1, 72, "bf16"), (1, 9001, 3, 17, "f32"),
])
def test_scan_stays_inside(B, L, H, D, dtype, how, ragged):
    r = torch.Generator(device="cuda")
    r.manual_seed(1)
    dt, n = DT[dtype], lens_for(B, L, ragged)
    cfg = gdn.make_scan_config(B, H, D, scale="complement", act=dtype)
    need = gdn.gdn_gated_scan_workspace_bytes(cfg, L)

    def filled(dtype, how="dense", shape=(B, L, H, D)):
        a = Guarded(shape, dtype, how)
        a.view.copy_(-torch.rand(shape, generator=r, device="cuda"))
        return a

    x, g, do = filled(dt, how), filled(torch.float32, how), filled(dt, how)
    o, hT, h0 = Guarded((B, L, H, D), dt, how), Guarded((B, H, D), torch.float32), filled(torch.float32, shape=(B, H, D))
    hist, ws = Guarded(gdn.gdn_scan_hist_shape(cfg, L), torch.float32), GuardedBytes(need)
    gdn.gdn_gated_scan(cfg, x.view, g.view, o.view, h0=h0.view, hT=hT.view, hist=hist.view, lens=n,
                       workspace=ws.get())
    clean(x=x, g=g, h0=h0, o=o, hT=hT, hist=hist, workspace=ws)
    dx, dg, dh0 = Guarded((B, L, H, D), dt, how), Guarded((B, L, H, D), torch.float32, how), Guarded((B, H, D), torch.float32)
    ws = GuardedBytes(need)
    gdn.gdn_gated_scan_backward(cfg, x.view, g.view, hist.view, do.view, dx.view, dg.view, dhT=h0.view,
                                dh0=dh0.view, lens=n, workspace=ws.get())
    clean(x=x, g=g, do=do, dx=dx, dg=dg, dh0=dh0, workspace=ws)


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("weight", ["head", "channel"])
@pytest.mark.parametrize("B,L,H,D,dtype,how", [
    (2, 9, 5, 36, "bf16", "wide"), (2, 50, 33, 8, "bf16", "tokens"), (3, 40, 6, 7, "bf16", "odd"),
    (8, 300, 32, 128, "bf16", "heads"), (1, 900, 2, 64, "f32", "tokens"), (2, 20, 9, 2, "f32", "heads"),
    # more than eight channels a lane: one CTA per SM, of few and of many heads
    (2, 300, 36, 512, "bf16", "tokens"), (2, 300, 40, 300, "bf16", "wide"), (1, 200, 60, 500, "f32", "heads"),
    (1, 100, 100, 260, "f32", "tokens"), (1, 64, 149, 1024, "bf16", "tokens"), (1, 7, 300, 333, "bf16", "odd"),
    (1, 5, 593, 264, "bf16", "tokens"),
    # a CTA a row
    (2, 33, 3, 1025, "bf16", "odd"), (1, 90, 40, 2048, "bf16", "tokens"), (1, 3, 1, 8192, "f32", "tokens"),
])
def test_norm_stays_inside(B, L, H, D, dtype, how, weight, ragged):
    r = torch.Generator(device="cuda")
    r.manual_seed(2)
    dt, n, s = DT[dtype], lens_for(B, L, ragged), (B, L, H, D)
    cfg = gdn.make_norm_config(B, H, D, center=True, activation="silu", weight=weight, act=dtype)
    p = (D,) if weight == "head" else (H, D)

    def filled(dtype, how="dense", shape=s):
        a = Guarded(shape, dtype, how)
        a.view.copy_(torch.randn(shape, generator=r, device="cuda"))
        return a

    x, z, dy = filled(dt, how), filled(dt, how), filled(dt, how)
    w, b = filled(torch.float32, shape=p), filled(torch.float32, shape=p)
    y, dx, dz = (Guarded(s, dt, how) for _ in range(3))
    dw, db = (Guarded(p, torch.float32) for _ in range(2))
    gdn.gdn_group_norm(cfg, x.view, w.view, y.view, b=b.view, z=z.view, lens=n)
    clean(x=x, z=z, w=w, b=b, y=y)
    for gated in (True, False):
        ws = GuardedBytes(gdn.gdn_group_norm_backward_workspace_bytes(cfg, L))
        gdn.gdn_group_norm_backward(cfg, x.view, w.view, dy.view, dx.view, dw.view, b=b.view,
                                    z=z.view if gated else None, dz=dz.view if gated else None,
                                    db=db.view, lens=n, workspace=ws.get())
        clean(x=x, z=z, dy=dy, dx=dx, dz=dz, dw=dw, db=db, workspace=ws)


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("how", ["tokens", "heads", "wide", "odd"])
@pytest.mark.parametrize("B,L,H,D,dtype,K", [
    (3, 1, 2, 20, "bf16", 4), (700, 1, 3, 50, "f32", 3), (5, 2, 1, 33, "bf16", 4), (4, 33, 2, 7, "bf16", 2),
    (40, 70, 4, 128, "bf16", 4), (2, 300, 1, 26, "f32", 4), (1, 5000, 1, 64, "bf16", 3), (3, 900, 5, 24, "f32", 2),
])
def test_conv_stays_inside(B, L, H, D, dtype, K, how, ragged):
    r = torch.Generator(device="cuda")
    r.manual_seed(3)
    dt, n, s, C = DT[dtype], lens_for(B, L, ragged), (B, L, H, D), H * D
    cfg = gdn.make_conv_config(B, H, D, K, act=dtype)

    def filled(dtype, how="dense", shape=s):
        a = Guarded(shape, dtype, how)
        a.view.copy_(torch.randn(shape, generator=r, device="cuda"))
        return a

    x, dy, w, b = filled(dt, how), filled(dt, how), filled(torch.float32, shape=(C, K)), filled(torch.float32, shape=(C,))
    si, dso = filled(dt, shape=(B, K - 1, C)), filled(dt, shape=(B, K - 1, C))
    y, so, dx, dsi = Guarded(s, dt, how), Guarded((B, K - 1, C), dt), Guarded(s, dt, how), Guarded((B, K - 1, C), dt)
    dw, db = Guarded((C, K), torch.float32), Guarded((C,), torch.float32)
    gdn.gdn_short_conv(cfg, x.view, w.view, y.view, bias=b.view, state_in=si.view, state_out=so.view, lens=n)
    clean(x=x, w=w, b=b, state_in=si, y=y, state_out=so)
    ws = GuardedBytes(gdn.gdn_short_conv_backward_workspace_bytes(cfg, L))
    gdn.gdn_short_conv_backward(cfg, x.view, w.view, dy.view, dx.view, dw.view, bias=b.view, db=db.view,
                                state_in=si.view, dstate_out=dso.view, dstate_in=dsi.view, lens=n,
                                workspace=ws.get())
    clean(x=x, dy=dy, state_in=si, dstate_out=dso, dx=dx, dstate_in=dsi, dw=dw, db=db, workspace=ws)
