"""What the operators around the recurrence read and write: states in place, nothing outside of an
output or a workspace, every partial sum counted once."""
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
