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
