"""Lengths beyond the C entry points' 32-bit token count are refused by the Python layer, not taken
modulo 2^32."""
import pytest
import torch

import bit_recurrent_state_gdn_b200 as gdn
from bit_recurrent_state_gdn_b200 import build

LENGTHS = [(1 << 30) + 1, 1 << 31, (1 << 32) + 1]


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


@pytest.mark.parametrize("L", LENGTHS)
def test_calls(L):
    x = torch.zeros((1, 1, 1, 4)).expand(1, L, 1, 4)
    w, k, d = torch.zeros(4), torch.zeros((4, 4)), torch.zeros((1, 1, 4))
    scan, norm, conv = (gdn.make_scan_config(1, 1, 4, act="f32"), gdn.make_norm_config(1, 1, 4, act="f32"),
                        gdn.make_conv_config(1, 1, 4, 4, act="f32"))
    for call in (lambda: gdn.gdn_gated_scan(scan, x, x, x), lambda: gdn.gdn_group_norm(norm, x, w, x),
                 lambda: gdn.gdn_gated_scan_backward(scan, x, x, d, x, x, x),
                 lambda: gdn.gdn_group_norm_backward(norm, x, w, x, x, w),
                 lambda: gdn.gdn_short_conv(conv, x, k, x),
                 lambda: gdn.gdn_short_conv_backward(conv, x, k, x, x, k)):
        with pytest.raises(ValueError, match="tokens"):
            call()


@pytest.mark.parametrize("L", LENGTHS + [-1, -(1 << 32) + 5000])
def test_workspaces_of_what_is_refused_are_empty(L):
    assert gdn.gdn_gated_scan_workspace_bytes(gdn.make_scan_config(1, 1, 64), L) == 0
    assert gdn.gdn_group_norm_backward_workspace_bytes(gdn.make_norm_config(1, 1, 64), L) == 0
    assert gdn.gdn_short_conv_backward_workspace_bytes(gdn.make_conv_config(1, 1, 64), L) == 0
