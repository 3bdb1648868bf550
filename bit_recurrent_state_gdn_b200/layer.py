"""Argument marshalling for the operators around the recurrence (include/gdnq_layer.h): torch
tensors -> pointers and strides, status codes -> exceptions. Same conventions as ``api``, and:

  - token arrays are [B][L][H][D] tensors with any strides whose last one is 1 (a transposed view
    of [B][H][L][D], a slice of wider rows); every other tensor is contiguous;
  - all tensors of a call are on one CUDA device, which need not be the current one; the call runs
    on that device's current stream (or ``stream``);
  - a workspace left out is allocated here, on the stream that the call runs on.
"""
from __future__ import annotations

import struct
from ctypes import byref, sizeof
from typing import Optional

import torch

from . import _abi
from .api import _DT, _TORCH_DT, GdnError

_SCALE = {"none": _abi.GDN_SCALE_NONE, "complement": _abi.GDN_SCALE_COMPLEMENT,
          "sqrt": _abi.GDN_SCALE_SQRT}
_ACTIVATION = {"none": _abi.GDN_ACT_NONE, "silu": _abi.GDN_ACT_SILU,
               "sigmoid": _abi.GDN_ACT_SIGMOID}
_WEIGHT = {"head": _abi.GDN_WEIGHT_HEAD, "channel": _abi.GDN_WEIGHT_CHANNEL}


def make_scan_config(B: int, H: int, D: int, scale: str = "none",
                     act: str = "bf16") -> _abi.gdn_scan_config:
    """scale: "none", "complement" (1 - a) or "sqrt" (sqrt(1 - a^2)), the factor of the input."""
    return _abi.gdn_scan_config(B, H, D, _SCALE[scale], _DT[act])


def make_norm_config(B: int, H: int, D: int, eps: float = 1e-6, center: bool = False,
                     activation: str = "none", weight: str = "head",
                     act: str = "bf16") -> _abi.gdn_norm_config:
    """center: take the mean off (group norm) or not (RMS norm). activation: "none", "silu" or
    "sigmoid", of the gate z where there is one, else of the normed values. weight: "head" ([D],
    shared) or "channel" ([H][D])."""
    return _abi.gdn_norm_config(B, H, D, int(center), _ACTIVATION[activation], _WEIGHT[weight],
                                _DT[act], eps)


def make_conv_config(B: int, H: int, D: int, K: int = 4, activation: str = "silu",
                     act: str = "bf16") -> _abi.gdn_conv_config:
    return _abi.gdn_conv_config(B, H, D, K, _ACTIVATION[activation], _DT[act])


def gdn_scan_hist_shape(cfg: _abi.gdn_scan_config, L: int) -> tuple:
    """Shape of the fp32 states that a forward scan of L tokens keeps for its backward pass."""
    return (cfg.B, -(-L // _abi.GDN_SCAN_CHUNK), cfg.H, cfg.D)


# The most tokens that the C entry points take: a longer count would reach them modulo 2^32.
_MAX_TOKENS = 1 << 30


def _shape(cfg, x: torch.Tensor):
    if x.dim() != 4:
        raise ValueError(f"x has {x.dim()} dimensions, expected [B][L][H][D]")
    if x.shape[1] > _MAX_TOKENS:
        raise ValueError(f"x has {x.shape[1]} tokens, at most 2^30 are taken")
    return (cfg.B, x.shape[1], cfg.H, cfg.D)


# A gdn_tokens as the bytes of its fields, which cost a third of a ctypes structure to make: the
# small calls of a decode step are bound by this layer.
_tokens_bytes = struct.Struct("@Pqqq").pack
assert struct.calcsize("@Pqqq") == sizeof(_abi.gdn_tokens)


# The current stream's handle without the object around it (3.2 us of a call, on the machine the
# decode step runs on; 0.1 us so); the public way where torch has no such function.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda index: torch.cuda.current_stream(index).cuda_stream)


class _Args:
    """Checks the tensors of one call: all on the device of the first."""

    __slots__ = ("shape", "index", "device", "channels")

    def __init__(self, cfg, x):
        self.shape = _shape(cfg, x)
        self.channels = cfg.D
        self.index = x.get_device()  # -1: not on a GPU
        self.device = x.device if self.index < 0 else None

    def on_device(self, t, name):
        if t.get_device() != self.index or (self.index < 0 and t.device != self.device):
            raise ValueError(f"{name} is on {t.device}, expected "
                             f"{self.device or torch.device('cuda', self.index)}")

    def tokens(self, t: Optional[torch.Tensor], name: str, dtype):
        if t is None:
            return None
        if t.shape != self.shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {self.shape}")
        if t.dtype is not dtype:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
        sb, sl, sh, sd = t.stride()
        if sd != 1 and self.channels > 1:
            raise ValueError(f"{name} must have contiguous channels")
        if t.get_device() != self.index or self.index < 0:
            self.on_device(t, name)
        return _tokens_bytes(t.data_ptr(), sb, sl, sh)

    def dense(self, t: Optional[torch.Tensor], name: str, dtype, numel: int):
        if t is None:
            return None
        if t.dtype is not dtype:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
        if t.numel() != numel:
            raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.get_device() != self.index or self.index < 0:
            self.on_device(t, name)
        return t.data_ptr() or None

    def lens(self, t):
        return None if t is None else self.dense(t, "lens", torch.int32, self.shape[0])

    def call(self, where: str, cfg, args, stream, workspace=None, need=None):
        """The C entry point ``where`` on cfg, L and args, the workspace (of ``need(cfg, L)`` bytes,
        in calls that have one) and the stream, with the tensors' device current."""
        if self.index < 0:
            raise ValueError(f"{where}: the tensors are on {self.device}, expected a CUDA device")
        if self.index != torch.cuda.current_device():
            with torch.cuda.device(self.index):
                return self.call(where, cfg, args, stream, workspace, need)
        if stream is None:
            handle = _current_stream(self.index)
        else:
            handle = stream if isinstance(stream, int) else stream.cuda_stream
        if need is not None:
            n = 0
            if workspace is None:
                n = need(cfg, self.shape[1])
            if n:
                on = None  # the current stream, which torch allocates for
                if stream is not None:
                    on = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
                with torch.cuda.stream(on):
                    workspace = torch.empty(n, dtype=torch.uint8, device="cuda")
            if workspace is None:
                args += (None, 0)
            else:
                self.on_device(workspace, "workspace")
                if not workspace.is_contiguous():
                    raise ValueError("workspace must be contiguous")
                args += (workspace.data_ptr() or None,
                         workspace.numel() * workspace.element_size())
        status = getattr(_abi.load(), where)(byref(cfg), self.shape[1], *args, handle)
        if status:
            raise GdnError(status, where)


def _bytes(which: str, cfg, L: int) -> int:
    return int(getattr(_abi.load(), which)(byref(cfg), L)) if 0 <= L <= _MAX_TOKENS else 0


def gdn_gated_scan_workspace_bytes(cfg, L: int) -> int:
    return _bytes("gdn_gated_scan_workspace_bytes", cfg, L)


def _scan_workspace(cfg, L: int) -> int:
    # a decode step does not pay for the question
    return 0 if L < _abi.GDN_SCAN_SPLIT else gdn_gated_scan_workspace_bytes(cfg, L)


def gdn_gated_scan(cfg, x, g, o, h0=None, hT=None, hist=None, lens=None, workspace=None,
                   stream=None):
    """x, o act [B][L][H][D]; g fp32 [B][L][H][D], the log of the gate; h0, hT fp32 [B][H][D] (may
    be the same);
    hist fp32 of gdn_scan_hist_shape(cfg, L), for the backward pass; lens int32 [B]. workspace: at
    least gdn_gated_scan_workspace_bytes(cfg, L) bytes on the device, made here when None."""
    a, act = _Args(cfg, x), _TORCH_DT[cfg.act_dtype]
    n = cfg.B * cfg.H * cfg.D
    f32, L = torch.float32, a.shape[1]
    a.call("gdn_gated_scan", cfg, (
        a.tokens(x, "x", act), a.tokens(g, "g", f32), a.tokens(o, "o", act),
        a.dense(h0, "h0", f32, n), a.dense(hT, "hT", f32, n),
        a.dense(hist, "hist", f32, n * -(-L // _abi.GDN_SCAN_CHUNK)), a.lens(lens)), stream,
        workspace, _scan_workspace)


def gdn_gated_scan_backward(cfg, x, g, hist, do, dx, dg, dhT=None, dh0=None, lens=None,
                            workspace=None, stream=None):
    """x, g, lens of the forward call and the hist that it wrote; do, dx act [B][L][H][D]; dg fp32
    [B][L][H][D]; dhT, dh0 fp32 [B][H][D] (may be the same); workspace as in the forward call."""
    a, act = _Args(cfg, x), _TORCH_DT[cfg.act_dtype]
    n = cfg.B * cfg.H * cfg.D
    f32, L = torch.float32, a.shape[1]
    a.call("gdn_gated_scan_backward", cfg, (
        a.tokens(x, "x", act), a.tokens(g, "g", f32),
        a.dense(hist, "hist", f32, n * -(-L // _abi.GDN_SCAN_CHUNK)), a.tokens(do, "do", act),
        a.dense(dhT, "dhT", f32, n), a.tokens(dx, "dx", act), a.tokens(dg, "dg", f32),
        a.dense(dh0, "dh0", f32, n), a.lens(lens)), stream, workspace, _scan_workspace)


def _norm_params(cfg) -> int:
    return cfg.D * (cfg.H if cfg.weight == _abi.GDN_WEIGHT_CHANNEL else 1)


def gdn_group_norm(cfg, x, w, y, b=None, z=None, lens=None, stream=None):
    """x, y and the gate z act [B][L][H][D]; w and the bias b fp32 [D] or [H][D]; lens int32 [B]."""
    a, act, n = _Args(cfg, x), _TORCH_DT[cfg.act_dtype], _norm_params(cfg)
    a.call("gdn_group_norm", cfg, (
        a.tokens(x, "x", act), a.dense(w, "w", torch.float32, n),
        a.dense(b, "b", torch.float32, n), a.tokens(z, "z", act), a.tokens(y, "y", act),
        a.lens(lens)), stream)


def gdn_group_norm_backward_workspace_bytes(cfg, L: int) -> int:
    return _bytes("gdn_group_norm_backward_workspace_bytes", cfg, L)


def gdn_group_norm_backward(cfg, x, w, dy, dx, dw, b=None, z=None, dz=None, db=None, lens=None,
                            workspace=None, stream=None):
    """x, w, b, z, lens of the forward call; dy, dx, dz act [B][L][H][D]; dw, db fp32 like w. dz
    goes with z and db with b. workspace: at least
    gdn_group_norm_backward_workspace_bytes(cfg, L) bytes on the device, made here when None."""
    a, act, n = _Args(cfg, x), _TORCH_DT[cfg.act_dtype], _norm_params(cfg)
    f32 = torch.float32
    a.call("gdn_group_norm_backward", cfg, (
        a.tokens(x, "x", act), a.dense(w, "w", f32, n), a.dense(b, "b", f32, n),
        a.tokens(z, "z", act), a.tokens(dy, "dy", act), a.tokens(dx, "dx", act),
        a.tokens(dz, "dz", act), a.dense(dw, "dw", f32, n), a.dense(db, "db", f32, n),
        a.lens(lens)), stream, workspace, gdn_group_norm_backward_workspace_bytes)


def gdn_short_conv(cfg, x, w, y, bias=None, state_in=None, state_out=None, lens=None,
                   stream=None):
    """x, y act [B][L][H][D]; w fp32 [H][D][K]; bias fp32 [H][D]; state_in, state_out act
    [B][K-1][H][D], the inputs before the first token and the last ones; lens int32 [B]."""
    a, act = _Args(cfg, x), _TORCH_DT[cfg.act_dtype]
    C, n = cfg.H * cfg.D, cfg.B * (cfg.K - 1) * cfg.H * cfg.D
    a.call("gdn_short_conv", cfg, (
        a.tokens(x, "x", act), a.dense(w, "w", torch.float32, C * cfg.K),
        a.dense(bias, "bias", torch.float32, C), a.dense(state_in, "state_in", act, n),
        a.tokens(y, "y", act), a.dense(state_out, "state_out", act, n), a.lens(lens)), stream)


def gdn_short_conv_backward_workspace_bytes(cfg, L: int) -> int:
    return _bytes("gdn_short_conv_backward_workspace_bytes", cfg, L)


def gdn_short_conv_backward(cfg, x, w, dy, dx, dw, bias=None, db=None, state_in=None,
                            dstate_out=None, dstate_in=None, lens=None, workspace=None,
                            stream=None):
    """x, w, bias, state_in, lens of the forward call; dy, dx act [B][L][H][D]; dw fp32 [H][D][K];
    db fp32 [H][D], which goes with bias; dstate_out, dstate_in act [B][K-1][H][D]. workspace: at
    least gdn_short_conv_backward_workspace_bytes(cfg, L) bytes on the device, made here when
    None."""
    a, act = _Args(cfg, x), _TORCH_DT[cfg.act_dtype]
    C, n = cfg.H * cfg.D, cfg.B * (cfg.K - 1) * cfg.H * cfg.D
    f32 = torch.float32
    a.call("gdn_short_conv_backward", cfg, (
        a.tokens(x, "x", act), a.dense(w, "w", f32, C * cfg.K),
        a.dense(bias, "bias", f32, C), a.dense(state_in, "state_in", act, n),
        a.tokens(dy, "dy", act), a.dense(dstate_out, "dstate_out", act, n),
        a.tokens(dx, "dx", act), a.dense(dw, "dw", f32, C * cfg.K), a.dense(db, "db", f32, C),
        a.dense(dstate_in, "dstate_in", act, n), a.lens(lens)), stream, workspace,
        gdn_short_conv_backward_workspace_bytes)
