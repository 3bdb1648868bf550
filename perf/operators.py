"""Cases that measure the operators around the recurrence: the gated scan, the group norm and the
short convolution, each forward and backward.

Every token array is [B][L][H][D] (sequences, tokens, heads, channels of a head), in one of three
places in memory: "tokens" (dense in that order), "heads" (dense as [B][H][L][D], as gdn_prefill
takes and leaves its arrays) or "wide" (a slice of a row that holds more, as a projection leaves
it). `run` with `own` false is the plain form in elementary torch operations; with `own` true the
library's entry points."""
import math
import random

import torch

own = False

CHUNK = 64  # tokens between the states that the forward scan keeps for its backward pass
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token of a mid-size decode batch through a gated recurrence
        dict(name="scan decode", op="scan", back=False, B=64, H=16, D=128, L=1, dtype="bf16",
             scale="sqrt", place="tokens", ragged=False, resets=False),
        # the prompt batch that the prefill is timed on, documents packed in it (the gate resets)
        dict(name="scan prompt", op="scan", back=False, B=8, H=32, D=128, L=4096, dtype="bf16",
             scale="sqrt", place="tokens", ragged=False, resets=True),
        # one long document, few channels, a length that no tile divides
        dict(name="scan long", op="scan", back=False, B=1, H=16, D=128, L=131071, dtype="bf16",
             scale="complement", place="tokens", ragged=False, resets=False),
        # the gradient of a padded training batch
        dict(name="scan train", op="scan", back=True, B=4, H=32, D=128, L=4096, dtype="bf16",
             scale="sqrt", place="tokens", ragged=True, resets=False),
        # the gradient in fp32 at odd sizes
        dict(name="scan train odd f32", op="scan", back=True, B=5, H=3, D=51, L=777, dtype="f32",
             scale="none", place="tokens", ragged=False, resets=True),
        # a layer's output norm and gate for one token of the mid-size decode batch
        dict(name="norm decode", op="norm", back=False, B=64, H=16, D=128, L=1, dtype="bf16",
             center=False, bias=False, gate=True, act="silu", weight="head", place="tokens",
             ragged=False),
        # the same for what the prefill leaves: head-major outputs, the gate a slice of a projection
        dict(name="norm prompt", op="norm", back=False, B=8, H=32, D=128, L=4096, dtype="bf16",
             center=False, bias=False, gate=True, act="silu", weight="head", place="heads",
             ragged=False),
        # group norm with mean, bias and activation, fp32, odd sizes
        dict(name="norm odd f32", op="norm", back=False, B=3, H=5, D=100, L=1999, dtype="f32",
             center=True, bias=True, gate=False, act="silu", weight="channel", place="tokens",
             ragged=False),
        # the gradient of the gated norm for a padded training batch
        dict(name="norm train", op="norm", back=True, B=4, H=32, D=128, L=4096, dtype="bf16",
             center=False, bias=False, gate=True, act="sigmoid", weight="head", place="heads",
             ragged=True),
        # one token of the serving batch through the short convolution
        dict(name="conv decode", op="conv", back=False, B=1024, H=32, D=128, L=1, dtype="bf16", K=4,
             bias=False, act="silu", place="tokens", ragged=False),
        # a prompt batch: a slice of the projection in, head-major out for the prefill
        dict(name="conv prompt", op="conv", back=False, B=8, H=32, D=128, L=4096, dtype="bf16", K=4,
             bias=False, act="silu", place="wide", ragged=False),
        # its gradient for a padded training batch
        dict(name="conv train", op="conv", back=True, B=4, H=32, D=128, L=4096, dtype="bf16", K=4,
             bias=True, act="silu", place="tokens", ragged=True),
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op, back = rng.choice(["scan", "norm", "conv"]), rng.random() < 0.4
    while True:
        D, H, B = _spread(rng, 4, 512), _spread(rng, 1, 64), _spread(rng, 1, 256)
        L = 1 if not back and rng.random() < 0.2 else _spread(rng, 1, 131072)
        if rng.random() < 0.5:
            D = -(-D // 16) * 16
        if 1 << 12 <= B * H * D * L <= 1 << 26:
            break
    case = dict(op=op, back=back, B=B, H=H, D=D, L=L, dtype=rng.choice(["bf16", "bf16", "f32"]),
                place=rng.choice(["tokens", "heads", "wide"]), ragged=rng.random() < 0.4)
    if op == "scan":
        case.update(scale=rng.choice(["none", "complement", "sqrt"]), resets=rng.random() < 0.4)
    elif op == "norm":
        case.update(center=rng.random() < 0.5, bias=rng.random() < 0.5, gate=rng.random() < 0.6,
                    act=rng.choice(["none", "silu", "sigmoid"]),
                    weight=rng.choice(["head", "channel"]))
    else:
        case.update(K=rng.choice([2, 3, 4, 4]), bias=rng.random() < 0.5,
                    act=rng.choice(["none", "silu", "silu"]))
    return case


def _lens(case):
    """Tokens of each sequence of a padded batch (some full, now and then one empty)."""
    r = random.Random(case["B"] * 1_000_003 + case["L"])
    L = case["L"]
    return [L if r.random() < 0.3 else r.randint(0 if r.random() < 0.1 else (L + 1) // 2, L)
            for _ in range(case["B"])]


def _empty(case, place, dtype):
    B, L, H, D = (case[n] for n in "BLHD")
    if place == "heads":
        return torch.zeros((B, H, L, D), dtype=dtype, device="cuda").transpose(1, 2)
    if place == "wide":
        return torch.zeros((B, L, 2 * H * D), dtype=dtype,
                           device="cuda")[..., :H * D].unflatten(-1, (H, D))
    return torch.zeros((B, L, H, D), dtype=dtype, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def tokens(place, dtype, mult=1.0):
        t = _empty(case, place, dtype)
        for b in range(case["B"]) if t.numel() > 1 << 27 else (slice(None),):
            t[b] = randn(*t[b].shape) * mult
        return t

    B, L, H, D = (case[n] for n in "BLHD")
    C, dt, place = H * D, DT[case["dtype"]], case["place"]
    s = dict(case=case, x=tokens(place, dt))
    s["lens"] = (torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
                 if case["ragged"] else None)
    if case["op"] == "scan":
        # per-channel rates of forgetting from a thousand tokens to one, modulated by the token
        rate = torch.exp(torch.rand((H, D), generator=gen, device="cuda") * math.log(700.0)) * 1e-3
        s["g"] = _empty(case, "tokens", torch.float32)
        for b in range(B) if s["g"].numel() > 1 << 27 else (slice(None),):
            s["g"][b] = torch.sigmoid(randn(*s["g"][b].shape)).mul_(rate).mul_(-2.0)
        if case["resets"]:  # a new document: the gate forgets everything before it
            at = torch.rand((B, L), generator=gen, device="cuda") < 1.0 / 500
            s["g"].masked_fill_(at[:, :, None, None], -math.inf)
        s["h0"] = randn(B, C)
        if case["back"]:
            s["do"], s["dhT"] = tokens(place, dt), randn(B, C)
            s["dx"], s["dg"] = _empty(case, place, dt), torch.zeros_like(s["g"])
            s["dh0"] = torch.zeros_like(s["h0"])
            # the states before every 64th token, which the forward pass keeps
            h = _scan_states(*_scan_terms(s)[:2], s["h0"])
            h = torch.cat([s["h0"].view(B, 1, C), h.reshape(B, L, C)], 1)
            s["hist"] = h[:, 0:L:CHUNK].contiguous()
        else:
            s["o"], s["hT"] = _empty(case, place, dt), torch.zeros_like(s["h0"])
    elif case["op"] == "norm":
        n = D if case["weight"] == "head" else C
        s["w"] = 1.0 + 0.2 * randn(n)
        s["b"] = 0.2 * randn(n) if case["bias"] else None
        # the gate comes out of a projection
        s["z"] = tokens("wide" if place == "heads" else place, dt) if case["gate"] else None
        if case["back"]:
            s["dy"], s["dx"] = tokens("tokens", dt), _empty(case, place, dt)
            s["dz"] = _empty(case, "tokens", dt) if case["gate"] else None
            s["dw"] = torch.zeros_like(s["w"])
            s["db"] = torch.zeros_like(s["w"]) if case["bias"] else None
        else:
            s["y"] = _empty(case, "tokens", dt)
    else:
        K = case["K"]
        s["w"] = randn(C, K) / math.sqrt(K)
        s["b"] = 0.2 * randn(C) if case["bias"] else None
        s["state"] = randn(B, K - 1, C).to(dt)
        if case["back"]:
            s["dy"], s["dx"] = tokens(place, dt), _empty(case, place, dt)
            s["dw"] = torch.zeros_like(s["w"])
            s["db"] = torch.zeros_like(s["b"]) if case["bias"] else None
            s["dstate_out"] = randn(B, K - 1, C).to(dt)
            s["dstate_in"] = torch.zeros_like(s["dstate_out"])
        else:
            s["y"] = _empty(case, "heads" if place == "wide" else place, dt)
            s["state_out"] = torch.zeros_like(s["state"])
    if own:
        _plan(s)
    return s


def _plan(s):
    """What a program keeps of the library beside its tensors: the configuration and a workspace."""
    import bit_recurrent_state_gdn_b200 as gdn

    case = s["case"]
    B, H, D, L, act = case["B"], case["H"], case["D"], case["L"], case["dtype"]
    n = 0
    if case["op"] == "scan":
        cfg = gdn.make_scan_config(B, H, D, scale=case["scale"], act=act)
    elif case["op"] == "norm":
        cfg = gdn.make_norm_config(B, H, D, eps=1e-6, center=case["center"],
                                   activation=case["act"], weight=case["weight"], act=act)
        if case["back"]:
            n = gdn.gdn_group_norm_backward_workspace_bytes(cfg, L)
    else:
        cfg = gdn.make_conv_config(B, H, D, case["K"], activation=case["act"], act=act)
        if case["back"]:
            n = gdn.gdn_short_conv_backward_workspace_bytes(cfg, L)
    s["cfg"] = cfg
    s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import bit_recurrent_state_gdn_b200 as gdn

    op, back, cfg, ws = s["case"]["op"], s["case"]["back"], s["cfg"], s["workspace"]
    if op == "scan" and not back:
        gdn.gdn_gated_scan(cfg, s["x"], s["g"], s["o"], h0=s["h0"], hT=s["hT"], lens=s["lens"])
        return s["o"], s["hT"]
    if op == "scan":
        gdn.gdn_gated_scan_backward(cfg, s["x"], s["g"], s["hist"], s["do"], s["dx"], s["dg"],
                                    dhT=s["dhT"], dh0=s["dh0"], lens=s["lens"])
        return s["dx"], s["dg"], s["dh0"]
    if op == "norm" and not back:
        gdn.gdn_group_norm(cfg, s["x"], s["w"], s["y"], b=s["b"], z=s["z"], lens=s["lens"])
        return s["y"]
    if op == "norm":
        gdn.gdn_group_norm_backward(cfg, s["x"], s["w"], s["dy"], s["dx"], s["dw"], b=s["b"],
                                    z=s["z"], dz=s["dz"], db=s["db"], lens=s["lens"], workspace=ws)
        return s["dx"], s["dz"], s["dw"], s["db"]
    if not back:
        gdn.gdn_short_conv(cfg, s["x"], s["w"], s["y"], bias=s["b"], state_in=s["state"],
                           state_out=s["state_out"], lens=s["lens"])
        return s["y"], s["state_out"]
    gdn.gdn_short_conv_backward(cfg, s["x"], s["w"], s["dy"], s["dx"], s["dw"], bias=s["b"],
                                db=s["db"], state_in=s["state"], dstate_out=s["dstate_out"],
                                dstate_in=s["dstate_in"], lens=s["lens"], workspace=ws)
    return s["dx"], s["dw"], s["db"], s["dstate_in"]


# ---- the plain forms ------------------------------------------------------------------------


def _mask(s):
    """[B][L][1][1]: the tokens that belong to a sequence; None where all do."""
    if s["lens"] is None:
        return None
    t = torch.arange(s["case"]["L"], device="cuda")
    return (t < s["lens"][:, None])[:, :, None, None]


def _f32(t, mask, fill=0.0):
    return t.float() if mask is None else torch.where(mask, t.float(), fill)


def _scan_terms(s):
    """Decay a, input s x, factor s and its derivative in g, [B][L][H][D]; tokens behind a
    sequence change nothing (a = 1, input 0)."""
    m, scale = _mask(s), s["case"]["scale"]
    g, x = _f32(s["g"], m), _f32(s["x"], m)
    a = torch.exp(g)
    if scale == "none":
        return a, x, None, None, x
    if scale == "complement":
        f, df = -torch.expm1(g), -a
    else:
        f = torch.sqrt(-torch.expm1(2 * g))
        df = torch.where(f > 0, -a * a / f, 0.0)
    return a, f * x, f, df, x


def _double(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from zero: each pass joins spans of twice the length,
    log2(L) passes in all. Overwrites both."""
    k = 1
    while k < b.shape[1]:
        b[:, k:] += a[:, k:] * b[:, :-k]
        a[:, k:] = a[:, k:] * a[:, :-k]
        k *= 2
    return b


def _scan_states(a, u, h0):
    a, u = a.clone(), u.clone()
    u[:, 0] += a[:, 0] * h0.view(u[:, 0].shape)
    return _double(a, u)


def _run_plain(s):
    case = s["case"]
    B, L, H, D = (case[n] for n in "BLHD")
    dt, m = DT[case["dtype"]], _mask(s)

    def rounded(t):
        return (t if m is None else torch.where(m, t, 0.0)).to(dt)

    if case["op"] == "scan":
        a, u, f, df, x = _scan_terms(s)
        h = _scan_states(a, u, s["h0"])
        if not case["back"]:
            return rounded(h), h[:, -1].reshape(B, H * D).clone()
        h = torch.cat([s["h0"].view(B, 1, H, D), h[:, :-1]], 1)
        dh = _f32(s["do"], m).clone()
        dh[:, -1] += s["dhT"].view(B, H, D)
        later = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
        dh = _double(later.flip(1), dh.flip(1)).flip(1)
        dg = a * h * dh
        if f is not None:
            dg = dg + dh * x * df
        dg = dg if m is None else torch.where(m, dg, 0.0)
        return rounded(dh if f is None else f * dh), dg, (a * dh)[:, 0].reshape(B, H * D)
    if case["op"] == "norm":
        return _norm_plain(s, m, rounded)
    return _conv_plain(s, m, rounded)


def _act(name, u):
    """The activation and its derivative."""
    if name == "none":
        return u, torch.ones_like(u)
    q = 1.0 / (1.0 + torch.exp(-u))
    return (q, q * (1 - q)) if name == "sigmoid" else (u * q, q * (1 + u * (1 - q)))


def _norm_plain(s, m, rounded):
    case = s["case"]
    x = _f32(s["x"], m)
    shape = (case["D"],) if case["weight"] == "head" else (case["H"], case["D"])
    w = s["w"].view(shape)
    x = x - x.mean(-1, keepdim=True) if case["center"] else x
    rstd = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    n = x * rstd
    u = n * w if s["b"] is None else n * w + s["b"].view(shape)
    z = None if s["z"] is None else _f32(s["z"], m)
    act, dact = _act(case["act"], u if z is None else z)
    if not case["back"]:
        return rounded(act if z is None else u * act)
    dy = _f32(s["dy"], m)
    du = dy * (dact if z is None else act)
    dims = (0, 1, 2) if case["weight"] == "head" else (0, 1)
    dn = du * w
    dx = dn - n * (dn * n).mean(-1, keepdim=True)
    if case["center"]:
        dx = dx - dn.mean(-1, keepdim=True)
    return (rounded(dx * rstd), None if z is None else rounded(dy * u * dact),
            (du * n).sum(dims).view(-1), None if s["b"] is None else du.sum(dims).view(-1))


def _conv_plain(s, m, rounded):
    case = s["case"]
    B, L, H, D = (case[n] for n in "BLHD")
    K, C, dt = case["K"], H * D, DT[case["dtype"]]
    xs = torch.cat([s["state"].float(), _f32(s["x"], m).reshape(B, L, C)], 1)
    pre = (xs.unfold(1, K, 1) * s["w"]).sum(-1)
    if s["b"] is not None:
        pre = pre + s["b"]
    act, dact = _act(case["act"], pre)
    lens = torch.full((B,), L, device="cuda") if s["lens"] is None else s["lens"].long()
    # rows of xs that are the K - 1 inputs before the sequence's end
    last = (lens[:, None] + torch.arange(K - 1, device="cuda"))[:, :, None].expand(B, K - 1, C)
    if not case["back"]:
        return rounded(act.view(B, L, H, D)), torch.gather(xs, 1, last).to(dt)
    dpre = _f32(s["dy"], m).reshape(B, L, C) * dact
    pad = torch.zeros((B, K - 1, C), device="cuda")
    dxs = (torch.cat([pad, dpre, pad], 1).unfold(1, K, 1) * s["w"].flip(1)).sum(-1)
    dxs = dxs.scatter_add(1, last, s["dstate_out"].float())
    dw = (xs.unfold(1, K, 1) * dpre[..., None]).sum((0, 1))
    return (rounded(dxs[:, K - 1:].view(B, L, H, D)), dw,
            None if s["b"] is None else dpre.sum((0, 1)), dxs[:, :K - 1].to(dt))


# ---- the definitions in 64 bits ---------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    B, L, H, D = (case[n] for n in "BLHD")
    live = torch.ones((B, L, 1), dtype=torch.bool, device="cuda")
    if s["lens"] is not None:
        live = torch.arange(L, device="cuda").view(1, L, 1) < s["lens"].view(B, 1, 1)

    def flat(t):
        """[B][L][C] in 64 bits, zero behind the sequences."""
        return t.reshape(B, L, H * D).double().masked_fill_(~live, 0.0)

    def out(t):
        return t.masked_fill(~live, 0.0).view(B, L, H, D)

    if case["op"] == "scan":
        return _scan_exact(s, case, flat, out)
    if case["op"] == "norm":
        return _norm_exact(s, case, flat, out, live)
    return _conv_exact(s, case, flat, out)


def _walk(a, u, h):
    """States of h <- a h + u along dim 1 of [B][L][C] from h [B][C]: all spans of about sqrt(L)
    tokens side by side, token by token; then span after span."""
    B, L, C = u.shape
    m = max(1, math.isqrt(L))
    n = -(-L // m)
    u = torch.cat([u, u.new_zeros(B, n * m - L, C)], 1).view(B, n, m, C)
    a = torch.cat([a, a.new_ones(B, n * m - L, C)], 1).view(B, n, m, C).clone()
    u = u.clone()
    for j in range(1, m):
        u[:, :, j] += a[:, :, j] * u[:, :, j - 1]
        a[:, :, j] *= a[:, :, j - 1]
    for i in range(n):
        u[:, i] += a[:, i] * h[:, None]
        h = u[:, i, -1]
    return u.view(B, n * m, C)[:, :L]


def _scan_exact(s, case, flat, out):
    B, L, H, D = (case[n] for n in "BLHD")
    g, x = flat(s["g"]), flat(s["x"])
    a = g.exp()
    one_a2 = -torch.expm1(2 * g)
    f = {"none": torch.ones_like(g), "complement": -torch.expm1(g), "sqrt": one_a2.sqrt()}[case["scale"]]
    h0 = s["h0"].double()
    h = _walk(a, f * x, h0)
    if not case["back"]:
        return out(h), h[:, -1].clone()
    dh = flat(s["do"])
    # gradients run from the last token to the first: token t takes a_{t+1} of what follows
    after = torch.ones_like(a)
    after[:, 1:] = a[:, 1:].flip(1)
    dh = _walk(after, dh.flip(1), s["dhT"].double()).flip(1)
    before = torch.cat([h0[:, None], h[:, :-1]], 1)
    dg = a * before * dh
    if case["scale"] == "complement":
        dg = dg - dh * x * a
    elif case["scale"] == "sqrt":
        dg = dg - torch.where(one_a2 > 0, dh * x * a * a / f, 0.0)
    return out(f * dh), out(dg), a[:, 0] * dh[:, 0]


def _slope(name, u):
    """Activation and derivative in 64 bits."""
    if name == "none":
        return u, torch.ones_like(u)
    q = torch.sigmoid(u)
    return (q, q - q * q) if name == "sigmoid" else (u * q, q + u * (q - q * q))


def _norm_exact(s, case, flat, out, live):
    B, L, H, D = (case[n] for n in "BLHD")
    x = flat(s["x"]).view(-1, H, D)
    w = s["w"].double().expand(H * D) if case["weight"] == "channel" else s["w"].double().repeat(H)
    b = torch.zeros_like(w) if s["b"] is None else s["b"].double().repeat(H * D // s["b"].numel())
    w, b = w.view(H, D), b.view(H, D)
    mean = x.sum(-1, keepdim=True) / D if case["center"] else torch.zeros_like(x[..., :1])
    sd = ((x - mean).square().sum(-1, keepdim=True) / D + 1e-6).sqrt()
    n = (x - mean) / sd
    u = n * w + b
    z = None if s["z"] is None else flat(s["z"]).view(-1, H, D)
    v, slope = _slope(case["act"], u if z is None else z)
    if not case["back"]:
        return out((v if z is None else u * v).view(B, L, H * D))
    dy = flat(s["dy"]).view(-1, H, D)
    du = dy * (slope if z is None else v)
    dn = du * w
    # d n_i / d x_j = (delta_ij - [center] / D - n_i n_j / D) / sd
    dx = (dn - n * (dn * n).sum(-1, keepdim=True) / D) / sd
    if case["center"]:
        dx = dx - dn.sum(-1, keepdim=True) / (D * sd)
    dw, db = (du * n).sum(0), du.sum(0)
    if case["weight"] == "head":
        dw, db = dw.sum(0), db.sum(0)
    return (out(dx.view(B, L, H * D)),
            None if z is None else out((dy * u * slope).view(B, L, H * D)), dw.reshape(-1),
            None if s["b"] is None else db.reshape(-1))


def _conv_exact(s, case, flat, out):
    B, L, H, D = (case[n] for n in "BLHD")
    K, C = case["K"], H * D
    w = s["w"].double()
    rows = torch.cat([s["state"].double(), flat(s["x"])], 1)  # token t is row t + K - 1
    pre = torch.zeros((B, L, C), dtype=torch.float64, device="cuda")
    if s["b"] is not None:
        pre += s["b"].double()
    for j in range(K):
        pre += w[:, j] * rows[:, j:j + L]
    v, slope = _slope(case["act"], pre)
    ends = [L] * B if s["lens"] is None else s["lens"].tolist()
    if not case["back"]:
        return out(v), torch.stack([rows[b, e:e + K - 1] for b, e in enumerate(ends)])
    dpre = flat(s["dy"]) * slope
    drows = torch.zeros_like(rows)
    dw = torch.zeros_like(w)
    for j in range(K):
        drows[:, j:j + L] += w[:, j] * dpre
        dw[:, j] = (rows[:, j:j + L] * dpre).sum((0, 1))
    for b, e in enumerate(ends):
        drows[b, e:e + K - 1] += s["dstate_out"][b].double()
    return (out(drows[:, K - 1:]), dw, None if s["b"] is None else dpre.sum((0, 1)),
            drows[:, :K - 1])


def work(case):
    B, L, H, D = (case[n] for n in "BLHD")
    C, e = H * D, 2 if case["dtype"] == "bf16" else 4
    n = C * (sum(_lens(case)) if case["ragged"] else B * L)  # elements of the live tokens
    if case["op"] == "scan":
        if case["back"]:  # x, g, do in; dx, dg out; kept states, and the states' gradients
            return {"bytes": n * (3 * e + 8) + B * C * (8 + 4 * -(-L // CHUNK)), "flops": 12 * n}
        return {"bytes": n * (2 * e + 4) + 8 * B * C, "flops": 4 * n}
    if case["op"] == "norm":
        z, w = int(case["gate"]), (D if case["weight"] == "head" else C) * (1 + int(case["bias"]))
        if case["back"]:  # x, dy, z in; dx, dz out
            return {"bytes": n * e * (3 + 2 * z) + 8 * w, "flops": 24 * n}
        return {"bytes": n * e * (2 + z) + 4 * w, "flops": 10 * n}
    K = case["K"]
    w = 4 * C * (K + int(case["bias"]))
    if case["back"]:  # x, dy, both states in; dx, the state's gradient, dw out
        return {"bytes": n * e * 3 + 3 * e * B * (K - 1) * C + 2 * w, "flops": (6 * K + 8) * n}
    return {"bytes": n * e * 2 + 2 * e * B * (K - 1) * C + w, "flops": (2 * K + 4) * n}
