"""Plain 64-bit forms of the operators around the recurrence, and bounds on how far fp32
arithmetic with one rounding at the end may be from them.

U = 2^-24 is fp32's half step. A bound is a sum of (relative error) x (magnitude of the terms that
carry it): N_OPS counts the half steps that the roundings between an input and a result can add
up to for one term (an exponential of 2 steps, a factor 1 - a or its root of 4, products, sums,
joins of spans)."""
import torch

U = 2.0 ** -24
# The hardware's exponential returns zero for e^g below fp32's smallest normal number: what such a
# gate multiplies is then lost, at most 2^-126 of it.
FLUSH = 2.0 ** -126
N_OPS = 24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def lens_of(lens, B, L):
    return [L] * B if lens is None else [min(max(int(v), 0), L) for v in lens.tolist()]


def live_mask(lens, B, L):
    return torch.arange(L)[None, :] < torch.tensor(lens_of(lens, B, L))[:, None]


def close(got, want, bound, dtype, where=""):
    """|got - want| within bound plus the rounding to dtype, everywhere."""
    got, want = got.detach().cpu().double(), want.double()
    tol = bound.double() + half_step(dtype) * want.abs() + 1e-37
    off = (got - want).abs()
    bad = ~((off <= tol) | (got == want))
    assert not bad.any(), (where, int(bad.sum()), float((off - tol).max()),
                           got[bad][:4].tolist(), want[bad][:4].tolist())


# ---- gated scan ---------------------------------------------------------------------------


def scan_factor(g, scale):
    if scale == "none":
        return torch.ones_like(g)
    return -torch.expm1(g) if scale == "complement" else torch.sqrt(-torch.expm1(2 * g))


def scan(x, g, h0, scale, lens=None):
    """o, hT, the state before every token, and the bound on each state, on [B][L][H][D]."""
    B, L = x.shape[:2]
    x, g = x.double(), g.double()
    h = h0.double().clone()
    size, err = h.abs(), torch.zeros_like(h)  # sum of the terms' magnitudes; bound
    o, before, errs, errs_before = (torch.zeros_like(x) for _ in range(4))
    live = live_mask(lens, B, L)
    for t in range(L):
        m = live[:, t].view(B, 1, 1)
        before[:, t], errs_before[:, t] = h, err
        a, u = g[:, t].exp(), scan_factor(g[:, t], scale) * torch.where(m, x[:, t], 0.0)
        n_h, n_s = a * h + u, a * size + u.abs()
        h, size = torch.where(m, n_h, h), torch.where(m, n_s, size)
        err = torch.where(m, a * err + N_OPS * U * n_s + FLUSH * before[:, t].abs(), err)
        o[:, t], errs[:, t] = h, err
    return o, h, before, errs, errs_before, err


def scan_backward(x, g, h0, do, dhT, scale, lens=None):
    """dx, dg, dh0 and their bounds."""
    B, L = x.shape[:2]
    x, g, do = x.double(), g.double(), do.double()
    _, _, before, _, err_before, _ = scan(x, g, h0, scale, lens)
    carry = dhT.double().clone()
    size, err = carry.abs(), torch.zeros_like(carry)
    dx, dg, e_dx, e_dg = (torch.zeros_like(x) for _ in range(4))
    live = live_mask(lens, B, L)
    for t in reversed(range(L)):
        m = live[:, t].view(B, 1, 1)
        a, s = g[:, t].exp(), scan_factor(g[:, t], scale)
        if scale == "none":
            ds = torch.zeros_like(a)
        elif scale == "complement":
            ds = -a
        else:
            ds = torch.where(s > 0, -a * a / s, 0.0)
        xt, dot = torch.where(m, x[:, t], 0.0), torch.where(m, do[:, t], 0.0)
        dh, n_s = dot + carry, dot.abs() + size
        e = err + N_OPS * U * n_s
        dx[:, t], e_dx[:, t] = s * dh, s * (e + N_OPS * U * n_s)
        k, ek = a * before[:, t] + ds * xt, a * err_before[:, t]
        mag = a * before[:, t].abs() + (ds * xt).abs()
        dg[:, t] = k * dh
        e_dg[:, t] = mag * e + ek * n_s + N_OPS * U * mag * n_s + FLUSH * before[:, t].abs() * n_s
        carry = torch.where(m, a * dh, carry)
        size, err = torch.where(m, a * n_s, size), torch.where(m, a * e + FLUSH * n_s, err)
    return dx, dg, carry, e_dx, e_dg, err + N_OPS * U * size


# ---- activations --------------------------------------------------------------------------


def act(name, u):
    """act, act' and a bound on the relative error of either from fp32's sigmoid, whose
    exponential is off by up to 2 + 1.2 |u| steps (two half steps each)."""
    if name == "none":
        return u, torch.ones_like(u), torch.zeros_like(u)
    q = torch.sigmoid(u)
    # 1 - q and 1 + u (1 - q) lose up to |u| more
    rel = U * (16 + 8 * u.abs())
    if name == "sigmoid":
        return q, q * (1 - q), rel
    return u * q, q * (1 + u * (1 - q)), rel


# ---- group norm ---------------------------------------------------------------------------


def norm_terms(x, w, b, z, activation, center, eps):
    x = x.double()
    D = x.shape[-1]
    m = x.mean(-1, keepdim=True) if center else torch.zeros_like(x[..., :1])
    rstd = 1 / torch.sqrt(((x - m) ** 2).mean(-1, keepdim=True) + eps)
    n = (x - m) * rstd
    # D terms added in fp32, at most 40 of them one after another
    c = U * (N_OPS + min(D, 40))
    big = c * x.abs().amax(-1, keepdim=True) * rstd if center else torch.zeros_like(rstd)
    e_n = big + n.abs() * (c + big)
    w = w.double()
    bias = torch.zeros_like(w) if b is None else b.double()
    u = n * w + bias
    e_u = w.abs() * e_n + N_OPS * U * ((n * w).abs() + bias.abs())
    return rstd, n, e_n, w, u, e_u, c, big


def norm(x, w, b, z, activation, center, eps):
    """y and its bound. w, b broadcast against [B][L][H][D]."""
    _, _, _, _, u, e_u, _, _ = norm_terms(x, w, b, z, activation, center, eps)
    if z is None:
        v, _, rel = act(activation, u)
        return v, 1.2 * e_u + rel * v.abs().clamp_min(1e-30)
    v, _, rel = act(activation, z.double())
    return u * v, e_u * v.abs() + (rel + N_OPS * U) * (u * v).abs()


def norm_backward(x, w, b, z, dy, activation, center, eps):
    """dx, dz, and the terms of dw and db per row, each with its bound."""
    rstd, n, e_n, w, u, e_u, c, big = norm_terms(x, w, b, z, activation, center, eps)
    dy = dy.double()
    v, slope, rel = act(activation, u if z is None else z.double())
    if z is None:
        # act'' is at most 1/2 for SiLU and the sigmoid; act' itself may cancel
        du = dy * slope
        e_du = dy.abs() * (0.5 * e_u + rel * (slope.abs() + 0.5))
        if activation == "none":
            e_du = torch.zeros_like(du)
        dz = e_dz = None
    else:
        du, e_du = dy * v, (dy * v).abs() * (rel + U)
        dz = dy * u * slope
        e_dz = dy.abs() * (e_u * slope.abs() + u.abs() * rel * (slope.abs() + 0.5)
                           + N_OPS * U * (u * slope).abs())
    dn, e_dn = du * w, e_du * w.abs() + U * (du * w).abs()

    def mean(t):
        return t.mean(-1, keepdim=True)

    m1 = mean(dn) if center else torch.zeros_like(rstd)
    m2 = mean(dn * n)
    dx = rstd * (dn - m1 - n * m2)
    e_m2 = mean(e_dn * n.abs() + dn.abs() * e_n + c * (dn * n).abs())
    e_dx = rstd * (e_dn + mean(e_dn) + c * mean(dn.abs()) + n.abs() * e_m2 + e_n * m2.abs()
                   + (c + big) * (dn.abs() + mean(dn.abs()) + n.abs() * mean((dn * n).abs())))
    return dx, e_dx, dz, e_dz, (du * n, e_du * n.abs() + du.abs() * e_n), (du, e_du)


def summed(term, err, dims, n):
    """A sum in fp32 of n terms, at most n after one another, and its bound."""
    return term.sum(dims), err.sum(dims) + U * (n + N_OPS) * term.abs().sum(dims)


# ---- short convolution ----------------------------------------------------------------------


def conv(x, w, b, state, activation, lens=None):
    """y, state_out, and y's bound, on [B][L][C]; state [B][K-1][C]."""
    B, L, C = x.shape
    K = w.shape[1]
    rows = torch.cat([state.double(), x.double()], 1)
    p = torch.zeros((B, L, C), dtype=torch.float64) + (0.0 if b is None else b.double())
    size = p.abs()
    for j in range(K):
        p = p + w[:, j].double() * rows[:, j:j + L]
        size = size + (w[:, j].double() * rows[:, j:j + L]).abs()
    v, _, rel = act(activation, p)
    ends = lens_of(lens, B, L)
    out = torch.stack([rows[i, e:e + K - 1] for i, e in enumerate(ends)]) if B else state.double()
    return v, out, 1.2 * N_OPS * U * size + rel * v.abs()


def conv_backward(x, w, b, state, dy, dstate_out, activation, lens=None):
    """dx, dw, db, dstate_in, each with its bound. Inputs behind a sequence are taken as zero."""
    B, L, C = x.shape
    K = w.shape[1]
    live = live_mask(lens, B, L)[:, :, None]
    x, dy = torch.where(live, x.double(), 0.0), torch.where(live, dy.double(), 0.0)
    w = w.double()
    rows = torch.cat([state.double(), x], 1)
    p = torch.zeros((B, L, C), dtype=torch.float64) + (0.0 if b is None else b.double())
    size = p.abs()
    for j in range(K):
        p = p + w[:, j] * rows[:, j:j + L]
        size = size + (w[:, j] * rows[:, j:j + L]).abs()
    _, slope, rel = act(activation, p)
    dp = dy * slope
    e_dp = dy.abs() * (0.5 * N_OPS * U * size + rel * (slope.abs() + 0.5))
    drows, e_rows = torch.zeros_like(rows), torch.zeros_like(rows)
    dw, e_dw = torch.zeros_like(w), torch.zeros_like(w)
    n = B * L
    for j in range(K):
        drows[:, j:j + L] += w[:, j] * dp
        e_rows[:, j:j + L] += w[:, j].abs() * (e_dp + N_OPS * U * dp.abs())
        term = rows[:, j:j + L] * dp
        dw[:, j], e_dw[:, j] = summed(term, rows[:, j:j + L].abs() * e_dp, (0, 1), n)
    for i, e in enumerate(lens_of(lens, B, L)):
        drows[i, e:e + K - 1] += dstate_out[i].double()
        e_rows[i, e:e + K - 1] += N_OPS * U * dstate_out[i].double().abs()
    db, e_db = summed(dp, e_dp, (0, 1), n)
    return ((drows[:, K - 1:], e_rows[:, K - 1:]), (dw, e_dw), (db, e_db),
            (drows[:, :K - 1], e_rows[:, :K - 1]))
