"""Plain 64-bit forms of the block operators, with error bounds for fp32 kernels.

Each function returns the exact values and, beside each, a bound on how far an
fp32 evaluation may be off.  The bounds follow the arithmetic: U = 2^-24 is the
relative error of one fp32 operation, and sums of magnitudes ("the same formula
on absolute values") carry it through.  ``ROUND[dtype]`` is the half step of the
output's own rounding, added by ``allowed``.
"""
import torch

U = 2.0 ** -24
ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def allowed(value, bound, dtype):
    """Largest |got - value| for an output of ``dtype``: the fp32 bound and the
    rounding of the (possibly off) value."""
    return bound + ROUND[dtype] * (value.abs() + bound) + 1e-37


def assert_close(name, got, value, bound, dtype=None):
    dtype = dtype or got.dtype
    got, value, bound = got.double().cpu(), value.cpu(), bound.cpu()
    assert got.shape == value.shape, (name, got.shape, value.shape)
    if got.numel() == 0:
        return
    assert torch.isfinite(got).all(), f"{name}: not finite"
    over = (got - value).abs() / allowed(value, bound, dtype)
    worst = over.argmax()
    assert over.max() <= 1.0, (f"{name}: {over.max():.3g} x the bound at {tuple(torch.unravel_index(worst, over.shape))}, "
                               f"got {got.flatten()[worst]}, want {value.flatten()[worst]}")


def d64(t):
    return None if t is None else t.detach().double().cpu()


# ---------------------------------------------------------------- gated recurrence
# Per step, a and u carry a relative error of a few operations: exp (2 units in
# the last place of its result, plus the rounding of its argument, |f| log2(e)
# U), an add, a divide (2), a multiply; the recurrence adds one rounded
# multiply-add, and the joins of partial scans (one per 8 steps, per 8 warps and
# per tile) a few more.  STEP U covers them with |f| counted separately.

STEP = 16.0


def gated(gate, x, gate_bias=None, initial_state=None, seqlens=None, log_decay=False, layout="bdl",
          dout=None, dlast_state=None):
    """Values and bounds of every output: a dict name -> (value, bound)."""
    f, x = d64(gate), d64(x)
    if layout == "bdl":
        f, x = f.transpose(1, 2), x.transpose(1, 2)
    B, L, D = f.shape
    if gate_bias is not None:
        f = f + d64(gate_bias)
    n = torch.full((B,), L) if seqlens is None else seqlens.cpu().long().clamp(0, L)
    inside = (torch.arange(L)[None] < n[:, None])[:, :, None]
    zero = torch.zeros((), dtype=torch.float64)
    f, x = torch.where(inside, f, zero), torch.where(inside, x, zero)
    if log_decay:
        a, g = torch.exp(f), torch.ones_like(f)
        delta = STEP * U + 2 * U * torch.where(torch.isfinite(f), f.abs(), zero)
    else:
        a, g = torch.sigmoid(-f), torch.sigmoid(f)
        delta = STEP * U + 2 * U * f.abs()
    a = torch.where(inside, a, zero + 1)
    g = torch.where(inside, g, zero)
    u = g * x
    h = torch.zeros(B, D, dtype=torch.float64) if initial_state is None else d64(initial_state).clone()
    h0 = h.clone()
    M, E = h.abs(), torch.zeros_like(h)
    hs, Ms, Es = torch.empty_like(f), torch.empty_like(f), torch.empty_like(f)
    enter = []
    for t in range(L):
        if t % 64 == 0:
            enter.append((h, E))
        dt = torch.where(inside[:, t], delta[:, t], zero + STEP * U)
        E = a[:, t] * E + dt * (a[:, t] * M + u[:, t].abs())
        M = a[:, t] * M + u[:, t].abs()
        h = a[:, t] * h + u[:, t]
        hs[:, t], Ms[:, t], Es[:, t] = h, M, E
    lay = (lambda t: t) if layout == "bld" else (lambda t: t.transpose(1, 2).contiguous())
    out = {"out": (lay(torch.where(inside, hs, zero)), lay(torch.where(inside, Es, zero))),
           "last_state": (h, E)}
    if layout == "bld":
        shape = (B, -(-L // 64), D)
        out["checkpoints"] = tuple(torch.stack([e[k] for e in enter], 1) if enter else
                                   torch.zeros(shape, dtype=torch.float64) for k in (0, 1))
    if dout is None:
        return out
    dy = d64(dout)
    dy = dy if layout == "bld" else dy.transpose(1, 2)
    dy = torch.where(inside, dy, zero)
    r = torch.zeros(B, D, dtype=torch.float64) if dlast_state is None else d64(dlast_state).clone()
    N, F = r.abs(), torch.zeros_like(r)                  # magnitude and error of r
    dx, df = torch.zeros_like(f), torch.zeros_like(f)
    bx, bf = torch.zeros_like(f), torch.zeros_like(f)
    for t in range(L - 1, -1, -1):
        at, gt, dt = a[:, t], g[:, t], delta[:, t]
        l, lm, le = dy[:, t] + r, dy[:, t].abs() + N, F + STEP * U * (dy[:, t].abs() + N)
        before = hs[:, t - 1] if t > 0 else h0
        bm = Ms[:, t - 1] if t > 0 else h0.abs()
        be = Es[:, t - 1] if t > 0 else torch.zeros_like(h0)
        if log_decay:
            dx[:, t], bx[:, t] = l, le
            df[:, t] = l * at * before
            bf[:, t] = at * (le * bm + lm * be + 4 * dt * lm * bm)
        else:
            dx[:, t], bx[:, t] = gt * l, gt * (le + dt * lm)
            df[:, t] = l * (x[:, t] - before) * gt * at
            xm = x[:, t].abs() + bm
            bf[:, t] = gt * at * (le * xm + lm * be + 4 * dt * lm * xm)
        r, N, F = at * l, at * lm, at * le + dt * at * lm
    dx, df = torch.where(inside, dx, zero), torch.where(inside, df, zero)
    bx, bf = torch.where(inside, bx, zero), torch.where(inside, bf, zero)
    out["dx"], out["dgate"] = (lay(dx), lay(bx)), (lay(df), lay(bf))
    # sums of B L terms, in at most B L roundings
    terms = df.abs().sum((0, 1))
    out["dgate_bias"] = (df.sum((0, 1)), bf.sum((0, 1)) + (B * L + 64) * U * (terms + bf.sum((0, 1))))
    out["dinitial_state"] = (r, F)
    return out


# ---------------------------------------------------------------- layer norm

def norm_fwd(x, weight=None, bias=None, residual=None, eps=1e-5, rms=False):
    s = d64(x) if residual is None else d64(x) + d64(residual)
    D = s.shape[-1]
    mean = torch.zeros_like(s[..., :1]) if rms else s.mean(-1, keepdim=True)
    c = s - mean
    rstd = (c.square().mean(-1, keepdim=True) + eps).rsqrt()
    w = torch.ones(D, dtype=torch.float64) if weight is None else d64(weight)
    b = torch.zeros(D, dtype=torch.float64) if bias is None else d64(bias)
    # s is rounded once, the mean is a tree sum over at most D / 8 + 16 roundings
    # of which the errors stay below 16 U times the mean magnitude for the team
    # sizes used (16 or 8 elements in a thread, then two 5-level trees)
    serr = 0.0 if residual is None else U * s.abs()
    wide = 16 + 2 * (D // 8192) * 8
    merr = torch.zeros_like(mean) if rms else (wide + 16) * U * s.abs().mean(-1, keepdim=True)
    cerr = serr + merr + U * c.abs()
    # relative error of rstd: half that of the mean square
    ms = c.square().mean(-1, keepdim=True)
    rel = ((2 * c.abs() * cerr + cerr * cerr).mean(-1, keepdim=True) + (wide + 16) * U * ms) / (2 * (ms + eps)) + 4 * U
    y = c * rstd * w + b
    bound = rstd * w.abs() * (cerr + c.abs() * (rel + 4 * U)) + 2 * U * (y.abs() + b.abs())
    out = {"out": (y, bound), "rstd": (rstd[..., 0], (rstd * rel)[..., 0]),
           "mean": (mean[..., 0], merr[..., 0]), "residual_out": (s, serr + torch.zeros_like(s))}
    return out


def norm_bwd(dout, s, rstd, mean=None, weight=None, dresidual_out=None, rms=False):
    """Gradients given the fp32 statistics as they are."""
    s, dy, r = d64(s), d64(dout), d64(rstd)[..., None]
    m = torch.zeros_like(r) if rms else d64(mean)[..., None]
    D = s.shape[-1]
    xh = (s - m) * r
    w = torch.ones(D, dtype=torch.float64) if weight is None else d64(weight)
    q = dy * w
    c1 = torch.zeros_like(r) if rms else q.mean(-1, keepdim=True)
    c2 = (q * xh).mean(-1, keepdim=True)
    ds = r * (q - c1 - xh * c2)
    # the same formula on magnitudes; every product and sum below has at most
    # `wide` roundings (as in the forward)
    wide = 48 + 4 * (D // 8192) * 8
    mag = r * (q.abs() + q.abs().mean(-1, keepdim=True) + xh.abs() * (q * xh).abs().mean(-1, keepdim=True))
    bound = wide * U * mag
    if dresidual_out is not None:
        ds = ds + d64(dresidual_out)
        bound = bound + U * (d64(dresidual_out).abs() + mag)
    rows = dy.numel() // max(D, 1)
    flat = lambda t: t.reshape(-1, D).sum(0)  # noqa: E731
    k = rows + 64
    return {"dx": (ds, bound), "dresidual": (ds, bound),
            "dweight": (flat(dy * xh), k * U * flat((dy * xh).abs())),
            "dbias": (flat(dy), k * U * flat(dy.abs()))}


# ---------------------------------------------------------------- convolution

def conv_bwd(x, weight, dout, bias=None, initial_conv_state=None, dfinal_conv_state=None, silu=True, depth=None):
    """depth: roundings that a term of the sums over batch and time goes through, at most (default:
    one per term)."""
    x, w, dy = d64(x), d64(weight), d64(dout)
    B, D, L = x.shape
    W = w.shape[1]
    init = torch.zeros(B, D, W, dtype=torch.float64) if initial_conv_state is None else d64(initial_conv_state)
    seq = torch.cat([init, x], 2)
    tap = lambda k: seq[:, :, 1 + k:1 + k + L]  # noqa: E731
    b = torch.zeros(D, dtype=torch.float64) if bias is None else d64(bias)
    pre = b[:, None] + sum(w[:, k, None] * tap(k) for k in range(W))
    mag = b.abs()[:, None] + sum(w[:, k, None].abs() * tap(k).abs() for k in range(W))
    perr = 2 * W * U * mag
    if silu:
        sg = torch.sigmoid(pre)
        fac = sg * (1 + pre * (1 - sg))
        # |silu''| <= 1/2; sigmoid to 8 units relative to 1 at most, |pre| (1 - sg) sg <= 0.3 |..|
        ferr = 0.5 * perr + 16 * U * (sg + (pre * sg).abs())
    else:
        fac, ferr = torch.ones_like(pre), torch.zeros_like(pre)
    dp, derr = dy * fac, dy.abs() * ferr + U * (dy * fac).abs()
    ds, se = torch.zeros_like(seq), torch.zeros_like(seq)
    for k in range(W):
        ds[:, :, 1 + k:1 + k + L] += w[:, k, None] * dp
        se[:, :, 1 + k:1 + k + L] += w[:, k, None].abs() * (derr + 2 * W * U * dp.abs())
    if dfinal_conv_state is not None:
        f = d64(dfinal_conv_state)
        se[:, :, L:] += 2 * U * (f.abs() + ds[:, :, L:].abs())
        ds[:, :, L:] += f
    depth = B * L + 64 if depth is None else depth
    terms = [dp * tap(k) for k in range(W)]
    dw = torch.stack([t.sum((0, 2)) for t in terms], 1)
    we = torch.stack([(derr * tap(k).abs()).sum((0, 2)) + depth * U * terms[k].abs().sum((0, 2))
                      for k in range(W)], 1)
    return {"dx": (ds[:, :, W:], se[:, :, W:]), "dinitial_conv_state": (ds[:, :, :W], se[:, :, :W]),
            "dweight": (dw, we),
            "dbias": (dp.sum((0, 2)), derr.sum((0, 2)) + depth * U * dp.abs().sum((0, 2)))}
