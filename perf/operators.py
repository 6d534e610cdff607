"""Cases, plain forms and 64-bit definitions of the operators around a recurrent block's projections.

Operators: layer norm with the residual add (forward and backward), the gated
linear recurrence (forward, backward and one token) and the backward pass of
the short causal convolution.

``run`` computes a case with elementary torch operations in 32 bits, or, with
``own`` set, through ``selective_state_space_55_b200.ops``.  ``exact`` computes
the same outputs in 64 bits straight from the definitions: step by step over
time, or as the derivative of the 64-bit forward.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BLOCK = 64                     # steps between the states that a training forward keeps


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # A block's entry in a decode step: eight sequences, the residual stream in fp32, d_model 2560.
        dict(name="norm_fwd_decode_8x2560", op="norm_fwd", rows=8, dim=2560, dtype="bf16",
             res="fp32", rms=False, bias=True),
        # The same entry over a training batch of 16 x 2048 tokens.
        dict(name="norm_fwd_train_32768x2560", op="norm_fwd", rows=32768, dim=2560, dtype="bf16",
             res="same", rms=False, bias=True),
        # Its backward: the gradient of the residual stream joins, weight and bias gradients are reduced.
        dict(name="norm_bwd_train_32768x2560", op="norm_bwd", rows=32768, dim=2560, dtype="bf16",
             res="same", rms=False, bias=True),
        # A narrow model of odd width in fp32 with the root-mean-square form, a ragged number of rows.
        dict(name="norm_bwd_ragged_4099x1001", op="norm_bwd", rows=4099, dim=1001, dtype="fp32",
             res="none", rms=True, bias=False),
        # Training forward of one layer: 8 x 2048 tokens, 4096 channels, channels fastest (as the
        # projections leave them), the gate as a sigmoid.
        dict(name="gated_fwd_bld_8x2048x4096", op="gated_fwd", batch=8, dim=4096, seqlen=2048,
             layout="bld", dtype="bf16", log_decay=False, bias=True, start=False, ragged=False),
        # One long document, few channels: time has to be split.  Log decays, a start state.
        dict(name="gated_fwd_bld_1x131072x1536", op="gated_fwd", batch=1, dim=1536, seqlen=131072,
             layout="bld", dtype="bf16", log_decay=True, bias=False, start=True, ragged=False),
        # Training backward of the 4096-channel layer.
        dict(name="gated_bwd_bld_8x2048x4096", op="gated_bwd", batch=8, dim=4096, seqlen=2048,
             layout="bld", dtype="bf16", log_decay=False, bias=True, start=False, ragged=False),
        # A padded batch with time fastest, odd sizes, fp32, a start state.
        dict(name="gated_bwd_bdl_5x777x1003", op="gated_bwd", batch=5, dim=777, seqlen=1003,
             layout="bdl", dtype="fp32", log_decay=True, bias=True, start=True, ragged=True),
        # One token of generation for one sequence: the smallest call.
        dict(name="gated_update_1x4096", op="gated_update", batch=1, dim=4096, dtype="bf16",
             log_decay=False, bias=True),
        # One token for 128 sequences.
        dict(name="gated_update_128x4096", op="gated_update", batch=128, dim=4096, dtype="bf16",
             log_decay=False, bias=True),
        # The convolution's backward in the 5120-channel training layer.
        dict(name="conv_bwd_16x5120x2048", op="conv_bwd", batch=16, dim=5120, seqlen=2048, width=4,
             dtype="bf16", silu=True, bias=True, state=False),
        # A short odd sequence continued from a conv state, three taps, fp32.
        dict(name="conv_bwd_3x1000x333", op="conv_bwd", batch=3, dim=1000, seqlen=333, width=3,
             dtype="fp32", silu=True, bias=True, state=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _shrink(sizes, order, limit):
    """Halves the sizes named in ``order`` in turn until their product is within ``limit``."""
    i = 0
    while math.prod(sizes.values()) > limit:
        k = order[i % len(order)]
        sizes[k] = max(1, sizes[k] // 2)
        i += 1
    return sizes


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "gated_fwd", "gated_fwd", "gated_bwd", "gated_bwd",
                     "gated_update", "conv_bwd"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("norm_fwd", "norm_bwd"):
        dim = _log_int(rng, 48, 16384)
        if flag():
            dim = max(8, dim // 8 * 8)
        s = _shrink(dict(rows=_log_int(rng, 1, 32768), dim=dim), ["rows"], 32768 * 2560 // 2)
        return dict(op=op, rows=s["rows"], dim=s["dim"], dtype=dtype,
                    res=rng.choice(["none", "same", "fp32"]), rms=flag(), bias=flag())
    if op in ("gated_fwd", "gated_bwd"):
        dim = _log_int(rng, 16, 5120)
        if flag():
            dim = max(8, dim // 8 * 8)
        s = _shrink(dict(batch=_log_int(rng, 1, 16), seqlen=_log_int(rng, 1, 65536), dim=dim),
                    ["batch", "seqlen"], 8 * 2048 * 4096 // 2)
        return dict(op=op, batch=s["batch"], dim=s["dim"], seqlen=s["seqlen"],
                    layout=rng.choice(["bld", "bld", "bdl"]), dtype=dtype, log_decay=flag(),
                    bias=flag(), start=flag(), ragged=flag())
    if op == "gated_update":
        return dict(op=op, batch=_log_int(rng, 1, 512), dim=_log_int(rng, 16, 5120), dtype=dtype,
                    log_decay=flag(), bias=flag())
    s = _shrink(dict(batch=_log_int(rng, 1, 16), seqlen=_log_int(rng, 1, 65536),
                     dim=_log_int(rng, 16, 5120)), ["batch", "seqlen"], 8 * 2048 * 4096 // 2)
    return dict(op=op, batch=s["batch"], dim=s["dim"], seqlen=s["seqlen"], width=rng.randint(1, 4),
                dtype=dtype, silu=flag(), bias=flag(), state=flag())


# ------------------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    g = _generator(seed)
    dt = DTYPES[case["dtype"]]
    randn = lambda *shape: torch.randn(*shape, generator=g, device=DEV)  # noqa: E731
    st = {"case": case}
    if case["op"] in ("norm_fwd", "norm_bwd"):
        R, D = case["rows"], case["dim"]
        rdt = torch.float32 if case["res"] == "fp32" else dt
        # activations with an offset and a few large channels, as residual streams have
        scale = torch.exp(0.5 * randn(D))
        st["weight"] = 1.0 + 0.1 * randn(D)
        st["bias"] = 0.1 * randn(D) if case["bias"] else None
        if case["op"] == "norm_fwd":
            st["x"] = (randn(R, D) * scale).to(dt)
            st["residual"] = None if case["res"] == "none" else (randn(R, D) * scale + 0.5).to(rdt)
        else:
            st["s"] = (randn(R, D) * scale + 0.5).to(rdt)
            st["dout"] = randn(R, D).to(dt)
            st["dresidual_out"] = None if case["res"] == "none" else randn(R, D).to(rdt)
            # the forward's statistics, which a training step keeps
            s = st["s"].double()
            mean = s.mean(1)
            if case["rms"]:
                mean = torch.zeros_like(mean)
            st["rstd"] = torch.rsqrt((s - mean[:, None]).square().mean(1) + 1e-5).float()
            st["mean"] = None if case["rms"] else mean.float()
        return st
    B, D = case["batch"], case["dim"]
    if case["op"] == "gated_update":
        st["state"] = randn(B, D)
        st["gate"], st["x"] = _gates(case, randn, (B, D), g).to(dt), randn(B, D).to(dt)
        st["gate_bias"] = _gate_bias(case, randn, D, g)
        return st
    L = case["seqlen"]
    if case["op"] in ("gated_fwd", "gated_bwd"):
        shape = (B, L, D) if case["layout"] == "bld" else (B, D, L)
        st["gate"] = _gates(case, randn, shape, g).to(dt)
        st["x"] = randn(*shape).to(dt)
        st["gate_bias"] = _gate_bias(case, randn, D, g)
        st["initial_state"] = randn(B, D) if case["start"] else None
        st["seqlens"] = None
        if case["ragged"]:
            st["seqlens"] = torch.randint(0, L + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        if case["op"] == "gated_bwd":
            st["dout"] = randn(*shape).to(dt)
            st["dlast_state"] = randn(B, D) if case["start"] else None
            st["checkpoints"] = None
            if case["layout"] == "bld":     # the forward's states at block starts, which a training step keeps
                a, b, _ = _terms(st)
                h = _scan(a, b, _start(st))
                h = torch.cat([_start(st)[:, None], h[:, :-1]], dim=1)
                st["checkpoints"] = h[:, ::BLOCK].contiguous()
        return st
    W = case["width"]
    st["x"] = randn(B, D, L).to(dt)
    st["dout"] = randn(B, D, L).to(dt)
    st["weight"] = randn(D, W) / W
    st["bias"] = randn(D) if case["bias"] else None
    st["initial_conv_state"] = randn(B, D, W).to(dt) if case["state"] else None
    st["dfinal_conv_state"] = randn(B, D, W).to(dt) if case["state"] else None
    return st


def _gates(case, randn, shape, g):
    if not case["log_decay"]:
        return randn(*shape)
    # decays of 2 to 1000 steps' memory, and a reset (decay 0) at about one step in 2000
    f = -torch.exp(1.5 * randn(*shape).clamp(-2, 2) - 3.5)
    reset = torch.rand(shape, generator=g, device=DEV) < 1.0 / 2000
    return f.masked_fill(reset, float("-inf"))


def _gate_bias(case, randn, D, g):
    if not case["bias"]:
        return None
    if case["log_decay"]:
        return -0.05 * torch.rand(D, generator=g, device=DEV)
    return randn(D) - 2.0


# ------------------------------------------------------------------------------ plain forms

def _start(st):
    if st["initial_state"] is not None:
        return st["initial_state"]
    return torch.zeros(st["case"]["batch"], st["case"]["dim"], device=DEV)


def _time_second(t, case):
    """(batch, L, dim) in fp32, whatever the layout."""
    t = t.float()
    return t if case["layout"] == "bld" else t.transpose(1, 2)


def _layout_of(t, case, dtype):
    return (t if case["layout"] == "bld" else t.transpose(1, 2)).to(dtype).contiguous()


def _live(st):
    """(batch, L, 1): which steps are inside their sequence; None when all are."""
    if st["seqlens"] is None:
        return None
    t = torch.arange(st["case"]["seqlen"], device=DEV)
    return (t[None, :] < st["seqlens"][:, None])[:, :, None]


def _terms(st):
    """Decay a, input term b and gate g of every step, (batch, L, dim) fp32."""
    case = st["case"]
    f, x = _time_second(st["gate"], case), _time_second(st["x"], case)
    if st["gate_bias"] is not None:
        f = f + st["gate_bias"]
    if case["log_decay"]:
        a, b, g = torch.exp(f), x, None
    else:
        g = 1.0 / (1.0 + torch.exp(-f))
        a, b = 1.0 / (1.0 + torch.exp(f)), g * x
    live = _live(st)
    if live is not None:
        a, b = torch.where(live, a, 1.0), torch.where(live, b, 0.0)
    return a, b, g


def _scan(a, b, h0):
    """h_t = a_t h_{t-1} + b_t along dimension 1, by doubling the reach of each step's pair (a, b)."""
    A, H = a.clone(), b.clone()
    L, d = a.shape[1], 1
    while d < L:
        H[:, d:] += A[:, d:] * H[:, :-d]
        A[:, d:] *= A[:, :-d].clone()
        d *= 2
    return H + A * h0[:, None]


def _plain_norm_fwd(st):
    case = st["case"]
    s = st["x"].float()
    if st["residual"] is not None:
        s = s + st["residual"].float()
    mean = torch.zeros_like(s[:, :1]) if case["rms"] else s.mean(1, keepdim=True)
    c = s - mean
    rstd = 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5)
    y = c * rstd * st["weight"]
    if st["bias"] is not None:
        y = y + st["bias"]
    out = {"out": y.to(st["x"].dtype), "rstd": rstd[:, 0]}
    if not case["rms"]:
        out["mean"] = mean[:, 0]
    if st["residual"] is not None:
        out["residual_out"] = s.to(st["residual"].dtype)
    return out


def _plain_norm_bwd(st):
    case = st["case"]
    s, dy, rstd = st["s"].float(), st["dout"].float(), st["rstd"][:, None]
    xh = (s if case["rms"] else s - st["mean"][:, None]) * rstd
    q = dy * st["weight"]
    c2 = (q * xh).mean(1, keepdim=True)
    ds = q - xh * c2
    if not case["rms"]:
        ds = ds - q.mean(1, keepdim=True)
    ds = ds * rstd
    if st["dresidual_out"] is not None:
        ds = ds + st["dresidual_out"].float()
    out = {"dx": ds.to(st["dout"].dtype), "dweight": (dy * xh).sum(0)}
    if st["bias"] is not None:
        out["dbias"] = dy.sum(0)
    if st["s"].dtype != st["dout"].dtype:
        out["dresidual"] = ds.to(st["s"].dtype)
    return out


def _plain_gated_fwd(st):
    case = st["case"]
    a, b, _ = _terms(st)
    h = _scan(a, b, _start(st))
    last = h[:, -1].contiguous()
    live = _live(st)
    if live is not None:
        h = torch.where(live, h, 0.0)
    return {"out": _layout_of(h, case, st["x"].dtype), "last_state": last}


def _plain_gated_bwd(st):
    case = st["case"]
    a, b, g = _terms(st)
    h0 = _start(st)
    h = _scan(a, b, h0)
    before = torch.cat([h0[:, None], h[:, :-1]], dim=1)
    dout, x = _time_second(st["dout"], case), _time_second(st["x"], case)
    live = _live(st)
    if live is not None:
        dout = torch.where(live, dout, 0.0)
    # lambda_t = dout_t + a_{t+1} lambda_{t+1}: the same scan backwards in time
    nxt = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], dim=1)
    end = st["dlast_state"] if st["dlast_state"] is not None else torch.zeros_like(h0)
    lam = _scan(nxt.flip(1), dout.flip(1), end).flip(1)
    if case["log_decay"]:
        dx, df = lam, lam * a * before
    else:
        dx, df = lam * g, lam * (x - before) * g * a
    if live is not None:
        dx, df = torch.where(live, dx, 0.0), torch.where(live, df, 0.0)
    out = {"dgate": _layout_of(df, case, st["x"].dtype), "dx": _layout_of(dx, case, st["x"].dtype)}
    if st["gate_bias"] is not None:
        out["dgate_bias"] = df.sum((0, 1))
    if st["initial_state"] is not None:
        out["dinitial_state"] = a[:, 0] * lam[:, 0]
    return out


def _plain_gated_update(st):
    f, x = st["gate"].float(), st["x"].float()
    if st["gate_bias"] is not None:
        f = f + st["gate_bias"]
    if st["case"]["log_decay"]:
        h = torch.exp(f) * st["state"] + x
    else:
        h = st["state"] / (1.0 + torch.exp(f)) + x / (1.0 + torch.exp(-f))
    st["state"].copy_(h)
    return {"out": h.to(st["x"].dtype), "state": st["state"]}


def _plain_conv_bwd(st):
    case = st["case"]
    W, L = case["width"], case["seqlen"]
    x, dout, w = st["x"].float(), st["dout"].float(), st["weight"]
    before = st["initial_conv_state"]
    before = torch.zeros_like(x[:, :, :1]).expand(-1, -1, W) if before is None else before.float()
    xp = torch.cat([before, x], dim=2)                      # x_t at index t + W
    dpre = dout
    if case["silu"]:
        pre = sum(w[:, k, None] * xp[:, :, 1 + k:1 + k + L] for k in range(W))
        if st["bias"] is not None:
            pre = pre + st["bias"][:, None]
        sg = 1.0 / (1.0 + torch.exp(-pre))
        dpre = dout * (sg + pre * sg * (1.0 - sg))
    dxp = torch.zeros_like(xp)
    for k in range(W):
        dxp[:, :, 1 + k:1 + k + L] += w[:, k, None] * dpre
    if st["dfinal_conv_state"] is not None:                 # the final state is the last W of xp
        dxp[:, :, L:] += st["dfinal_conv_state"].float()
    out = {"dx": dxp[:, :, W:].to(st["x"].dtype),
           "dweight": torch.stack([(dpre * xp[:, :, 1 + k:1 + k + L]).sum((0, 2)) for k in range(W)], 1)}
    if st["bias"] is not None:
        out["dbias"] = dpre.sum((0, 2))
    if st["initial_conv_state"] is not None:
        out["dinitial_conv_state"] = dxp[:, :, :W].to(st["x"].dtype)
    return out


# ------------------------------------------------------------------------------ the framework's calls

def _own(st):
    from selective_state_space_55_b200 import ops

    case = st["case"]
    op = case["op"]
    if op == "norm_fwd":
        r = ops.layer_norm_fwd(st["x"], weight=st["weight"], bias=st["bias"],
                               residual=st["residual"], eps=1e-5, rms=case["rms"],
                               return_stats=True)
        out = {"out": r[0], "rstd": r[-1]}
        if not case["rms"]:
            out["mean"] = r[-2]
        if st["residual"] is not None:
            out["residual_out"] = r[1]
        return out
    if op == "norm_bwd":
        return ops.layer_norm_bwd(st["dout"], st["s"], st["rstd"], mean=st["mean"],
                                  weight=st["weight"], bias=st["bias"],
                                  dresidual_out=st["dresidual_out"], rms=case["rms"])
    if op == "gated_fwd":
        out, last = ops.gated_scan_fwd(st["gate"], st["x"], gate_bias=st["gate_bias"],
                                       initial_state=st["initial_state"], seqlens=st["seqlens"],
                                       log_decay=case["log_decay"], return_last_state=True,
                                       layout=case["layout"])
        return {"out": out, "last_state": last}
    if op == "gated_bwd":
        return ops.gated_scan_bwd(st["gate"], st["x"], st["dout"], gate_bias=st["gate_bias"],
                                  initial_state=st["initial_state"], seqlens=st["seqlens"],
                                  dlast_state=st["dlast_state"], checkpoints=st["checkpoints"],
                                  log_decay=case["log_decay"], layout=case["layout"])
    if op == "gated_update":
        out = ops.gated_state_update(st["state"], st["gate"], st["x"], gate_bias=st["gate_bias"],
                                     log_decay=case["log_decay"])
        return {"out": out, "state": st["state"]}
    return ops.causal_conv1d_bwd(st["x"], st["weight"], st["dout"], bias=st["bias"],
                                 initial_conv_state=st["initial_conv_state"],
                                 dfinal_conv_state=st["dfinal_conv_state"], silu=case["silu"])


_PLAIN = {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "gated_fwd": _plain_gated_fwd,
          "gated_bwd": _plain_gated_bwd, "gated_update": _plain_gated_update,
          "conv_bwd": _plain_conv_bwd}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------------------ floors

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        R, D = case["rows"], case["dim"]
        r = 4 if case["res"] == "fp32" else e
        params = 4 * D * (1 + case["bias"])
        stats = 4 * R * (1 if case["rms"] else 2)
        if op == "norm_fwd":        # x, out, and with a residual its read and the sum's write
            per = 2 * e + (0 if case["res"] == "none" else 2 * r)
            return {"bytes": R * D * per + params + stats, "flops": 8 * R * D}
        per = 2 * e + r             # dout, dx, s; the residual's gradient in (and out, when its type differs)
        per += 0 if case["res"] == "none" else r
        per += r if r != e else 0
        return {"bytes": R * D * per + 2 * params - (4 * D if case["bias"] else 0) + stats,
                "flops": 14 * R * D}
    n = case["batch"] * case["dim"]
    if op == "gated_update":
        return {"bytes": n * (8 + 3 * e) + (4 * case["dim"] if case["bias"] else 0), "flops": 8 * n}
    L = case["seqlen"]
    if op == "gated_fwd":
        return {"bytes": 3 * e * n * L + 4 * n * (1 + case["start"]) +
                (4 * case["dim"] if case["bias"] else 0), "flops": 8 * n * L}
    if op == "gated_bwd":
        kept = -(-L // BLOCK) if case["layout"] == "bld" else 0
        return {"bytes": 5 * e * n * L + 4 * n * (kept + 3 * case["start"]) +
                (8 * case["dim"] if case["bias"] else 0), "flops": 16 * n * L}
    W = case["width"]
    state = 3 * e * n * W if case["state"] else 0
    return {"bytes": 3 * e * n * L + state + 8 * case["dim"] * (W + case["bias"]),
            "flops": (6 * W + (10 if case["silu"] else 0)) * n * L}


# ------------------------------------------------------------------------------ 64-bit definitions

def _exact_norm_fwd(st):
    case = st["case"]
    s = st["x"].double()
    if st["residual"] is not None:
        s = s + st["residual"].double()
    D = s.shape[1]
    mean = s.sum(1) / D * (0.0 if case["rms"] else 1.0)
    var = ((s - mean[:, None]) ** 2).sum(1) / D
    rstd = (var + 1e-5) ** -0.5
    y = (s - mean[:, None]) * (rstd[:, None] * st["weight"].double())
    if st["bias"] is not None:
        y = y + st["bias"].double()
    out = {"out": y, "rstd": rstd}
    if not case["rms"]:
        out["mean"] = mean
    if st["residual"] is not None:
        out["residual_out"] = s
    return out


def _exact_norm_bwd(st):
    """The derivative of the 64-bit forward, rows in slices."""
    case = st["case"]
    R, D = st["s"].shape
    w = st["weight"].double().requires_grad_()
    b = torch.zeros(D, dtype=torch.float64, device=DEV, requires_grad=True)
    dw, db, ds = torch.zeros_like(w), torch.zeros_like(b), []
    step = max(1, (1 << 24) // D)
    for r in range(0, R, step):
        s = st["s"][r:r + step].double().requires_grad_()
        c = s if case["rms"] else s - s.mean(1, keepdim=True)
        y = c * (c.square().mean(1, keepdim=True) + 1e-5).rsqrt() * w + b
        gs, gw, gb = torch.autograd.grad(y, (s, w, b), st["dout"][r:r + step].double())
        if st["dresidual_out"] is not None:
            gs = gs + st["dresidual_out"][r:r + step].double()
        ds.append(gs)
        dw, db = dw + gw, db + gb
    ds = torch.cat(ds)
    out = {"dx": ds, "dweight": dw.detach()}
    if st["bias"] is not None:
        out["dbias"] = db.detach()
    if st["s"].dtype != st["dout"].dtype:
        out["dresidual"] = ds
    return out


def _exact_steps(st):
    """Per-step tensors with time first, (L, batch, dim) in 64 bits, and the lengths."""
    case = st["case"]
    order = (1, 0, 2) if case["layout"] == "bld" else (2, 0, 1)
    f = st["gate"].permute(order).double().contiguous()
    x = st["x"].permute(order).double().contiguous()
    if st["gate_bias"] is not None:
        f = f + st["gate_bias"].double()
    L, B = f.shape[:2]
    n = st["seqlens"].long() if st["seqlens"] is not None else torch.full((B,), L, device=DEV)
    return f, x, n.clamp(0, L), order


def _back(order):
    return (1, 0, 2) if order == (1, 0, 2) else (1, 2, 0)


def _exact_gated_forward(st):
    f, x, n, order = _exact_steps(st)
    log_decay = st["case"]["log_decay"]
    a = torch.exp(f) if log_decay else torch.sigmoid(-f)
    u = x if log_decay else torch.sigmoid(f) * x
    L = f.shape[0]
    inside = (torch.arange(L, device=DEV)[:, None] < n[None, :])[:, :, None]
    whole = bool((n == L).all())
    h = _start(st).double()
    hs = torch.empty_like(f)
    for t in range(L):
        new = torch.addcmul(u[t], a[t], h)
        h = new if whole else torch.where(inside[t], new, h)
        hs[t] = h
    return f, x, a, hs, h, inside, order


def _exact_gated_fwd(st):
    _, _, _, hs, h, inside, order = _exact_gated_forward(st)
    out = torch.where(inside, hs, 0.0).permute(_back(order)).contiguous()
    return {"out": out, "last_state": h}


def _exact_gated_bwd(st):
    f, x, a, hs, _, inside, order = _exact_gated_forward(st)
    log_decay = st["case"]["log_decay"]
    dout = torch.where(inside, st["dout"].permute(order).double(), 0.0)
    a = torch.where(inside, a, 1.0)
    # dLoss/dh_t, from the last step to the first
    lam = torch.zeros_like(f)
    nxt = st["dlast_state"].double() if st["dlast_state"] is not None else torch.zeros_like(f[0])
    for t in range(f.shape[0] - 1, -1, -1):
        lam[t] = dout[t] + nxt
        nxt = a[t] * lam[t]
    before = torch.cat([_start(st).double()[None], hs[:-1]])
    if log_decay:
        dx, da = lam, lam * before
        df = da * a
    else:
        g = torch.sigmoid(f)
        dx = lam * g
        df = lam * (x - before) * (g * torch.sigmoid(-f))
    dx, df = torch.where(inside, dx, 0.0), torch.where(inside, df, 0.0)
    out = {"dgate": df.permute(_back(order)).contiguous(), "dx": dx.permute(_back(order)).contiguous()}
    if st["gate_bias"] is not None:
        out["dgate_bias"] = df.sum((0, 1))
    if st["initial_state"] is not None:
        out["dinitial_state"] = nxt
    return out


def _exact_gated_update(st):
    f = st["gate"].double()
    if st["gate_bias"] is not None:
        f = f + st["gate_bias"].double()
    if st["case"]["log_decay"]:
        h = torch.exp(f) * st["state"].double() + st["x"].double()
    else:
        h = torch.sigmoid(-f) * st["state"].double() + torch.sigmoid(f) * st["x"].double()
    return {"out": h, "state": h}


def _exact_conv_bwd(st):
    """The derivative of the 64-bit convolution, one batch row at a time."""
    case = st["case"]
    B, D, W, L = case["batch"], case["dim"], case["width"], case["seqlen"]
    w = st["weight"].double().requires_grad_()
    b = torch.zeros(D, dtype=torch.float64, device=DEV)
    b = (b if st["bias"] is None else b + st["bias"].double()).requires_grad_()
    dw, db, dx, dinit = torch.zeros_like(w), torch.zeros_like(b), [], []
    for i in range(B):
        x = st["x"][i].double().requires_grad_()
        init = st["initial_conv_state"]
        init = torch.zeros(D, W, dtype=torch.float64, device=DEV) if init is None else init[i].double()
        init = init.requires_grad_()
        seq = torch.cat([init, x], 1)
        taps = torch.stack([seq[:, 1 + k:1 + k + L] for k in range(W)], 2)      # (D, L, W)
        y = (taps * w[:, None, :]).sum(2) + b[:, None]
        if case["silu"]:
            y = y * torch.sigmoid(y)
        total = (y * st["dout"][i].double()).sum()
        if st["dfinal_conv_state"] is not None:
            total = total + (seq[:, L:] * st["dfinal_conv_state"][i].double()).sum()
        gx, gi, gw, gb = torch.autograd.grad(total, (x, init, w, b), allow_unused=True)
        dx.append(gx)
        dinit.append(gi if gi is not None else torch.zeros_like(init))
        dw, db = dw + gw, db + gb
    out = {"dx": torch.stack(dx), "dweight": dw.detach()}
    if st["bias"] is not None:
        out["dbias"] = db.detach()
    if st["initial_conv_state"] is not None:
        out["dinitial_conv_state"] = torch.stack(dinit)
    return out


_EXACT = {"norm_fwd": _exact_norm_fwd, "norm_bwd": _exact_norm_bwd, "gated_fwd": _exact_gated_fwd,
          "gated_bwd": _exact_gated_bwd, "gated_update": _exact_gated_update,
          "conv_bwd": _exact_conv_bwd}


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))
