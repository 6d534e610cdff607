"""The block operators together, as a recurrent block uses them: layer norm with the residual
add, projection, short convolution, gated recurrence, projection; trained and served.

Reference: the same block in 64 bits on the CPU, its gradients by torch's autograd.
Tolerance: every operator and fp32 product is good to about 1e-5 of the magnitudes that
enter it (a product over 192 columns: 192 * 2^-24 = 1.1e-5), and some ten of them follow one
another: 2e-4 of each result's largest magnitude.
"""
import pytest
import torch

from selective_state_space_55_b200 import ops

pytestmark = pytest.mark.gpu

DEV = "cuda"
B, L, M, D, W = 3, 90, 64, 96, 4          # batch, steps, model width, channels, taps
TOL = 2e-4


def params(seed):
    g = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(norm_w=1 + 0.1 * randn(M), norm_b=0.1 * randn(M), w_in=randn(M, 2 * D) / M ** 0.5,
                conv_w=randn(D, W) / 2, conv_b=0.1 * randn(D), gate_b=randn(D) - 1,
                w_out=randn(D, M) / D ** 0.5, x=randn(B, L, M), res=randn(B, L, M),
                dy=randn(B, L, M), ds=randn(B, L, M))


def reference(p):
    q = {k: v.double().requires_grad_(k not in ("dy", "ds")) for k, v in p.items()}
    s = q["x"] + q["res"]
    c = s - s.mean(-1, keepdim=True)
    y = c * (c.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * q["norm_w"] + q["norm_b"]
    gate, u = (y @ q["w_in"]).split(D, -1)
    up = torch.cat([torch.zeros(B, W - 1, D, dtype=torch.float64), u], 1)
    pre = q["conv_b"] + sum(q["conv_w"][:, k] * up[:, k:k + L] for k in range(W))
    v = pre * torch.sigmoid(pre)
    a, g = torch.sigmoid(-(gate + q["gate_b"])), torch.sigmoid(gate + q["gate_b"])
    h, hs = torch.zeros(B, D, dtype=torch.float64), []
    for t in range(L):
        h = a[:, t] * h + g[:, t] * v[:, t]
        hs.append(h)
    out = torch.stack(hs, 1) @ q["w_out"]
    ((out * q["dy"]).sum() + (s * q["ds"]).sum()).backward()
    return out.detach(), h.detach(), {k: t.grad for k, t in q.items() if t.requires_grad}


def close(name, got, want):
    err = (got.double().cpu() - want).abs().max().item()
    assert err <= TOL * want.abs().max().item(), f"{name}: {err}"


@pytest.mark.parametrize("layout", ["bdl", "bld"])
def test_training_step(layout):
    p = params(1)
    out, _, grads = reference(p)
    c = {k: v.to(DEV) for k, v in p.items()}
    y, s, mean, rstd = ops.layer_norm_fwd(c["x"], c["norm_w"], c["norm_b"], residual=c["res"], return_stats=True)
    proj = y @ c["w_in"]
    u = proj[..., D:].transpose(1, 2).contiguous()
    v = ops.causal_conv1d_fwd(u, c["conv_w"], bias=c["conv_b"])
    lay = (lambda t: t) if layout == "bdl" else (lambda t: t.transpose(1, 2).contiguous())
    gate = proj[..., :D] if layout == "bld" else proj[..., :D].transpose(1, 2).contiguous()
    h = ops.gated_scan_fwd(gate, lay(v), c["gate_b"], layout=layout, return_checkpoints=layout == "bld")
    h, ck = h if layout == "bld" else (h, None)
    ht = h if layout == "bld" else h.transpose(1, 2)
    close("out", ht @ c["w_out"], out)

    g = {"w_out": ht.reshape(-1, D).T @ c["dy"].reshape(-1, M)}
    dh = c["dy"] @ c["w_out"].T
    dproj = torch.empty_like(proj)
    if layout == "bld":
        gs = ops.gated_scan_bwd(gate, lay(v), dh, c["gate_b"], checkpoints=ck, dgate=dproj[..., :D], layout="bld")
        dv = gs["dx"].transpose(1, 2).contiguous()
    else:
        gs = ops.gated_scan_bwd(gate, v, dh.transpose(1, 2).contiguous(), c["gate_b"])
        dproj[..., :D] = gs["dgate"].transpose(1, 2)
        dv = gs["dx"]
    gc = ops.causal_conv1d_bwd(u, c["conv_w"], dv, bias=c["conv_b"])
    dproj[..., D:] = gc["dx"].transpose(1, 2)
    g.update(gate_b=gs["dgate_bias"], conv_w=gc["dweight"], conv_b=gc["dbias"],
             w_in=y.reshape(-1, M).T @ dproj.reshape(-1, 2 * D))
    gn = ops.layer_norm_bwd(dproj @ c["w_in"].T, s, rstd, mean=mean, weight=c["norm_w"], bias=c["norm_b"],
                            dresidual_out=c["ds"])
    g.update(norm_w=gn["dweight"], norm_b=gn["dbias"], x=gn["dx"], res=gn["dx"])
    for k in grads:
        close(k, g[k], grads[k])


def test_prefill_then_tokens():
    """30 steps at once, then the rest one by one, equals the whole sequence."""
    p = params(2)
    out, last, _ = reference(p)
    c = {k: v.to(DEV) for k, v in p.items()}
    T = 30
    y, _ = ops.layer_norm_fwd(c["x"][:, :T].contiguous(), c["norm_w"], c["norm_b"],
                              residual=c["res"][:, :T].contiguous())
    proj = y @ c["w_in"]
    u = proj[..., D:].transpose(1, 2).contiguous()
    v, conv_state = ops.causal_conv1d_fwd(u, c["conv_w"], bias=c["conv_b"], return_final_state=True)
    h, state = ops.gated_scan_fwd(proj[..., :D], v.transpose(1, 2).contiguous(), c["gate_b"],
                                  return_last_state=True, layout="bld")
    outs = [h @ c["w_out"]]
    for t in range(T, L):
        y, _ = ops.layer_norm_fwd(c["x"][:, t], c["norm_w"], c["norm_b"], residual=c["res"][:, t])
        proj = y @ c["w_in"]
        v = ops.causal_conv1d_update(conv_state, proj[:, D:].contiguous(), c["conv_w"], bias=c["conv_b"])
        outs.append((ops.gated_state_update(state, proj[:, :D], v, c["gate_b"]) @ c["w_out"])[:, None])
    close("out", torch.cat(outs, 1), out)
    close("state", state, last)


def test_refusals():
    """What the operators do not take is refused before anything is launched."""
    f32 = torch.zeros(4, 6, 64, device=DEV)
    bf = f32.bfloat16()
    row, state = f32[0, 0], torch.zeros(4, 64, device=DEV)
    stats = torch.ones(4, 6, device=DEV)
    taps = torch.zeros(6, 4, device=DEV)
    bad = [
        lambda: ops.layer_norm_fwd(f32.cpu()),
        lambda: ops.layer_norm_fwd(f32.half()),
        lambda: ops.layer_norm_fwd(row.expand(6, 64)),                      # rows that overlap
        lambda: ops.layer_norm_fwd(f32.transpose(1, 2)),                    # last dimension not contiguous
        lambda: ops.layer_norm_fwd(f32, weight=row.bfloat16()),
        lambda: ops.layer_norm_fwd(f32, weight=row[:63]),
        lambda: ops.layer_norm_fwd(f32, residual=bf),                       # fp32 rows, bf16 residual
        lambda: ops.layer_norm_fwd(f32, eps=-1.0),
        lambda: ops.layer_norm_fwd(f32, residual=f32.clone(), residual_out=f32),
        lambda: ops.layer_norm_bwd(f32, f32, stats),                        # mean missing
        lambda: ops.layer_norm_bwd(f32, f32, stats[:3], mean=stats),
        lambda: ops.layer_norm_bwd(bf, f32, stats, mean=stats, dresidual_out=bf),
        lambda: ops.layer_norm_bwd(f32, f32, stats, mean=stats, weight=row,
                                   workspace=torch.empty(16, dtype=torch.uint8, device=DEV)),
        lambda: ops.gated_scan_fwd(f32, bf),
        lambda: ops.gated_scan_fwd(f32, f32[:, :5]),
        lambda: ops.gated_scan_fwd(f32, f32, layout="dbl"),
        lambda: ops.gated_scan_fwd(f32[0], f32[0]),
        lambda: ops.gated_scan_fwd(f32, f32, out=f32),
        lambda: ops.gated_scan_fwd(f32, f32[0].expand(4, 6, 64)),           # one batch row for all
        lambda: ops.gated_scan_fwd(f32, f32, out=f32[:1].clone().expand(4, 6, 64)),
        lambda: ops.gated_scan_fwd(f32, f32, return_checkpoints=True),      # layout "bdl"
        lambda: ops.gated_scan_fwd(f32, f32, seqlens=torch.ones(4, dtype=torch.int64, device=DEV)),
        lambda: ops.gated_scan_fwd(f32, f32, flags=1 << 20),
        lambda: ops.gated_scan_bwd(f32, f32, f32.clone(), dx=f32),
        lambda: ops.gated_scan_bwd(f32, f32, f32.clone(), checkpoints=state),
        lambda: ops.gated_state_update(state.bfloat16(), bf[:, 0], bf[:, 0]),
        lambda: ops.gated_state_update(state[:, :63], f32[:, 0], f32[:, 0]),
        lambda: ops.gated_state_update(state, f32[:, 0], bf[:, 0]),
        lambda: ops.causal_conv1d_bwd(f32, taps, bf),
        lambda: ops.causal_conv1d_bwd(f32, taps.new_zeros(6, 5), f32.clone()),
        lambda: ops.causal_conv1d_bwd(f32.transpose(1, 2), taps.new_zeros(64, 4), f32.transpose(1, 2)),
        lambda: ops.causal_conv1d_bwd(f32, taps, f32[:, :5]),
    ]
    for i, call in enumerate(bad):
        try:
            call()
        except (ValueError, RuntimeError):
            continue
        pytest.fail(f"call {i} was not refused")
    torch.cuda.synchronize()
    assert ops.device_status() == 0
