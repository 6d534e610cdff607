"""Gated linear recurrence (forward, backward, one token) against its 64-bit form."""
import ctypes
import time

import pytest
import torch

import block_reference as ref
from block_reference import assert_close
from selective_state_space_55_b200 import ops

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def make(batch, dim, L, layout, dtype, log_decay, seed, bias=True, start=True, ragged=False):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    shape = (batch, L, dim) if layout == "bld" else (batch, dim, L)
    gate = randn(*shape)
    if log_decay:
        gate = -torch.exp(1.5 * gate - 3.0)
        gate[torch.rand(shape, generator=g, device=DEV) < 0.01] = float("-inf")    # resets
    v = dict(gate=gate.to(dtype), x=randn(*shape).to(dtype),
             gate_bias=(-0.05 * randn(dim).abs() if log_decay else randn(dim)) if bias else None,
             initial_state=randn(batch, dim) if start else None, seqlens=None)
    if ragged:
        n = torch.randint(0, L + 1, (batch,), generator=g, device=DEV, dtype=torch.int32)
        n[0] = 0
        v["seqlens"] = n
    back = dict(dout=randn(*shape).to(dtype), dlast_state=randn(batch, dim) if start else None)
    return v, back


def check(v, back, layout, log_decay, checkpoints="given", fwd_kw=None, bwd_kw=None):
    want = ref.gated(**v, log_decay=log_decay, layout=layout, **back)
    got = ops.gated_scan_fwd(**v, log_decay=log_decay, layout=layout, return_last_state=True,
                             return_checkpoints=layout == "bld", **(fwd_kw or {}))
    ck = None
    if layout == "bld":
        assert_close("checkpoints", got[2], *want["checkpoints"])
        ck = got[2] if checkpoints == "given" else None
    grads = ops.gated_scan_bwd(**v, **back, checkpoints=ck, log_decay=log_decay, layout=layout,
                               **(bwd_kw or {}))
    assert ops.device_status() == 0
    assert_close("out", got[0], *want["out"])
    assert_close("last_state", got[1], *want["last_state"])
    for name in grads:
        assert_close(name, grads[name], *want[name])
    assert ("dgate_bias" in grads) == (v["gate_bias"] is not None)
    assert ("dinitial_state" in grads) == (v["initial_state"] is not None)
    return got, grads


@pytest.mark.parametrize("L", [1, 7, 8, 63, 64, 65, 200, 511, 512, 513, 1003])
@pytest.mark.parametrize("log_decay", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["bld", "bdl"])
def test_lengths(layout, dtype, log_decay, L):
    v, back = make(3, 70, L, layout, dtype, log_decay, seed=L)
    check(v, back, layout, log_decay)


@pytest.mark.parametrize("dim", [1, 2, 3, 63, 64, 65, 129, 256])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["bld", "bdl"])
def test_channel_counts(layout, dtype, dim):
    v, back = make(2, dim, 150, layout, dtype, False, seed=dim)
    check(v, back, layout, False)


@pytest.mark.parametrize("L", [255, 256, 257, 505, 512, 1024, 1030, 2041, 2048, 2049, 4100])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_layout_tile_borders(dtype, L):
    """1, 2, 4 and 8 warps per chain, one tile and several, aligned and shifted rows."""
    v, back = make(2, 5, L, "bdl", dtype, True, seed=L)
    check(v, back, "bdl", True)


@pytest.mark.parametrize("log_decay", [False, True])
@pytest.mark.parametrize("layout", ["bld", "bdl"])
def test_many_tiles(layout, log_decay):
    """20,000 steps: 40 segments in two join groups (10 tiles in the rows layout)."""
    v, back = make(1, 66, 20000, layout, BF, log_decay, seed=5)
    check(v, back, layout, log_decay)


def test_more_segments_than_the_gpu_holds():
    """CTAs work through several segments, chains in all stages at once."""
    v, back = make(6, 2100, 2100, "bld", BF, False, seed=6)
    check(v, back, "bld", False)


@pytest.mark.parametrize("checkpoints", ["given", "recomputed"])
@pytest.mark.parametrize("bias,start", [(True, False), (False, True), (False, False)])
def test_options(bias, start, checkpoints):
    v, back = make(2, 130, 300, "bld", BF, False, seed=7, bias=bias, start=start)
    check(v, back, "bld", False, checkpoints)
    v, back = make(2, 33, 300, "bdl", BF, False, seed=7, bias=bias, start=start)
    check(v, back, "bdl", False, checkpoints)


@pytest.mark.parametrize("L", [50, 64, 333, 2500])
@pytest.mark.parametrize("log_decay", [False, True])
@pytest.mark.parametrize("layout", ["bld", "bdl"])
def test_padded_batch(layout, log_decay, L):
    """Lengths from 0 to L; NaN and infinity in the padding change nothing, outputs there are 0."""
    v, back = make(6, 40, L, layout, BF, log_decay, seed=L, ragged=True)
    outside = (torch.arange(L, device=DEV)[None] >= v["seqlens"][:, None])
    outside = outside[:, :, None] if layout == "bld" else outside[:, None, :]
    for t, bad in ((v["gate"], float("nan")), (v["x"], float("inf")), (back["dout"], float("nan"))):
        t.copy_(torch.where(outside, torch.full_like(t, bad), t))
    got, grads = check(v, back, layout, log_decay)
    for t in (got[0], grads["dgate"], grads["dx"]):
        assert (torch.where(outside, t, torch.zeros_like(t)) == 0).all()
    assert torch.equal(got[1][0], v["initial_state"][0])          # a row of length 0


def test_lengths_beyond_the_batch_are_clamped():
    v, back = make(3, 40, 90, "bld", BF, False, seed=8)
    v["seqlens"] = torch.tensor([-5, 1000, 90], dtype=torch.int32, device=DEV)
    check(v, back, "bld", False)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["bld", "bdl"])
@pytest.mark.parametrize("dim,L", [(48, 100), (51, 101)])
def test_strided_and_shifted_views(layout, dtype, dim, L):
    """gate and x as halves of one projection's output, gradients into halves of another;
    then every tensor at its own element offset."""
    v, back = make(2, dim, L, layout, dtype, False, seed=9)
    inner = v["gate"].shape[-1]
    both = torch.cat([v["gate"], v["x"]], dim=-1)
    dboth = torch.full_like(both, 7.0)
    v2 = dict(v, gate=both[..., :inner], x=both[..., inner:])
    _, g = check(v2, back, layout, False,
                 bwd_kw=dict(dgate=dboth[..., :inner], dx=dboth[..., inner:]))
    assert torch.equal(dboth[..., :inner], g["dgate"])

    def at(t, offset):
        if t is None:
            return None
        buf = torch.empty(t.numel() + offset, dtype=t.dtype, device=DEV)
        w = buf[offset:].view(t.shape)
        w.copy_(t)
        return w

    v3 = {k: at(t, i + 1) for i, (k, t) in enumerate(v.items())}
    b3 = {k: at(t, i + 2) for i, (k, t) in enumerate(back.items())}
    check(v3, b3, layout, False, fwd_kw=dict(out=at(v["x"], 5)),
          bwd_kw=dict(dgate=at(v["x"], 3), dx=at(v["x"], 6)))


def test_time_major_batch():
    """(L, batch, dim) in memory, seen as (batch, L, dim)."""
    v, back = make(3, 64, 130, "bld", BF, False, seed=10)
    tm = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    v["gate"], v["x"], back["dout"] = tm(v["gate"]), tm(v["x"]), tm(back["dout"])
    out = tm(torch.zeros_like(v["x"]))
    got, _ = check(v, back, "bld", False, fwd_kw=dict(out=out))
    assert got[0] is out


def test_gaps_between_rows_stay_untouched():
    v, back = make(2, 64, 70, "bld", BF, False, seed=11)
    wide = torch.full((2, 70, 96), 3.0, dtype=BF, device=DEV)
    ops.gated_scan_fwd(**v, layout="bld", out=wide[..., 16:80])
    torch.cuda.synchronize()
    assert (wide[..., :16] == 3.0).all() and (wide[..., 80:] == 3.0).all()


@pytest.mark.parametrize("layout", ["bld", "bdl"])
def test_empty_sequence_and_batch(layout):
    shape = (2, 0, 5) if layout == "bld" else (2, 5, 0)
    z = torch.zeros(shape, device=DEV)
    h0, dl = torch.randn(2, 5, device=DEV), torch.randn(2, 5, device=DEV)
    bias = torch.randn(5, device=DEV)
    out, last = ops.gated_scan_fwd(z, z, initial_state=h0, return_last_state=True, layout=layout)
    assert out.shape == shape and torch.equal(last, h0)
    _, last = ops.gated_scan_fwd(z, z, return_last_state=True, layout=layout)
    assert (last == 0).all()
    g = ops.gated_scan_bwd(z, z, z, gate_bias=bias, initial_state=h0, dlast_state=dl, layout=layout)
    assert torch.equal(g["dinitial_state"], dl) and (g["dgate_bias"] == 0).all()
    e = torch.zeros((0, 4, 5), device=DEV)
    g = ops.gated_scan_bwd(e, e, e, gate_bias=bias[:5 if layout == "bld" else 4], layout=layout)
    assert (g["dgate_bias"] == 0).all()


def test_state_in_place_and_pieces():
    """last_state into initial_state's buffer; two pieces equal one call to the bound."""
    v, _ = make(2, 96, 300, "bld", F32, False, seed=12)
    want = ref.gated(**v, layout="bld")
    state = v["initial_state"].clone()
    first = ops.gated_scan_fwd(v["gate"][:, :130], v["x"][:, :130], v["gate_bias"],
                               initial_state=state, last_state=state, layout="bld")
    second = ops.gated_scan_fwd(v["gate"][:, 130:], v["x"][:, 130:], v["gate_bias"],
                                initial_state=state, last_state=state, layout="bld")
    assert_close("out", torch.cat([first[0], second[0]], 1), *want["out"])
    assert_close("last", state, *want["last_state"])


@pytest.mark.parametrize("layout", ["bld", "bdl"])
def test_repeats_bit_for_bit(layout):
    v, back = make(2, 200, 5000, layout, BF, False, seed=13)
    runs = []
    for _ in range(3):
        o = ops.gated_scan_fwd(**v, layout=layout)
        runs.append((o, ops.gated_scan_bwd(**v, **back, layout=layout)))
    for o, g in runs[1:]:
        assert torch.equal(o, runs[0][0])
        for k in g:
            assert torch.equal(g[k], runs[0][1][k])


def test_large_decay_products_and_saturated_gates():
    """Gates of +-100 and -inf/+inf: g is exactly 0 or 1, states pass or are replaced."""
    L = 130
    gate = torch.full((1, L, 64), -100.0, device=DEV)
    gate[:, 20] = 100.0
    gate[:, 60] = float("inf")
    gate[:, 61:] = float("-inf")
    x = torch.randn(1, L, 64, device=DEV)
    out = ops.gated_scan_fwd(gate, x, layout="bld")
    torch.testing.assert_close(out[:, 20:60], x[:, 20:21].expand(-1, 40, -1), rtol=0, atol=1e-6)
    assert torch.equal(out[:, 60:], x[:, 60:61].expand(-1, L - 60, -1))


@pytest.mark.parametrize("log_decay", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("batch,dim", [(1, 1), (1, 4096), (3, 7), (5, 64), (128, 4096), (2, 1001)])
def test_update(batch, dim, dtype, log_decay):
    v, _ = make(batch, dim, 1, "bld", dtype, log_decay, seed=dim + batch)
    want = ref.gated(**v, log_decay=log_decay, layout="bld")
    state = v["initial_state"].clone()
    out = ops.gated_state_update(state, v["gate"][:, 0], v["x"][:, 0], v["gate_bias"], log_decay=log_decay)
    assert_close("out", out, want["out"][0][:, 0], want["out"][1][:, 0])
    assert_close("state", state, *want["last_state"])


def test_update_strided_and_in_place():
    v, _ = make(6, 128, 1, "bld", BF, False, seed=14, bias=False)
    want = ref.gated(**v, layout="bld")
    both = torch.cat([v["gate"][:, 0], v["x"][:, 0]], -1)
    gate, x = both[:, :128], both[:, 128:]
    state = v["initial_state"].clone()
    ops.gated_state_update(state, gate, x, out=x)
    assert_close("out", x, want["out"][0][:, 0], want["out"][1][:, 0])
    assert torch.equal(both[:, :128], v["gate"][:, 0])


def test_updates_continue_a_scan():
    v, _ = make(4, 96, 40, "bld", BF, False, seed=15)
    want = ref.gated(**v, layout="bld")
    _, state = ops.gated_scan_fwd(v["gate"][:, :30], v["x"][:, :30], v["gate_bias"],
                                  initial_state=v["initial_state"], return_last_state=True, layout="bld")
    outs = [ops.gated_state_update(state, v["gate"][:, t], v["x"][:, t], v["gate_bias"]) for t in range(30, 40)]
    assert_close("out", torch.stack(outs, 1), want["out"][0][:, 30:], want["out"][1][:, 30:])
    assert_close("state", state, *want["last_state"])


def test_gradients_match_differences():
    """Central differences of the 64-bit forward agree with its 64-bit gradients, and those
    with the kernel's: a slip shared by formula and kernel would show in the first."""
    v, back = make(1, 3, 9, "bld", F32, False, seed=16)
    want = ref.gated(**v, layout="bld", **back)
    _, g = check(v, back, "bld", False)

    def loss(w):
        o = ref.gated(**w, layout="bld")
        return ((o["out"][0] * back["dout"].double().cpu()).sum()
                + (o["last_state"][0] * back["dlast_state"].double().cpu()).sum())

    for name, grad in (("gate", "dgate"), ("x", "dx"), ("gate_bias", "dgate_bias"),
                       ("initial_state", "dinitial_state")):
        for i in range(v[name].numel()):
            step = torch.zeros(v[name].numel(), dtype=torch.float64)
            step[i] = 1e-5
            base = v[name].double().cpu()
            d = (loss({**v, name: base + step.view(base.shape)})
                 - loss({**v, name: base - step.view(base.shape)})) / 2e-5
            assert abs(d - want[grad][0].flatten()[i]) <= 1e-8 * (1 + abs(d)), (name, i)


def test_two_streams_at_once():
    """Two calls side by side, each with its own workspace, on streams of their own."""
    a, ab = make(2, 512, 1000, "bld", BF, False, seed=17)
    b, bb = make(2, 512, 1000, "bld", BF, True, seed=18)
    wa, wb = (ref.gated(**v, layout="bld", log_decay=ld, **k) for v, ld, k in ((a, False, ab), (b, True, bb)))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    results = []
    for _ in range(5):
        results.append((ops.gated_scan_fwd(**a, layout="bld", stream=s1),
                        ops.gated_scan_bwd(**a, **ab, layout="bld", stream=s1),
                        ops.gated_scan_fwd(**b, layout="bld", log_decay=True, stream=s2),
                        ops.gated_scan_bwd(**b, **bb, layout="bld", log_decay=True, stream=s2)))
    torch.cuda.synchronize()
    assert ops.device_status() == 0
    for oa, ga, ob, gb in results:
        assert_close("out a", oa, *wa["out"])
        assert_close("out b", ob, *wb["out"])
        for k in ga:
            assert_close(k, ga[k], *wa[k])
        for k in gb:
            assert_close(k, gb[k], *wb[k])


def test_captured_and_replayed():
    """A captured training step, replayed on new inputs, one workspace for both calls."""
    v, back = make(2, 192, 1500, "bld", BF, False, seed=19)
    ws = torch.empty(32 << 20, dtype=torch.uint8, device=DEV)
    run = lambda: (ops.gated_scan_fwd(**v, layout="bld", return_checkpoints=True, workspace=ws),  # noqa: E731
                   ops.gated_scan_bwd(**v, **back, layout="bld", workspace=ws))
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (out, ck), g = run()
    for seed in (20, 21):
        v2, b2 = make(2, 192, 1500, "bld", BF, False, seed=seed)
        for k in ("gate", "x", "gate_bias", "initial_state"):
            v[k].copy_(v2[k])
        for k in back:
            back[k].copy_(b2[k])
        graph.replay()
        torch.cuda.synchronize()
        want = ref.gated(**v, layout="bld", **back)
        assert_close("out", out, *want["out"])
        assert_close("checkpoints", ck, *want["checkpoints"])
        for k in g:
            assert_close(k, g[k], *want[k])


def test_withheld_handoff_is_reported():
    """Segments that never publish: the waits run out, the call ends and the status says so."""
    v, _ = make(1, 64, 1100, "bld", BF, False, seed=22)
    ops.device_status()
    ops.gated_scan_fwd(**v, layout="bld", flags=ops.MAMBA_FLAG_TEST_WITHHOLD_HANDOFF)
    assert ops.STATUS_NAMES[ops.device_status()] == "MAMBA_ERR_TIMEOUT"
    assert ops.device_status() == 0
    want = ref.gated(**v, layout="bld")
    assert_close("out", ops.gated_scan_fwd(**v, layout="bld"), *want["out"])


@pytest.mark.parametrize("ragged,log_decay", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_plentiful_chains(dtype, ragged, log_decay):
    """(batch, dim, seqlen) with so many pairs of chains that one warp walks a pair's three
    tiles forward; an odd dim leaves pairs with one chain."""
    v, back = make(2, 2961, 701, "bdl", dtype, log_decay, seed=17, ragged=ragged)
    if ragged:
        outside = (torch.arange(701, device=DEV)[None] >= v["seqlens"][:, None])[:, None, :]
        for t in (v["gate"], v["x"], back["dout"]):
            t.copy_(torch.where(outside, torch.full_like(t, float("nan")), t))
    check(v, back, "bdl", log_decay)


@pytest.mark.parametrize("log_decay", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("batch,dim,L", [(1, 64, 7000), (2, 200, 513), (3, 72, 257), (1, 1536, 300), (5, 16, 31)])
def test_few_chains(batch, dim, L, dtype, log_decay):
    """Too few groups for a CTA each, rows on 16-byte boundaries: segments of a chain kept on chip
    while they are joined; 7000 steps are more segments than one join group holds."""
    v, back = make(batch, dim, L, "bld", dtype, log_decay, seed=L + dim)
    check(v, back, "bld", log_decay)


CHAINED = [(4, 2048, 1100), (2, 4160, 700), (130, 64, 70), (3, 2728, 130), (9, 1000, 600),
           (10, 2048, 1100), (5, 4160, 700), (321, 64, 70), (8, 2728, 130), (21, 1000, 600)]


@pytest.mark.parametrize("log_decay", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("batch,dim,L", CHAINED)
def test_many_chains(batch, dim, L, dtype, log_decay):
    """From 192 groups of 64 channels on (bf16 forward: 320) stretches of a chain are handed
    from CTA to CTA; sizes on both sides of that."""
    v, back = make(batch, dim, L, "bld", dtype, log_decay, seed=L)
    check(v, back, "bld", log_decay)


@pytest.mark.parametrize("checkpoints", ["given", "recomputed"])
@pytest.mark.parametrize("L", [1, 63, 65, 577])
@pytest.mark.parametrize("batch", [10, 25])
def test_many_chains_padded(L, checkpoints, batch):
    v, back = make(batch, 840, L, "bld", BF, False, seed=L, ragged=True)
    outside = (torch.arange(L, device=DEV)[None] >= v["seqlens"][:, None])[:, :, None]
    for t, bad in ((v["gate"], float("nan")), (v["x"], float("inf")), (back["dout"], float("nan"))):
        t.copy_(torch.where(outside, torch.full_like(t, bad), t))
    got, grads = check(v, back, "bld", False, checkpoints)
    for t in (got[0], grads["dgate"], grads["dx"]):
        assert (torch.where(outside, t, torch.zeros_like(t)) == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("batch", [4, 11])
def test_many_chains_strided(dtype, batch):
    """Halves of one tensor in and out, time-major memory, neighbours untouched."""
    v, back = make(batch, 2048, 140, "bld", dtype, False, seed=30)
    both = torch.cat([v["gate"], v["x"]], dim=-1)
    dboth = torch.full((batch, 140, 4096 + 16), 7.0, dtype=dtype, device=DEV)
    v2 = dict(v, gate=both[..., :2048], x=both[..., 2048:])
    _, g = check(v2, back, "bld", False,
                 bwd_kw=dict(dgate=dboth[..., :2048], dx=dboth[..., 2056:4104]))
    assert (dboth[..., 2048:2056] == 7.0).all() and (dboth[..., 4104:] == 7.0).all()
    tm = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    v3 = dict(v, gate=tm(v["gate"]), x=tm(v["x"]))
    check(v3, dict(back, dout=tm(back["dout"])), "bld", False, fwd_kw=dict(out=tm(torch.zeros_like(v["x"]))))


@pytest.mark.parametrize("batch", [3, 5])
def test_many_chains_repeat_bit_for_bit_and_replay(batch):
    v, back = make(batch, 4096, 1300, "bld", BF, False, seed=31)
    run = lambda: (ops.gated_scan_fwd(**v, layout="bld"), ops.gated_scan_bwd(**v, **back, layout="bld"))  # noqa: E731
    o, g = run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2, g2 = run()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, o2)
        for k in g:
            assert torch.equal(g[k], g2[k])
    assert ops.device_status() == 0


@pytest.mark.parametrize("batch", [4, 6])
def test_many_chains_state_in_place(batch):
    v, _ = make(batch, 2048, 700, "bld", F32, False, seed=32)
    want = ref.gated(**v, layout="bld")
    state = v["initial_state"].clone()
    out, _ = ops.gated_scan_fwd(v["gate"], v["x"], v["gate_bias"], initial_state=state, last_state=state, layout="bld")
    assert_close("out", out, *want["out"])
    assert_close("last", state, *want["last_state"])


@pytest.mark.parametrize("batch", [4, 10])
def test_many_chains_withheld_handoff_is_reported(batch):
    v, _ = make(batch, 2048, 2000, "bld", BF, False, seed=33)
    ops.device_status()
    ops.gated_scan_fwd(**v, layout="bld", flags=ops.MAMBA_FLAG_TEST_WITHHOLD_HANDOFF)
    assert ops.STATUS_NAMES[ops.device_status()] == "MAMBA_ERR_TIMEOUT"
    assert ops.device_status() == 0
    want = ref.gated(**v, layout="bld")
    assert_close("out", ops.gated_scan_fwd(**v, layout="bld"), *want["out"])


@pytest.mark.parametrize("L", [5, 100, 700, 2100])
@pytest.mark.parametrize("batch,dim", [(1, 1), (3, 5), (5, 13)])
def test_rows_layout_odd_chain_counts(batch, dim, L):
    """A pair of chains with a missing second one, and pairs across two batch rows."""
    v, back = make(batch, dim, L, "bdl", BF, False, seed=L + dim, ragged=batch > 1)
    check(v, back, "bdl", False)


def test_distances_of_extent_one():
    """A tensor's distance along an axis of one element says nothing."""
    v, back = make(3, 64, 1, "bld", BF, False, seed=40)
    odd = lambda t: torch.as_strided(t.clone(), t.shape, (64, 1, 1))  # noqa: E731
    v2 = dict(v, gate=odd(v["gate"]), x=odd(v["x"]))
    check(v2, back, "bld", False)
    v, back = make(1, 64, 90, "bld", BF, False, seed=41)
    odd = lambda t: torch.as_strided(t.clone(), t.shape, (1, 64, 1))  # noqa: E731
    v2 = dict(v, gate=odd(v["gate"]), x=odd(v["x"]))
    check(v2, back, "bld", False)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim,L", [(64, 90), (67, 90), (2048, 90), (67, 1300), (256, 1300), (1536, 1300)])
def test_concurrent_streams(dim, L, dtype):
    """Two calls at once on streams of their own, each with its own workspace."""
    sides = [make(11, dim, L, "bld", dtype, False, seed=s) for s in (50, 51)]
    streams = [torch.cuda.Stream() for _ in sides]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for (v, back), stream in zip(sides, streams):
            with torch.cuda.stream(stream):
                got.append((ops.gated_scan_fwd(**v, layout="bld"), ops.gated_scan_bwd(**v, **back, layout="bld")))
    torch.cuda.synchronize()
    for i, (out, g) in enumerate(got):
        v, back = sides[i % 2]
        want = ref.gated(**v, layout="bld", **back)
        assert_close("out", out, *want["out"])
        for k in g:
            assert_close(k, g[k], *want[k])


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("layout,batch,dim,L", [("bld", 5, 96, 65), ("bld", 5, 96, 512), ("bld", 3, 70, 300),
                                                ("bld", 2, 64, 7000), ("bld", 25, 840, 577), ("bdl", 3, 70, 300),
                                                ("bdl", 2, 5, 4100)])
def test_state_gradient_in_place(layout, batch, dim, L, ragged):
    """dinitial_state in dlast_state's buffer (the C entry point): the warps of a short chain, the
    segments of a long one and the chained stretches all read it before it is replaced."""
    v, back = make(batch, dim, L, layout, BF, False, seed=L + dim, ragged=ragged)
    want = ref.gated(**v, **back, layout=layout)
    lib, flags = ops.library(), ops.MAMBA_FLAG_LAYOUT_BLD if layout == "bld" else 0
    dims = ops.GatedDims(batch=batch, dim=dim, seqlen=L, io_dtype=ops.MAMBA_BF16, flags=flags,
                         seqlens=v["seqlens"].data_ptr() if ragged else None)
    need = lib.mamba_gated_scan_bwd_workspace_bytes(ctypes.byref(dims), 0)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    dims.workspace, dims.workspace_bytes = ws.data_ptr(), need
    for _ in range(3):
        state, dgate, dx = back["dlast_state"].clone(), torch.empty_like(v["x"]), torch.empty_like(v["x"])
        rc = lib.mamba_gated_scan_bwd(
            v["gate"].data_ptr(), v["x"].data_ptr(), v["gate_bias"].data_ptr(), v["initial_state"].data_ptr(), None,
            back["dout"].data_ptr(), state.data_ptr(), dgate.data_ptr(), dx.data_ptr(), None, state.data_ptr(),
            ctypes.byref(dims), torch.cuda.current_stream().cuda_stream)
        assert rc == ops.MAMBA_OK
        torch.cuda.synchronize()
        assert_close("dinitial_state", state, *want["dinitial_state"])
        assert_close("dgate", dgate, *want["dgate"])
        assert_close("dx", dx, *want["dx"])
    assert ops.device_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout,batch,dim,L", [("bld", 2, 64, 7000), ("bld", 2, 67, 7000), ("bld", 3, 96, 257),
                                                ("bld", 25, 840, 1300), ("bdl", 3, 70, 5000)])
def test_long_state_in_place(layout, batch, dim, L, dtype):
    """last_state in initial_state's buffer where many segments or stretches read the start: each
    has read it before the last of them replaces it."""
    v, _ = make(batch, dim, L, layout, dtype, False, seed=L + dim)
    want = ref.gated(**v, layout=layout)
    for _ in range(3):
        state = v["initial_state"].clone()
        out, _ = ops.gated_scan_fwd(v["gate"], v["x"], v["gate_bias"], initial_state=state, last_state=state,
                                    layout=layout)
        assert_close("out", out, *want["out"])
        assert_close("last", state, *want["last_state"])
    assert ops.device_status() == 0


WITHHELD = [("fwd", 1, 8, 1 << 21, True), ("fwd", 1, 7, 1 << 21, True), ("bwd", 1, 8, 1 << 21, True),
            ("bwd", 1, 8, 1 << 21, False), ("bwd", 2, 7, 1 << 20, True), ("bwd", 10, 2048, 2000, True)]


@pytest.mark.parametrize("call,batch,dim,L,checkpoints", WITHHELD)
def test_withheld_handoff_ends_the_whole_call(call, batch, dim, L, checkpoints):
    """Thousands of segments that never hand on (thousands of waits of some 0.3 s, were each to run
    out by itself): the call ends soon, the status says so, and the next call is right again."""
    v, back = make(batch, dim, L, "bld", BF, True, seed=dim)

    def run(flags=0):
        if call == "fwd":
            return {"out": ops.gated_scan_fwd(**v, log_decay=True, layout="bld", flags=flags)}
        return ops.gated_scan_bwd(**v, **back, checkpoints=ck, log_decay=True, layout="bld", flags=flags)

    ck = ops.gated_scan_fwd(**v, log_decay=True, layout="bld", return_checkpoints=True)[1] if checkpoints else None
    good = run()
    assert ops.device_status() == 0
    start = time.perf_counter()
    run(ops.MAMBA_FLAG_TEST_WITHHOLD_HANDOFF)
    torch.cuda.synchronize()
    took = time.perf_counter() - start
    assert ops.STATUS_NAMES[ops.device_status()] == "MAMBA_ERR_TIMEOUT"
    assert took < 1.5, took
    again = run()
    assert ops.device_status() == 0
    for k in good:
        assert torch.equal(good[k], again[k]), k


@pytest.mark.parametrize("layout,batch,dim,L,ragged", [
    ("bld", 25, 840, 577, True), ("bld", 13, 1024, 200, False), ("bld", 4, 67, 700, False), ("bld", 2, 64, 5000, True),
    ("bld", 9, 300, 64, False), ("bdl", 3, 70, 1000, True), ("bdl", 5, 33, 2047, False), ("bdl", 2, 3, 5000, False),
    ("bdl", 40, 65, 30, True)])
def test_bias_gradient_holds_every_step_once(layout, batch, dim, L, ragged):
    """In fp32 dgate_bias is the sum of the dgate that the call returns, to the roundings of a sum
    in which no term passes more than L + batch + 64 of them."""
    v, back = make(batch, dim, L, layout, F32, False, seed=L, ragged=ragged)
    g = ops.gated_scan_bwd(**v, **back, layout=layout)
    terms = g["dgate"].double().sum(1 if layout == "bld" else 2), g["dgate"].double().abs().sum(1 if layout == "bld" else 2)
    off = (g["dgate_bias"].double() - terms[0].sum(0)).abs()
    assert (off <= (L + batch + 64) * ref.U * terms[1].sum(0)).all()


@pytest.mark.parametrize("layout,shape", [("bld", (70, 8192, 4096)), ("bld", (70, 8192, 4095)), ("bld", (1, 1 << 24, 136)),
                                          ("bdl", (2, 35001, 32760))])
def test_offsets_beyond_32_bits(layout, shape):
    """More than 2^31 elements per tensor: the last channels of the last batch row."""
    g = torch.Generator(device=DEV)
    g.manual_seed(60)
    gate, x, dout = (torch.randn(shape, generator=g, device=DEV, dtype=BF) for _ in range(3))
    dim = shape[2] if layout == "bld" else shape[1]
    assert gate.numel() > 2 ** 31
    bias = torch.full((dim,), 1.0, device=DEV)
    out, last = ops.gated_scan_fwd(gate, x, bias, layout=layout, return_last_state=True)
    grads = ops.gated_scan_bwd(gate, x, dout, layout=layout)
    # gates around 1 forget within some 30 steps: the last 1000 steps tell nothing of those before
    tail = (lambda t: t[-1:, -1000:, -3:]) if layout == "bld" else (lambda t: t[-1:, -3:, -1000:])
    late = (lambda t: t[:, 500:]) if layout == "bld" else (lambda t: t[..., 500:])
    want = ref.gated(tail(gate), tail(x), bias[-3:], layout=layout)
    assert_close("out", late(tail(out)), *(late(t) for t in want["out"]))
    assert_close("last", last[-1:, -3:], *want["last_state"])
    want = ref.gated(tail(gate), tail(x), layout=layout, dout=tail(dout))
    for k in ("dgate", "dx"):
        assert_close(k, late(tail(grads[k])), *(late(t) for t in want[k]))
    assert ops.device_status() == 0
