"""Backward of the short causal convolution against its 64-bit form."""
import ctypes

import pytest
import torch

import block_reference as ref
from block_reference import assert_close
from selective_state_space_55_b200 import ops

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def make(batch, dim, L, W, dtype, seed, bias=True, state=True):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return dict(x=randn(batch, dim, L).to(dtype), weight=randn(dim, W), dout=randn(batch, dim, L).to(dtype),
                bias=randn(dim) if bias else None,
                initial_conv_state=randn(batch, dim, W).to(dtype) if state else None,
                dfinal_conv_state=randn(batch, dim, W).to(dtype) if state else None)


def check(v, silu=True):
    want = ref.conv_bwd(**v, silu=silu)
    g = ops.causal_conv1d_bwd(**v, silu=silu)
    assert ("dbias" in g) == (v["bias"] is not None)
    assert ("dinitial_conv_state" in g) == (v["initial_conv_state"] is not None)
    for k in g:
        assert_close(k, g[k], *want[k])
    return g


@pytest.mark.parametrize("L", [1, 2, 3, 4, 7, 8, 9, 255, 256, 257, 333, 1001])
@pytest.mark.parametrize("W", [1, 2, 3, 4])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_lengths_and_widths(dtype, W, L):
    check(make(3, 37, L, W, dtype, seed=10 * L + W))


@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("silu", [True, False])
def test_options(silu, state, bias):
    check(make(2, 50, 300, 4, BF, seed=1, bias=bias, state=state), silu=silu)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("L", [40000, 39999])
def test_long_rows_are_cut_into_stretches(L, dtype):
    """Few chains: stretches of a row meet at tile borders, aligned or shifted."""
    check(make(2, 3, L, 4, dtype, seed=2))


def test_many_chains():
    check(make(4, 3000, 96, 4, BF, seed=3))


def test_empty_sequence():
    v = make(2, 6, 0, 4, F32, seed=4)
    g = check(v)
    assert torch.equal(g["dinitial_conv_state"], v["dfinal_conv_state"])
    assert (g["dweight"] == 0).all()


def test_empty_batch():
    v = make(0, 6, 9, 4, F32, seed=5)
    g = ops.causal_conv1d_bwd(**v)
    assert (g["dweight"] == 0).all() and (g["dbias"] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_shifted_buffers(dtype):
    """Each tensor starts at its own element offset."""
    v = make(2, 9, 530, 4, dtype, seed=6)
    for i, k in enumerate(("x", "dout", "initial_conv_state", "dfinal_conv_state", "weight", "bias")):
        buf = torch.empty(v[k].numel() + i + 1, dtype=v[k].dtype, device=DEV)
        w = buf[i + 1:].view(v[k].shape)
        w.copy_(v[k])
        v[k] = w
    check(v)


def test_forward_then_backward():
    """The gradient of the forward kernel's own result, by 64-bit differences of its formula."""
    v = make(1, 2, 6, 3, F32, seed=7)
    want = ref.conv_bwd(**v)
    x, w, b = (v[k].double().cpu() for k in ("x", "weight", "bias"))
    init, dy, df = (v[k].double().cpu() for k in ("initial_conv_state", "dout", "dfinal_conv_state"))

    def loss(x, w, b, init):
        seq = torch.cat([init, x], 2)
        pre = b[:, None] + sum(w[:, k, None] * seq[:, :, 1 + k:7 + k] for k in range(3))
        return (pre * torch.sigmoid(pre) * dy).sum() + (seq[:, :, 6:] * df).sum()

    for k, name in enumerate(("dx", "dweight", "dbias", "dinitial_conv_state")):
        args = [x, w, b, init]
        for i in range(args[k].numel()):
            e = torch.zeros(args[k].numel(), dtype=torch.float64)
            e[i] = 1e-6
            hi, lo = list(args), list(args)
            hi[k] = args[k] + e.view(args[k].shape)
            lo[k] = args[k] - e.view(args[k].shape)
            d = (loss(*hi) - loss(*lo)) / 2e-6
            assert abs(d - want[name][0].flatten()[i]) <= 1e-7 * (1 + abs(d))
    check(v)


def test_repeats_bit_for_bit():
    v = make(3, 200, 2000, 4, BF, seed=8)
    runs = [ops.causal_conv1d_bwd(**v) for _ in range(3)]
    for g in runs[1:]:
        for k in g:
            assert torch.equal(g[k], runs[0][k])


def test_saturated_activation():
    """pre of +-300: silu' is 1 or 0, never NaN."""
    v = make(1, 8, 64, 1, F32, seed=9, state=False)
    v["x"] = v["x"].sign() * 100.0
    v["weight"].fill_(3.0)
    v["bias"].zero_()
    g = check(v)
    assert torch.isfinite(g["dx"]).all()


def test_longest_rows():
    """The documented limit, 2^31 - 65536 steps: the last stretch of a row ends at 2^31.  Small
    whole numbers in the last 2.2 million steps and zeros before them, so every product and
    partial sum (below 2^24) is exact."""
    L, n, W = 2 ** 31 - 65536, 2_200_000, 4
    g = torch.Generator(device=DEV)
    g.manual_seed(10)
    x, dout = (torch.zeros(1, 2, L, dtype=BF, device=DEV) for _ in range(2))
    xt = torch.randint(0, 3, (2, n), generator=g, device=DEV).double()
    dt = torch.randint(0, 2, (2, n), generator=g, device=DEV).double()
    x[0, :, L - n:], dout[0, :, L - n:] = xt.to(BF), dt.to(BF)
    w = torch.tensor([[1.0, -2.0, 1.0, 2.0], [2.0, 1.0, -1.0, 1.0]], device=DEV)
    got = ops.causal_conv1d_bwd(x, w, dout, bias=torch.zeros(2, device=DEV), silu=False)
    seq, after = (torch.nn.functional.pad(t, p) for t, p in ((xt, (W - 1, 0)), (dt, (0, W - 1))))
    dw = torch.stack([(dt * seq[:, k:k + n]).sum(1) for k in range(W)], 1)
    dx = sum(w[:, k:k + 1].double() * after[:, W - 1 - k:W - 1 - k + n] for k in range(W))
    assert torch.equal(got["dweight"].double(), dw)
    assert torch.equal(got["dbias"].double(), dt.sum(1))
    assert torch.equal(got["dx"][0, :, L - n:].double(), dx)
    # the gradient reaches W - 1 steps further back, no more
    assert not got["dx"][0, :, :L - n - W + 1].any()


RING = 4                       # tiles of 256 steps on their way to a warp, at most


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("batch,dim,L,W,state", [
    (5, 1000, 1300, 4, True), (5, 1000, 2048, 4, False), (1, 3001, 2300, 3, True), (1, 5120, 2047, 4, True),
    (3, 700, 4000, 2, True), (1, 1001, 8003, 4, True), (1, 301, 20001, 4, False), (2, 1200, 4096, 1, True)])
def test_many_tiles_per_stretch(batch, dim, L, W, state, dtype):
    """A warp walks more tiles than its ring holds, in one stretch per row or several: what one tile
    leaves for the next, the neighbours taken from the ring's next stage and the reuse of its slots."""
    v = make(batch, dim, L, W, dtype, seed=L + W, state=state)
    dims = ops.make_scan_dims(batch=batch, dim=dim, dstate=1, seqlen=L, io_dtype=dtype, bc_dtype=dtype)
    room = ops.library().mamba_causal_conv1d_bwd_workspace_bytes(ctypes.byref(dims), W)
    stretches = room // (batch * (W + 1) * dim * 4)           # one row of sums for each
    phase = 0 if (L * v["x"].element_size()) % 16 == 0 else 16 // v["x"].element_size() - 1
    tiles = -(-(L + phase) // 256) // stretches
    assert tiles > RING, (tiles, stretches)
    # a lane's eight steps of every tile (the tensors' phase adds one at most), five joins of
    # lanes, the stretches' rows by 32 warps and the sum of those
    depth = 8 * (tiles + 2) + 5 + batch * stretches // 32 + 1 + 32
    want = ref.conv_bwd(**v, depth=depth)
    g = ops.causal_conv1d_bwd(**v)
    for k in g:
        assert_close(k, g[k], *want[k])


@pytest.mark.parametrize("L", [32768, 32763])
def test_offsets_beyond_32_bits(L):
    """More than 2^31 elements per tensor: the last channels."""
    g = torch.Generator(device=DEV)
    g.manual_seed(60)
    x, dout = (torch.randn(2, 35001, L, generator=g, device=DEV, dtype=BF) for _ in range(2))
    assert x.numel() > 2 ** 31
    w, b = torch.randn(35001, 4, generator=g, device=DEV), torch.randn(35001, generator=g, device=DEV)
    got = ops.causal_conv1d_bwd(x, w, dout, bias=b)
    want = ref.conv_bwd(x[:, -3:], w[-3:], dout[:, -3:], b[-3:], depth=8 * (L // 256 + 2) + 64)
    assert_close("dx", got["dx"][:, -3:], *want["dx"])
    assert_close("dweight", got["dweight"][-3:], *want["dweight"])
    assert_close("dbias", got["dbias"][-3:], *want["dbias"])
