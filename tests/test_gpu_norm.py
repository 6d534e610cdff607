"""Layer norm with the residual add, forward and backward, against its 64-bit form."""
import ctypes

import pytest
import torch

import block_reference as ref
from block_reference import assert_close
from selective_state_space_55_b200 import ops

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def make(rows, dim, dtype, res, seed, offset=0.5):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    rdt = {"none": None, "same": dtype, "fp32": F32}[res]
    x = (randn(rows, dim) + offset).to(dtype)
    return dict(x=x, residual=None if rdt is None else randn(rows, dim).to(rdt),
                weight=1.0 + 0.2 * randn(dim), bias=0.3 * randn(dim), dout=randn(rows, dim).to(dtype),
                ds=None if rdt is None else randn(rows, dim).to(rdt))


def check(v, rms=False, eps=1e-5, weight=True, bias=True, fwd_kw=None, bwd_kw=None):
    w, b = v["weight"] if weight else None, v["bias"] if bias else None
    want = ref.norm_fwd(v["x"], w, b, v["residual"], eps, rms)
    r = ops.layer_norm_fwd(v["x"], weight=w, bias=b, residual=v["residual"], eps=eps, rms=rms,
                           return_stats=True, **(fwd_kw or {}))
    out, mean, rstd = r[0], r[-2], r[-1]
    s = v["x"] if v["residual"] is None else r[1]
    assert_close("out", out, *want["out"])
    assert_close("rstd", rstd, *want["rstd"])
    if rms:
        assert mean is None
    else:
        assert_close("mean", mean, *want["mean"])
    if v["residual"] is not None:
        assert_close("residual_out", s, *want["residual_out"])
    gw = ref.norm_bwd(v["dout"], s, rstd, mean, w, v["ds"], rms)
    g = ops.layer_norm_bwd(v["dout"], s, rstd, mean=mean, weight=w, bias=b, dresidual_out=v["ds"],
                           rms=rms, **(bwd_kw or {}))
    assert ("dweight" in g) == weight and ("dbias" in g) == bias
    for k in g:
        assert_close(k, g[k], *gw[k])
    return r, g


@pytest.mark.parametrize("dim", [1, 7, 8, 31, 64, 100, 255, 256, 257, 500, 512, 513, 520, 768, 1001,
                                 2560, 4096, 5000, 8192])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rms", [False, True])
def test_widths(rms, dtype, dim):
    check(make(5, dim, dtype, "same", seed=dim), rms=rms)


@pytest.mark.parametrize("dim", [8193, 8200, 16384, 20001])
@pytest.mark.parametrize("dtype,res", [(BF, "none"), (BF, "fp32"), (F32, "same")])
def test_wide_rows(dtype, res, dim):
    check(make(7, dim, dtype, res, seed=dim))


@pytest.mark.parametrize("rows", [1, 2, 9, 147, 1185, 5000])
@pytest.mark.parametrize("dim", [96, 392, 1024])
@pytest.mark.parametrize("res", ["none", "same", "fp32"])
def test_row_counts(res, dim, rows):
    check(make(rows, dim, BF, res, seed=rows))


@pytest.mark.parametrize("dim", [4100, 6144, 8192])
@pytest.mark.parametrize("dtype,res", [(F32, "same"), (BF, "fp32"), (BF, "same")])
def test_widest_rows_in_registers(dtype, res, dim):
    """Many rows at the widths where the shared memory of a CTA is fullest."""
    check(make(700, dim, dtype, res, seed=dim))


@pytest.mark.parametrize("weight,bias", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("dim", [130, 640, 9000])
def test_without_weight_or_bias(dim, weight, bias):
    check(make(300, dim, BF, "same", seed=1), weight=weight, bias=bias)


def test_offset_far_above_the_spread():
    """Mean 1000, spread 1: the variance keeps its digits (two reductions, not E[s^2] - mean^2)."""
    check(make(33, 1024, F32, "none", seed=2, offset=1000.0))
    check(make(33, 384, F32, "none", seed=2, offset=1000.0))


@pytest.mark.parametrize("dim", [64, 1024, 8448])
def test_constant_rows(dim):
    v = make(4, dim, BF, "none", seed=3)
    v["x"].fill_(2.0)
    r, g = check(v)
    assert torch.equal(r[0].float(), v["bias"].to(BF).float().expand(4, -1))


def test_a_nan_row_stays_in_its_row():
    v = make(20, 512, BF, "none", seed=4)
    v["x"][7, 3] = float("nan")
    out = ops.layer_norm_fwd(v["x"], v["weight"], v["bias"])
    assert out[7].isnan().all() and not out[:7].isnan().any() and not out[8:].isnan().any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim", [128, 131, 1000, 9001])
def test_strided_rows_and_shapes(dtype, dim):
    """Rows as a slice of wider ones, at odd offsets, (batch, L, dim) in front."""
    v = make(24, dim, dtype, "same", seed=dim)
    wide = torch.full((24, 2 * dim + 3), 9.0, dtype=dtype, device=DEV)
    x = wide[:, 1:dim + 1]
    x.copy_(v["x"])
    out = torch.full((24, dim + 5), 4.0, dtype=dtype, device=DEV)
    v["x"] = x
    check(v, fwd_kw=dict(out=out[:, 2:dim + 2]))
    assert (out[:, :2] == 4.0).all() and (out[:, dim + 2:] == 4.0).all()
    y = ops.layer_norm_fwd(x.view(2, 3, 4, dim) if x.is_contiguous() else x.unflatten(0, (2, 3, 4)),
                           v["weight"], v["bias"], return_stats=True)
    assert y[0].shape == (2, 3, 4, dim) and y[1].shape == (2, 3, 4)
    assert_close("out", y[0].view(24, dim), *ref.norm_fwd(x, v["weight"], v["bias"])["out"])


@pytest.mark.parametrize("dim", [256, 2560, 9216])
def test_in_place(dim):
    v = make(40, dim, BF, "same", seed=5)
    want = ref.norm_fwd(v["x"], v["weight"], v["bias"], v["residual"])
    x, res = v["x"].clone(), v["residual"].clone()
    out, s, mean, rstd = ops.layer_norm_fwd(x, v["weight"], v["bias"], residual=res, out=x,
                                            residual_out=res, return_stats=True)
    assert out is x and s is res
    assert_close("out", x, *want["out"])
    assert_close("residual_out", res, *want["residual_out"])
    gw = ref.norm_bwd(v["dout"], s, rstd, mean, v["weight"], v["ds"])
    dout = v["dout"].clone()
    g = ops.layer_norm_bwd(dout, s, rstd, mean=mean, weight=v["weight"], bias=v["bias"],
                           dresidual_out=v["ds"], dx=dout)
    for k in g:
        assert_close(k, g[k], *gw[k])
    ds = v["ds"].clone()
    g = ops.layer_norm_bwd(v["dout"], s, rstd, mean=mean, weight=v["weight"], bias=v["bias"],
                           dresidual_out=ds, dx=ds)
    for k in g:
        assert_close(k, g[k], *gw[k])


def test_first_block_keeps_the_stream_in_fp32():
    """No residual yet, residual_out in fp32: s = x."""
    v = make(10, 320, BF, "none", seed=6)
    s = torch.empty(10, 320, device=DEV)
    out, s2 = ops.layer_norm_fwd(v["x"], v["weight"], residual_out=s)
    assert s2 is s and torch.equal(s, v["x"].float())


def test_no_rows():
    e = torch.empty(0, 64, device=DEV)
    st = torch.empty(0, device=DEV)
    w = torch.ones(64, device=DEV)
    assert ops.layer_norm_fwd(e, w).shape == (0, 64)
    g = ops.layer_norm_bwd(e, e, st, mean=st, weight=w, bias=w)
    assert (g["dweight"] == 0).all() and (g["dbias"] == 0).all()


def test_repeats_bit_for_bit():
    v = make(3000, 768, BF, "same", seed=7)
    _, s, mean, rstd = ops.layer_norm_fwd(v["x"], v["weight"], v["bias"], residual=v["residual"], return_stats=True)
    runs = [ops.layer_norm_bwd(v["dout"], s, rstd, mean=mean, weight=v["weight"], bias=v["bias"]) for _ in range(3)]
    for g in runs[1:]:
        for k in g:
            assert torch.equal(g[k], runs[0][k])


def test_gradients_match_differences():
    v = make(2, 5, F32, "none", seed=8)
    x, w, b = (v[k].double().cpu() for k in ("x", "weight", "bias"))
    dy = v["dout"].double().cpu()

    def loss(x, w, b):
        return (ref.norm_fwd(x, w, b)["out"][0] * dy).sum()

    o = ref.norm_fwd(x, w, b)
    g = ref.norm_bwd(dy, x, o["rstd"][0], o["mean"][0], w)
    for k, name in enumerate(("dx", "dweight", "dbias")):
        args = [x, w, b]
        for i in range(args[k].numel()):
            e = torch.zeros(args[k].numel(), dtype=torch.float64)
            e[i] = 1e-6
            hi, lo = list(args), list(args)
            hi[k] = args[k] + e.view(args[k].shape)
            lo[k] = args[k] - e.view(args[k].shape)
            d = (loss(*hi) - loss(*lo)) / 2e-6
            assert abs(d - g[name][0].flatten()[i]) <= 1e-7 * (1 + abs(d))
    check(v)


def test_stream_of_its_own():
    v = make(64, 512, BF, "same", seed=9)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    out, s = ops.layer_norm_fwd(v["x"], v["weight"], v["bias"], residual=v["residual"], stream=st)
    st.synchronize()
    assert_close("out", out, *ref.norm_fwd(v["x"], v["weight"], v["bias"], v["residual"])["out"])


@pytest.mark.parametrize("rms", [False, True])
def test_no_columns(rms):
    """The moments of empty rows are 0 / 0, not what the buffers held before."""
    x = torch.empty(3, 5, 0, device=DEV)
    stats = torch.full((2, 3, 5), 7.0, device=DEV)
    dims = ops.NormDims(rows=15, dim=0, rms=rms, eps=1e-5)
    rc = ops.library().mamba_layer_norm_fwd(None, None, None, None, None, None, stats[0].data_ptr(), stats[1].data_ptr(),
                                            ctypes.byref(dims), torch.cuda.current_stream().cuda_stream)
    assert rc == ops.MAMBA_OK
    assert stats[1].isnan().all() and ((stats[0] == 0).all() if rms else stats[0].isnan().all())
    out, mean, rstd = ops.layer_norm_fwd(x, rms=rms, return_stats=True)
    assert out.shape == (3, 5, 0) and rstd.isnan().all() and (mean is None if rms else mean.isnan().all())
    g = ops.layer_norm_bwd(x, x, rstd, mean=mean, weight=torch.empty(0, device=DEV), rms=rms)
    assert g["dx"].shape == (3, 5, 0) and g["dweight"].shape == (0,)


# columns that take 1, 2, 3, 4, 5, 6 and 8 chunks of 8 per lane with many rows, on vectors and
# element by element
CHUNKS = [256, 255, 512, 509, 768, 767, 1024, 1021, 1280, 1275, 1536, 1529, 2048, 2041, 2560, 2555]


@pytest.mark.parametrize("dim", CHUNKS)
@pytest.mark.parametrize("dtype,res", [(BF, "none"), (BF, "same"), (BF, "fp32"), (F32, "same")])
def test_many_rows_at_every_chunk_count(dtype, res, dim):
    check(make(331, dim, dtype, res, seed=dim), rms=dim % 3 == 0)


@pytest.mark.parametrize("rows,dim", [(13100, 512), (13100, 509), (6600, 1024), (6600, 1021), (2700, 2560), (2700, 2555),
                                      (1700, 4096)])
@pytest.mark.parametrize("dtype,res", [(BF, "same"), (BF, "fp32"), (F32, "same")])
def test_backward_of_many_rows(dtype, res, rows, dim):
    """So many rows that the backward takes two chunks per lane: 1, 2, 5 and 8 warps per row, 8 to
    1 rows side by side."""
    check(make(rows, dim, dtype, res, seed=dim))


@pytest.mark.parametrize("rows,dim", [(1, 8), (3, 2560), (331, 1280), (2000, 2555), (13100, 512), (13100, 509),
                                      (6600, 1024), (2700, 2560), (2700, 2555), (1700, 4096), (40000, 96), (3000, 9000),
                                      (1500, 8193)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_column_sums_hold_every_row_once(dtype, rows, dim):
    """Small whole numbers and rstd = 1: dweight and dbias are exact (far below 2^24)."""
    g = torch.Generator(device=DEV)
    g.manual_seed(rows + dim)
    pick = lambda: torch.randint(-2, 3, (rows, dim), generator=g, device=DEV)  # noqa: E731
    s, dout = pick(), pick()
    mean = torch.randint(-1, 2, (rows,), generator=g, device=DEV)
    got = ops.layer_norm_bwd(dout.to(dtype), s.to(dtype), torch.ones(rows, device=DEV), mean=mean.float(),
                             weight=torch.ones(dim, device=DEV), bias=torch.zeros(dim, device=DEV))
    assert torch.equal(got["dweight"].long(), (dout * (s - mean[:, None])).sum(0))
    assert torch.equal(got["dbias"].long(), dout.sum(0))


def test_offsets_beyond_32_bits():
    """More than 2^31 elements per tensor: the last rows, and every row once in the sums."""
    rows, dim = 1_100_000, 2048
    g = torch.Generator(device=DEV)
    g.manual_seed(60)
    x, dout = (torch.randn(rows, dim, generator=g, device=DEV, dtype=BF) for _ in range(2))
    res = torch.randn(rows, dim, generator=g, device=DEV, dtype=BF)
    out, s, mean, rstd = ops.layer_norm_fwd(x, residual=res, return_stats=True)
    want = ref.norm_fwd(x[-5:], residual=res[-5:])
    assert_close("out", out[-5:], *want["out"])
    assert_close("residual_out", s[-5:], *want["residual_out"])
    grad = ops.layer_norm_bwd(dout, s, rstd, mean=mean, bias=torch.zeros(dim, device=DEV))
    want = ref.norm_bwd(dout[-5:], s[-5:], rstd[-5:], mean[-5:])
    assert_close("dx", grad["dx"][-5:], *want["dx"])
    # bf16 whole numbers: exact sums
    dout = torch.randint(0, 3, (rows, dim), generator=g, device=DEV, dtype=torch.int8).to(BF)
    grad = ops.layer_norm_bwd(dout, s, rstd, mean=mean, bias=torch.zeros(dim, device=DEV))
    assert torch.equal(grad["dbias"].double(), sum(part.double().sum(0) for part in dout.split(100_000)))
