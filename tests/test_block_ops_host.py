"""Host-side checks of the block operators (no GPU): the C ABI refuses bad
arguments before it touches the device, and the binding refuses host tensors."""
import ctypes

import pytest
import torch

from selective_state_space_55_b200 import build, ops

FAKE = 0x10000          # never dereferenced: validation fails first
OTHER = 0x20000
INVALID, UNSUPPORTED, ALIGN, WORKSPACE = -1, -2, -3, -4
BLD = ops.MAMBA_FLAG_LAYOUT_BLD


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ops.library()


def gated_dims(**kw):
    d = ops.GatedDims(batch=2, dim=64, seqlen=1024, io_dtype=ops.MAMBA_BF16, flags=BLD)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def gated_fwd(lib, d, gate=FAKE, x=FAKE, bias=None, h0=None, out=OTHER, last=None, ck=None):
    return lib.mamba_gated_scan_fwd(gate, x, bias, h0, out, last, ck,
                                    ctypes.byref(d) if d is not None else None, None)


def gated_bwd(lib, d, gate=FAKE, x=FAKE, dout=FAKE, dgate=OTHER, dx=OTHER + 0x10000, db=None, dh0=None, ck=None):
    return lib.mamba_gated_scan_bwd(gate, x, None, None, ck, dout, None, dgate, dx, db, dh0,
                                    ctypes.byref(d) if d is not None else None, None)


@pytest.mark.parametrize("call", [gated_fwd, gated_bwd])
def test_gated_refuses_bad_arguments(lib, call):
    S = ops.Strides
    assert call(lib, None) == INVALID
    for k in ("batch", "dim", "seqlen"):
        assert call(lib, gated_dims(**{k: -1})) == INVALID
        assert call(lib, gated_dims(**{k: 1 << 31})) == INVALID
    assert call(lib, gated_dims(io_dtype=5)) == UNSUPPORTED
    assert call(lib, gated_dims(flags=BLD | ops.MAMBA_FLAG_ZOH)) == UNSUPPORTED
    assert call(lib, gated_dims(batch=1 << 20, dim=1 << 20, seqlen=1 << 20)) == UNSUPPORTED
    assert call(lib, gated_dims(), gate=None) == INVALID
    assert call(lib, gated_dims(), x=None) == INVALID
    assert call(lib, gated_dims(), gate=FAKE + 1) == ALIGN
    assert call(lib, gated_dims(seqlens=FAKE + 2)) == ALIGN
    assert call(lib, gated_dims(gate=S(128 * 64, 63))) == INVALID         # rows overlap
    assert call(lib, gated_dims(gate=S(0, 64))) == INVALID                # broadcast batch
    assert call(lib, gated_dims(x=S(-1, 64))) == INVALID
    assert call(lib, gated_dims(flags=0), ck=FAKE) == UNSUPPORTED         # checkpoints: (batch, seqlen, dim) only
    assert call(lib, gated_dims()) == WORKSPACE
    assert call(lib, gated_dims(workspace=FAKE, workspace_bytes=16)) == WORKSPACE
    assert call(lib, gated_dims(workspace=FAKE + 4, workspace_bytes=1 << 30)) == ALIGN


def test_gated_refuses_aliased_and_overlapping_outputs(lib):
    S = ops.Strides
    assert gated_fwd(lib, gated_dims(), out=FAKE) == INVALID
    assert gated_fwd(lib, gated_dims(), out=None) == INVALID
    assert gated_fwd(lib, gated_dims(out=S(64, 64))) == INVALID           # batch rows on one another
    assert gated_fwd(lib, gated_dims(out=S(127 * 64, 64))) == INVALID
    assert gated_bwd(lib, gated_dims(), dgate=OTHER, dx=OTHER) == INVALID
    assert gated_bwd(lib, gated_dims(), dx=FAKE) == INVALID
    assert gated_bwd(lib, gated_dims(), dout=None) == INVALID
    assert gated_bwd(lib, gated_dims(dx=S(64, 64))) == INVALID
    assert gated_fwd(lib, gated_dims(), h0=0x40000, last=0x40100) == INVALID     # partial overlap of the states
    # time-major rows do not overlap: the next check (the workspace) answers
    assert gated_fwd(lib, gated_dims(out=S(64, 2 * 64))) == WORKSPACE


def test_gated_empty_problems_need_nothing(lib):
    assert gated_fwd(lib, gated_dims(batch=0)) == 0
    assert gated_fwd(lib, gated_dims(dim=0)) == 0
    assert gated_fwd(lib, gated_dims(seqlen=0), gate=None, x=None, out=None) == 0
    assert gated_bwd(lib, gated_dims(dim=0)) == 0
    assert lib.mamba_gated_scan_workspace_bytes(ctypes.byref(gated_dims(seqlen=0))) == 0


def test_gated_workspace_sizes(lib):
    size = lambda **kw: lib.mamba_gated_scan_workspace_bytes(ctypes.byref(gated_dims(**kw)))  # noqa: E731
    bwd = lambda have, **kw: lib.mamba_gated_scan_bwd_workspace_bytes(ctypes.byref(gated_dims(**kw)), have)  # noqa: E731
    assert size(seqlen=256) == 0                   # one segment per chain: nothing to hand on
    assert size(flags=0, seqlen=100000) == 0       # a chain stays with its warps
    assert size(seqlen=257) > 0
    assert bwd(0) > bwd(1) > 0
    none = ctypes.c_size_t(-1).value
    assert size(batch=-1) == none and bwd(0, io_dtype=9) == none
    assert size(batch=1 << 20, dim=1 << 12, seqlen=1 << 16) == none       # more tiles than a counter holds


def test_gated_update_refuses_bad_arguments(lib):
    def call(d, state=FAKE, gate=FAKE, x=FAKE, out=OTHER, bias=None):
        return lib.mamba_gated_state_update(state, gate, x, bias, out, ctypes.byref(d) if d else None, None)
    S = ops.Strides
    assert call(None) == INVALID
    assert call(gated_dims(batch=-1)) == INVALID
    assert call(gated_dims(io_dtype=7)) == UNSUPPORTED
    for k in ("state", "gate", "x", "out"):
        assert call(gated_dims(), **{k: None}) == INVALID
    assert call(gated_dims(), state=FAKE + 2) == ALIGN
    assert call(gated_dims(), x=FAKE + 1) == ALIGN
    assert call(gated_dims(gate=S(63, 0))) == INVALID
    assert call(gated_dims(x=S(128, 0)), out=FAKE) == INVALID             # in place with another stride
    assert call(gated_dims(), out=FAKE, state=FAKE, x=OTHER, gate=OTHER) == INVALID
    assert call(gated_dims(batch=0)) == 0


def norm_dims(**kw):
    d = ops.NormDims(rows=4, dim=64, io_dtype=ops.MAMBA_BF16, residual_dtype=ops.MAMBA_BF16, eps=1e-5)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def norm_fwd(lib, d, x=FAKE, res=None, w=None, b=None, out=OTHER, res_out=None):
    return lib.mamba_layer_norm_fwd(x, res, w, b, out, res_out, None, None, ctypes.byref(d) if d else None, None)


def norm_bwd(lib, d, s=FAKE, w=None, mean=FAKE, rstd=FAKE, dout=FAKE, dres=None, dx=OTHER, dres_in=None,
             dw=None, db=None):
    return lib.mamba_layer_norm_bwd(s, w, mean, rstd, dout, dres, dx, dres_in, dw, db,
                                    ctypes.byref(d) if d else None, None)


@pytest.mark.parametrize("call", [norm_fwd, norm_bwd])
def test_norm_refuses_bad_sizes(lib, call):
    assert call(lib, None) == INVALID
    assert call(lib, norm_dims(rows=-1)) == INVALID
    assert call(lib, norm_dims(dim=-1)) == INVALID
    assert call(lib, norm_dims(dim=(1 << 28) + 1)) == UNSUPPORTED
    assert call(lib, norm_dims(io_dtype=3)) == UNSUPPORTED
    assert call(lib, norm_dims(io_dtype=ops.MAMBA_F32)) == UNSUPPORTED     # bf16 residual beside fp32
    for k in ("x_stride", "out_stride", "residual_stride", "residual_out_stride", "dx_stride"):
        assert call(lib, norm_dims(**{k: 63})) == INVALID
        assert call(lib, norm_dims(**{k: -64})) == INVALID


def test_norm_refuses_bad_pointers(lib):
    assert norm_fwd(lib, norm_dims(), x=None) == INVALID
    assert norm_fwd(lib, norm_dims(), out=None) == INVALID
    assert norm_fwd(lib, norm_dims(), x=FAKE + 1) == ALIGN
    assert norm_fwd(lib, norm_dims(), w=FAKE + 2) == ALIGN
    assert norm_fwd(lib, norm_dims(eps=-1.0)) == INVALID
    assert norm_fwd(lib, norm_dims(eps=float("nan"))) == INVALID
    assert norm_fwd(lib, norm_dims(x_stride=128), out=FAKE) == INVALID
    assert norm_fwd(lib, norm_dims(), res=OTHER, out=OTHER) == INVALID
    assert norm_fwd(lib, norm_dims(), res_out=OTHER) == INVALID
    assert norm_fwd(lib, norm_dims(residual_stride=128), res=0x30000, res_out=0x30000) == INVALID
    assert norm_bwd(lib, norm_dims(), s=None) == INVALID
    assert norm_bwd(lib, norm_dims(), mean=None) == INVALID
    assert norm_bwd(lib, norm_dims(), rstd=None) == INVALID
    assert norm_bwd(lib, norm_dims(), dx=None) == INVALID
    assert norm_bwd(lib, norm_dims(), dw=FAKE + 1) == ALIGN
    assert norm_fwd(lib, norm_dims(rows=0)) == 0
    assert norm_bwd(lib, norm_dims(dim=0)) == 0


def test_conv_backward_refuses_bad_arguments(lib):
    def call(d, x=FAKE, w=FAKE, width=4, dout=FAKE, dx=OTHER, dw=FAKE, init=None, dinit=None):
        return lib.mamba_causal_conv1d_bwd(x, w, None, init, width, 1, dout, None, dx, dw, None, dinit,
                                           ctypes.byref(d) if d is not None else None, None)

    def dims(**kw):
        base = dict(batch=2, dim=8, dstate=1, seqlen=16, io_dtype=torch.bfloat16, bc_dtype=torch.bfloat16)
        base.update(kw)
        return ops.make_scan_dims(**base)

    assert call(None) == INVALID
    assert call(dims(batch=-1)) == INVALID
    assert call(dims(seqlen=1 << 31)) == INVALID
    assert call(dims(), width=5) == UNSUPPORTED
    assert call(dims(), width=0) == UNSUPPORTED
    for k in ("x", "w", "dout", "dx", "dw"):
        assert call(dims(), **{k: None}) == INVALID
    assert call(dims(), x=FAKE + 1) == ALIGN
    assert call(dims(), dx=FAKE) == INVALID
    assert call(dims(), init=0x30000, dinit=0x30000) == INVALID
    assert call(dims(dim=0)) == 0


def test_binding_refuses_host_tensors_and_bad_shapes(lib):
    x = torch.zeros(2, 4, 8)
    with pytest.raises(ValueError):
        ops.gated_scan_fwd(x, x)
    with pytest.raises(ValueError):
        ops.gated_scan_bwd(x, x, x)
    with pytest.raises(ValueError):
        ops.gated_scan_fwd(x, x, layout="lbd")
    with pytest.raises(ValueError):
        ops.gated_scan_fwd(x[0], x[0])
    with pytest.raises(ValueError):
        ops.gated_state_update(x[0], x[0], x[0])
    with pytest.raises(ValueError):
        ops.layer_norm_fwd(x)
    with pytest.raises(ValueError):
        ops.layer_norm_bwd(x, x, x[..., 0])
    with pytest.raises(ValueError):
        ops.causal_conv1d_bwd(x, torch.zeros(4, 4), x)
