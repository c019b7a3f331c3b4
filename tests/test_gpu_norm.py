"""falqon_norm_fwd / falqon_norm_bwd against the float64 definitions.

Tolerances count roundings.  u is half a step of the output's type, e =
2^-24, D bounds the roundings of a row sum (a thread adds at most cols / 32
terms in turn, then the tree), R those of a sum over rows (at most 512 in
turn, then the tree)."""

import math

import pytest
import torch

import fp8_quantized_lora_b200 as F
from gpu_util import kernels_of
from oracle import block

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def _depth(cols):
    return cols / 32 + 16


def _u(dtype):
    return torch.finfo(dtype).eps / 2


def _make(seed, rows, cols, dtype, pdtype, affine, rms, dev="cuda"):
    g = torch.Generator(device=dev).manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    x = (rnd(rows, cols) * (0.5 + torch.rand(rows, 1, generator=g, device=dev)) + 0.3).to(dtype)
    gamma = (1 + 0.2 * rnd(cols)).to(pdtype) if affine else None
    beta = (0.2 * rnd(cols)).to(pdtype) if affine and not rms else None
    return x, gamma, beta, rnd(rows, cols).mul(1e-2).to(dtype), rnd(rows, cols).mul(1e-2).to(dtype)


def _check_fwd(x, gamma, beta, eps, rms, y, mean, rstd):
    Y, MU, RS = block.norm_fwd(x, gamma, beta, eps, rms)
    D = _depth(x.shape[1])
    xd = x.double()
    xh = (xd if rms else xd - MU[:, None]) * RS[:, None]
    dmu = torch.zeros_like(RS) if rms else (D + 2) * E * xd.abs().mean(1)
    rel = ((D + 4) / 2 + 6) * E + (dmu * RS) ** 2  # of rstd
    assert ((rstd - RS).abs() <= rel * RS).all()
    if not rms:
        assert ((mean - MU).abs() <= dmu).all()
    ga = 1.0 if gamma is None else gamma.double().abs()
    be = 0.0 if beta is None else beta.double().abs()
    err = ga * ((dmu * RS)[:, None] + xh.abs() * (rel[:, None] + 2 * E)) + 2 * E * ((xh * ga).abs() + be)
    tol = err * (1 + _u(x.dtype)) + _u(x.dtype) * Y.abs()
    assert ((y - Y).abs() <= tol).all(), float(((y - Y).abs() - tol).max())


SHAPES = [(1, 1), (1, 4096), (3, 8), (5, 17), (33, 257), (300, 1000), (65, 2050), (4, 16384), (2, 40001), (1000, 512),
          (9, 8192), (37, 12288), (3, 20000), (2, 65536)]
# more rows than the device holds at once, in each class of row lengths
MANY_ROWS = [(2000, 400), (2000, 515), (1900, 700), (1900, 1000), (1900, 1003), (1900, 1280), (1900, 1531),
             (1900, 1792), (1900, 1801), (1900, 2056), (1900, 3001), (1900, 4096)]


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dtype,pdtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(cuda_device, rows, cols, dtype, pdtype, rms):
    x, gamma, beta, _, _ = _make(rows + cols, rows, cols, dtype, pdtype, True, rms)
    # the rows behind the last one stay as they were
    buf = torch.full((rows + 2, cols), 7.0, dtype=dtype, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kind = F.NORM_RMS if rms else F.NORM_LAYER
    y, mean, rstd = F.falqon_norm_fwd(x, gamma, beta, 1e-5, kind, y=buf[:rows], dev_status=st)
    assert (mean is None) == rms
    _check_fwd(x, gamma, beta, 1e-5, rms, y, mean, rstd)
    assert (buf[rows:] == 7.0).all() and int(st.item()) == 0


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dtype,pdtype", [(BF, F32), (F32, BF)])
@pytest.mark.parametrize("rows,cols", [(10000, 24), (10000, 250), (10000, 400), (10001, 505), (10000, 515),
                                       (5000, 700), (5000, 1003), (5000, 1280), (5003, 1801), (3000, 2056),
                                       (3000, 3001), (3000, 4096), (1500, 8192), (1500, 8195), (600, 12001),
                                       (600, 16384)])
def test_forward_of_more_rows_than_fit(cuda_device, rows, cols, dtype, pdtype, rms):
    """Every block (or warp) takes several rows, the next one read ahead, in each class of row lengths."""
    x, gamma, beta, _, _ = _make(rows + cols, rows, cols, dtype, pdtype, True, rms)
    buf = torch.full((rows + 2, cols), 7.0, dtype=dtype, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kind = F.NORM_RMS if rms else F.NORM_LAYER

    def call():
        return F.falqon_norm_fwd(x, gamma, beta, 1e-5, kind, y=buf[:rows], dev_status=st)
    y, mean, rstd = call()
    _check_fwd(x, gamma, beta, 1e-5, rms, y, mean, rstd)
    assert (buf[rows:] == 7.0).all() and int(st.item()) == 0
    (name, grid, block), = kernels_of(call)
    assert "norm_fwd_row_kernel" in name
    held = grid[0] * (block[0] // 32 if cols <= 505 else 1)  # a warp or a block a row
    assert rows > held, (grid, block)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("cols", [48, 515, 4096])
def test_forward_without_parameters_or_statistics(cuda_device, cols, rms):
    kind = F.NORM_RMS if rms else F.NORM_LAYER
    x, _, _, _, _ = _make(cols, 17, cols, BF, BF, False, rms)
    y, mean, rstd = F.falqon_norm_fwd(x, kind=kind)
    _check_fwd(x, None, None, 1e-5, rms, y, mean, rstd)
    y2, m2, r2 = F.falqon_norm_fwd(x, kind=kind, mean=None, rstd=None)
    assert m2 is None and r2 is None and torch.equal(y2, y)
    if not rms:  # beta alone
        beta = torch.randn(cols, device="cuda")
        y3, m3, r3 = F.falqon_norm_fwd(x, None, beta)
        _check_fwd(x, None, beta, 1e-5, rms, y3, m3, r3)


@pytest.mark.parametrize("cols", [64, 1001, 4096, 30000])
def test_forward_offsets_and_small_values(cuda_device, cols):
    """A large common offset (the variance is taken about the mean), rows near
    float32's lower end (eps decides) and constant rows."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(6, cols, generator=g, device="cuda")
    x[0] = x[0] + 4096.0
    x[1] = x[1] * 1e-25
    x[2] = 3.5
    x[3] = 0.0
    x[4] = x[4] * 1e15
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, mean, rstd = F.falqon_norm_fwd(x, dev_status=st)
    _check_fwd(x, None, None, 1e-5, False, y, mean, rstd)
    assert (y[2] == 0).all() and (y[3] == 0).all() and int(st.item()) == 0


@pytest.mark.parametrize("cols", [40, 333, 4096, 20000])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_forward_non_finite_row(cuda_device, cols, bad):
    """A row with an infinity or NaN raises the status bit and leaves the other rows alone."""
    for rms in (False, True):
        kind = F.NORM_RMS if rms else F.NORM_LAYER
        x, gamma, _, _, _ = _make(cols, 9, cols, BF, BF, True, True)
        good = F.falqon_norm_fwd(x, gamma, None, kind=kind)[0].clone()
        x[4, cols - 1] = bad
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        y, _, _ = F.falqon_norm_fwd(x, gamma, None, kind=kind, dev_status=st)
        assert int(st.item()) == F.DEV_NONFINITE
        keep = [i for i in range(9) if i != 4]
        assert torch.equal(y[keep], good[keep])
        assert torch.isnan(y[4]).any()


def _check_bwd(x, gamma, dy, dres, mean, rstd, rms, dx, dgamma, dbeta):
    rows, cols = x.shape
    D, R = _depth(cols), min(rows, 512) + 64
    DX, DG, DB = block.norm_bwd(dy, x, gamma, mean, rstd, dres, rms)
    xd, rs = x.double(), rstd.double()[:, None]
    xh = (xd if rms else xd - mean.double()[:, None]) * rs
    g = dy.double() if gamma is None else dy.double() * gamma.double()
    if dx is not None:
        c1 = 0.0 if rms else g.mean(1, keepdim=True).abs()
        c2 = (g * xh).mean(1, keepdim=True).abs()
        dc1 = 0.0 if rms else (D + 3) * E * g.abs().mean(1, keepdim=True)
        dc2 = (D + 6) * E * (g * xh).abs().mean(1, keepdim=True)
        err = rs * (4 * E * (g.abs() + c1 + (xh * c2).abs()) + dc1 + xh.abs() * (dc2 + 3 * E * c2)) + 3 * E * DX.abs()
        err = err if dres is None else err + 2 * E * dres.double().abs()
        tol = err * (1 + _u(x.dtype)) + _u(x.dtype) * DX.abs()
        assert ((dx - DX).abs() <= tol).all(), float(((dx - DX).abs() - tol).max())
    if dgamma is not None:
        assert ((dgamma - DG).abs() <= (R + 5) * E * (dy.double() * xh).abs().sum(0)).all()
    if dbeta is not None:
        assert ((dbeta - DB).abs() <= R * E * dy.double().abs().sum(0)).all()


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dtype,pdtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("rows,cols", SHAPES + [(2000, 64), (1500, 24), (700, 1536)] + MANY_ROWS)
def test_backward(cuda_device, rows, cols, dtype, pdtype, rms):
    x, gamma, beta, dy, dres = _make(rows * 3 + cols, rows, cols, dtype, pdtype, True, rms)
    kind = F.NORM_RMS if rms else F.NORM_LAYER
    _, mean, rstd = F.falqon_norm_fwd(x, gamma, beta, 1e-5, kind)
    need = F.falqon_workspace_size(F.OP_NORM_BWD, rows, 0, cols)
    raw = torch.full((need // 4 + 64 + 64,), math.nan, device="cuda")  # what a workspace holds does not matter
    off = (-raw.data_ptr() // 4) % 64
    ws = raw[off:off + need // 4].view(torch.uint8)
    guard = raw[off + need // 4:]
    buf = torch.full((rows + 2, cols), 7.0, dtype=dtype, device="cuda")
    dx, dgamma, dbeta = F.falqon_norm_bwd(dy, x, gamma, mean, rstd, kind, dres=dres, dx=buf[:rows], workspace=ws)
    assert (dbeta is None) == rms
    _check_bwd(x, gamma, dy, dres, mean, rstd, rms, dx, dgamma, dbeta)
    assert (buf[rows:] == 7.0).all() and torch.isnan(guard).all()
    # the same call gives the same bits, and so does a call for each output alone
    again = F.falqon_norm_bwd(dy, x, gamma, mean, rstd, kind, dres=dres)
    for a, b in zip(again, (dx, dgamma, dbeta)):
        assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("want", ["dx", "dgamma", "dbeta", "dx+dbeta", "dgamma+dbeta"])
@pytest.mark.parametrize("cols", [96, 333, 2048, 20000])
def test_backward_output_subsets(cuda_device, cols, want):
    x, _, _, dy, _ = _make(cols, 41, cols, BF, F32, False, False)
    _, mean, rstd = F.falqon_norm_fwd(x)
    flags = {k: k in want.split("+") for k in ("dx", "dgamma", "dbeta")}
    out = F.falqon_norm_bwd(dy, x, None, mean, rstd, **flags)
    assert [o is not None for o in out] == list(flags.values())
    _check_bwd(x, None, dy, None, mean, rstd, False, *out)


@pytest.mark.parametrize("cols", [40, 333, 4096, 12000, 20000])
def test_backward_non_finite_row(cuda_device, cols):
    """An infinity or NaN in a row of dy raises the status bit; the other rows' dx keep their bits."""
    for rms in (False, True):
        kind = F.NORM_RMS if rms else F.NORM_LAYER
        x, gamma, beta, dy, _ = _make(cols, 9, cols, BF, BF, True, rms)
        _, mean, rstd = F.falqon_norm_fwd(x, gamma, beta, 1e-5, kind)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        good = F.falqon_norm_bwd(dy, x, gamma, mean, rstd, kind, dgamma=None, dbeta=None, dev_status=st)[0]
        assert int(st.item()) == 0
        for bad in (math.inf, math.nan):
            dy2 = dy.clone()
            dy2[4, cols - 1] = bad
            st.zero_()
            dx, dgamma, _ = F.falqon_norm_bwd(dy2, x, gamma, mean, rstd, kind, dev_status=st)
            assert int(st.item()) == F.DEV_NONFINITE
            keep = [i for i in range(9) if i != 4]
            assert torch.equal(dx[keep], good[keep])
            assert not torch.isfinite(dx[4]).all() and torch.isfinite(dgamma[:cols - 1]).all()


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("scale", [1e-30, 1e-20, 1e16, 1e18, 1e30])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(7, 200), (9, 515), (700, 1000), (500, 1536), (9, 4096), (2000, 4096), (3, 8192),
                                       (3, 12001), (3, 20000)])
def test_backward_far_magnitudes(cuda_device, rows, cols, dtype, scale, rms):
    """Statistics far from 1, whose squares leave float32 while no term of the gradients does.  The tolerance is that
    of the other sizes and, since dx goes down to 1e-36 and its small elements below the normal range, the absolute
    half step there: 2^-134 for a bf16 output, 2^-150 for a float32 one and for each float32 intermediate: b (two
    products), the sum with it, the sum with xh a, the sum with dres, and a (two products), which xh multiplies."""
    x, gamma, beta, dy, dres = _make(rows + cols, rows, cols, dtype, F32, True, rms)
    x, dy = (x.double() * scale).to(dtype), (dy.double() * 1e-4).to(dtype)
    dres = (dres.double() * 1e-4 / scale).to(dtype)
    _, mean, rstd = block.norm_fwd(x, gamma, beta, 0.0, rms)
    mean, rstd = None if rms else mean.float(), rstd.float()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dx, dgamma, dbeta = F.falqon_norm_bwd(dy, x, gamma, mean, rstd, F.NORM_RMS if rms else F.NORM_LAYER, dres=dres,
                                          dev_status=st)
    _check_bwd(x, gamma, dy, dres, mean, rstd, rms, None, dgamma, dbeta)
    xh = (x.double() if rms else x.double() - mean.double()[:, None]).abs() * rstd.double()[:, None]
    tiny = (2.0 ** -134 if dtype == BF else 2.0 ** -150) + (5 + 2 * xh) * 2.0 ** -150
    DX = block.norm_bwd(dy, x, gamma, mean, rstd, dres, rms)[0]
    off = dx.double() - DX
    rest = off.sign() * (off.abs() - tiny).clamp_min(0)  # beyond the absolute part
    _check_bwd(x, gamma, dy, dres, mean, rstd, rms, DX + rest, None, None)
    assert int(st.item()) == 0


def test_gradient_agrees_with_autograd(cuda_device):
    """The whole chain x -> y -> loss against torch's differentiation of the definition in float64."""
    for rms in (False, True):
        x, gamma, beta, dy, _ = _make(5, 60, 384, F32, F32, True, rms)
        kind = F.NORM_RMS if rms else F.NORM_LAYER
        _, mean, rstd = F.falqon_norm_fwd(x, gamma, beta, 1e-5, kind)
        dx, dgamma, dbeta = F.falqon_norm_bwd(dy, x, gamma, mean, rstd, kind)
        leaves = [t.double().requires_grad_() for t in (x, gamma) + (() if rms else (beta,))]
        y = block.norm_fwd(leaves[0], leaves[1], None if rms else leaves[2], 1e-5, rms)[0]
        want = torch.autograd.grad((y * dy.double()).sum(), leaves)
        for got, w in zip((dx, dgamma, dbeta), want):
            # statistics off by (D / 2 + 6) e, sums of 60 rows by 124 e of their terms' sizes: 2e-5 covers both
            assert float((got - w).norm() / w.norm()) < 2e-5


def test_rows_past_31_bits_of_elements(cuda_device):
    """2^31 + elements: offsets are 64-bit.  Sampled rows, the last among them."""
    rows, cols = 262400, 8192  # 2.15e9 elements, 4.3 GB in bf16
    x = torch.empty(rows, cols, dtype=BF, device="cuda").normal_()
    gamma = torch.ones(cols, dtype=BF, device="cuda")
    y, _, rstd = F.falqon_norm_fwd(x, gamma, None, 1e-5, F.NORM_RMS)
    pick = torch.tensor([0, 1, 131071, 262143, 262144, rows - 1], device="cuda")
    _check_fwd(x[pick], gamma, None, 1e-5, True, y[pick], None, rstd[pick])
    dx, dgamma, _ = F.falqon_norm_bwd(y, x, gamma, None, rstd, F.NORM_RMS)
    xh = x[pick].double() * rstd[pick].double()[:, None]
    g = y[pick].double()
    want = (g - xh * (g * xh).mean(1, keepdim=True)) * rstd[pick].double()[:, None]
    # y is xh rounded: dx is what the rounding left, so it is compared with the size of g
    assert float((dx[pick].double() - want).abs().max()) < 2.0 ** -8 * float(want.abs().max()) + 1e-3 * 2.0 ** -8 + 2e-5
    assert float((dgamma / rows - 1).abs().max()) < 0.05  # mean of xh^2 over 262400 rows: 1 +- 6 sqrt(2 / 262400)
