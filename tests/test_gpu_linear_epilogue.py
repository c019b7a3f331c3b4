"""falqon_linear_fwd_epilogue / falqon_linear_epilogue_bwd against the float64
definitions.

The forward's tolerance: K products and sums of one float32 rounding each
(2^-23 where the tensor core cuts rather than rounds) for Z, the activation's
own error, one rounding of bf16.  `exact` inputs are small whole numbers whose
sums every order gives exactly."""

import math

import pytest
import torch

import fp8_quantized_lora_b200 as F
from gpu_util import kernels_of
from oracle import block

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
U = 2.0 ** -8  # bf16
BF, F32 = torch.bfloat16, torch.float32


def _value_error(z, which):
    """Of act(z) in float32, beyond the error of z.  exp(-t) is off by 2 + 1.2 |t| ulp and by 4 |t| e through t;
    GELU's normal CDF may be an approximation within 1.5e-7."""
    z = z.abs()
    if which == 2:
        return z * 2.0 ** -21
    if which in (3, 4):
        t = z if which == 4 else 1.6 * (z + 0.045 * z ** 3)
        p = block.act(z, which).abs().clamp_min(1e-30)
        return p * (8 + 6 * t.clamp_max(90)) * 2 * E + 2.0 ** -100
    return 0 * z


def _slope_error(z, which):
    a = z.double().abs()
    if which == 2:
        return (1 + a) * 2.0 ** -21
    if which in (3, 4):
        t = a if which == 4 else 1.6 * (a + 0.045 * a ** 3)
        c = 1.0 if which == 4 else 1.6 * (1 + 0.135 * a ** 2)
        p = torch.sigmoid(t if which == 4 else t)
        near = torch.exp(-t.clamp_max(80))  # 1 - p on the large side, p on the other
        return (8 + 6 * t.clamp_max(90)) * 2 * E * (p * near + a * c * near) + 4 * E * (1 + a * c * 2.0 ** -20)
    return 0 * a


def _codes(g, shape, std):
    x = torch.randn(shape, generator=g, device="cuda") * std
    c, s, _ = F.falqon_quantize(x)
    return c, s


def _check_fwd(xq, s_x, wq, s_w, bias, which, res, y, z):
    K = xq.shape[1]
    Y, Z = block.linear_fwd_epilogue(xq, s_x.item(), wq, s_w.item(), bias, which, res)
    mag = block.decode_e4m3(xq).abs() @ block.decode_e4m3(wq).abs().T / (s_x.item() * s_w.item())
    dz = (K + 8) * 2 * E * mag + 4 * E * Z.abs() + (0 if bias is None else 2 * E * bias.double().abs())
    if z is not None:
        tol = dz * (1 + U) + U * Z.abs()
        assert ((z - Z).abs() <= tol).all(), float(((z - Z).abs() - tol).max())
    err = 1.13 * dz + _value_error(Z, which) + (0 if res is None else 2 * E * res.double().abs()) + 2 * E * Y.abs()
    tol = err * (1 + U) + U * Y.abs()
    assert ((y - Y).abs() <= tol).all(), float(((y - Y).abs() - tol).max())


SHAPES = [(1, 16, 16), (1, 4096, 512), (2, 272, 336), (17, 48, 1008), (64, 528, 256), (65, 256, 512), (130, 256, 128),
          (200, 272, 336), (256, 512, 512), (300, 208, 144), (600, 1040, 272)]


@pytest.mark.parametrize("which", range(5))
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_forward(cuda_device, M, N, K, which):
    g = torch.Generator(device="cuda").manual_seed(M * 7 + N + which)
    xq, s_x = _codes(g, (M, K), 1.0)
    wq, s_w = _codes(g, (N, K), 0.1)
    bias = torch.randn(N, generator=g, device="cuda").to(BF if which % 2 else F32)
    res = torch.randn(M, N, generator=g, device="cuda").to(BF)
    ybuf, zbuf = (torch.full((M + 2, N), 7.0, dtype=BF, device="cuda") for _ in range(2))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, z = F.falqon_linear_fwd_epilogue(xq, s_x, wq, s_w, bias, which, res, z=zbuf[:M], y=ybuf[:M], dev_status=st)
    assert int(st.item()) == 0
    _check_fwd(xq, s_x, wq, s_w, bias, which, res, y, z)
    assert (ybuf[M:] == 7.0).all() and (zbuf[M:] == 7.0).all()
    # each part may be left out
    y, z = F.falqon_linear_fwd_epilogue(xq, s_x, wq, s_w, act=which)
    assert z is None
    _check_fwd(xq, s_x, wq, s_w, None, which, None, y, None)
    y, z = F.falqon_linear_fwd_epilogue(xq, s_x, wq, s_w, bias=bias, act=which, z=True)
    _check_fwd(xq, s_x, wq, s_w, bias, which, None, y, z)


@pytest.mark.parametrize("M,N,K", [(300, 208, 144), (512, 1040, 640), (4736, 1280, 256)])
def test_nothing_in_the_epilogue_is_the_plain_forward(cuda_device, M, N, K):
    """The same product; where both run 256 x 256 tiles the same bits, else float32 sums in another order: each is
    within (K + 8) 2^-23 of its terms' sizes and half a step of bf16."""
    g = torch.Generator(device="cuda").manual_seed(M)
    xq, s_x = _codes(g, (M, K), 1.0)
    wq, s_w = _codes(g, (N, K), 0.02)
    y, _ = F.falqon_linear_fwd_epilogue(xq, s_x, wq, s_w)
    plain = F.falqon_linear_fwd(xq, s_x, wq, s_w)
    if M > 4096:
        assert torch.equal(y, plain)
    mag = block.decode_e4m3(xq).abs() @ block.decode_e4m3(wq).abs().T / (s_x.item() * s_w.item())
    tol = 2 * ((K + 8) * 2 * E * mag + U * plain.double().abs()) * (1 + U)
    assert ((y.double() - plain.double()).abs() <= tol).all()


@pytest.mark.parametrize("M,N,K", [(1, 16, 16), (1, 4096, 4096), (3, 176, 11008), (33, 4096, 2064), (64, 1040, 4096),
                                   (128, 4096, 1024), (257, 1040, 4096), (1024, 2048, 2048)])
def test_whole_numbers_are_exact(cuda_device, M, N, K):
    """Codes of -2 .. 2: Z is a whole number below 2^24, so Y is its rounding whatever the order of the sums."""
    g = torch.Generator(device="cuda").manual_seed(N + K)
    v = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").float()  # noqa: E731
    x, w, bias, res = v(M, K), v(N, K), v(N), v(M, N).to(BF)
    one = torch.ones(1, device="cuda")
    xq, wq = (t.to(torch.float8_e4m3fn).view(torch.uint8) for t in (x, w))
    for which in (0, 1):
        y, z = F.falqon_linear_fwd_epilogue(xq, one, wq, one, bias, which, res, z=True)
        Z = x.double() @ w.double().T + bias
        Y = (Z.clamp_min(0) if which else Z) + res
        assert torch.equal(z, Z.to(F32).to(BF)) and torch.equal(y, Y.to(F32).to(BF))


# Products that the rule leaves to 256 x 256 tiles on SM pairs (ragged rows, columns and K; a tile of 16 columns; more
# tiles than pairs, whose rest runs whole or, at 4736 x 1280 and 2304 x 2064, in halves), few-row plans of 128 rows a
# tile, which 64-row tiles are more than two an SM for, in more than one wave, and the largest plan of 64 rows (296
# tiles; 297 at 19000 rows).
PAIR, FEW128, FEW64 = "tc_gemm_pair_kernel", "6FewCfgILi128E", "6FewCfgILi64E"
TILED = [(PAIR, 2048, 1296, 512), (PAIR, 4736, 1280, 256), (PAIR, 4700, 1296, 272), (PAIR, 2304, 2064, 1040),
         (PAIR, 700, 2064, 8192), (FEW128, 300, 11008, 128), (FEW128, 20000, 128, 512), (FEW128, 19000, 128, 272),
         (FEW64, 18900, 128, 272)]


@pytest.mark.parametrize("which", range(5))
@pytest.mark.parametrize("kernel,M,N,K", TILED)
def test_forward_of_each_kernel(cuda_device, kernel, M, N, K, which):
    """test_forward's checks where the rule takes the kernel named."""
    g = torch.Generator(device="cuda").manual_seed(M * 7 + N + which)
    xq, s_x = _codes(g, (M, K), 1.0)
    wq, s_w = _codes(g, (N, K), 0.1)
    res = torch.randn(M, N, generator=g, device="cuda").to(BF)
    ybuf, zbuf = (torch.full((M + 2, N), 7.0, dtype=BF, device="cuda") for _ in range(2))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dtype in (BF, F32):
        bias = torch.randn(N, generator=g, device="cuda").to(dtype)
        ybuf[:M], zbuf[:M] = math.nan, math.nan

        def call():
            return F.falqon_linear_fwd_epilogue(xq, s_x, wq, s_w, bias, which, res, z=zbuf[:M], y=ybuf[:M],
                                                dev_status=st)
        y, z = call()
        assert int(st.item()) == 0
        _check_fwd(xq, s_x, wq, s_w, bias, which, res, y, z)
        assert (ybuf[M:] == 7.0).all() and (zbuf[M:] == 7.0).all()
        launched = kernels_of(call)
        assert len(launched) == 1 and kernel in launched[0][0], launched
    # without the residual or Z, and the activation alone
    y, none = F.falqon_linear_fwd_epilogue(xq, s_x, wq, s_w, bias, which)
    assert none is None
    _check_fwd(xq, s_x, wq, s_w, bias, which, None, y, None)
    y, _ = F.falqon_linear_fwd_epilogue(xq, s_x, wq, s_w, act=which)
    _check_fwd(xq, s_x, wq, s_w, None, which, None, y, None)
    y, z = F.falqon_linear_fwd_epilogue(xq, s_x, wq, s_w, act=which, residual=res, z=True)
    _check_fwd(xq, s_x, wq, s_w, None, which, res, y, z)


@pytest.mark.parametrize("kernel,M,N,K", TILED)
def test_whole_numbers_are_exact_in_each_kernel(cuda_device, kernel, M, N, K):
    """test_whole_numbers_are_exact's checks where the rule takes the kernel named."""
    g = torch.Generator(device="cuda").manual_seed(N + K)
    v = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").float()  # noqa: E731
    x, w, bias, res = v(M, K), v(N, K), v(N), v(M, N).to(BF)
    one = torch.ones(1, device="cuda")
    xq, wq = (t.to(torch.float8_e4m3fn).view(torch.uint8) for t in (x, w))
    for which in (0, 1):
        y, z = F.falqon_linear_fwd_epilogue(xq, one, wq, one, bias, which, res, z=True)
        Z = x.double() @ w.double().T + bias
        Y = (Z.clamp_min(0) if which else Z) + res
        assert torch.equal(z, Z.to(F32).to(BF)) and torch.equal(y, Y.to(F32).to(BF))


def test_codes_may_be_float8_tensors_and_large_values_stay(cuda_device):
    g = torch.Generator(device="cuda").manual_seed(1)
    xq, s_x = _codes(g, (40, 64), 1.0)
    wq, s_w = _codes(g, (32, 64), 1.0)
    bias = torch.zeros(32, device="cuda")
    bias[0], bias[1], bias[2], bias[3] = 200.0, -200.0, 1e30, -1e30
    for which in range(1, 5):
        y, _ = F.falqon_linear_fwd_epilogue(xq.view(torch.float8_e4m3fn), s_x, wq.view(torch.float8_e4m3fn), s_w,
                                            bias, which)
        _check_fwd(xq, s_x, wq, s_w, bias, which, None, y, None)
        assert torch.isfinite(y).all()
        assert (y[:, 1] == 0).all() and (y[:, 3] == 0).all()


def test_wrong_shapes_are_refused(cuda_device):
    g = torch.Generator(device="cuda").manual_seed(1)
    xq, s = _codes(g, (8, 32), 1.0)
    wq, _ = _codes(g, (16, 32), 1.0)
    for kw in (dict(bias=torch.zeros(15, device="cuda")), dict(bias=torch.zeros(16, device="cuda").double()),
               dict(residual=torch.zeros(8, 16, device="cuda")), dict(residual=torch.zeros(7, 16, device="cuda").to(BF)),
               dict(y=torch.zeros(8, 15, device="cuda").to(BF)), dict(z=torch.zeros(16, 8, device="cuda").to(BF).t())):
        with pytest.raises(ValueError):
            F.falqon_linear_fwd_epilogue(xq, s, wq, s, **kw)
    with pytest.raises(ValueError):
        F.falqon_linear_fwd_epilogue(xq, s, wq[:, :16].contiguous(), s)
    with pytest.raises(F.FalqonError):
        F.falqon_linear_fwd_epilogue(xq, s, wq, s, act=5)


def _check_bwd(dy, z, which, dz, dbias):
    DZ, DB = block.linear_epilogue_bwd(dy, z, which)
    err = 0 if which == 0 else dy.double().abs() * _slope_error(z, which) + 2 * E * DZ.abs()
    if dz is not None:
        tol = err * (1 + U) + U * DZ.abs() + 1e-40
        assert ((dz - DZ).abs() <= tol).all(), float(((dz - DZ).abs() - tol).max())
    if dbias is not None:
        R = min(dy.shape[0], 2048) + 64
        tol = (err.sum(0) if which else 0) + R * E * DZ.abs().sum(0)
        assert ((dbias - DB).abs() <= tol).all()


@pytest.mark.parametrize("which", range(5))
@pytest.mark.parametrize("M,N", [(1, 16), (7, 48), (8, 256), (9, 272), (200, 272), (1000, 1008), (3001, 528),
                                 (2, 11008), (5000, 16)])
def test_backward(cuda_device, M, N, which):
    g = torch.Generator(device="cuda").manual_seed(M + N + which)
    dy = torch.randn(M, N, generator=g, device="cuda").to(BF)
    z = (2.5 * torch.randn(M, N, generator=g, device="cuda")).to(BF)
    z[0, :8] = torch.tensor([0.0, -0.0, 30.0, -30.0, 1000.0, -1000.0, 1e-30, -1e-30], device="cuda").to(BF)
    buf = torch.full((M + 2, N), 7.0, dtype=BF, device="cuda")
    need = F.falqon_workspace_size(F.OP_LINEAR_EPILOGUE_BWD, M, N)
    raw = torch.full((need // 4 + 128,), math.nan, device="cuda")
    off = (-raw.data_ptr() // 4) % 64
    dz, dbias = F.falqon_linear_epilogue_bwd(dy, z, which, dz=buf[:M],
                                             workspace=raw[off:off + need // 4].view(torch.uint8))
    _check_bwd(dy, z, which, dz, dbias)
    assert (buf[M:] == 7.0).all() and torch.isnan(raw[off + need // 4:]).all()
    a, none = F.falqon_linear_epilogue_bwd(dy, z, which, dbias=None)
    none2, b = F.falqon_linear_epilogue_bwd(dy, z, which, dz=None)
    assert none is None and none2 is None and torch.equal(a, dz) and torch.equal(b, dbias)
    if which == 0:
        assert torch.equal(dz, dy)
        assert torch.equal(F.falqon_linear_epilogue_bwd(dy, None, which, dz=None)[1], dbias)


@pytest.mark.parametrize("which", range(1, 5))
def test_backward_up_to_the_largest_pre_activation(cuda_device, which):
    """Past |z| = 1000 every slope is 1 or 0 (the rest is below 1e-400), so dz is dy or 0 without a rounding, and
    the sums of a few powers of two are exact; a NaN stays one."""
    big = torch.tensor([1e3, 1e10, 1.8e19, 1e25, 1e30, 3.8e36, 4e36, 1e37, 1e38, 3.3e38, 3.38e38], device="cuda")
    z = torch.zeros(70, 32, device="cuda")
    z[:, :11], z[:, 11:22] = big, -big
    z = z.to(BF)
    dy = torch.full_like(z, 2.0 ** -6)
    dz, dbias = F.falqon_linear_epilogue_bwd(dy, z, which)
    assert torch.equal(dz[:, :11], dy[:, :11]) and (dz[:, 11:22] == 0).all()
    assert (dbias[:11] == 70 * 2.0 ** -6).all() and (dbias[11:22] == 0).all()
    z[3, 5] = math.nan
    if which != 1:  # ReLU's slope is a comparison
        dz, dbias = F.falqon_linear_epilogue_bwd(dy, z, which)
        assert torch.isnan(dz[3, 5]) and torch.isnan(dbias[5]) and int(torch.isnan(dz).sum()) == 1


@pytest.mark.parametrize("which", range(1, 5))
@pytest.mark.parametrize("M", [3, 2304])
def test_columns_masked_by_the_lowest_bias(cuda_device, M, which):
    """A float32 bias of its type's lowest value switches a column off: y is 0 there, the bf16 Z that is kept is
    -infinity (the lowest float32 is past bf16's by 3/4 of a step), and the gradient is 0, not NaN.  The greatest is
    +infinity with slope 1."""
    g = torch.Generator(device="cuda").manual_seed(which)
    N, K = 272, 64
    (xq, s_x), (wq, s_w) = _codes(g, (M, K), 1.0), _codes(g, (N, K), 0.1)
    bias = torch.randn(N, generator=g, device="cuda")
    off, on = torch.arange(0, N, 5, device="cuda"), torch.arange(1, N, 5, device="cuda")
    bias[off], bias[on] = torch.finfo(F32).min, torch.finfo(F32).max
    y, z = F.falqon_linear_fwd_epilogue(xq, s_x, wq, s_w, bias, which, z=True)
    assert (y[:, off] == 0).all() and (z[:, off] == -math.inf).all() and (z[:, on] == math.inf).all()
    rest = torch.ones(N, dtype=torch.bool, device="cuda")
    rest[off] = rest[on] = False
    dy = torch.full((M, N), 2.0 ** -6, dtype=BF, device="cuda")
    dz, dbias = F.falqon_linear_epilogue_bwd(dy, z, which)
    assert (dz[:, off] == 0).all() and (dbias[off] == 0).all()
    assert torch.equal(dz[:, on], dy[:, on]) and (dbias[on] == M * 2.0 ** -6).all()
    zr, dyr = z[:, rest], dy[:, rest]
    _check_bwd(dyr, zr, which, dz[:, rest], dbias[rest])


def test_gradient_against_differences(cuda_device):
    """The slope that the backward applies against differences of the forward's own activation: N(0, 1)
    pre-activations, one sample per element.  The forward's outputs are bf16, so the differences are taken of the
    float64 definition that the forward is held to, and the step is 2^-10."""
    z = torch.linspace(-6, 6, 16 * 64, device="cuda").reshape(64, 16).to(BF)
    dy = torch.ones_like(z)
    h = 2.0 ** -10
    for which in range(1, 5):
        zz = z + 0.0625 if which == 1 else z
        dz, _ = F.falqon_linear_epilogue_bwd(dy, zz, which)
        num = (block.act(zz.double() + h, which) - block.act(zz.double() - h, which)) / (2 * h)
        # h^2 f''' / 6 < 2^-20, one rounding of a value up to 1.13
        assert float((dz.double() - num).abs().max()) < 1.13 * U + 2.0 ** -20
