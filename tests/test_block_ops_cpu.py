"""CPU checks of the operators around the linear layer: argument errors of the
C calls (returned before any CUDA call), refusals of the binding, and the
float64 definitions against differences and an independent decoding."""

import ctypes as C
import math

import pytest
import torch

import fp8_quantized_lora_b200 as F
from oracle import block

# Fake, 256-byte aligned addresses: a call is refused before any is read.
P = C.c_void_p(1 << 20)
P8 = C.c_void_p((1 << 20) + 8)
BF, F32 = 0, 1
LAYER, RMS = 0, 1
NAN, INF = math.nan, math.inf


def test_workspace_sizes():
    for op, args in ((F.OP_NORM_BWD, (4096, 0, 4096)), (F.OP_NORM_BWD, (1, 0, 1)), (F.OP_NORM_BWD, (3, 0, 70001)),
                     (F.OP_LINEAR_EPILOGUE_BWD, (1, 16)), (F.OP_LINEAR_EPILOGUE_BWD, (8192, 11008)),
                     (F.OP_CLIP_GRADS, ())):
        n = F.falqon_workspace_size(op, *args)
        assert n > 0 and n % 256 == 0, (op, args)
    assert F.falqon_workspace_size(F.OP_NORM_BWD, 0, 0, 4096) == 0
    assert F.falqon_workspace_size(F.OP_LINEAR_EPILOGUE_BWD, 16, 0) == 0


def test_norm_fwd_argument_errors():
    f = F.lib().falqon_norm_fwd

    def call(x=P, dt=BF, gamma=P, beta=P, pt=BF, kind=LAYER, rows=4, cols=24, eps=1e-5, y=P, mean=P, rstd=P):
        return f(x, dt, gamma, beta, pt, kind, rows, cols, eps, y, mean, rstd, None, None)
    assert call(x=None) == 1 and call(y=None) == 1
    assert call(dt=2) == 1 and call(pt=-1) == 1 and call(kind=2) == 1
    assert call(rows=0) == 1 and call(cols=0) == 1 and call(rows=-4) == 1
    assert call(eps=-1e-5) == 1 and call(eps=NAN) == 1 and call(eps=INF) == 1
    assert call(kind=RMS) == 1                       # beta
    assert call(kind=RMS, beta=None) == 1            # mean
    assert call(rows=1 << 31) == 2 and call(cols=1 << 31) == 2
    for name in ("x", "y", "gamma", "beta", "mean", "rstd"):
        assert call(**{name: P8}) == 2, name


def test_norm_bwd_argument_errors():
    f = F.lib().falqon_norm_bwd

    def call(dy=P, x=P, dt=BF, gamma=P, pt=BF, kind=LAYER, mean=P, rstd=P, dres=P, rows=4, cols=24, dx=P, dgamma=P,
             dbeta=P, ws=P, wsb=1 << 20):
        return f(dy, x, dt, gamma, pt, kind, mean, rstd, dres, rows, cols, dx, dgamma, dbeta, None, ws, wsb, None)
    assert call(dx=None, dgamma=None, dbeta=None) == 1
    assert call(dy=None) == 1 and call(x=None) == 1 and call(rstd=None) == 1 and call(mean=None) == 1
    assert call(dt=7) == 1 and call(pt=7) == 1 and call(kind=5) == 1 and call(rows=0) == 1 and call(cols=-1) == 1
    assert call(kind=RMS) == 1                                   # a mean
    assert call(kind=RMS, mean=None) == 1                        # a dbeta
    assert call(dx=None) == 1                                    # dres without dx
    for name in ("dy", "x", "gamma", "mean", "rstd", "dres", "dx", "dgamma", "dbeta"):
        assert call(**{name: P8}) == 2, name
    need = F.falqon_workspace_size(F.OP_NORM_BWD, 4, 0, 24)
    assert call(ws=None, wsb=0) == 3 and call(wsb=need - 1) == 3 and call(ws=P8) == 3


def test_linear_epilogue_argument_errors():
    f = F.lib().falqon_linear_fwd_epilogue

    def call(xq=P, sx=P, wq=P, sw=P, bias=P, bt=BF, act=1, res=P, M=4, N=32, K=48, z=P, y=P):
        return f(xq, sx, wq, sw, bias, bt, act, res, M, N, K, z, y, None, None)
    for name in ("xq", "sx", "wq", "sw", "y"):
        assert call(**{name: None}) == 1, name
    assert call(act=5) == 1 and call(act=-1) == 1 and call(bt=3) == 1
    assert call(M=0) == 1 and call(N=-16) == 1 and call(K=0) == 1
    assert call(N=24) == 2 and call(K=40) == 2 and call(M=1 << 31) == 2
    for name in ("xq", "wq", "bias", "res", "z", "y"):
        assert call(**{name: P8}) == 2, name
    b = F.lib().falqon_linear_epilogue_bwd

    def bwd(dy=P, z=P, act=4, M=4, N=32, dz=P, db=P, ws=P, wsb=1 << 20):
        return b(dy, z, act, M, N, dz, db, ws, wsb, None)
    assert bwd(dz=None, db=None) == 1 and bwd(dy=None) == 1 and bwd(z=None) == 1 and bwd(act=9) == 1
    assert bwd(M=0) == 1 and bwd(N=0) == 1 and bwd(N=24) == 2 and bwd(M=1 << 31) == 2
    for name in ("dy", "z", "dz", "db"):
        assert bwd(**{name: P8}) == 2, name
    assert bwd(ws=None, wsb=0) == 3 and bwd(wsb=64) == 3 and bwd(ws=P8) == 3


def test_outputs_over_inputs_or_one_another_are_refused():
    def at(i):
        return C.c_void_p((1 << 20) + (i << 12))

    def refused(f, args, outs, ins):
        # each output moved onto each input and each other output, and onto its last bytes
        for o, size in outs.items():
            for other, n in {**ins, **outs}.items():
                if other == o:
                    continue
                for where in (0, (n - 1) // 16 * 16):
                    moved = dict(args, **{o: C.c_void_p(args[other].value + where)})
                    assert f(**moved) == 1, (o, other, where)

    ws, wsb = C.c_void_p(1 << 28), 1 << 24
    L = F.lib()
    rows, cols = 8, 24
    mat, par, per_row, per_col = rows * cols * 2, cols * 2, rows * 4, cols * 4
    args = {k: at(i) for i, k in enumerate(("x", "gamma", "beta", "y", "mean", "rstd"))}
    refused(lambda x, gamma, beta, y, mean, rstd: L.falqon_norm_fwd(
        x, BF, gamma, beta, BF, LAYER, rows, cols, 1e-5, y, mean, rstd, None, None),
        args, dict(y=mat, mean=per_row, rstd=per_row), dict(x=mat, gamma=par, beta=par))
    args = {k: at(i) for i, k in enumerate(("dy", "x", "gamma", "mean", "rstd", "dres", "dx", "dg", "db"))}
    refused(lambda dy, x, gamma, mean, rstd, dres, dx, dg, db: L.falqon_norm_bwd(
        dy, x, BF, gamma, BF, LAYER, mean, rstd, dres, rows, cols, dx, dg, db, None, ws, wsb, None),
        args, dict(dx=mat, dg=per_col, db=per_col),
        dict(dy=mat, x=mat, gamma=par, mean=per_row, rstd=per_row, dres=mat))
    M, N, K = 4, 32, 48
    args = {k: at(i) for i, k in enumerate(("xq", "sx", "wq", "sw", "bias", "res", "z", "y"))}
    refused(lambda xq, sx, wq, sw, bias, res, z, y: L.falqon_linear_fwd_epilogue(
        xq, sx, wq, sw, bias, BF, 1, res, M, N, K, z, y, None, None),
        args, dict(z=M * N * 2, y=M * N * 2), dict(xq=M * K, wq=N * K, bias=N * 2, res=M * N * 2, sx=4, sw=4))
    args = {k: at(i) for i, k in enumerate(("dy", "z", "dz", "db"))}
    refused(lambda dy, z, dz, db: L.falqon_linear_epilogue_bwd(dy, z, 4, M, N, dz, db, ws, wsb, None),
            args, dict(dz=M * N * 2, db=N * 4), dict(dy=M * N * 2, z=M * N * 2))


def _clip(ptrs=(1 << 20, 1 << 21), dtypes=(BF, F32), numel=(100, 50), max_norm=1.0, factor=1.0, outs=None, norm=P,
          ws=P, wsb=1 << 20, n=None):
    k = len(ptrs)
    vp = lambda v: None if v is None else (C.c_void_p * len(v))(*v)  # noqa: E731
    return F.lib().falqon_clip_grads(k if n is None else n, vp(ptrs), (C.c_int * k)(*dtypes), (C.c_int64 * k)(*numel),
                                     max_norm, factor, vp(outs), norm, None, None, ws, wsb, None)


def test_clip_argument_errors():
    A, B = 1 << 20, 1 << 21
    assert _clip(n=0) == 1 and _clip(n=-1) == 1 and _clip(norm=None) == 1
    assert _clip(max_norm=0.0) == 1 and _clip(max_norm=-1.0) == 1 and _clip(max_norm=NAN) == 1
    assert _clip(factor=NAN) == 1 and _clip(factor=INF) == 1
    assert _clip(dtypes=(BF, 2)) == 1 and _clip(numel=(100, -1)) == 1
    assert _clip(ptrs=(None, B)) == 1 and _clip(outs=(A, None)) == 1
    assert _clip(ptrs=(A + 8, B)) == 2 and _clip(outs=(A, B + 4)) == 2
    assert _clip(numel=(1 << 43, 1)) == 2 and _clip(numel=(1 << 42, 1 << 42)) == 3 - 1
    assert _clip(ws=None, wsb=0) == 3 and _clip(wsb=16) == 3 and _clip(ws=P8) == 3
    # a refused size comes before the workspace, so these get that far: no overlap
    bad_ws = dict(ws=None, wsb=0)
    assert _clip(outs=(A, B), **bad_ws) == 3                        # in place
    assert _clip(outs=(A + 4096, B + 4096), **bad_ws) == 3          # apart
    assert _clip(ptrs=(A, A), dtypes=(BF, BF), numel=(100, 100), **bad_ws) == 3  # counted twice, nothing written
    assert _clip(ptrs=(A, None), numel=(100, 0), outs=(A, None), **bad_ws) == 3  # no elements: pointers unused


def test_clip_refuses_overlapping_outputs():
    A, B = 1 << 20, 1 << 21
    same = dict(dtypes=(BF, BF), numel=(100, 100))
    assert _clip(ptrs=(A, A), outs=(A, A), **same) == 1            # the same tensor twice, in place
    assert _clip(ptrs=(A, B), outs=(B + 4096, B + 4096), **same) == 1  # two outputs in one place
    assert _clip(ptrs=(A, B), outs=(B + 4096, B + 4112), **same) == 1  # overlapping outputs
    assert _clip(ptrs=(A, B), outs=(B, A), **same) == 1            # outputs swapped with the gradients
    assert _clip(ptrs=(A, B), outs=(A + 16, B), **same) == 1       # an output that begins inside its gradient
    assert _clip(ptrs=(A, A + 208), outs=(A + 208, B), numel=(104, 8), dtypes=(BF, BF)) == 1  # onto the next one
    assert _clip(ptrs=(A, A + 208), outs=(A, A + 208), numel=(104, 8), dtypes=(BF, BF), ws=None, wsb=0) == 3


def test_clip_refuses_results_over_tensors_or_one_another():
    """norm and coef are outputs like the others: each at the first and the last float of a gradient, of an output,
    and in one place, with and without outputs."""
    A, B, O, Q, R = (v << 20 for v in (1, 2, 3, 4, 5))
    ws = C.c_void_p(1 << 28)
    vp = lambda v: None if v is None else (C.c_void_p * len(v))(*v)  # noqa: E731
    dtypes, numel = (C.c_int * 2)(BF, F32), (C.c_int64 * 2)(100, 50)  # 200 bytes each

    def call(norm, coef=None, outs=None):
        return F.lib().falqon_clip_grads(2, vp((A, B)), dtypes, numel, 1.0, 1.0, vp(outs), C.c_void_p(norm),
                                         None if coef is None else C.c_void_p(coef), None, ws, 1 << 20, None)
    for outs in (None, (O, Q), (A, B)):
        assert call(R, R, outs) == 1
        for begin in (A, B) + (outs or ()):
            for at in (begin, begin + 196):
                assert call(at, R, outs) == 1 and call(R, at, outs) == 1 and call(at, None, outs) == 1
        assert call(R + 2, None, outs) == 2 and call(R, R + 5, outs) == 2


def test_a_gradient_list_keeps_or_follows_its_memory(monkeypatch):
    """The pointers that reach the C call, recorded in its place: always of memory that is alive, whatever became of
    the tensors, and a refusal where that memory was given back."""
    seen = []

    class Recorder:
        @staticmethod
        def falqon_clip_grads(n, grads, dtypes, numel, max_norm, factor, outs, *rest):
            seen.append([(grads[i], numel[i], None if outs is None else outs[i]) for i in range(n)])
            return 0
    monkeypatch.setattr(F, "lib", Recorder)
    monkeypatch.setattr(F, "_ptr", lambda t: C.c_void_p(t.data_ptr()))
    monkeypatch.setattr(F, "_elsewhere", lambda dev, stream: None)
    monkeypatch.setattr(F, "_raw_stream", lambda dev: None)
    monkeypatch.setattr(F, "falqon_workspace_size", lambda *a: 256)
    flat = torch.zeros(64)
    grads = [torch.zeros(40), flat[8:16], flat[24:64], torch.zeros(0)]
    outs = [torch.zeros(n) for n in (40, 8, 40, 0)]
    g, o = F.GradList(grads), F.GradList(outs)

    def pointers(out):
        F.falqon_clip_grads(g, 1.0, out=out)
        return [(p, q) for p, _, q in seen[-1]]

    first = [t.data_ptr() for t in grads[:3]] + [None]
    outs_at = [t.data_ptr() for t in outs[:3]] + [None]
    assert pointers(None) == [(p, None) for p in first] and [n for _, n, _ in seen[-1]] == [40, 8, 40, 0]
    assert pointers(o) == list(zip(first, outs_at)) and pointers(g) == list(zip(first, first))
    # other memory for a tensor: the list still stands for, and holds, the old
    grads[0].data = torch.ones(40)
    grads[1].set_(torch.ones(8))
    again = [torch.full((40,), 2.0) for _ in range(50)]  # none of which may get the old memory
    assert first[0] not in [t.data_ptr() for t in again]
    assert pointers(o) == list(zip(first, outs_at))
    # a storage that moves takes its tensors along
    flat.resize_(1 << 18)
    assert flat.data_ptr() != first[1] - 32
    moved = [first[0], flat.data_ptr() + 32, flat.data_ptr() + 96, None]
    assert pointers(None) == [(p, None) for p in moved] and pointers(o) == list(zip(moved, outs_at))
    outs[2].resize_(1 << 18)
    outs_at[2] = outs[2].data_ptr()
    assert pointers(o) == list(zip(moved, outs_at))
    # given back: refused, and so are the calls after it
    flat.untyped_storage().resize_(0)
    for _ in range(2):
        with pytest.raises(ValueError):
            F.falqon_clip_grads(g, 1.0)
    with pytest.raises(ValueError):
        F.falqon_clip_grads(o, 1.0, out=g)


def test_binding_refuses_wrong_tensors():
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    for call in (lambda: F.falqon_norm_fwd(x), lambda: F.falqon_norm_fwd(x[0]),
                 lambda: F.falqon_norm_bwd(x, x, None, torch.zeros(4), torch.zeros(4)),
                 lambda: F.falqon_linear_fwd_epilogue(x, torch.ones(1), x, torch.ones(1)),
                 lambda: F.falqon_linear_epilogue_bwd(x, x, F.ACT_RELU),
                 lambda: F.falqon_clip_grads([x], 1.0), lambda: F.GradList([]),
                 lambda: F.GradList([x.half()])):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("rms", [False, True])
def test_norm_gradient_against_differences(rms):
    g = torch.Generator().manual_seed(3)
    x, dy = (torch.randn(3, 7, generator=g, dtype=torch.float64) for _ in range(2))
    gamma, beta = (torch.randn(7, generator=g, dtype=torch.float64) for _ in range(2))
    beta = None if rms else beta
    _, mean, rstd = block.norm_fwd(x, gamma, beta, 1e-3, rms)
    dx, dgamma, dbeta = block.norm_bwd(dy, x, gamma, mean, rstd, None, rms)

    def slope(t, i, h=1e-5):
        keep = t.view(-1)[i].item()
        v = []
        for s in (h, -h):
            t.view(-1)[i] = keep + s
            v.append((block.norm_fwd(x, gamma, beta, 1e-3, rms)[0] * dy).sum())
        t.view(-1)[i] = keep
        return float(v[0] - v[1]) / (2 * h)
    # central differences: error h^2 f''' / 6 + 2^-53 |f| / h, below 1e-8 here
    for t, d in ((x, dx), (gamma, dgamma)) + (() if rms else ((beta, dbeta),)):
        for i in range(t.numel()):
            assert abs(slope(t, i) - d.view(-1)[i].item()) < 1e-7


@pytest.mark.parametrize("which", range(5))
def test_activation_slopes_against_differences_and_torch(which):
    z = torch.linspace(-9, 9, 361, dtype=torch.float64) + 0.0125  # not at ReLU's corner
    h = 1e-5
    num = (block.act(z + h, which) - block.act(z - h, which)) / (2 * h)
    assert float((num - block.act_slope(z, which)).abs().max()) < 1e-8
    f = torch.nn.functional
    ref = (lambda v: v, f.relu, f.gelu, lambda v: f.gelu(v, approximate="tanh"), f.silu)[which]
    assert float((ref(z) - block.act(z, which)).abs().max()) < 1e-12


def test_decoding_matches_the_format():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double()
    got = block.decode_e4m3(codes)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(got[ok], want[ok])


def test_clip_definition():
    g = [torch.tensor([3.0, 0.0]), torch.tensor([4.0])]
    outs, norm, coef = block.clip_grads(g, 2.5, -0.1)
    assert norm == 5.0 and coef == 0.5 and torch.allclose(outs[0], torch.tensor([-0.15, 0.0], dtype=torch.float64))
    assert block.clip_grads(g, 5.0)[2] == 1.0 and block.clip_grads(g, INF)[2] == 1.0
    outs, norm, coef = block.clip_grads([torch.tensor([1.0, INF])], 1.0)
    assert norm == INF and coef == 0.0 and not outs[0].any()
