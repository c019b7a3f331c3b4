"""The norm, the linear layer's epilogue and the gradient clip together, around
the quantized linear layers, as a fine-tuning step of an MLP block uses them:

  x -> RMS norm -> quantize -> linear (bias, GELU) -> quantize -> linear (bias, + x)
  and back: bias gradients, adapter gradients, the norm's gradient joined by the
  residual's, the global clip, the increments into the proxy update.

Every step is held to its definition on the inputs that it got."""

import math
import pathlib
import subprocess
import sys
import threading
import types

import pytest
import torch

import fp8_quantized_lora_b200 as F
from oracle import block

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
U = 2.0 ** -8
E = 2.0 ** -24
LR, MAX_NORM = 1e-2, 1e-3


class Block:
    """Buffers of one MLP block of width K, hidden N, adapters of rank r, for M tokens."""

    def __init__(self, M, K, N, r, seed=0, dev="cuda"):
        g = torch.Generator(device=dev).manual_seed(seed)
        rnd = lambda *s, std=1.0: torch.randn(s, generator=g, device=dev) * std  # noqa: E731
        self.M, self.K, self.N, self.r = M, K, N, r
        self.x, self.dy = rnd(M, K).to(BF), rnd(M, K, std=1e-3).to(BF)
        self.gamma = (1 + rnd(K, std=0.1)).to(BF)
        self.b1, self.b2 = rnd(N, std=0.1).to(BF), rnd(K, std=0.1)
        (self.w1, self.s1, _), (self.w2, self.s2, _) = (F.falqon_quantize(rnd(N, K, std=0.05)),
                                                        F.falqon_quantize(rnd(K, N, std=0.05)))
        self.A1, self.B1 = rnd(r, K, std=0.01).to(BF), rnd(N, r, std=1e-3).to(BF)
        self.A2, self.B2 = rnd(r, N, std=0.01).to(BF), rnd(K, r, std=1e-3).to(BF)
        self.P1, self.P2 = torch.zeros(N, K, device=dev), torch.zeros(K, N, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        ws = lambda op, *s: F.workspace(op, *s)  # noqa: E731
        self.ws = dict(q1=ws(F.OP_QUANTIZE, M, K), q2=ws(F.OP_QUANTIZE, M, N), q3=ws(F.OP_QUANTIZE, M, K),
                       q4=ws(F.OP_QUANTIZE, M, N), e1=ws(F.OP_LINEAR_EPILOGUE_BWD, M, N),
                       e2=ws(F.OP_LINEAR_EPILOGUE_BWD, M, K), n=ws(F.OP_NORM_BWD, M, 0, K),
                       l1=ws(F.OP_LINEAR_BWD, M, N, K, r), l2=ws(F.OP_LINEAR_BWD, M, K, N, r),
                       c=ws(F.OP_CLIP_GRADS), p1=ws(F.OP_PROXY_UPDATE, 0, N, K), p2=ws(F.OP_PROXY_UPDATE, 0, K, N))

    def step(self):
        st, ws, o = self.status, self.ws, {}
        o["h"], _, o["rstd"] = F.falqon_norm_fwd(self.x, self.gamma, kind=F.NORM_RMS, dev_status=st)
        o["hq"], o["sh"], _ = F.falqon_quantize(o["h"], dev_status=st, workspace=ws["q1"])
        o["a"], o["z"] = F.falqon_linear_fwd_epilogue(o["hq"], o["sh"], self.w1, self.s1, self.b1, F.ACT_GELU_TANH,
                                                      z=True, dev_status=st)
        o["aq"], o["sa"], _ = F.falqon_quantize(o["a"], dev_status=st, workspace=ws["q2"])
        o["y"], _ = F.falqon_linear_fwd_epilogue(o["aq"], o["sa"], self.w2, self.s2, self.b2, residual=self.x,
                                                 dev_status=st)
        # backward: dy is the gradient of y, and of the residual branch
        _, o["db2"] = F.falqon_linear_epilogue_bwd(self.dy, None, F.ACT_NONE, dz=None, workspace=ws["e2"])
        o["dyq"], o["sdy"], _ = F.falqon_quantize(self.dy, dev_status=st, workspace=ws["q3"])
        o["da"], _, o["dB2"] = F.falqon_linear_bwd(o["dyq"], o["sdy"], self.w2, self.s2, o["aq"], o["sa"], self.A2,
                                                   self.B2, dA=None, dev_status=st, workspace=ws["l2"])
        o["dz"], o["db1"] = F.falqon_linear_epilogue_bwd(o["da"], o["z"], F.ACT_GELU_TANH, workspace=ws["e1"])
        o["dzq"], o["sdz"], _ = F.falqon_quantize(o["dz"], dev_status=st, workspace=ws["q4"])
        o["dh"], _, o["dB1"] = F.falqon_linear_bwd(o["dzq"], o["sdz"], self.w1, self.s1, o["hq"], o["sh"], self.A1,
                                                   self.B1, dA=None, dev_status=st, workspace=ws["l1"])
        o["dx"], o["dgamma"], _ = F.falqon_norm_bwd(o["dh"], self.x, self.gamma, None, o["rstd"], F.NORM_RMS,
                                                    dres=self.dy, dev_status=st, workspace=ws["n"])
        grads = [o["dB1"], o["dB2"], o["db1"], o["db2"], o["dgamma"]]
        o["inc"], o["norm"], o["coef"] = F.falqon_clip_grads(grads, MAX_NORM, -LR, out=True, dev_status=st,
                                                             workspace=ws["c"])
        o["m1"], o["n1"] = F.falqon_proxy_update(self.w1, self.s1, self.P1, o["inc"][0], self.A1, dev_status=st,
                                                 workspace=ws["p1"])
        o["m2"], o["n2"] = F.falqon_proxy_update(self.w2, self.s2, self.P2, o["inc"][1], self.A2, dev_status=st,
                                                 workspace=ws["p2"])
        return o


def _near(got, want, rel, what):
    """Within `rel` of the value, or of the root mean square where the value is smaller: what sums of products leave."""
    floor = want.double().square().mean().sqrt()
    off = ((got.double() - want).abs() / torch.maximum(want.abs(), floor)).max()
    assert float(off) < rel, (what, float(off))


@pytest.mark.parametrize("M,K,N,r", [(64, 128, 256, 16), (300, 336, 528, 16), (1024, 512, 1024, 64)])
def test_step_against_definitions(cuda_device, M, K, N, r):
    b = Block(M, K, N, r)
    w1, w2 = b.w1.clone(), b.w2.clone()
    o = b.step()
    assert int(b.status.item()) == 0
    # one rounding to bf16 of a float32 result whose own error is far below it
    h, _, rstd = block.norm_fwd(b.x, b.gamma, rms=True)
    _near(o["h"], h, 1.1 * U, "h")
    a, z = block.linear_fwd_epilogue(o["hq"], o["sh"], w1, b.s1, b.b1, F.ACT_GELU_TANH)
    _near(o["z"], z, 1.1 * U, "z")
    _near(o["a"], a, 1.1 * U, "a")
    y, _ = block.linear_fwd_epilogue(o["aq"], o["sa"], w2, b.s2, b.b2, F.ACT_NONE, b.x)
    _near(o["y"], y, 1.1 * U, "y")
    _near(o["db2"], b.dy.double().sum(0), 1e-4, "db2")
    dz, db1 = block.linear_epilogue_bwd(o["da"], o["z"], F.ACT_GELU_TANH)
    _near(o["dz"], dz, 1.1 * U, "dz")
    _near(o["db1"], db1, 1e-4, "db1")
    dx, dgamma, _ = block.norm_bwd(o["dh"], b.x, b.gamma, None, o["rstd"], b.dy, True)
    _near(o["dx"], dx, 1.1 * U, "dx")
    _near(o["dgamma"], dgamma, 1e-4, "dgamma")
    grads = [o["dB1"], o["dB2"], o["db1"], o["db2"], o["dgamma"]]
    inc, norm, coef = block.clip_grads(grads, MAX_NORM, -LR)
    assert abs(o["norm"].item() - norm) < 6 * E * norm and abs(o["coef"].item() - coef) < 8 * E * coef
    assert coef < 1  # the clip is in force
    for got, want in zip(o["inc"], inc):
        _near(got, want, 1.1 * U if got.dtype == BF else 1e-6, "increment")
    # the clipped gradients' norm is the bound, up to the outputs' roundings
    after = math.sqrt(sum(float(v.double().square().sum()) for v in o["inc"])) / LR
    assert abs(after / MAX_NORM - 1) < U


def test_gradient_of_the_block_against_differences(cuda_device):
    """The whole chain against differences of the float64 definition with the same (fixed) weights and without the
    quantization of activations: the E4M3 roundings of h, a, dy and dz are off by at most 2^-4 of a value each and
    average out over the sums, so the directional derivative agrees within a few hundredths."""
    M, K, N, r = 256, 256, 512, 16
    b = Block(M, K, N, r, seed=3)
    w1, w2 = block.decode_e4m3(b.w1) / b.s1.double(), block.decode_e4m3(b.w2) / b.s2.double()
    o = b.step()

    def loss(x, gamma):
        h = block.norm_fwd(x, gamma, rms=True)[0]
        y = block.act(h @ w1.T + b.b1.double(), F.ACT_GELU_TANH) @ w2.T + b.b2.double() + x.double()
        return (y * b.dy.double()).sum()
    x, gamma = b.x.double(), b.gamma.double()
    for name, t, got in (("x", x, o["dx"]), ("gamma", gamma, o["dgamma"])):
        # along the gradient itself: the directional derivative is its squared norm
        d = got.double()
        step = 1e-4 * float(t.norm() / d.norm())
        lo, hi = [(loss(x + s * step * d, gamma) if name == "x" else loss(x, gamma + s * step * d)) for s in (-1, 1)]
        slope = float(hi - lo) / (2 * step)
        assert abs(slope / float(d.square().sum()) - 1) < 0.03, name


def test_captured_step_replays_on_new_inputs(cuda_device):
    """The step captured into a graph on another stream and replayed on other inputs gives the bits of the eager step."""
    shape = (320, 256, 512, 16)
    b = Block(*shape, seed=1)
    keep = {k: getattr(b, k).clone() for k in ("w1", "w2", "x", "dy")}
    other = Block(*shape, seed=2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            o = b.step()
    torch.cuda.current_stream().wait_stream(s)
    for x, dy in ((keep["x"], keep["dy"]), (other.x, other.dy)):
        eager = Block(*shape, seed=1)
        eager.x.copy_(x)
        eager.dy.copy_(dy)
        b.x.copy_(x)
        b.dy.copy_(dy)
        b.w1.copy_(keep["w1"])
        b.w2.copy_(keep["w2"])
        b.P1.zero_()
        b.P2.zero_()
        want = eager.step()
        graph.replay()
        torch.cuda.synchronize()
        for k in ("h", "rstd", "z", "a", "y", "db2", "dz", "db1", "dx", "dgamma", "norm", "coef", "m1", "m2"):
            assert torch.equal(o[k], want[k]), k
        assert all(torch.equal(p, q) for p, q in zip(o["inc"], want["inc"]))
        assert torch.equal(b.w1, eager.w1) and torch.equal(b.P2, eager.P2)
    assert int(b.status.item()) == 0


def test_two_streams_at_once(cuda_device):
    """Steps of two blocks side by side, each with workspaces of its own."""
    shape = (512, 512, 1024, 16)
    alone = [Block(*shape, seed=s).step() for s in (5, 6)]
    torch.cuda.synchronize()
    blocks = [Block(*shape, seed=s) for s in (5, 6)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    outs = [None, None]
    for i, (b, s) in enumerate(zip(blocks, streams)):
        with torch.cuda.stream(s):
            outs[i] = b.step()
    torch.cuda.synchronize()
    for o, want in zip(outs, alone):
        for k in ("y", "dx", "dgamma", "norm"):
            assert torch.equal(o[k], want[k]), k


def test_stream_argument(cuda_device):
    """A call on a stream that is not current: what it allocates and launches belongs to that stream."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(2048, 1024, generator=g, device="cuda").to(BF)
    gamma = torch.ones(1024, device="cuda")
    want = F.falqon_norm_fwd(x, gamma)
    wantb = F.falqon_norm_bwd(x, x, gamma, want[1], want[2])
    wantc = F.falqon_clip_grads([x], 1.0, out=True)
    wante = F.falqon_linear_epilogue_bwd(x, x, F.ACT_SILU)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = F.falqon_norm_fwd(x, gamma, stream=s)
        gotb = F.falqon_norm_bwd(x, x, gamma, got[1], got[2], stream=s)
        gotc = F.falqon_clip_grads([x], 1.0, out=True, stream=s)
        gote = F.falqon_linear_epilogue_bwd(x, x, F.ACT_SILU, stream=s)
    s.synchronize()
    for a, b in zip(got + gotb + gote, want + wantb + wante):
        assert torch.equal(a, b)
    assert torch.equal(gotc[0][0], wantc[0][0]) and torch.equal(gotc[1], wantc[1])


@pytest.mark.parametrize("M,N,K", [(2048, 1296, 512), (40, 272, 256), (4736, 1280, 256)])
def test_outputs_aligned_to_16_bytes_only(cuda_device, M, N, K):
    """Every tensor 16-byte but not 32-byte aligned."""
    g = torch.Generator(device="cuda").manual_seed(M)

    def off(t):
        """A copy of t that begins 16 bytes past a multiple of 32."""
        raw = torch.empty(t.numel() * t.element_size() + 64, dtype=torch.uint8, device="cuda")
        at = (-raw.data_ptr()) % 32 + 16
        v = raw[at:at + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
        assert v.data_ptr() % 32 == 16
        return v.copy_(t)
    (xq, sx, _), (wq, sw, _) = (F.falqon_quantize(torch.randn(M, K, generator=g, device="cuda")),
                                F.falqon_quantize(torch.randn(N, K, generator=g, device="cuda")))
    bias, res = torch.randn(N, generator=g, device="cuda"), torch.randn(M, N, generator=g, device="cuda").to(BF)
    y, z = F.falqon_linear_fwd_epilogue(xq, sx, wq, sw, bias, F.ACT_SILU, res, z=True)
    y2, z2 = F.falqon_linear_fwd_epilogue(off(xq), sx, off(wq), sw, off(bias), F.ACT_SILU, off(res),
                                          z=off(torch.zeros_like(z)), y=off(torch.zeros_like(y)))
    assert torch.equal(y, y2) and torch.equal(z, z2)
    dz, db = F.falqon_linear_epilogue_bwd(res, z, F.ACT_SILU)
    dz2, db2 = F.falqon_linear_epilogue_bwd(off(res), z2, F.ACT_SILU, dz=off(torch.zeros_like(dz)))
    assert torch.equal(dz, dz2) and torch.equal(db, db2)
    n = F.falqon_norm_fwd(res, None, None)
    n2 = F.falqon_norm_fwd(off(res), None, None, y=off(torch.zeros_like(res)))
    assert all(torch.equal(a, b) for a, b in zip(n, n2))
    c, c2 = F.falqon_clip_grads([res, bias], 1.0, out=True), F.falqon_clip_grads([off(res), off(bias)], 1.0, out=True)
    assert torch.equal(c[0][0], c2[0][0]) and torch.equal(c[1], c2[1])


def test_tensors_side_by_side(cuda_device):
    """Every tensor of a call in one allocation, end to end: apart for the
    overlap checks, and nothing is written past an output's last element."""
    g = torch.Generator(device="cuda").manual_seed(2)
    rows, cols = 40, 1000  # 2 000-byte rows; 160-byte statistics
    x, dy, dres = (torch.randn(rows, cols, generator=g, device="cuda").to(BF) for _ in range(3))
    gamma = torch.randn(cols, generator=g, device="cuda").to(BF)
    mean, rstd = F.falqon_norm_fwd(x, gamma)[1:]
    want = F.falqon_norm_bwd(dy, x, gamma, mean, rstd, dres=dres)
    parts = [dy, x, dres, gamma, mean, rstd, *want]
    sizes = [t.numel() * t.element_size() for t in parts]
    assert all(s % 16 == 0 for s in sizes)
    buf = torch.full((sum(sizes) + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    views, at = [], 0
    for t, s in zip(parts, sizes):
        views.append(buf[at:at + s].view(t.dtype).view(t.shape))
        at += s
    for v, t in zip(views[:6], parts):
        v.copy_(t)
    F.falqon_norm_bwd(views[0], views[1], views[3], views[4], views[5], dres=views[2], dx=views[6], dgamma=views[7],
                      dbeta=views[8])
    for v, t in zip(views, parts):
        assert torch.equal(v, t)
    assert bool((buf[at:] == 0x5A).all())


def test_a_stream_of_another_device_is_refused(cuda_device):
    x = torch.ones(16, 16, device="cuda", dtype=BF)
    other = types.SimpleNamespace(device=torch.device("cuda", x.device.index + 1))
    v = torch.ones(16, device="cuda")
    codes = x.to(torch.float8_e4m3fn)
    for call in (lambda: F.falqon_norm_fwd(x, stream=other), lambda: F.falqon_norm_bwd(x, x, None, v, v, stream=other),
                 lambda: F.falqon_linear_fwd_epilogue(codes, v[:1], codes, v[:1], stream=other),
                 lambda: F.falqon_linear_epilogue_bwd(x, x, F.ACT_RELU, stream=other),
                 lambda: F.falqon_clip_grads([x], 1.0, stream=other)):
        with pytest.raises(ValueError):
            call()


def test_calls_from_several_threads(cuda_device):
    """Threads of one process, each with a stream of its own, from their first call on."""
    g = torch.Generator(device="cuda").manual_seed(3)
    xs = [torch.randn(300 + 77 * i, 1040, generator=g, device="cuda").to(BF) for i in range(4)]
    w = (torch.randn(528, 1040, generator=g, device="cuda") / 32).to(torch.float8_e4m3fn)
    one = torch.ones(1, device="cuda")
    gamma = torch.randn(1040, generator=g, device="cuda")

    def calls(x):
        y, mean, rstd = F.falqon_norm_fwd(x, gamma)
        z = F.falqon_linear_fwd_epilogue(y.to(torch.float8_e4m3fn), one, w, one, act=F.ACT_GELU_ERF, z=True)
        b = F.falqon_linear_epilogue_bwd(z[0], z[1], F.ACT_GELU_ERF)
        n = F.falqon_norm_bwd(y, x, gamma, mean, rstd)
        c, norm, _ = F.falqon_clip_grads([n[0], b[1]], 1.0, out=True)
        return [y, *z, *b, *n, *c, norm]

    got = [None] * len(xs)
    torch.cuda.synchronize()

    def run(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(5):
                got[i] = calls(xs[i])
        s.synchronize()

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(xs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i, x in enumerate(xs):
        for a, b in zip(got[i], calls(x), strict=True):
            assert torch.equal(a, b)


FIRST_CALL_CAPTURED = """
import torch
import fp8_quantized_lora_b200 as F
x = torch.randn(300, 1040, device="cuda").to(torch.bfloat16)
w = (torch.randn(528, 1040, device="cuda") / 32).to(torch.float8_e4m3fn)
xq = x.to(torch.float8_e4m3fn)
one, gamma = torch.ones(1, device="cuda"), torch.randn(1040, device="cuda")
def calls():
    y, mean, rstd = F.falqon_norm_fwd(x, gamma)
    o, z = F.falqon_linear_fwd_epilogue(xq, one, w, one, act=F.ACT_SILU, z=True)
    dz, db = F.falqon_linear_epilogue_bwd(o, z, F.ACT_SILU)
    n = F.falqon_norm_bwd(y, x, gamma, mean, rstd)
    c, norm, coef = F.falqon_clip_grads([n[0], db], 1.0, out=True)
    return [y, mean, rstd, o, z, dz, db, *n, *c, norm, coef]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, calls(), strict=True))
print("same")
"""


def test_first_call_of_a_process_inside_a_capture(cuda_device):
    p = subprocess.run([sys.executable, "-c", FIRST_CALL_CAPTURED], capture_output=True, text=True, timeout=300,
                       cwd=pathlib.Path(F.__file__).resolve().parents[1])
    assert p.returncode == 0 and p.stdout.strip() == "same", p.stderr[-2000:]
