"""falqon_clip_grads against the float64 definition.

A vector's float32 sum of up to eight squares is off by 8 e of itself (e =
2^-24), the root halves that, one rounding gives the float32 norm: 6 e.  The
outputs add the rounding of the factor, of the product and of the type."""

import math

import pytest
import torch

import fp8_quantized_lora_b200 as F
from oracle import block

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def _tensors(seed, sizes, dtypes, std=1e-3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(std * (1 + i % 5) * torch.randn(n, generator=g, device="cuda")).to(dtypes[i % len(dtypes)])
            for i, n in enumerate(sizes)]


def _check(grads, max_norm, factor, outs, norm, coef):
    O, NORM, COEF = block.clip_grads(grads, max_norm, factor)
    assert abs(norm.item() - NORM) <= 6 * E * NORM
    assert abs(coef.item() - COEF) <= 8 * E * COEF
    for o, want in zip(outs or [], O):
        u = torch.finfo(o.dtype).eps / 2
        tiny = 2.0 ** -134 if o.dtype == BF else 2.0 ** -150
        assert ((o - want).abs() <= (u + 9 * E) * want.abs() + tiny).all()


SIZES = [[1], [7], [8], [4096], [4097], [1, 2, 3, 4, 5], [0, 100, 0, 33], [65536, 3, 4095, 8192, 12345, 16],
         [262144, 262144, 4096, 4097], [17] * 511, [33] * 512, [9] * 513, [5000] * 1100]


@pytest.mark.parametrize("dtypes", [(BF,), (F32,), (BF, F32)])
@pytest.mark.parametrize("sizes", SIZES, ids=[f"{len(s)}x{s[-1]}" for s in SIZES])
def test_clip(cuda_device, sizes, dtypes):
    grads = _tensors(len(sizes), sizes, dtypes)
    keep = [g.clone() for g in grads]
    _, norm64, _ = block.clip_grads(grads, 1.0)
    for max_norm, factor in ((norm64 / 3, -1e-2), (norm64 * 2, 1.0), (math.inf, 0.5)):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        outs, norm, coef = F.falqon_clip_grads(grads, max_norm, factor, out=True, dev_status=st)
        mn = torch.tensor(max_norm, dtype=F32).item()  # the call takes a float
        fa = torch.tensor(factor, dtype=F32).item()
        _check(grads, mn, fa, outs, norm, coef)
        assert int(st.item()) == 0 and all(torch.equal(a, b) for a, b in zip(grads, keep))
        alone, n2, c2 = F.falqon_clip_grads(grads, max_norm)
        assert alone is None and torch.equal(n2, norm) and torch.equal(c2, coef)
        inplace = [g.clone() for g in grads]
        plan = F.GradList(inplace)
        _, n3, _ = F.falqon_clip_grads(plan, max_norm, factor, out=plan)
        assert torch.equal(n3, norm) and all(torch.equal(a, b) for a, b in zip(inplace, outs))


@pytest.mark.parametrize("n,size", [(40, 700000), (100, 300000), (600, 60000)])
def test_long_runs_across_many_tensors(cuda_device, n, size):
    """More than four 16 KB chunks a block, of odd lengths: each block's run goes on from tensor to tensor, of both
    types; 600 tensors take two launches each way."""
    sizes = [size + 997 * i % 4001 for i in range(n)]
    for dtypes in ((BF, F32), (BF, BF, F32)):
        grads = _tensors(n, sizes, dtypes)
        chunks = sum(-(-g.numel() * g.element_size() // 16384) for g in grads)
        assert chunks > 4 * 740
        _, norm64, _ = block.clip_grads(grads, 1.0)
        mn = torch.tensor(norm64 / 3, dtype=F32).item()
        outs, norm, coef = F.falqon_clip_grads(grads, mn, -0.5, out=True)
        _check(grads, mn, -0.5, outs, norm, coef)
        inplace = [g.clone() for g in grads]
        _, n2, c2 = F.falqon_clip_grads(inplace, mn, -0.5, out=inplace)
        assert torch.equal(n2, norm) and torch.equal(c2, coef)
        assert all(torch.equal(a, b) for a, b in zip(inplace, outs))


def test_neighbours_stay_as_they_were(cuda_device):
    """Views of one buffer, each of an odd length: what lies between them is neither read nor written."""
    flat = torch.full((40000,), math.nan, dtype=BF, device="cuda")
    out = torch.full((40000,), 7.0, dtype=BF, device="cuda")
    at, views, outs = 0, [], []
    for n in (1, 9, 4099, 8191, 77, 16385):
        views.append(flat[at:at + n].copy_(torch.randn(n, device="cuda")))
        outs.append(out[at:at + n])
        at += (n + 7) // 8 * 8 + 8
    mask = torch.zeros(40000, dtype=torch.bool, device="cuda")
    for v in outs:
        mask[v.storage_offset():v.storage_offset() + v.numel()] = True
    _, norm, coef = F.falqon_clip_grads(views, 1.0, 2.0, out=outs)
    _check(views, 1.0, 2.0, outs, norm, coef)
    assert (out[~mask] == 7.0).all()


@pytest.mark.parametrize("std", [1e-30, 1e-25, 1e-19, 1e15, 1e20, 1e30])
def test_far_magnitudes(cuda_device, std):
    """Squares that leave float32 on either side."""
    for dtypes in ((BF,), (F32,)):
        grads = [t / 1e-3 * std for t in _tensors(3, [10000, 77, 8], dtypes)]
        _, norm64, _ = block.clip_grads(grads, 1.0)
        mn = torch.tensor(norm64 / 4, dtype=F32).item()
        outs, norm, coef = F.falqon_clip_grads(grads, mn, 1.0, out=True)
        _check(grads, mn, 1.0, outs, norm, coef)


def test_zero_gradients(cuda_device):
    grads = [torch.zeros(1000, dtype=BF, device="cuda"), torch.zeros(0, device="cuda"), torch.zeros(5, device="cuda")]
    outs, norm, coef = F.falqon_clip_grads(grads, 1.0, -1.0, out=True)
    assert norm.item() == 0.0 and coef.item() == 1.0 and all((o == 0).all() for o in outs)
    empty = [torch.zeros(0, device="cuda")]
    outs, norm, coef = F.falqon_clip_grads(empty, 1.0, out=True)
    assert norm.item() == 0.0 and coef.item() == 1.0


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("where", [0, 4095, 4096, 8999])
def test_non_finite_gradient_voids_the_step(cuda_device, bad, where):
    grads = _tensors(5, [9000, 64], (BF, F32))
    grads[0][where] = bad
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs, norm, coef = F.falqon_clip_grads(grads, 1.0, -1.0, out=True, dev_status=st)
    assert int(st.item()) == F.DEV_NONFINITE and coef.item() == 0.0 and not math.isfinite(norm.item())
    for o in outs:
        assert (o == 0).all() and not torch.signbit(o).any()


def test_refusals(cuda_device):
    a, b = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    with pytest.raises(F.FalqonError) as e:
        F.falqon_clip_grads([a, a], 1.0, out=[a, a])
    assert e.value.status == 1
    with pytest.raises(F.FalqonError) as e:
        F.falqon_clip_grads([a, b], 1.0, out=[b, a])
    assert e.value.status == 1
    with pytest.raises(F.FalqonError):
        F.falqon_clip_grads([a], 0.0)
    with pytest.raises(F.FalqonError) as e:
        F.falqon_clip_grads([a[1:]], 1.0)  # not 16-byte aligned
    assert e.value.status == 2
    for out in ([a], [a, b[:32]], [a, b.to(BF)]):
        with pytest.raises(ValueError):
            F.falqon_clip_grads([a, b], 1.0, out=out)
    with pytest.raises(ValueError):
        F.GradList([torch.ones(8, 8, device="cuda").t()])
    _, norm, _ = F.falqon_clip_grads([a, a], 100.0)  # read twice: counted twice
    assert abs(norm.item() - math.sqrt(128)) < 1e-5


def test_a_list_keeps_or_follows_its_memory(cuda_device):
    """Tensors that get other memory leave the list's as it was; a storage that resize_ moves is followed; one that
    is given back is refused."""
    grads, outs = _tensors(7, [5000, 64, 777], (BF, F32)), [torch.zeros(n, device="cuda") for n in (5000, 64, 777)]
    outs = [o.to(g.dtype) for o, g in zip(outs, grads)]
    g, o = F.GradList(grads), F.GradList(outs)
    keep = [t.clone() for t in grads]
    _check(keep, 1.0, -2.0, *F.falqon_clip_grads(g, 1.0, -2.0, out=o))
    grads[0].data = 3 * grads[0]
    grads[1].set_(5 * grads[1])
    fill = [torch.full((5000,), math.nan, dtype=BF, device="cuda") for _ in range(20)]  # none in the list's memory
    grads[2].resize_(100000)
    _check(keep, 1.0, -2.0, *F.falqon_clip_grads(g, 1.0, -2.0, out=o))
    assert torch.equal(grads[2][:777], keep[2]) and len(fill) == 20
    grads[2].untyped_storage().resize_(0)
    with pytest.raises(ValueError):
        F.falqon_clip_grads(g, 1.0)


def test_results_beside_the_gradients(cuda_device):
    """norm and coef right behind a gradient and right before the next are apart; on one of their elements, or in one
    place, they are refused."""
    flat = torch.zeros(1000, device="cuda")
    a, norm, coef, b = flat[:100], flat[100:101], flat[103:104], flat[104:200]
    keep = [t.copy_(torch.randn(t.numel(), device="cuda")).clone() for t in (a, b)]
    for out in (None, True, [a, b]):
        for t, k in zip((a, b), keep):
            t.copy_(k)
        outs = F.falqon_clip_grads([a, b], 1.0, 2.0, out=out, norm=norm, coef=coef)[0]
        _check(keep, 1.0, 2.0, outs, norm, coef)
        assert (flat[101:103] == 0).all() and (flat[200:] == 0).all()
        for at in (a[:1], a[99:], b[:1], b[95:]):
            for kw in (dict(norm=at), dict(norm=norm, coef=at), dict(norm=norm, coef=norm)):
                with pytest.raises(F.FalqonError) as e:
                    F.falqon_clip_grads([a, b], 1.0, 2.0, out=out, **kw)
                assert e.value.status == 1


def test_more_than_2_31_elements(cuda_device):
    n = (1 << 31) + 12345
    g = torch.zeros(n, dtype=BF, device="cuda")
    g[0], g[1 << 31], g[n - 1] = 3.0, 4.0, 12.0
    plan = F.GradList([g])
    _, norm, coef = F.falqon_clip_grads(plan, 6.5, 1.0, out=plan)
    assert norm.item() == 13.0 and coef.item() == 0.5
    assert g[0].item() == 1.5 and g[1 << 31].item() == 2.0 and g[n - 1].item() == 6.0
