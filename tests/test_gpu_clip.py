"""GPU: the global gradient norm and clipping, against fp64 sums.

At most 128 squares are added in fp32 before fp64 takes over, so the norm is
within 2^-18 of itself (half of 128 * 2^-24, and its rounding); expected 2^-24."""
import math

import pytest
import torch

import workloads
from tests import _encoder_ref as ref

pytestmark = pytest.mark.gpu
m = pytest.importorskip("maxsim_scoring_02_gb300")
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.load_library()


def _norm(grads):
    return math.sqrt(math.fsum((g.double() ** 2).sum().item() for g in grads))


def _check(grads, outs, norm, max_norm, before=None):
    before = grads if before is None else before
    want = _norm(before)
    assert abs(norm.item() - want) <= 2.0 ** -18 * want
    f = min(1.0, max_norm / (want + 1e-6))
    for g, o in zip(before, outs):
        # the factor is off by the norm's error and its own rounding, the product is rounded once
        small = 2.0 ** -24 if g.dtype == torch.float16 else 0.0   # fp16 results below its smallest normal number
        assert ((o.double() - g.double() * f).abs() <= g.double().abs() * f * (ref.U[g.dtype] + 2.0 ** -17) + small).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sizes", [[1], [7, 0, 33], [16384], [16385, 3, 32768, 40000], [1_000_003]])
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_sizes_and_types(dtype, sizes, max_norm):
    grads = [workloads.normal((n,), seed=n + 1, device=DEV).to(dtype) for n in sizes]
    before = [g.clone() for g in grads]
    outs = [torch.empty_like(g) for g in grads]
    norm = m.maxsim_clip_grad_norm(grads, max_norm, out=outs)
    _check(grads, outs, norm, max_norm)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    again = m.maxsim_clip_grad_norm(grads, max_norm)             # in place
    assert torch.equal(again, norm) and all(torch.equal(a, b) for a, b in zip(grads, outs))


def test_mixed_types_and_odd_addresses():
    """Tensors that lie back to back in a buffer start at any element."""
    sizes = [5, 1001, 64, 3, 70001, 12, 1]
    for dtype in (torch.bfloat16, torch.float32):
        flat = workloads.normal((sum(sizes),), seed=9, device=DEV).to(dtype)
        same = list(torch.split(flat.clone(), sizes))
        shifted = list(torch.split(torch.empty(sum(sizes) + 1, dtype=dtype, device=DEV)[1:], sizes))
        grads = list(torch.split(flat, sizes))
        norm = m.maxsim_clip_grad_norm(grads, 1.0, out=same)
        _check(grads, same, norm, 1.0)
        m.maxsim_clip_grad_norm(grads, 1.0, out=shifted)
        assert all(torch.equal(a, b) for a, b in zip(same, shifted))
    mixed = [workloads.normal((n, 3), seed=n, device=DEV).to(t)
             for n, t in ((50, torch.float32), (9000, torch.bfloat16), (70, torch.float16))]
    outs = [torch.empty_like(g) for g in mixed]
    _check(mixed, outs, m.maxsim_clip_grad_norm(mixed, 2.0, out=outs), 2.0)


@pytest.mark.parametrize("count", [32, 33, 256, 257, 1024, 1025, 2600])
def test_many_tensors(count):
    flat = workloads.normal((count * 40,), seed=count, device=DEV)
    grads = list(torch.split(flat, 40))
    before = flat.clone()
    norm = m.maxsim_clip_grad_norm(grads, 1.0)
    _check(grads, [flat], norm, 1.0, before=[before])


def test_extreme_values():
    """Squares beyond fp32's range, zeros, infinities and NaN."""
    for value in (1e30, 1e-30, 3e38):
        g = torch.full((5000,), value, device=DEV)
        g[::2] = 0
        want = value * math.sqrt(2500.0)
        norm = m.maxsim_clip_grad_norm([g], 1e38)
        if want < 3.4e38:
            assert abs(norm.item() / want - 1) <= 2.0 ** -18
        else:
            assert math.isinf(norm.item())
            assert abs(g[1].item() / (1e38 / 50) - 1) <= 1e-5     # the factor is made before the norm is rounded
    z = torch.zeros(100_000, device=DEV)
    assert m.maxsim_clip_grad_norm([z], 1.0).item() == 0 and (z == 0).all()
    g = torch.ones(300, device=DEV)
    g[7] = float("inf")
    assert math.isinf(m.maxsim_clip_grad_norm([g], 1.0).item())
    assert torch.isnan(g[7]) and (g[:7] == 0).all() and (g[8:] == 0).all()
    h = torch.ones(300, device=DEV, dtype=torch.bfloat16)
    h[299] = float("nan")
    assert math.isnan(m.maxsim_clip_grad_norm([h, z], 1.0).item())
    assert torch.isnan(h).all() and torch.isnan(z).all()


def test_more_than_32_bits_of_elements():
    n = (1 << 32) + 12345
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    g[-1], g[1 << 31], g[5] = 2, 2, 1
    assert abs(m.maxsim_clip_grad_norm([g], 1.5).item() - 3) <= 1e-6
    assert [g[i].item() for i in (-1, 1 << 31, 5, 6)] == [1, 1, 0.5, 0]


def test_repeatable_and_no_tensors():
    g = workloads.normal((3_000_001,), seed=1, device=DEV)
    o = torch.empty_like(g)
    first = m.maxsim_clip_grad_norm([g], 1.0, out=[o]).clone()
    assert all(torch.equal(m.maxsim_clip_grad_norm([g], 1.0, out=[o]), first) for _ in range(3))
    assert m.maxsim_clip_grad_norm([], 1.0).item() == 0


def test_refusals():
    g = torch.ones(8, 8, device=DEV)
    with pytest.raises(ValueError):
        m.maxsim_clip_grad_norm([g.t()[1:]], 1.0)
    with pytest.raises(ValueError):
        m.maxsim_clip_grad_norm([g.cpu()], 1.0)
    with pytest.raises(TypeError):
        m.maxsim_clip_grad_norm([g.double()], 1.0)
    with pytest.raises(ValueError):
        m.maxsim_clip_grad_norm([g], 1.0, out=[g.half()])
    with pytest.raises(m.MaxSimError) as e:
        m.maxsim_clip_grad_norm([g], -1.0)
    assert e.value.status == 1
    with pytest.raises(m.MaxSimError) as e:
        m.maxsim_clip_grad_norm([g], 1.0, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
    assert e.value.status == 5
