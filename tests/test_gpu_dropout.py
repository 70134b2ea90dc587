"""GPU: dropout from the counter-based generator, against the plain form: the mask
exactly, values to their rounding."""
import pytest
import torch

import workloads
from tests import _layer_ref as ref

pytestmark = pytest.mark.gpu
m = pytest.importorskip("maxsim_scoring_02_gb300")
DEV = "cuda"
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.load_library()


def rows(n, d, seed, dtype, pad=0, shift=0):
    """[n, d] values as a slice of rows `pad` longer, `shift` elements in."""
    t = workloads.normal((n, d + pad), seed=seed, device=DEV).to(dtype)
    return t[:, shift:shift + d]


def _rng(seed=0x1234567890ABCDEF, call=(7 << 32) + 5):
    return torch.tensor([seed, call], dtype=torch.int64, device=DEV)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d", [(1, 1), (1, 8), (3, 7), (5, 255), (2, 256), (33, 257), (70, 768), (9, 1001), (4, 2056)])
@pytest.mark.parametrize("residual", [False, True])
def test_sizes_and_types(dtype, n, d, residual):
    x, rng = rows(n, d, 1, dtype), _rng()
    res = rows(n, d, 2, dtype) if residual else None
    got = m.encoder_dropout(x, 0.3, rng, residual=res)
    want, tol = ref.dropout(x, 0.3, rng, res)
    ref.within(got, want, tol)
    if not residual:
        assert torch.equal(got != 0, ref.kept(n, d, 0.3, rng, DEV)[0] & (x != 0))


@pytest.mark.parametrize("p", [0.0, 1e-6, 2.0 ** -16, 0.5, 0.99997])
def test_chances(p):
    """p = 1e-6 is no multiple of 2^-16 and rounds to 0; 0.99997 keeps two lots of 65536."""
    x, rng = torch.ones((64, 4096), device=DEV), _rng(seed=-3)
    got = m.encoder_dropout(x, p, rng)
    want, tol = ref.dropout(x, p, rng)
    ref.within(got, want, tol)
    if round(p * 65536) == 0:
        assert torch.equal(got, x) and torch.equal(m.encoder_dropout(x, p, None if p == 0 else rng), x)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (3, 0), (3, 1), (9, 1)])
def test_strides_and_addresses_do_not_change_values(dtype, pad, shift):
    n, d, rng = 50, 320, _rng()
    x, res = rows(n, d, 1, dtype, pad, shift), rows(n, d, 2, dtype, pad, shift)
    want = m.encoder_dropout(x.contiguous(), 0.25, rng, residual=res.contiguous())
    wide = torch.full((n, d + pad), 7.0, dtype=dtype, device=DEV)
    got = m.encoder_dropout(x, 0.25, rng, residual=res, out=wide[:, shift:shift + d])
    assert torch.equal(got, want)
    wide[:, shift:shift + d] = 7.0
    assert (wide == 7.0).all()                       # what lies between the rows stays


def test_one_row_for_all():
    """A stride of 0: every row is the same, its mask is not."""
    x, rng = rows(1, 512, 1, torch.bfloat16).expand(40, 512), _rng()
    want, tol = ref.dropout(x.contiguous(), 0.5, rng)
    ref.within(m.encoder_dropout(x, 0.5, rng), want, tol)


@pytest.mark.parametrize("d", [512, 77])
def test_in_place_and_the_gradient(d):
    x, res, rng = rows(60, d, 1, torch.bfloat16), rows(60, d, 2, torch.bfloat16), _rng()
    want = m.encoder_dropout(x, 0.1, rng, residual=res)
    a, b = x.clone(), res.clone()
    assert m.encoder_dropout(a, 0.1, rng, residual=res, out=a) is a and torch.equal(a, want)
    m.encoder_dropout(x, 0.1, rng, residual=b, out=b)
    assert torch.equal(b, want)
    keep, f = ref.kept(60, d, 0.1, rng, DEV)
    dy = rows(60, d, 3, torch.float32)
    got = m.encoder_dropout(dy, 0.1, rng)
    assert ((got.double() - dy.double() * keep * f).abs() <= 2.0 ** -22 * dy.double().abs() * f).all()


def test_what_is_dropped_may_be_anything():
    rng = _rng()
    keep, _ = ref.kept(30, 264, 0.4, rng, DEV)
    x = torch.where(keep, 1.0, torch.where(torch.arange(264, device=DEV) % 2 == 0, float("nan"), float("inf"))).bfloat16()
    got = m.encoder_dropout(x, 0.4, rng)
    assert torch.isfinite(got).all() and torch.equal(got != 0, keep)


def test_calls_differ_and_repeat():
    x = torch.ones((100, 1000), device=DEV)
    a = m.encoder_dropout(x, 0.5, _rng(1, 1))
    assert torch.equal(a, m.encoder_dropout(x, 0.5, _rng(1, 1)))
    for other in (_rng(1, 2), _rng(2, 1), _rng(1, 1 + (1 << 32)), _rng(1 + (1 << 32), 1)):
        b = m.encoder_dropout(x, 0.5, other)
        # 10^5 independent pairs agree half the time, to 6 standard deviations
        assert abs((a == b).double().mean().item() - 0.5) <= 6 * 0.5 / 100000 ** 0.5
    # 10^5 lots, and those of each of the eight places of a group
    stay = a != 0
    assert abs(stay.double().mean().item() - 0.5) <= 6 * 0.5 / 100000 ** 0.5
    assert ((stay.view(-1, 8).double().mean(0) - 0.5).abs() <= 6 * 0.5 / 12500 ** 0.5).all()


def test_many_rows():
    """Rows whose offsets pass 32 bits; the last ones against the oracle's."""
    n, d = (1 << 21) + 5, 1032
    x, rng = torch.ones((n, d), dtype=torch.bfloat16, device=DEV), _rng()
    got = m.encoder_dropout(x, 0.5, rng, out=x)
    seed, call = (int(v) & (2 ** 64 - 1) for v in rng.tolist())
    for first in (0, n // 2, n - 7):
        want = (ref.lots(7, d, seed, call, first=first) >= 32768).to(DEV)
        assert torch.equal(got[first:first + 7] != 0, want)


def test_refusals():
    x, rng = rows(4, 64, 1, torch.bfloat16), _rng()
    wide = torch.zeros((4, 100), dtype=torch.bfloat16, device=DEV)
    for bad in (lambda: m.encoder_dropout(wide[:, :64], 0.5, rng, out=wide[:, 8:72]), lambda: m.encoder_dropout(x, 1.0, rng),
                lambda: m.encoder_dropout(x, 0.5, rng, out=x[:1].expand(4, 64))):
        with pytest.raises(m.MaxSimError) as e:
            bad()
        assert e.value.status == 1
    with pytest.raises(ValueError):
        m.encoder_dropout(x.cpu(), 0.5, rng)
    with pytest.raises(ValueError):
        m.encoder_dropout(x, 0.5, rng.cpu())
    assert m.encoder_dropout(x[:0], 0.5, rng).shape == (0, 64)
