"""GPU: cross entropy over a vocabulary and its gradients, against fp64."""
import math

import pytest
import torch

import workloads
from tests import _layer_ref as ref

pytestmark = pytest.mark.gpu
m = pytest.importorskip("maxsim_scoring_02_gb300")
DEV = "cuda"
DTYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.load_library()
    yield
    assert m.maxsim_device_status() == (0, 0)


def _inputs(T, V, d, dtype, seed=1, pad=0, spread=2.0, ignored=True):
    x = workloads.normal((T, d + pad), seed=seed, device=DEV).to(dtype)[:, :d]
    w = (workloads.normal((V, d + pad), seed=seed + 1, device=DEV) * (spread / math.sqrt(d))).to(dtype)[:, :d]
    g = torch.Generator().manual_seed(seed)
    t = torch.randint(0, V, (T,), generator=g)
    if ignored and T > 2:
        t[torch.rand(T, generator=g) < 0.2] = -100
    dloss = torch.rand(T, generator=g) * 2 - 0.5
    return x, w, t.to(DEV), (dloss / T).to(DEV)


def _check(x, w, t, dloss, scale=1.0):
    loss, lse = m.encoder_cross_entropy(x, w, t, scale=scale)
    want = ref.cross_entropy(x, w, t, scale, dloss)
    ref.within(lse, want["lse"], want["lse_tol"], "lse")
    ref.within(loss, want["loss"], want["loss_tol"], "loss")
    assert (loss[t < 0] == 0).all()
    if dloss is None:
        return loss, lse
    dx, dw = m.encoder_cross_entropy_backward(dloss, x, w, t, lse, scale=scale)
    ref.within(dx, want["dx"], want["dx_tol"], "dx")
    ref.within(dw, want["dw"], want["dw_tol"], "dw")
    assert (dx[t < 0] == 0).all()
    return loss, lse, dx, dw


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V,d", [
    (1, 1, 8), (1, 2, 64), (2, 31, 16), (31, 127, 72), (33, 128, 128), (128, 129, 64), (129, 255, 264), (257, 257, 200),
    (256, 256, 256), (300, 1000, 520), (600, 5003, 136), (40, 30011, 768), (1531, 700, 1000), (7, 70001, 48)])
def test_sizes_and_types(dtype, T, V, d):
    _check(*_inputs(T, V, d, dtype))


@pytest.mark.parametrize("scale", [2.0 ** -10, 0.05, 3.0, 40.0])
def test_scales(scale):
    _check(*_inputs(100, 900, 64, torch.bfloat16), scale=scale)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("factor", [1e-12, 1.0, 1e12])
def test_small_and_large_gradients_keep_their_bits(dtype, factor):
    """dz is held divided by the largest dloss: what a row gets does not depend on the sizes
    of all (results beyond the type's range excepted)."""
    x, w, t, dloss = _inputs(90, 800, 64, torch.bfloat16 if dtype == torch.bfloat16 else dtype)
    if dtype == torch.float16:
        factor = min(factor, 10.0)
    _check(x, w, t, dloss * factor)
    if factor == 1.0:
        wide = dloss.clone()
        wide[::2] *= 1e-4
        _check(x, w, t, wide)


def test_strides():
    x, w, t, dloss = _inputs(150, 600, 96, torch.bfloat16, pad=24)
    a = _check(x, w, t, dloss)
    b = _check(x.contiguous(), w.contiguous(), t, dloss)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    wide_x = torch.full((150, 120), 7.0, dtype=torch.bfloat16, device=DEV)
    wide_w = torch.full((600, 104), 7.0, dtype=torch.bfloat16, device=DEV)
    m.encoder_cross_entropy_backward(dloss, x, w, t, a[1], dx=wide_x[:, 16:112], dweight=wide_w[:, :96])
    assert torch.equal(wide_x[:, 16:112], a[2]) and torch.equal(wide_w[:, :96], a[3])
    assert (wide_x[:, :16] == 7).all() and (wide_x[:, 112:] == 7).all() and (wide_w[:, 96:] == 7).all()


def test_several_pieces_of_the_vocabulary():
    """dz of 8192 rows and 20000 columns takes two pieces, that of 600000 rows two of
    256 columns; rows that are the same in all pieces' sums."""
    _check(*_inputs(8192, 20000, 64, torch.bfloat16))
    _check(*_inputs(600001, 300, 8, torch.float16))


def test_several_pieces_of_the_rows():
    """The parts of 60000 rows and 40000 columns take two pieces in the forward (rows
    against the fp64 form, some of them); a vocabulary of 2^31 elements."""
    x, w, t, _ = _inputs(60000, 40000, 64, torch.bfloat16)
    loss, lse = m.encoder_cross_entropy(x, w, t)
    for a in (0, 20000, 59000):
        want = ref.cross_entropy(x[a:a + 999], w, t[a:a + 999])
        ref.within(lse[a:a + 999], want["lse"], want["lse_tol"], "lse")
        ref.within(loss[a:a + 999], want["loss"], want["loss_tol"], "loss")


def test_more_than_31_bits_of_elements():
    """Columns whose rows of weight lie beyond 2^31 elements: their gradients, and a
    target there."""
    T, V, d, n = 5, (1 << 20) + 777, 2056, 300
    x = workloads.normal((T, d), seed=1, device=DEV).bfloat16()
    w = torch.zeros((V, d), dtype=torch.bfloat16, device=DEV)
    w[-n:] = (workloads.normal((n, d), seed=2, device=DEV) * 0.1).bfloat16()
    t = torch.tensor([V - 1, 3, V - n, -1, V - 7], device=DEV)
    dloss = torch.rand(T, generator=torch.Generator().manual_seed(3)).to(DEV)
    loss, lse = m.encoder_cross_entropy(x, w, t)
    # V - n columns have logit 0
    z = x.double() @ w[-n:].double().T
    want = torch.logaddexp(torch.logsumexp(z, 1), torch.full((T,), math.log(V - n), device=DEV, dtype=torch.float64))
    off = (x.double().abs() @ w[-n:].double().abs().T).amax(1) * d * 2.0 ** -23 + 2.0 ** -16 + 2.0 ** -22 * want
    assert ((lse.double() - want).abs() <= off).all()
    dx, dw = m.encoder_cross_entropy_backward(dloss, x, w, t, lse)
    part = torch.where(t >= 0, dloss.double(), 0.0)[:, None]
    for cols, zz in ((slice(V - n, V), z), (slice(0, 64), torch.zeros((T, 64), dtype=torch.float64, device=DEV))):
        p = torch.exp(zz - want[:, None])
        dz = p * part - part * (torch.arange(V, device=DEV)[cols][None] == t[:, None])
        E = 2.0 ** -8 * dz.abs() + p * part * (4 * off[:, None] + 2.0 ** -17) + 2.0 ** -20 * dz.abs()
        ref.within(dw[cols], dz.T @ x.double(), E.T @ x.double().abs() + 2.0 ** -8 * (dz.T @ x.double()).abs())
        if cols.start:  # the other columns' weights are 0
            ref.within(dx, dz @ w[cols].double(), E @ w[cols].double().abs() + 2.0 ** -8 * (dz @ w[cols].double()).abs()
                       + 2.0 ** -15 * (dz.abs() @ w[cols].double().abs()))


def test_rows_off_line_boundaries():
    """Rows of 2000 bytes are copied into aligned ones where products are long; the
    same rows 2048 bytes apart, or from a wider buffer, give the same numbers."""
    T, V, d = 700, 20001, 1000
    x, w, t, dloss = _inputs(T, V, d, torch.bfloat16)
    want = _check(x, w, t, dloss)
    for wide, first in ((1024, 0), (1016, 8), (1024, 16)):
        y = torch.full((T, wide), float("nan"), dtype=torch.bfloat16, device=DEV)
        y[:, first:first + d] = x
        y = y[:, first:first + d]
        loss, lse = m.encoder_cross_entropy(y, w, t)
        got = (loss, lse) + m.encoder_cross_entropy_backward(dloss, y, w, t, lse)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_many_columns_for_one_row():
    _check(*_inputs(1, (1 << 20) + 3, 64, torch.bfloat16))


@pytest.mark.parametrize("T,V,d", [(40000, 3, 64), (20001, 300, 136), (5000, 40, 520)])
def test_many_rows_for_few_columns(T, V, d):
    """dW's sums over the rows are cut, too."""
    _check(*_inputs(T, V, d, torch.bfloat16))


def test_no_targets_and_bad_ones():
    x, w, t, dloss = _inputs(70, 300, 64, torch.bfloat16)
    none = torch.full_like(t, -100)
    loss, lse, dx, dw = _check(x, w, none, dloss)
    assert (loss == 0).all() and (dx == 0).all() and (dw == 0).all()
    bad = t.clone()
    bad[3], bad[5], bad[7] = 300, 1 << 40, -(1 << 40)
    ok = t.clone()
    ok[3] = ok[5] = ok[7] = -1
    want = _check(x, w, ok, dloss)
    loss, lse = m.encoder_cross_entropy(x, w, bad)
    assert m.maxsim_device_status() == (1, m.DEVERR_BAD_INPUT)
    dx, dw = m.encoder_cross_entropy_backward(dloss, x, w, bad, lse)
    assert m.maxsim_device_status() == (1, m.DEVERR_BAD_INPUT)
    assert all(torch.equal(a, b) for a, b in zip((loss, lse, dx, dw), want))


def test_infinities_and_nan():
    """A row that is not finite has no loss; the others keep theirs."""
    x, w, t, dloss = _inputs(40, 500, 64, torch.bfloat16, ignored=False)
    loss, lse = m.encoder_cross_entropy(x, w, t)
    bad = x.clone()
    bad[3, 0], bad[9, 5] = float("nan"), float("inf")
    l2, e2 = m.encoder_cross_entropy(bad, w, t)
    rows = torch.ones(40, dtype=torch.bool, device=DEV)
    rows[[3, 9]] = False
    assert torch.equal(l2[rows], loss[rows]) and torch.equal(e2[rows], lse[rows])
    assert torch.isnan(l2[~rows]).all() and torch.isnan(e2[~rows]).all()
    dx, _ = m.encoder_cross_entropy_backward(dloss, x, w, t, lse)
    d2, dw = m.encoder_cross_entropy_backward(dloss, bad, w, t, e2)
    assert torch.equal(d2[rows], dx[rows]) and torch.isnan(d2[~rows]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [40, 33000])
def test_a_gradient_that_is_not_finite(dtype, T):
    """It spoils its own row of dx alone."""
    x, w, t, dloss = _inputs(T, 300, 64, dtype, ignored=False)
    dloss = dloss * 100
    rows = torch.ones(T, dtype=torch.bool, device=DEV)
    rows[[3, 9]] = False
    dloss[~rows] = 0.0
    _, lse = m.encoder_cross_entropy(x, w, t)
    dx, _ = m.encoder_cross_entropy_backward(dloss, x, w, t, lse)
    dloss[3], dloss[9] = float("inf"), float("nan")
    d2, _ = m.encoder_cross_entropy_backward(dloss, x, w, t, lse)
    assert torch.equal(d2[rows], dx[rows]) and torch.isfinite(d2[rows]).all()
    assert torch.isnan(d2[9]).all() and not torch.isfinite(d2[3]).any()


def test_large_logits():
    """Logits of thousands: one column has all the weight, exponentials of the others vanish."""
    x, w, t, dloss = _inputs(60, 400, 64, torch.bfloat16, spread=2000.0)
    _check(x, w, t, dloss)


def test_one_side_alone():
    x, w, t, dloss = _inputs(300, 2000, 128, torch.bfloat16)
    _, lse, dx, dw = _check(x, w, t, dloss)
    a, none = m.encoder_cross_entropy_backward(dloss, x, w, t, lse, want_dweight=False)
    assert none is None and torch.equal(a, dx)
    none, b = m.encoder_cross_entropy_backward(dloss, x, w, t, lse, want_dx=False)
    assert none is None and torch.equal(b, dw)
    assert m.encoder_cross_entropy_backward(dloss, x, w, t, lse, want_dx=False, want_dweight=False) == (None, None)


def test_no_rows():
    x, w, t, dloss = _inputs(4, 50, 64, torch.bfloat16)
    loss, lse = m.encoder_cross_entropy(x[:0], w, t[:0])
    assert loss.shape == lse.shape == (0,)
    wide = torch.full((50, 72), 7.0, dtype=torch.bfloat16, device=DEV)
    dx, dw = m.encoder_cross_entropy_backward(dloss[:0], x[:0], w, t[:0], lse, dweight=wide[:, :64])
    assert dx.shape == (0, 64) and (dw == 0).all() and (wide[:, 64:] == 7).all()


def test_gradients_against_differences():
    """Along random directions: bf16 values moved by whole steps of their own type,
    so that the moved inputs are exact; loss differences in fp64 sums of fp32 losses."""
    T, V, d = 64, 300, 64
    x, w, t, dloss = _inputs(T, V, d, torch.float16, ignored=False)
    _, lse = m.encoder_cross_entropy(x, w, t)
    grads = m.encoder_cross_entropy_backward(dloss, x, w, t, lse)
    for k, g in enumerate(grads):
        v = torch.where(workloads.normal(tuple(g.shape), seed=30 + k, device=DEV) > 0, 1.0, -1.0)
        s = 2.0 ** -6 if k == 0 else 2.0 ** -9
        ends, moves = [], []
        for sign in (s, -s):
            args = [x, w]
            args[k] = (args[k].float() + sign * v).half()
            moves.append(args[k].double())
            loss, _ = m.encoder_cross_entropy(args[0], args[1], t)
            ends.append((loss.double() * dloss.double()).sum().item())
        step = moves[0] - moves[1]                     # as it was rounded
        want = (g.double() * step).sum().item()
        size = (g.double().abs() * step.abs()).sum().item()
        # the gradient's rounding 2^-11, losses to 2^-17 each, and the third derivative along the step
        err = 2.0 ** -10 * size + 2 * 2.0 ** -16 * dloss.abs().sum().item() + 0.02 * abs(want)
        assert abs(ends[0] - ends[1] - want) <= err


def test_repeatable():
    x, w, t, dloss = _inputs(3000, 9001, 256, torch.bfloat16)
    first = None
    for _ in range(3):
        loss, lse = m.encoder_cross_entropy(x, w, t)
        got = (loss, lse) + m.encoder_cross_entropy_backward(dloss, x, w, t, lse)
        first = first or [a.clone() for a in got]
        assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_refusals():
    x, w, t, dloss = _inputs(40, 500, 64, torch.bfloat16)
    loss, lse = m.encoder_cross_entropy(x, w, t)
    with pytest.raises(m.MaxSimError) as e:
        m.encoder_cross_entropy(x[:, :60], w[:, :60], t)
    assert e.value.status == 2
    for bad in (lambda: m.encoder_cross_entropy(x, w, t, scale=0.0), lambda: m.encoder_cross_entropy_backward(dloss, x, w, t, lse, dx=x),
                lambda: m.encoder_cross_entropy(x[:1].expand(40, 64), w, t)):
        with pytest.raises(m.MaxSimError) as e:
            bad()
        assert e.value.status == 1
    need = m.encoder_cross_entropy_backward_workspace_size(x, w, t)
    for call in (lambda ws: m.encoder_cross_entropy_backward(dloss, x, w, t, lse, workspace=ws),
                 lambda ws: m.encoder_cross_entropy(x, w, t, workspace=ws)):
        with pytest.raises(m.MaxSimError) as e:
            call(torch.empty(min(need - 1, m.encoder_cross_entropy_workspace_size(x, w, t) - 1), dtype=torch.uint8, device=DEV))
        assert e.value.status == 5
