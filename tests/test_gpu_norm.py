"""GPU: root-mean-square norms, forward and backward, against fp64."""
import math

import pytest
import torch

import workloads
from tests import _layer_ref as ref
from tests.test_gpu_dropout import _rng, rows

pytestmark = pytest.mark.gpu
m = pytest.importorskip("maxsim_scoring_02_gb300")
DEV = "cuda"
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
EPS = 1e-6
# widths at and around each change of the threads of a row
WIDTHS = [1, 8, 31, 128, 136, 256, 264, 512, 513, 768, 1024, 1032, 1025, 2048, 2056, 4096, 4104, 4099, 8192, 8200, 16384, 16383]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.load_library()


def _weight(d, dtype, seed=9):
    return (1 + 0.3 * workloads.normal((d,), seed=seed, device=DEV)).to(dtype)


def _check_forward(x, h, y, weight, eps=EPS):
    want, _ = ref.norm(h, weight, eps)
    ref.within(y, want, (ref.U[x.dtype] + ref.ROW) * want.abs() + ref.TINY[x.dtype], "y")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", WIDTHS)
def test_forward_widths(dtype, d):
    n = 37
    x, res, w = rows(n, d, 1, dtype), rows(n, d, 2, dtype), _weight(d, torch.float32)
    y = m.encoder_rms_norm(x, w)
    _check_forward(x, x, y, w)
    y, h = m.encoder_rms_norm(x, w, residual=res, want_sum=True)
    want, tol = x.double() + res.double(), 0.0
    ref.within(h, want, ref.U[dtype] * want.abs() + ref.TINY[dtype], "h")
    _check_forward(x, h, y, w)
    assert torch.equal(m.encoder_rms_norm(x, w, residual=res), y)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", WIDTHS)
def test_backward_widths(dtype, d):
    n = 300 if d < 3000 else 41
    _backward(rows(n, d, 1, dtype), rows(n, d, 2, dtype), rows(n, d, 3, dtype), _weight(d, torch.float32), 0.2)


def _backward(dy, h, dsum, w, p, eps=EPS, **views):
    dtype, n = h.dtype, h.shape[0]
    rng = _rng()
    dx, dres, dw = m.encoder_rms_norm_backward(dy, h, w, dsum=dsum, eps=eps, p=p, rng=rng, **views)
    back, tol, dw64, size = ref.norm_backward(dy, h, w, eps, dsum)
    u, tiny = ref.U[dtype], ref.TINY[dtype]
    ref.within(dres, back, tol + u * back.abs() + tiny, "dresidual")
    if p:
        keep, f = ref.kept(*h.shape, p, rng, DEV)
        want = torch.where(keep, back * f, 0.0)
        ref.within(dx, want, torch.where(keep, tol * f, 0.0) + (u + 2.0 ** -23) * want.abs() + tiny, "dx")
    else:
        assert torch.equal(dx, dres)
    if w is not None:
        # a block's rows one after another, 16 teams, 38 blocks a warp, 5 steps: at most n / 1216 + 60 additions
        ref.within(dw, dw64, (ref.ROW + (n / 1216 + 60) * 2.0 ** -24) * size + ref.U[w.dtype] * dw64.abs() + ref.TINY[w.dtype], "dw")
    return dx, dres, dw


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d", [(1, 64), (2, 768), (1217, 128), (5000, 48), (20011, 264), (1500, 1032), (3001, 200)])
def test_row_counts(dtype, n, d):
    x, w = rows(n, d, 1, dtype), _weight(d, dtype)
    _check_forward(x, x, m.encoder_rms_norm(x, w), w)
    _backward(rows(n, d, 2, dtype), x, None, w, 0.0)


@pytest.mark.parametrize("residual,p,weight,dsum", [(a, b, c, e) for a in (False, True) for b in (0.0, 0.15)
                                                    for c in ("none", "fp32", "same") for e in (False, True)])
def test_optional_parts(residual, p, weight, dsum):
    n, d, dtype, rng = 70, 392, torch.bfloat16, _rng()
    w = None if weight == "none" else _weight(d, torch.float32 if weight == "fp32" else dtype)
    x, res = rows(n, d, 1, dtype), rows(n, d, 2, dtype) if residual else None
    y, h = m.encoder_rms_norm(x, w, residual=res, p=p, rng=rng, want_sum=True)
    if p:  # the same numbers as the two calls
        assert torch.equal(h, m.encoder_dropout(x, p, rng, residual=res))
    assert torch.equal(y, m.encoder_rms_norm(h, w))
    _check_forward(x, h, y, w)
    _backward(rows(n, d, 3, dtype), h, rows(n, d, 4, dtype) if dsum else None, w, p)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,pad,shift", [(320, 8, 8), (320, 3, 1), (771, 5, 0), (1500, 4, 4)])
def test_strides_and_in_place(dtype, d, pad, shift):
    n, w, rng = 45, _weight(d, torch.float32), _rng()
    x, res, dy = (rows(n, d, s, dtype, pad, shift) for s in (1, 2, 3))
    plain = [t.contiguous() for t in (x, res, dy)]
    y, h = m.encoder_rms_norm(plain[0], w, residual=plain[1], p=0.1, rng=rng, want_sum=True)
    close = lambda a, b: ref.within(a, b.double(), 2 * (ref.U[dtype] + ref.ROW) * b.double().abs())  # noqa: E731
    wide = torch.full((n, d + pad), 7.0, dtype=dtype, device=DEV)
    got, hh = m.encoder_rms_norm(x, w, residual=res, p=0.1, rng=rng, want_sum=True, out=wide[:, shift:shift + d])
    close(got, y)                                       # sums may be added in another order
    assert torch.equal(hh, h)
    wide[:, shift:shift + d] = 7.0
    assert (wide == 7.0).all()
    back = m.encoder_rms_norm_backward(plain[2], h, w, p=0.1, rng=rng)
    # in place: h over the residual, y over x; the gradients over dy and what reaches the sum
    a, b = x.clone(), res.clone()
    m.encoder_rms_norm(a, w, residual=b, p=0.1, rng=rng, out=a, sum_out=b)
    assert torch.equal(b, h)
    close(a, y)
    g, more = plain[2].clone(), torch.zeros_like(h)
    m.encoder_rms_norm_backward(g, h, w, dsum=more, p=0.1, rng=rng, dx=g, dresidual=more)
    assert torch.equal(g, back[0]) and torch.equal(more, back[1])
    # views of one buffer's columns
    both = torch.empty((n, 2 * d), dtype=dtype, device=DEV)
    m.encoder_rms_norm(plain[0], w, residual=plain[1], p=0.1, rng=rng, out=both[:, :d], sum_out=both[:, d:])
    close(both[:, :d], y)
    assert torch.equal(both[:, d:], h)


@pytest.mark.parametrize("fmt,top", [("int8", 127.0), ("e4m3", 448.0)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d", [(1, 8), (40, 128), (33, 100), (20, 768), (9, 1001), (7, 4096), (3, 16384)])
def test_eight_bits(fmt, top, dtype, n, d):
    x, res, w = rows(n, d, 1, dtype), rows(n, d, 2, dtype), _weight(d, torch.float32)
    q, scale, h = m.encoder_rms_norm(x, w, residual=res, fmt=fmt, want_sum=True)
    y, _ = ref.norm(h, w, EPS)
    want = y.abs().amax(1) / top
    assert ((scale.double() - want).abs() <= 2 * ref.ROW * want).all()
    v = y / want[:, None]                   # to 2^-18 and a few roundings of itself
    step = 0.5 if fmt == "int8" else (v.abs() * 2.0 ** -4).clamp_min(2.0 ** -10)
    assert q.dtype == (torch.int8 if fmt == "int8" else torch.float8_e4m3fn)
    ref.within(q.float(), v, step + 2.0 ** -20 * v.abs())
    assert (q.float().abs().amax(1) == top).all()
    assert torch.equal(h, m.encoder_rms_norm(x, w, residual=res, want_sum=True)[1])


def test_eight_bit_rows_are_what_scoring_takes():
    """Embeddings normed into int8 documents and a query, scored: within the codes'
    rounding of the fp64 scores of the normed rows."""
    d, lens = 128, [100, 1, 333]
    T, w = sum(lens), torch.full((d,), d ** -0.5, device=DEV)   # unit vectors
    off = workloads.csr_offsets(torch.tensor(lens, dtype=torch.int64)).to(DEV)
    D, Q = rows(T, d, 1, torch.bfloat16), rows(32, d, 2, torch.bfloat16)
    (dq, ds), (qq, qs) = m.encoder_rms_norm(D, w, fmt="int8"), m.encoder_rms_norm(Q, w, fmt="int8")
    got = m.maxsim_score_i8(qq, qs, dq, ds, off)
    Dn, Qn = ref.norm(D, w, EPS)[0], ref.norm(Q, w, EPS)[0]
    # each element is off by half a step, at most: <q, d> by half a step of each times the other's 1-norm
    off_by = (0.5 * qs.double()[:, None] * Dn.abs().sum(1)[None] + 0.5 * ds.double()[None] * Qn.abs().sum(1)[:, None]
              + 0.25 * d * qs.double()[:, None] * ds.double()[None]) * (1 + 2.0 ** -15)
    sim, a = Qn @ Dn.T, 0
    for b, n in enumerate(lens):
        want, tol = sim[:, a:a + n].amax(1).sum(), off_by[:, a:a + n].amax(1).sum()
        assert abs(got.view(-1)[b].double() - want) <= tol + 1e-5
        a += n


def test_extreme_values():
    """Squares beyond fp32's range in one of two rows of a warp, zeros, infinities and NaN."""
    d = 128
    x = rows(6, d, 1, torch.float32).contiguous()
    usual = m.encoder_rms_norm(x)
    x[1], x[3] = x[1] * 1e30, 0.0
    y = m.encoder_rms_norm(x)
    _check_forward(x, x, y, None)
    for r in (0, 2, 4, 5):
        assert torch.equal(y[r], usual[r])
    assert (y[3] == 0).all()
    q, s = m.encoder_rms_norm(x, fmt="int8")
    assert (q[3] == 0).all() and 0 < s[3] <= 1e-30
    dy = rows(6, d, 2, torch.float32)
    _backward(dy, x, None, None, 0.0)
    big = x.clone()
    big[0, 5], big[2, 7] = float("inf"), float("nan")
    y = m.encoder_rms_norm(big)
    assert torch.isnan(y[0, 5]) and (y[0, :5] == 0).all() and torch.isnan(y[2]).all() and torch.equal(y[4], usual[4])
    q, s = m.encoder_rms_norm(big, fmt="int8")
    assert not torch.isfinite(s[[0, 2]]).any() and torch.isfinite(s[[1, 3, 4, 5]]).all()
    tiny = torch.full((2, 64), 1e-25, device=DEV)
    _check_forward(tiny, tiny, m.encoder_rms_norm(tiny), None)
    assert math.isclose(m.encoder_rms_norm(torch.full((1, 64), 3.0, device=DEV), eps=16.0)[0, 0].item(), 3 / 5, rel_tol=1e-6)


@pytest.mark.parametrize("fmt,top", [("int8", 127.0), ("e4m3", 448.0)])
@pytest.mark.parametrize("d", [64, 100, 768, 2048])
def test_eight_bits_of_large_rows_and_weights(fmt, top, d):
    """Up to the end of fp32's range; a row whose |h w| is beyond it has no scale, beside usual rows."""
    x, w = rows(6, d, 1, torch.float32).contiguous(), _weight(d, torch.float32)
    x[1], x[4] = x[1] * 2.0 ** 120, x[4] * 2.0 ** 64
    for weight in (w * 2.0 ** 10, w * 2.0 ** 64, w * 2.0 ** 110, w * 2.0 ** 124):
        q, scale = m.encoder_rms_norm(x, weight, fmt=fmt)
        y, _ = ref.norm(x, weight, EPS)
        there = torch.isfinite((x * weight).abs().amax(1))
        assert there[[0, 2, 3, 5]].all() and not torch.isfinite(scale[~there]).any()
        q, scale, y = q.float()[there], scale[there], y[there]
        want = y.abs().amax(1) / top
        assert ((scale.double() - want).abs() <= 2 * ref.ROW * want).all()
        v = y / want[:, None]
        step = 0.5 if fmt == "int8" else (v.abs() * 2.0 ** -4).clamp_min(2.0 ** -10)
        ref.within(q, v, step + 2.0 ** -20 * v.abs())
        assert (q.abs().amax(1) == top).all()


def test_gradients_against_differences():
    """In fp32, along random directions: the change of <dy, y> + <more, h> for a
    step s is s times the gradient's product, to s^2 and the forward's rounding."""
    n, d, p, rng = 12, 200, 0.25, _rng()
    x, res, dy, more = (rows(n, d, s, torch.float32).contiguous() for s in (1, 2, 3, 4))
    w = _weight(d, torch.float32)

    def value(x, res, w):
        y, h = m.encoder_rms_norm(x, w, residual=res, p=p, rng=rng, want_sum=True)
        return ((dy.double() * y.double()).sum() + (more.double() * h.double()).sum()).item()

    _, h = m.encoder_rms_norm(x, w, residual=res, p=p, rng=rng, want_sum=True)
    grads = m.encoder_rms_norm_backward(dy, h, w, dsum=more, p=p, rng=rng)
    for k, g in enumerate(grads):
        v = workloads.normal(tuple(g.shape), seed=20 + k, device=DEV)
        args, s = [x, res, w], 1e-2
        ends = []
        for sign in (s, -s):
            moved = list(args)
            moved[k] = args[k] + sign * v
            ends.append(value(*moved))
        want = (g.double() * v.double()).sum().item()
        size = (g.double().abs() * v.double().abs()).sum().item()
        # third derivatives of a normed row's elements are below 10, steps 1e-2: 1e-4 * 10 / 6; rounding 2^-22 / 1e-2
        assert abs((ends[0] - ends[1]) / (2 * s) - want) <= (2e-4 + 1e-4) * size


def test_many_rows():
    """Rows whose offsets pass 32 bits: some of them against fp64, forward and backward."""
    n, d = (1 << 21) + 5, 1032
    x, w = torch.empty((n, d), dtype=torch.bfloat16, device=DEV), _weight(d, torch.float32)
    for a in range(0, n, 1 << 19):
        b = min(n, a + (1 << 19))
        x[a:b] = workloads.normal((b - a, d), seed=a + 1, device=DEV).bfloat16()
    y = m.encoder_rms_norm(x, w)
    for a in (0, n // 2, n - 9):
        _check_forward(x, x[a:a + 9], y[a:a + 9], w)
    dx, _, _ = m.encoder_rms_norm_backward(y, x, w)
    for a in (0, n // 2, n - 9):
        back, tol, _, _ = ref.norm_backward(y[a:a + 9], x[a:a + 9], w, EPS)
        ref.within(dx[a:a + 9], back, tol + 2.0 ** -8 * back.abs())
    q, s = m.encoder_rms_norm(x, w, fmt="int8")
    want, _ = ref.norm(x[-9:], w, EPS)
    ref.within(q[-9:].float(), want / s[-9:, None].double(), 0.5 + 2.0 ** -20 * (want / s[-9:, None].double()).abs() + 2 * ref.ROW * 127)


def test_repeatable_and_no_rows():
    dy, h, w = rows(3000, 520, 1, torch.bfloat16), rows(3000, 520, 2, torch.bfloat16), _weight(520, torch.float32)
    first = [t.clone() for t in m.encoder_rms_norm_backward(dy, h, w)]
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(m.encoder_rms_norm_backward(dy, h, w), first))
    dx, dres, dw = m.encoder_rms_norm_backward(dy[:0], h[:0], w)
    assert dx.shape == (0, 520) and (dw == 0).all() and m.encoder_rms_norm(h[:0], w).shape == (0, 520)
    assert m.encoder_rms_norm_backward(dy, h)[2] is None
    need = m.encoder_rms_norm_backward_workspace_size(h, w)
    small = torch.empty(need - 1, dtype=torch.uint8, device=DEV)
    with pytest.raises(m.MaxSimError) as e:
        m.encoder_rms_norm_backward(dy, h, w, workspace=small)
    assert e.value.status == 5
