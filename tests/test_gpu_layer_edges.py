"""GPU: small rows in 8 bits, confident rows and long rows of the cross entropy,
gradients whose sums do not cancel, and scales at the ends of their ranges."""
import pytest
import torch

import workloads
from tests import _layer_ref as ref
from tests.test_gpu_dropout import rows
from tests.test_gpu_loss import _check, _inputs

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


def _uniform(shape, seed, lo=0.5, hi=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.rand(shape, generator=g) * (hi - lo) + lo).to(DEV)


# ------------------------------------------------------------ rows in 8 bits

@pytest.mark.parametrize("fmt,top", [("int8", 127.0), ("e4m3", 448.0)])
@pytest.mark.parametrize("eps", [1e-6, 1e-12, 2.0 ** -60])
@pytest.mark.parametrize("d", [64, 100, 200, 768, 2048])
def test_eight_bits_of_small_rows(fmt, top, eps, d):
    """Rows of zeros and of small numbers, beside usual ones, whatever eps; weights that
    are zero or small."""
    x, w = rows(7, d, 1, torch.float32).contiguous(), 1 + 0.3 * workloads.normal((d,), seed=9, device=DEV)
    x[1] = 0.0
    x[2], x[3], x[4], x[5] = x[2] * 1e-9, x[3] * 1e-20, x[4] * 1e-30, x[5] * 1e-37
    holes = torch.where(torch.arange(d, device=DEV) % 3 == 0, 0.0, w)
    for weight in (None, w, holes, w * 1e-20, torch.zeros_like(w)):
        q, scale = m.encoder_rms_norm(x, weight, eps=eps, fmt=fmt)
        y, rstd = ref.norm(x, weight, eps)
        reach = y.abs().amax(1).clamp_min(1e-30)
        assert ((scale.double() - reach / top).abs() <= 2 * ref.ROW * reach / top).all()
        v = y / (reach / top)[:, None]
        step = 0.5 if fmt == "int8" else (v.abs() * 2.0 ** -4).clamp_min(2.0 ** -10)
        # products h w below the smallest normal number are multiples of 2^-149
        below = 2.0 ** -149 * rstd / reach[:, None] * top
        ref.within(q.float(), v, step + 2.0 ** -18 * v.abs() + below)
        assert (q.float()[y == 0] == 0).all()


# -------------------------------------------------- logits, losses, gradients

def _confident(d, V, z, dtype, seed=1, T=33):
    """Rows whose target, column 0, has a logit of some z, the others of z - 17: all
    products of one sign. The last element is the target's alone: what dx has there is q - 1
    times dloss."""
    x = _uniform((T, d), seed)
    w = _uniform((V, d), seed + 1, 0.9, 1.1) * (z / d)
    w[1:] *= (z - 17.0) / z
    x, w = x.to(dtype), w.to(dtype)
    x[:, -1], w[:, -1] = 0.0, 0.0
    w[0, -1] = 1.0
    return x, w, torch.zeros(T, dtype=torch.int64, device=DEV)


# The sum of 300 exponentials, the largest of them 1, in fp32: an accumulator adds 32 (to 1 or
# more, where what is small loses up to 2^-24 each time), two steps join four of them, one a
# warp's parts, five the warps; the exponential of the largest is off by 2^-22, the logarithm
# by 2^-23, the difference and its product with ln 2 by less: 32 + 2 + 1 + 5 + 4 + 2 + 2.
SUMS = 48 * 2.0 ** -24


def _softmax(x, w, scale=1.0):
    z = x.double() @ w.double().T * scale
    return z, torch.logsumexp(z, 1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,z", [(64, 30.0), (2048, 30.0), (2048, 100.0), (8192, 100.0), (65536, 60.0)])
def test_gradient_of_confident_rows(dtype, d, z):
    """The backward's logits are the forward's to the last bit, so q = exp(z - lse) near 1
    is off by the rounding of numbers of lse's size alone: the sum, its product with ln 2, the
    product with 1 / ln 2 (2^-24 each), both constants (2^-25); and by SUMS. What else q has is
    off by 2^-17 of the logits. With all of d in one sum, cut towards zero, q was off
    by 1e-4 at d = 2048 and z = 100."""
    x, w, t = _confident(d, 300, z, dtype)
    _, lse = m.encoder_cross_entropy(x, w, t)
    dx, dw = m.encoder_cross_entropy_backward(torch.ones(33, device=DEV), x, w, t, lse)
    zz, lse64 = _softmax(x, w)
    want = torch.expm1(zz[:, 0] - lse64)
    assert (want < 0).all() and (want > -0.01).all()
    off = 4 * 2.0 ** -24 * lse64.abs() + SUMS
    ref.within(dx[:, -1], want, off + (2 * ref.U[dtype] + 2.0 ** -17 * z) * want.abs() + 2 * ref.TINY[dtype])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,z", [(64, 30.0), (2048, 100.0), (2048, 1000.0)])
def test_loss_of_confident_rows(dtype, d, z):
    """A loss near 0 is no difference of two rounded numbers of lse's size: off by SUMS,
    whatever the logits."""
    x, w, t = _confident(d, 300, z, dtype)
    loss, _ = m.encoder_cross_entropy(x, w, t)
    zz, lse = _softmax(x, w)
    want = torch.log1p(torch.exp(zz[:, 1:] - zz[:, :1]).sum(1))
    # the others' logits, and the target's, are off by 2^-18 of themselves at most
    ref.within(loss, want, SUMS + want * 2.0 ** -17 * z)


@pytest.mark.parametrize("d", [512, 1024, 2048, 8192, 65536])
def test_long_rows(d):
    """All products of one sign, evenly: a part of 512 is 32 additions cut towards zero,
    each by up to 2^-23 of a sum that grows evenly, 33 / 2 steps of its whole; n parts are added with
    rounding, (n + 1) / 2 steps of 2^-24. All of d = 8192 in one cut sum was off by 5e-6 of itself."""
    T, V = 40, 9
    x, w = _uniform((T, d), 3).bfloat16(), (_uniform((V, d), 4) * 60.0 / d).bfloat16()
    t = torch.arange(T, device=DEV) % V
    loss, lse = m.encoder_cross_entropy(x, w, t)
    z, want = _softmax(x, w)
    of = 33 / 2 * 2.0 ** -23 + (d / 512 + 1) / 2 * 2.0 ** -24
    ref.within(lse, want, of * z.amax(1) + 2.0 ** -22 * want + 2.0 ** -20, "lse")
    ref.within(loss, want - z.gather(1, t[:, None])[:, 0], 2 * of * z.amax(1) + 2.0 ** -20, "loss")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [4104, 65536])
def test_gradients_of_long_rows(dtype, d):
    """Random signs: the parts' cut is at most 32 * 2^-23 of the sizes' sum, and n steps of 2^-24."""
    T, V = 40, 300
    x, w, t, dloss = _inputs(T, V, d, dtype)
    _, lse = m.encoder_cross_entropy(x, w, t)
    dx, dw = m.encoder_cross_entropy_backward(dloss, x, w, t, lse)
    z, want = _softmax(x, w)
    X, W, u = x.double(), w.double(), ref.U[dtype]
    off = (32 * 2.0 ** -23 + d / 512 * 2.0 ** -24) * (X.abs() @ W.abs().T).amax(1) + 2.0 ** -17 + 2.0 ** -22 * want.abs()
    ref.within(lse, want, off, "lse")
    part = torch.where(t >= 0, dloss.double(), 0.0)[:, None]
    p = torch.exp(z - want[:, None])
    hit = torch.nn.functional.one_hot(t.clamp_min(0), V).double()
    dz = (p - hit) * part
    E = u * dz.abs() + p * part.abs() * (2 * off[:, None] + 2.0 ** -18) + ref.TINY[dtype] * 2.0 ** -13 * dloss.abs().max().item()
    ref.within(dx, dz @ W, (E + V * 2.0 ** -23 * dz.abs()) @ W.abs() + u * (dz @ W).abs() + ref.TINY[dtype], "dx")
    ref.within(dw, dz.T @ X, (E + T * 2.0 ** -23 * dz.abs()).T @ X.abs() + u * (dz.T @ X).abs() + ref.TINY[dtype], "dw")


def test_a_large_dloss_times_a_large_scale():
    """Their product leaves fp32's range, results do not: they are what the formula says, and
    0 in rows without a target."""
    _check(*_many(90, 700, 64, torch.bfloat16, 2.0 ** -30, 2.0 ** 96), scale=2.0 ** 60)
    _check(*_many(5000, 40, 64, torch.bfloat16, 2.0 ** -30, 2.0 ** 96), scale=2.0 ** 60)


def test_a_small_dloss_times_a_small_scale():
    """Their product is below the normal numbers, results are not."""
    _check(*_many(90, 700, 64, torch.bfloat16, 2.0 ** 30, 2.0 ** -80), scale=2.0 ** -60)
    _check(*_many(5000, 40, 64, torch.bfloat16, 2.0 ** 30, 2.0 ** -80), scale=2.0 ** -60)


def _many(T, V, d, dtype, of, times):
    x, w, t, dloss = _inputs(T, V, d, dtype)
    return x * of, w * of, t, dloss * times


# Rows by blocks, each of which has an element of its own, and one target: no sum of dW cancels.
@pytest.mark.parametrize("T,V,d,dtype", [(40000, 3, 64, torch.bfloat16), (40000, 300, 64, torch.float16), (20001, 300, 136, torch.bfloat16),
                                         (5000, 40, 520, torch.bfloat16), (600001, 300, 8, torch.float16), (9000, 17000, 64, torch.bfloat16)])
def test_sums_that_do_not_cancel(T, V, d, dtype):
    """dW[v, j] is the sum of dz[t, v] over the rows of block j: a part of the rows that is
    lost, or added to another, changes an element by a part of itself. dz is rounded (u), n
    additions of one sign cut by 2^-23 at most of what they have reached, (n + 1) / 2 of the
    whole, and the result rounded (u)."""
    block = torch.arange(T, device=DEV) * d // T
    x = torch.nn.functional.one_hot(block, d).to(dtype)
    w = (workloads.normal((V, d), seed=3, device=DEV)).to(dtype)
    t = torch.where(torch.arange(T, device=DEV) % 5 == 4, -1, V // 2)
    dloss = torch.full((T,), 0.75 * d / T, device=DEV)
    _, lse = m.encoder_cross_entropy(x, w, t)
    dx, dw = m.encoder_cross_entropy_backward(dloss, x, w, t, lse)
    z = w.double().T                                   # of block j: all its rows are the same
    p = torch.softmax(z, 1)
    dz = (p - (torch.arange(V, device=DEV) == V // 2).double()) * dloss[0].double()
    n = torch.zeros(d, dtype=torch.float64, device=DEV).index_add_(0, block, (t >= 0).double())
    u, tiny = ref.U[dtype], ref.TINY[dtype]
    E = u * dz.abs() + p * dloss[0].double() * 2.0 ** -15 + tiny * 2.0 ** -13 * dloss[0].double()
    want = (dz * n[:, None]).T
    fp = ((n + 1) / 2 * 2.0 ** -23)[None] * want.abs()
    ref.within(dw, want, (E * n[:, None]).T + fp + u * want.abs() + tiny, "dw")
    back = torch.where((t >= 0)[:, None], (dz @ w.double())[block], 0.0)
    tol = ((E + (V + 1) / 2 * 2.0 ** -23 * dz.abs()) @ w.double().abs())[block]
    ref.within(dx, back, torch.where((t >= 0)[:, None], tol, 0.0) + u * back.abs() + tiny, "dx")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [514, 40000])
def test_columns_that_every_row_has_to_add_up(dtype, T):
    """dx[t, j] is the sum of dz[t, v] over the columns of block j of the vocabulary: parts of the
    columns (few rows) and pieces of it (a dloss a row)."""
    V, d = (70001, 64) if T < 1000 else (9001, 16)
    block = torch.arange(V, device=DEV) * d // V
    w = torch.nn.functional.one_hot(block, d).to(dtype)
    x = workloads.normal((T, d), seed=4, device=DEV).to(dtype)
    t = torch.where(torch.arange(T, device=DEV) % 5 == 4, -1, V // 2)
    dloss = _uniform((T,), 5)
    _, lse = m.encoder_cross_entropy(x, w, t)
    dx, _ = m.encoder_cross_entropy_backward(dloss, x, w, t, lse, want_dweight=False)
    n = torch.bincount(block, minlength=d).double()
    z = x.double()
    each = torch.exp(z - torch.logsumexp(z + n.log(), 1)[:, None])       # p of a column of block j
    part = torch.where(t >= 0, dloss.double(), 0.0)[:, None]
    hit = (torch.arange(d, device=DEV) == block[V // 2]).double()
    want = (each * n - hit) * part
    u, tiny = ref.U[dtype], ref.TINY[dtype]
    E = (each * n + hit) * part * (u + 2.0 ** -15) + tiny * 2.0 ** -13 * dloss.max().double() * n * (part > 0)
    ref.within(dx, want, E + (n + 1) / 2 * 2.0 ** -23 * (each * n + hit) * part + u * want.abs() + tiny, "dx")


@pytest.mark.parametrize("dtype,steps", [(torch.bfloat16, 257), (torch.float16, 2049)])
def test_targets_of_equal_rows_are_exact(dtype, steps):
    """dloss = (n + 1) / n is next to 1 in the inputs' type; n rows of it are n + 1, a number of
    that type, and n (1 or its neighbour) if dz held dloss itself. Softmax's part, 1 / V a row, is
    less than half a step there."""
    V, d = 20000, 64
    x = torch.zeros((steps, d), dtype=dtype, device=DEV)
    x[:, 0] = 1.0
    w = torch.zeros((V, d), dtype=dtype, device=DEV)
    w[:, 1] = 1.0                                      # logits 0
    t = torch.full((steps,), 777, device=DEV)
    dloss = torch.full((steps,), (steps + 1) / steps, device=DEV)
    _, lse = m.encoder_cross_entropy(x, w, t)
    _, dw = m.encoder_cross_entropy_backward(dloss, x, w, t, lse)
    assert dw[777, 0].item() == -(steps + 1)


def test_a_few_rows_of_a_long_vocabulary():
    """More columns than 256 MB hold the parts of for 256 rows: the workspace has room for the rows there are."""
    x, w, t, _ = _inputs(3, (1 << 25) + 5, 8, torch.bfloat16)
    assert m.encoder_cross_entropy_workspace_size(x, w, t) <= 3 * ((1 << 18) + 1) * 8 + 512
    _check(x, w, t, None)
