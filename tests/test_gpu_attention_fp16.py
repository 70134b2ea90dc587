"""GPU: the fp16 backward over the range that its gradients have: long documents,
whose weights are small, and small or large gradients of the output.

Every weight, dS and result is rounded to 2^-11 of itself at most, and scores of
N(0,1) inputs move weights by less than as much on average; the roundings of
thousands of terms do not add up. Together no more than 4 * 2^-11 of the result,
in the 2-norm, where nothing is too small or too large for fp16."""
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


def _inputs(lengths, d, seed, q_times=1.0, k_times=1.0, dO_times=1.0):
    T = sum(lengths)
    new = lambda s, f: (workloads.normal((T, 1, d), seed=seed + s, device=DEV) * f).half()  # noqa: E731
    return new(0, q_times), new(1, k_times), new(2, 1.0), new(3, dO_times)


def _run(lengths, q, k, v, dO, **how):
    off = workloads.csr_offsets(torch.tensor(lengths, dtype=torch.int64)).to(DEV)
    out, lse = m.maxsim_attention(q, k, v, off, want_lse=True, **how)
    got = dict(zip(("dq", "dk", "dv"), m.maxsim_attention_backward(dO, q, k, v, out, lse, off, **how)))
    torch.cuda.synchronize()
    assert m.maxsim_device_status() == (0, 0)
    return got, out, lse


def _near(got, want, name):
    err = ((got.double() - want).norm() / want.norm()).item()
    assert err <= 4 * 2.0 ** -11, f"{name}: {err:.2e} of its norm"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("times", [1e-3, 1e3])
def test_small_and_large_gradients_of_long_documents(d, times):
    """12001 keys: a weight is 2^-13.5. Keys 64 times as large as their queries are
    small bring dq to fp16's normal numbers, and queries dk; scores are N(0,1)."""
    n = [12001]
    small = 1.0 / 64 if times < 1 else 1.0
    for which, q_times, k_times in (("dq", small, 1 / small), ("dk", 1 / small, small)):
        q, k, v, dO = _inputs(n, d, 5, q_times, k_times, times)
        got, _, _ = _run(n, q, k, v, dO)
        r = ref.attention(q, k, v, n, dO=dO)
        assert torch.isfinite(got[which]).all()
        _near(got[which], r[which], which)
    _near(got["dv"], r["dv"], "dv")


def test_each_document_has_its_own_range():
    """Gradients of 10^4 beside ones of 10^-4, and hidden values as large as fp16
    has: every document's gradients are what they are alone, to the bit."""
    n, hide = [700, 300, 900], [700, 300, 500]
    q, k, v, dO = _inputs(n, 64, 17)
    dO[:700] *= 1e-4
    dO[700:1000] *= 1e4
    dO[1000:] *= 1e-4
    k[1500:], v[1500:] = 6e4, 6e4
    got, _, _ = _run(n, q, k, v, dO, key_len=torch.tensor(hide, dtype=torch.int32, device=DEV))
    s = 0
    for length, keys in zip(n, hide):
        part = slice(s, s + length)
        alone, _, _ = _run([length], *(t[part].contiguous() for t in (q, k, v, dO)),
                           key_len=torch.tensor([keys], dtype=torch.int32, device=DEV))
        assert all(torch.equal(got[x][part], alone[x]) for x in got)
        s += length


@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_hidden_values_never_reach_a_row(poison):
    n, hide = [90, 150, 40, 300], [60, 150, 40, 170]
    q, k, v, dO = _inputs(n, 64, 23)
    kl = torch.tensor(hide, dtype=torch.int32, device=DEV)
    want, _, _ = _run(n, q, k, v, dO, key_len=kl)
    for t in (k, v):
        t[60:90] = poison
        t[280 + 170:] = poison
    for t in (k, v, q, dO):
        t[240:280] = poison
    got, _, _ = _run(n, q, k, v, dO, key_len=kl)
    rows = torch.ones(sum(n), dtype=torch.bool, device=DEV)
    rows[240:280] = False
    assert all(torch.equal(got[x][rows], want[x][rows]) for x in got)


def test_no_gradient_at_all():
    n = [200, 31]
    q, k, v, dO = _inputs(n, 64, 29, dO_times=0.0)
    got, _, _ = _run(n, q, k, v, dO)
    assert all((t == 0).all() for t in got.values())
