"""GPU: calls with ``stream=`` while the current stream still has work that
writes memory which has been freed there."""
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu
m = pytest.importorskip("maxsim_scoring_02_gb300")
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.load_library()


def _encoder_calls():
    n = [300, 41]
    T, H, G, d = sum(n), 4, 2, 64
    x = workloads.normal((T, H + 2 * G, d), seed=1, device=DEV).to(torch.bfloat16)
    dO = workloads.normal((T, H, d), seed=2, device=DEV).to(torch.bfloat16)
    q, k, v = x[:, :H], x[:, H:H + G], x[:, H + G:]
    off = workloads.csr_offsets(torch.tensor(n, dtype=torch.int64)).to(DEV)
    freq, _ = m.maxsim_rotary_frequencies(d)
    out, lse = m.maxsim_attention(q, k, v, off, want_lse=True)
    grads = [workloads.normal((5000,), seed=3 + i, device=DEV) for i in range(3)]
    clipped = [torch.empty_like(g) for g in grads]
    return {
        "rotary": lambda **kw: m.maxsim_rotary(q, freq, offsets=off, **kw),
        "attention": lambda **kw: m.maxsim_attention(q, k, v, off, want_lse=True, **kw),
        "attention_backward": lambda **kw: m.maxsim_attention_backward(dO, q, k, v, out, lse, off, **kw),
        "clip": lambda **kw: (m.maxsim_clip_grad_norm(grads, 1.0, out=clipped, **kw), *clipped),
    }


def _busy():
    """Some tens of milliseconds of work on the current stream."""
    a = torch.ones((8192, 8192), dtype=torch.bfloat16, device=DEV)
    for _ in range(40):
        torch.mm(a, a)


def _freed_but_pending():
    """Blocks of every small size, freed, which the current stream will yet overwrite."""
    blocks = [torch.empty(512 << i, dtype=torch.uint8, device=DEV) for i in range(11) for _ in range(6)]
    torch.cuda.synchronize()
    _busy()
    for b in blocks:
        b.fill_(255)


@pytest.mark.parametrize("name", ["rotary", "attention", "attention_backward", "clip"])
def test_pending_writes_of_the_current_stream_reach_no_call_on_another(name):
    call = _encoder_calls()[name]
    want = call()
    want = [t.clone() for t in (want if isinstance(want, tuple) else (want,))]
    s = torch.cuda.Stream()
    call(stream=s)
    for _ in range(3):
        torch.cuda.synchronize()
        _freed_but_pending()
        got = call(stream=s)
        got = got if isinstance(got, tuple) else (got,)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert m.maxsim_device_status() == (0, 0)
