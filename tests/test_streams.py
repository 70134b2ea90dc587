"""Where a call runs and what it makes there: on its tensors' device, whichever
is current; and with ``stream=`` its workspace and its results come from that
stream's memory, not from the current stream's, whose freed blocks may still be
written by work that has yet to run."""
import inspect

import pytest
import torch

import maxsim_scoring_02_gb300 as m
from tests import _fake_cuda as fake

BF, F32, I8, I32, I64, U8 = torch.bfloat16, torch.float32, torch.int8, torch.int32, torch.int64, torch.uint8


@pytest.fixture
def cuda(monkeypatch):
    return fake.Cuda(monkeypatch, m)


def _calls(cuda, index=0):
    """Every entry point that makes something: (call, tensors that it makes)."""
    t = lambda shape, dtype: cuda.tensor(shape, dtype, index)  # noqa: E731
    q, k, x = t((6, 4, 64), BF), t((6, 2, 64), BF), t((6, 4, 64), BF)
    Q, D, pq = t((1, 3, 64), BF), t((5, 8, 64), BF), (t((3, 64), F32), t((8, 16, 8), F32), t((9, 8), U8), t((3,), I64))
    off, lse, freq = t((3,), I64), t((4, 6), F32), t((32,), I64)
    return {
        "rotary": (lambda **kw: m.maxsim_rotary(x, freq, offsets=off, **kw), 1),
        "attention": (lambda **kw: m.maxsim_attention(q, k, k, off, want_lse=True, **kw), 2),
        "attention_backward": (lambda **kw: m.maxsim_attention_backward(x, q, k, k, x, lse, off, **kw), 4),
        "clip": (lambda **kw: m.maxsim_clip_grad_norm([t((8,), F32), t((9,), BF)], 1.0, **kw), 2),
        "score": (lambda **kw: m.maxsim_score(Q, D, want_argmax=True, **kw), 2),
        "length_order": (lambda **kw: m.maxsim_length_order(doc_len=t((5,), I32), nd=8, **kw), 2),
        "score_ordered": (lambda **kw: m.maxsim_score_ordered(Q, D, t((5,), I32), want_argmax=True, **kw), 2),
        "score_streamed": (lambda **kw: m.maxsim_score_streamed(Q, torch.zeros((5, 8, 64), dtype=BF), want_argmax=True, **kw), 3),
        "score_varlen": (lambda **kw: m.maxsim_score_varlen(Q, t((9, 64), BF), off, want_argmax=True, **kw), 2),
        "score_pq": (lambda **kw: m.maxsim_score_pq(*pq, want_argmax=True, **kw), 3),
        "score_pq_noalloc": (lambda **kw: m.maxsim_score_pq_noalloc(*pq, want_argmax=True, **kw), 2),
        "score_i8": (lambda **kw: m.maxsim_score_i8(t((3, 64), I8), t((3,), F32), t((9, 64), I8), t((9,), F32), off,
                                                    want_details=True, **kw), 4),
        "backward": (lambda **kw: m.maxsim_backward(Q, D, t((1, 5, 3), I32), t((1, 5), F32), **kw), 3),
        "backward_dq": (lambda **kw: m.maxsim_backward_dq(D, t((1, 5, 3), I32), t((1, 5), F32), **kw), 2),
        "backward_dd": (lambda **kw: m.maxsim_backward_dd(Q, t((1, 5, 3), I32), t((1, 5), F32), 8, **kw), 1),
    }


ENTRIES = ["rotary", "attention", "attention_backward", "clip", "score", "length_order", "score_ordered",
           "score_streamed", "score_varlen", "score_pq", "score_pq_noalloc", "score_i8", "backward", "backward_dq",
           "backward_dd"]


@pytest.mark.parametrize("name", ENTRIES)
def test_a_call_on_another_stream_makes_its_memory_there(cuda, name):
    call, count = _calls(cuda)[name]
    other, outer = fake.Stream(0, 0x77), cuda.streams[0]
    result = call(stream=other)
    result = result if isinstance(result, tuple) else (result,)
    assert len(cuda.made) == count and all(t.pool is other for t in cuda.made)
    # results are read by the caller's stream; a workspace is not
    for t in cuda.made:
        assert (outer in t.users) == any(t is r for r in result)
    launches = [c for c in cuda.lib.calls]
    assert len(launches) == 1 and 0x77 in [getattr(a, "value", a) for a in launches[0][2]]
    assert cuda.streams[0] is outer


@pytest.mark.parametrize("name", ENTRIES)
def test_a_call_on_the_current_stream(cuda, name):
    call, count = _calls(cuda)[name]
    call()
    assert len(cuda.made) == count and all(t.pool is cuda.streams[0] and not t.users for t in cuda.made)


def test_the_stream_may_be_given_by_position(cuda):
    other = fake.Stream(0, 0x77)
    x, freq = cuda.tensor((6, 4, 64), BF), cuda.tensor((32,), I64)
    m.maxsim_rotary(x, freq, None, None, False, 1.0, False, None, other)
    assert [t.pool for t in cuda.made] == [other]


@pytest.mark.parametrize("name", ENTRIES)
def test_a_call_runs_on_its_tensors_device(cuda, name):
    call, count = _calls(cuda, 1)[name]
    call()
    assert [device for _, device, _ in cuda.lib.calls] == [1] and cuda.device == 0
    assert len(cuda.made) == count and all(t.index == 1 and t.pool is cuda.streams[1] for t in cuda.made)
    other = fake.Stream(1, 0x99)
    call(stream=other)
    assert cuda.lib.calls[-1][1] == 1 and 0x99 in [getattr(a, "value", a) for a in cuda.lib.calls[-1][2]]


@pytest.mark.parametrize("name", ENTRIES)
def test_a_stream_of_another_device_is_refused(cuda, name):
    call, _ = _calls(cuda, 1)[name]
    with pytest.raises(ValueError):
        call(stream=fake.Stream(0, 0x77))
    assert not cuda.lib.calls


ARGUMENTS = {
    "maxsim_rotary": dict(x=((6, 4, 64), BF), freq=((32,), I64), offsets=((3,), I64), out=((6, 4, 64), BF)),
    "maxsim_attention": dict(q=((6, 4, 64), BF), k=((6, 2, 64), BF), v=((6, 2, 64), BF), offsets=((3,), I64),
                             key_len=((2,), I32), prefix_len=((2,), I32), slopes=((4,), F32), out=((6, 4, 64), BF),
                             lse=((4, 6), F32)),
    "maxsim_attention_backward": dict(dO=((6, 4, 64), BF), q=((6, 4, 64), BF), k=((6, 2, 64), BF), v=((6, 2, 64), BF),
                                      out=((6, 4, 64), BF), lse=((4, 6), F32), offsets=((3,), I64),
                                      key_len=((2,), I32), prefix_len=((2,), I32), slopes=((4,), F32),
                                      dq=((6, 4, 64), BF), dk=((6, 2, 64), BF), dv=((6, 2, 64), BF),
                                      workspace=((64,), U8)),
    "maxsim_score": dict(Q=((1, 3, 64), BF), D=((5, 8, 64), BF), doc_len=((5,), I32), out=((1, 5), F32)),
    "maxsim_backward": dict(Q=((1, 3, 64), BF), D=((5, 8, 64), BF), argmax=((1, 5, 3), I32), dS=((1, 5), F32)),
}


@pytest.mark.parametrize("name", ARGUMENTS)
def test_tensors_of_two_devices_are_refused(cuda, name):
    f, shapes = getattr(m, name), ARGUMENTS[name]
    how = {"mask": "prefix"} if "prefix_len" in shapes else {}
    every = lambda odd: {k: cuda.tensor(*v, 0 if k == odd else 1) for k, v in shapes.items()}  # noqa: E731
    f(**every(None), **how)
    assert len(cuda.lib.calls) == 1
    for odd in shapes:
        with pytest.raises(ValueError):
            f(**every(odd), **how)
    assert len(cuda.lib.calls) == 1


def test_clipping_refuses_tensors_of_two_devices(cuda):
    g = [cuda.tensor((8,), F32, 1), cuda.tensor((9,), F32, 1)]
    for kw in ({"norm": cuda.tensor((1,), F32, 0)}, {"workspace": cuda.tensor((64,), U8, 0)},
               {"out": [cuda.tensor((8,), F32, 0), cuda.tensor((9,), F32, 0)]}):
        with pytest.raises(ValueError):
            m.maxsim_clip_grad_norm(g, 1.0, **kw)
    with pytest.raises(ValueError):
        m.maxsim_clip_grad_norm([g[0], cuda.tensor((9,), F32, 0)], 1.0)
    assert not cuda.lib.calls


def test_every_entry_point_with_a_stream_is_covered():
    with_stream = {n[len("maxsim_"):] for n in dir(m) if n.startswith("maxsim_") and n != "maxsim_device_status"
                   and "stream" in inspect.signature(getattr(m, n)).parameters}
    assert with_stream == {"clip_grad_norm" if n == "clip" else n for n in ENTRIES}
