"""Host side of the token-encoder operators: the frequency table and the
argument checks, which reject before any CUDA call."""
import ctypes
import math

import pytest
import torch

import maxsim_scoring_02_gb300 as m
from maxsim_scoring_02_gb300 import build as mbuild
from tests import _encoder_ref as ref


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return m.load_library()


@pytest.mark.parametrize("rot,base,scaling,factor,original", [
    (64, 10000.0, "none", 1.0, 0), (128, 500000.0, "linear", 8.0, 0), (96, 10000.0, "ntk", 4.0, 0),
    (128, 10000.0, "yarn", 16.0, 8192), (32, 10000.0, "yarn", 2.0, 512), (2, 10000.0, "none", 1.0, 0)])
def test_frequencies(lib, rot, base, scaling, factor, original):
    freq, amp = m.maxsim_rotary_frequencies(rot, base, scaling, factor, original, device="cpu")
    angles, amplitude = ref.rotary_angles(torch.ones(1), rot, base, scaling, factor, original)
    want = angles[0] * (2.0 ** 64 / (2 * math.pi))
    assert freq.shape == (rot // 2,) and (freq > 0).all()
    # whole units of 2^-64 of a turn, made in fp64
    assert ((freq.double() - want).abs() <= 1 + want * 1e-14).all()
    assert abs(amp - amplitude) <= 1e-7 * amplitude


def test_frequency_refusals(lib):
    for args in ((63,), (0,), (64, 1.0), (64, float("inf")), (2, 1e4, "ntk", 2.0), (64, 1e4, "linear", 0.5),
                 (64, 1e4, "yarn", 2.0, 0)):
        with pytest.raises(m.MaxSimError):
            m.maxsim_rotary_frequencies(*args, device="cpu")
    with pytest.raises(ValueError):
        m.maxsim_rotary_frequencies(64, scaling="other", device="cpu")


def _heads(p=0x1000, token=256, head=64):
    return m._Heads(p, token, head)


def _spec(**change):
    v = dict(T=100, B=2, heads=4, kv_heads=2, d=64, dtype=0, mask=0, scale=0.1, cap=0.0, offsets=0x1000, key_len=None,
             prefix_len=None, slopes=None)
    v.update(change)
    return m._AttentionSpec(*v.values())


@pytest.mark.parametrize("change,status", [
    ({"T": -1}, 1), ({"B": -1}, 1), ({"heads": 0}, 1), ({"kv_heads": 3}, 1), ({"dtype": 9}, 1), ({"mask": 3}, 1),
    ({"mask": 2}, 1), ({"scale": 0.0}, 1), ({"scale": float("nan")}, 1), ({"cap": float("inf")}, 1),
    ({"offsets": None}, 1), ({"offsets": 0x1004}, 1), ({"key_len": 0x1002}, 1), ({"dtype": 2}, 2), ({"d": 60}, 2),
    ({"d": 136}, 2), ({"T": 2 ** 31}, 2), ({"heads": 70000, "kv_heads": 1}, 2)])
def test_attention_spec_refusals(lib, change, status):
    h = _heads()
    assert lib.maxsim_attention(_spec(**change), h, h, h, h, None, None) == status
    assert lib.maxsim_attention_backward(_spec(**change), h, h, h, h, h, 0x1000, h, h, h, 0x1000, 1 << 30, None) == status
    assert lib.maxsim_attention_backward_workspace_size(_spec(**change)) >= 0


@pytest.mark.parametrize("bad", [_heads(0), _heads(0x1008), _heads(token=100), _heads(token=0), _heads(head=-64),
                                 _heads(head=4)])
def test_attention_view_refusals(lib, bad):
    h = _heads()
    for i in range(4):
        views = [h] * 4
        views[i] = bad
        assert lib.maxsim_attention(_spec(), *views, None, None) == 1
    for i in range(8):
        views = [h] * 8
        views[i] = bad
        assert lib.maxsim_attention_backward(_spec(), *views[:5], 0x1000, *views[5:], 0x1000, 1 << 30, None) == 1


def test_attention_workspace(lib):
    h = _heads()
    need = lib.maxsim_attention_backward_workspace_size(_spec())
    assert need >= 100 * 4 * 4
    for ws, n in ((None, 1 << 30), (0x1000, need - 1), (0x1008, need)):
        assert lib.maxsim_attention_backward(_spec(), h, h, h, h, h, 0x1000, h, h, h, ws, n, None) == 5
    assert lib.maxsim_attention_backward(_spec(), h, h, h, h, h, None, h, h, h, 0x1000, need, None) == 1
    assert lib.maxsim_attention(_spec(T=0), h, h, h, h, None, None) == 0
    assert lib.maxsim_attention(None, h, h, h, h, None, None) == 1


def test_rotary_refusals(lib):
    h = _heads()
    call = lambda x=h, T=10, heads=2, d=64, rot=64, freq=0x1000, off=None, B=0, pos=None, dt=0, out=h: \
        lib.maxsim_rotary(x, T, heads, d, rot, freq, off, B, pos, 0, 1.0, 0, dt, out, None)  # noqa: E731
    assert call(T=0) == 0
    for kw in (dict(T=-1), dict(heads=0), dict(rot=63), dict(rot=66), dict(rot=0), dict(freq=None), dict(dt=5),
               dict(x=_heads(0x1001)), dict(off=0x1000, B=0), dict(off=0x1000, B=2, pos=0x1000),
               dict(out=_heads(token=512)), dict(x=_heads(token=-1)), dict(x=_heads(0))):
        assert call(**kw) == 1, kw
    assert call(d=5000, rot=64) == 2


def test_clip_refusals(lib):
    A = lambda t, *v: (t * len(v))(*v)  # noqa: E731
    ptr, n, dt = A(ctypes.c_void_p, 0x1000), A(ctypes.c_int64, 8), A(ctypes.c_int32, 2)
    ws = m.maxsim_clip_grad_norm_workspace_size(1)
    assert ws > 0 and m.maxsim_clip_grad_norm_workspace_size(-1) == 0
    call = lambda g=ptr, o=ptr, s=n, d=dt, k=1, mx=1.0, norm=0x1000, w=0x1000, b=ws: \
        lib.maxsim_clip_grad_norm(g, o, s, d, k, mx, norm, w, b, None)  # noqa: E731
    for kw in (dict(k=-1), dict(g=None), dict(s=A(ctypes.c_int64, -1)), dict(d=A(ctypes.c_int32, 3)), dict(mx=-1.0),
               dict(mx=float("nan")), dict(norm=None), dict(g=A(ctypes.c_void_p, 0x1002)), dict(o=A(ctypes.c_void_p, None))):
        assert call(**kw) == 1, kw
    assert call(w=None) == 5 and call(b=ws - 1) == 5 and call(w=0x1008) == 5
