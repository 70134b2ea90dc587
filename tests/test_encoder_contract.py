"""Host side of the token-encoder operators: calls that their contract rules
out are refused before any CUDA call."""
import pytest

import maxsim_scoring_02_gb300 as m
from maxsim_scoring_02_gb300 import build as mbuild

INVALID = 1


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return m.load_library()


def _heads(p=0x1000, token=256, head=64):
    return m._Heads(p, token, head)


def _spec(**change):
    v = dict(T=100, B=2, heads=4, kv_heads=2, d=64, dtype=0, mask=0, scale=0.1, cap=0.0, offsets=0x1000, key_len=None,
             prefix_len=None, slopes=None)
    v.update(change)
    return m._AttentionSpec(*v.values())


def _forward(lib, views=None, **change):
    return lib.maxsim_attention(_spec(**change), *(views or [_heads()] * 4), None, None)


def _backward(lib, views=None, **change):
    views = views or [_heads()] * 8
    return lib.maxsim_attention_backward(_spec(**change), *views[:5], 0x1000, *views[5:], 0x1000, 1 << 30, None)


def test_tokens_without_a_document_are_refused(lib):
    """Nothing would be written, and the results would be what the memory held."""
    assert _forward(lib, B=0) == INVALID and _backward(lib, B=0) == INVALID
    assert _forward(lib, T=0, B=0) == 0 and _backward(lib, T=0, B=0) == 0
