"""Host side of the token-encoder operators: calls that their contract rules
out are refused before any CUDA call."""
import pytest

import maxsim_scoring_02_gb300 as m
from maxsim_scoring_02_gb300 import build as mbuild

INVALID, UNSUPPORTED = 1, 2


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


@pytest.mark.parametrize("change", [{"cap": 3e38}, {"cap": 2.0 ** 61}, {"cap": 1e-39}, {"cap": 2.0 ** -61},
                                    {"scale": 2.0 ** 61}, {"scale": 3e38}, {"scale": 1e-39}])
def test_scales_and_caps_out_of_the_kernels_range_are_refused(lib, change):
    """3e38 log2(e) is infinite and scale / 1e-39 too: a score of 0 became NaN."""
    assert _forward(lib, **change) == UNSUPPORTED and _backward(lib, **change) == UNSUPPORTED


def test_the_ends_of_the_range_are_taken(lib):
    for change in ({"cap": 2.0 ** 60}, {"cap": 2.0 ** -60}, {"scale": 2.0 ** 60}, {"scale": 2.0 ** -60}, {"cap": -1.0}):
        assert lib.maxsim_attention_backward(_spec(**change), *[_heads()] * 5, 0x1000, *[_heads()] * 3, None, 0, None) == 5


def test_tokens_without_a_document_are_refused(lib):
    """Nothing would be written, and the results would be what the memory held."""
    assert _forward(lib, B=0) == INVALID and _backward(lib, B=0) == INVALID
    assert _forward(lib, T=0, B=0) == 0 and _backward(lib, T=0, B=0) == 0


# (token stride, head stride) of 100 tokens with 4 heads of 64 (2 of them for keys)
APART = [(256, 64), (64, 6400), (64, 6408), (512, 128), (264, 64), (288, 72)]
SHARED = [(64, 64), (248, 64), (64, 6328), (128, 64), (256, 56), (8, 6400), (256, 256), (96, 64)]



@pytest.mark.parametrize("token,head", SHARED)
def test_results_whose_rows_share_elements_are_refused(lib, token, head):
    """Which block wrote such an element last would decide its value."""
    bad, good = _heads(token=token, head=head), _heads()
    assert _forward(lib, [good, good, good, bad]) == INVALID
    for i in (5, 6, 7):
        views = [good] * 8
        views[i] = bad
        if i == 5 or (token, head) not in ((128, 64), (248, 64)):   # two key-value heads of 64 lie within 128
            assert _backward(lib, views) == INVALID, i
    assert lib.maxsim_rotary(_heads(0x8000), 100, 4, 64, 64, 0x1000, None, 0, None, 0, 1.0, 0, 0, bad, None) == INVALID


def test_rotary_results_without_a_stride_are_refused(lib):
    for bad in (_heads(token=0), _heads(head=0)):
        assert lib.maxsim_rotary(_heads(0x8000), 100, 4, 64, 64, 0x1000, None, 0, None, 0, 1.0, 0, 0, bad, None) == INVALID


def test_rows_that_lie_apart_pass_that_check(lib):
    """Past it comes the workspace's check, which these calls fail."""
    for token, head in APART:
        v = _heads(token=token, head=head)
        assert lib.maxsim_attention_backward(_spec(), *[_heads()] * 5, 0x1000, v, v, v, None, 0, None) == 5
    one = _heads(token=8, head=64)
    assert lib.maxsim_attention_backward(_spec(T=1), *[_heads()] * 5, 0x1000, one, one, one, None, 0, None) == 5
