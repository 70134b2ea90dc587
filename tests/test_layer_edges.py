"""Host side of the layer and loss operators: sizes beyond what they count in, memory that
overlaps what is written, and calls that want nothing."""
import pytest
import torch

import maxsim_scoring_02_gb300 as m
from maxsim_scoring_02_gb300 import build as mbuild
from tests import _fake_cuda as fake
from tests.test_layer_contract import (BF, BIG, F32, I64, INVALID, UNSUPPORTED, WORKSPACE, _backward, _dropout, _forward, _loss,
                                       _norm, _norm_bwd, _spec, _v)


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return m.load_library()


@pytest.mark.parametrize("d", [2 ** 31 - 257, 2 ** 31 - 256, 2 ** 31 - 1])
def test_rows_too_long_for_dropout(lib, d):
    """Parts of 256 columns, and the columns of the last of them, are counted in 31 bits."""
    assert _dropout(lib, T=1, d=d, x=_v(0x100000, 1 << 32), out=_v(1 << 40, 1 << 32)) == UNSUPPORTED


def test_widths_beyond_32_bits_are_refused(monkeypatch):
    """ctypes passes on the lower 32 bits of a width, and a row of 2^32 + 64 columns would be one of 64."""
    cuda = fake.Cuda(monkeypatch, m)
    wide = lambda dtype: fake.dress(torch.empty((1, 2 ** 32 + 64), dtype=dtype, device="meta"), 0, cuda.streams[0])  # noqa: E731
    rng, row = cuda.tensor((2,), I64), cuda.tensor((1,), F32)
    target = cuda.tensor((1,), I64)
    for call in (lambda: m.encoder_dropout(wide(BF), 0.5, rng), lambda: m.encoder_rms_norm(wide(BF)),
                 lambda: m.encoder_rms_norm_backward(wide(BF), wide(BF)), lambda: m.encoder_rms_norm_backward_workspace_size(wide(BF)),
                 lambda: m.encoder_cross_entropy(wide(BF), wide(BF), target),
                 lambda: m.encoder_cross_entropy_backward(row, wide(BF), wide(BF), target, row)):
        with pytest.raises(m.MaxSimError) as e:
            call()
        assert e.value.status == UNSUPPORTED
    assert not cuda.lib.calls


# The views' places: x (or dy) at 0x100000, out at 0x900000, h at 0x600000; 10 rows of 64 bf16, 512 bytes apart.

def test_rng_and_scale_overlap_nothing_that_is_written(lib):
    assert _dropout(lib, rng=0x900010) == INVALID
    assert _dropout(lib, rng=0x900000 + 9 * 512 + 120) == INVALID
    for kw in (dict(rng=0x900010), dict(rng=0x800008, sum=_v(0x800000)), dict(rng=0x4000, format=1, scale=0x4008),
               dict(weight=0x4000, format=1, scale=0x4000), dict(weight=0x4000, format=2, scale=0x40fc),
               dict(weight=0x4000, format=1, scale=0x4000 - 36)):
        assert _norm(lib, **kw) == INVALID, kw
    for kw in (dict(dx=_v(0x900000), rng=0x900008), dict(dres=_v(0x900000), rng=0x900008),
               dict(dw=0x7000, rng=0x70f8, ws=0x10000, n=BIG)):
        assert _norm_bwd(lib, **kw) == INVALID, kw


def test_workspaces_overlap_nothing_else(lib):
    """A workspace that begins within what is read or written, or ends there."""
    need = lib.maxsim_rms_norm_backward_workspace_size(_spec())
    last = (need - 1) // 16 * 16
    out, other = _v(0x900000), _v(0xa00000)
    for at in (0x500000, 0x600000, 0x700000, 0x900000, 0xa00000, 0x3000, 0x7000, 0x2000):
        for ws in (at, at - last):
            assert _norm_bwd(lib, dsum=_v(0x700000), dx=out, dres=other, dw=0x7000, ws=ws, n=BIG) == INVALID, hex(ws)
    need = lib.maxsim_cross_entropy_workspace_size(_loss())
    last = (need - 1) // 16 * 16
    for at in (0x100000, 0x900000, 0x2000, 0x3000, 0x4000):
        for ws in (at, at - last):
            assert _forward(lib, ws=ws, n=BIG) == INVALID, hex(ws)
    need = lib.maxsim_cross_entropy_backward_workspace_size(_loss())
    last = (need - 1) // 256 * 256
    for at in (0x100000, 0x900000, 0x1100000, 0x1900000, 0x20000, 0x30000, 0x40000):
        for ws in (at, at - last):
            assert _backward(lib, dloss=0x30000, lse=0x40000, targets=0x20000, ws=ws, n=BIG) == INVALID, hex(ws)


def test_gradients_that_nobody_wants(lib, monkeypatch):
    """Neither dx nor dweight: the arguments are looked at, nothing is launched and no memory made."""
    both = lambda **kw: lib.maxsim_cross_entropy_backward(_loss(**kw), 0x3000, _v(), _v(0x900000), 0x4000, None, None,  # noqa: E731
                                                          None, 0, None)
    assert both() == 0 and both(d=60) == UNSUPPORTED and both(targets=None) == INVALID
    assert _backward(lib, ws=None, n=0) == WORKSPACE
    cuda = fake.Cuda(monkeypatch, m)
    x, w, t, row = cuda.tensor((6, 64), BF), cuda.tensor((9, 64), BF), cuda.tensor((6,), I64), cuda.tensor((6,), F32)
    assert m.encoder_cross_entropy_backward(row, x, w, t, row, want_dx=False, want_dweight=False) == (None, None)
    assert not cuda.made


@pytest.mark.parametrize("T,V", [(1, 2 ** 31 - 300), (3, 1 << 25), (255, 1 << 26), (256, 1 << 26), (1000, 1 << 26), (1, 1000)])
def test_the_forwards_workspace_is_bounded(lib, T, V):
    """A pair of numbers for 128 columns of a row: of all rows, of 256, or of what 256 MB hold."""
    per = (V + 127) // 128 * 8
    need = lib.maxsim_cross_entropy_workspace_size(_loss(T=T, V=V))
    assert 0 < need <= max(min(T, 256) * per, min(T * per, 256 << 20)) + 4 * T + 512
