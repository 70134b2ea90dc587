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
