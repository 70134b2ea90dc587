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
