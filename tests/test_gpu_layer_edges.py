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
