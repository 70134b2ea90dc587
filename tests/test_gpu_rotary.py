"""GPU: rotary positions against the fp64 definition.

The angle is off by at most 2^-24 * pi (its fp32 value of up to half a turn)
plus sincospif's own 2 ulp, the two products and their sum by 2^-23 each, so
|y - ref| <= u |ref| + 1.2e-6 * amplitude * (|x1| + |x2|)."""
import pytest
import torch

import workloads
from tests import _encoder_ref as ref

pytestmark = pytest.mark.gpu
m = pytest.importorskip("maxsim_scoring_02_gb300")
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.load_library()


def _check(y, x, angles, amplitude, rot, **how):
    r = ref.rotary(x, angles, amplitude, rot, **how)
    size = ref.rotary(x.abs(), torch.full_like(angles, 0.25 * torch.pi), amplitude * 2 ** 0.5, rot, **dict(how, inverse=False))
    mirrored = ref.rotary(x.abs(), torch.full_like(angles, 0.25 * torch.pi), amplitude * 2 ** 0.5, rot, **dict(how, inverse=True))
    around = torch.maximum(size, mirrored)  # amplitude * (|x1| + |x2|) in both places of a pair
    tol = ref.U[x.dtype] * r.abs() + 1.2e-6 * around
    assert ((y.double() - r).abs() <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (128, 64), (96, 48), (40, 36), (10, 6), (2, 2), (256, 32)])
def test_packed_documents(dtype, interleaved, d, rot):
    lengths = [1, 0, 33, 128, 5, 0, 200]
    off = workloads.csr_offsets(torch.tensor(lengths)).to(DEV)
    pos = torch.cat([torch.arange(n) for n in lengths]).to(DEV)
    x = workloads.normal((len(pos), 5, d), seed=d + rot, device=DEV).to(DT[dtype])
    freq, amp = m.maxsim_rotary_frequencies(rot)
    angles, _ = ref.rotary_angles(pos, rot)
    for inverse in (False, True):
        y = m.maxsim_rotary(x, freq, offsets=off, interleaved=interleaved, inverse=inverse)
        _check(y, x, angles, amp, rot, interleaved=interleaved, inverse=inverse)
        assert torch.equal(y[..., rot:], x[..., rot:])
        z = x.clone()
        assert m.maxsim_rotary(z, freq, offsets=off, interleaved=interleaved, inverse=inverse, out=z) is z
        assert torch.equal(z, y)
    assert m.maxsim_device_status() == (0, 0)


@pytest.mark.parametrize("scaling,factor,original", [("none", 1.0, 0), ("linear", 4.0, 0), ("ntk", 8.0, 0),
                                                     ("yarn", 16.0, 8192), ("yarn", 1.0, 100)])
def test_long_positions(scaling, factor, original):
    pos = torch.tensor([0, 1, 4095, 8191, 100_003, 1_048_575, 16_777_217, 2_000_000_011, 7], dtype=torch.int32, device=DEV)
    x = workloads.normal((9, 3, 128), seed=3, device=DEV)
    freq, amp = m.maxsim_rotary_frequencies(128, scaling=scaling, factor=factor, original_length=original)
    angles, amplitude = ref.rotary_angles(pos, 128, scaling=scaling, factor=factor, original_length=original)
    assert abs(amp - amplitude) <= 1e-7 * amplitude
    # fp64 angles of 2e9 rad are themselves off by 2e-7, the table by 2^-53 of a turn per position
    y = m.maxsim_rotary(x, freq, positions=pos, amplitude=amp)
    _check(y, x, angles, amp, 128)


def test_views_and_token_index():
    """Query and key heads rotated together in a fused projection, in place; and
    addresses that are not multiples of 16 bytes."""
    buf = workloads.normal((77, 9, 64), seed=5, device=DEV).to(torch.bfloat16)
    freq, amp = m.maxsim_rotary_frequencies(64)
    angles, _ = ref.rotary_angles(torch.arange(77, device=DEV), 64)
    before = buf.clone()
    heads = buf[:, :6]
    assert m.maxsim_rotary(heads, freq, out=heads) is heads
    _check(buf[:, :6], before[:, :6], angles, amp, 64)
    assert torch.equal(buf[:, 6:], before[:, 6:])
    odd = workloads.normal((77 * 3 * 65 + 1,), seed=6, device=DEV).to(torch.bfloat16)[1:].view(77, 3, 65)[..., :64]
    _check(m.maxsim_rotary(odd, freq), odd, angles, amp, 64)


def test_bad_offsets_are_reported():
    x = workloads.normal((10, 1, 64), seed=7, device=DEV)
    freq, _ = m.maxsim_rotary_frequencies(64)
    m.maxsim_rotary(x, freq, offsets=torch.tensor([0, 4, 8], device=DEV))   # two tokens outside
    assert m.maxsim_device_status()[0] == 1


def test_refusals():
    x = workloads.normal((10, 2, 64), seed=8, device=DEV)
    freq, _ = m.maxsim_rotary_frequencies(64)
    big, _ = m.maxsim_rotary_frequencies(66)
    with pytest.raises(TypeError):
        m.maxsim_rotary(x.double(), freq)
    with pytest.raises(TypeError):
        m.maxsim_rotary(x, freq.float())
    with pytest.raises(ValueError):
        m.maxsim_rotary(x.cpu(), freq)
    with pytest.raises(ValueError):
        m.maxsim_rotary(x.transpose(1, 2), freq)
    with pytest.raises(ValueError):
        m.maxsim_rotary(x, freq, positions=torch.zeros(9, dtype=torch.int32, device=DEV))
    with pytest.raises(m.MaxSimError):
        m.maxsim_rotary(x, big)
    with pytest.raises(m.MaxSimError):
        m.maxsim_rotary(x, freq, offsets=torch.tensor([0, 10], device=DEV),
                        positions=torch.zeros(10, dtype=torch.int32, device=DEV))
    assert m.maxsim_rotary(x[:0], freq).shape == (0, 2, 64)
