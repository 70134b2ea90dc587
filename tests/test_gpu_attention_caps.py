"""GPU: capped scores of every size against the fp64 plain form, within the
bounds of tests/_encoder_ref.py.

Those are for inputs N(0,1), whose scores are off by 1.4e-4 at most; a query
`times` as large makes scores off by `times` as much, and FP with them. A capped
score adds 2^-22 of its cap (caps up to 128: 3e-5) or 2^-20 of itself."""
import pytest
import torch

import workloads
from tests import _encoder_ref as ref

pytestmark = pytest.mark.gpu
m = pytest.importorskip("maxsim_scoring_02_gb300")
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.load_library()


@pytest.fixture
def run(monkeypatch):
    def call(lengths, H, G, d, dtype, seed, times=1.0, slopes=False, key_len=None, prefix_len=None, **how):
        monkeypatch.setattr(ref, "FP", 4e-4 * max(1.0, times))
        T = sum(lengths)
        x = workloads.normal((T, H + 2 * G, d), seed=seed, device=DEV)
        x[:, :H] *= times
        x = x.to(DT[dtype])
        dO = workloads.normal((T, H, d), seed=seed + 1, device=DEV).to(DT[dtype])
        q, k, v = x[:, :H], x[:, H:H + G], x[:, H + G:]
        off = workloads.csr_offsets(torch.tensor(lengths, dtype=torch.int64)).to(DEV)
        if slopes:
            how["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device=DEV)
        if key_len is not None:
            how["key_len"] = torch.tensor(key_len, dtype=torch.int32, device=DEV)
        if prefix_len is not None:
            how["prefix_len"] = torch.tensor(prefix_len, dtype=torch.int32, device=DEV)
        out, lse = m.maxsim_attention(q, k, v, off, want_lse=True, **how)
        got = dict(zip(("dq", "dk", "dv"), m.maxsim_attention_backward(dO, q, k, v, out, lse, off, **how)), out=out)
        torch.cuda.synchronize()
        assert m.maxsim_device_status() == (0, 0)
        r = ref.attention(q, k, v, lengths, dO=dO, **how)
        for name, t in got.items():
            ref.check(t, r, name)
        some = ~torch.isinf(r["lse"])
        assert torch.equal(torch.isinf(lse), ~some)
        assert ((lse.double() - r["lse"])[some].abs() <= ref.FP / 2 + 2.0 ** -21 * r["lse"][some].abs()).all()
    return call


@pytest.mark.parametrize("cap", [300.0, 1e4, 1e6])
@pytest.mark.parametrize("d", [64, 128])
def test_wide_caps_leave_small_scores_alone(run, cap, d):
    run([140, 3, 290], 2, 2, d, "bf16", 1, cap=cap)
    run([1030], 2, 1, d, "fp16", 3, cap=cap, mask="causal")
    run([300, 1, 77, 513], 2, 1, d, "bf16", 5, cap=cap, slopes=True, key_len=[250, 0, 77, 513])


@pytest.mark.parametrize("d", [64, 128])
def test_wide_caps_that_scores_reach(run, d):
    """Scores of 0.3 caps on average: most tiles hold small ones and bent ones."""
    run([140, 3, 290], 2, 2, d, "bf16", 7, times=60.0, cap=200.0)
    run([500], 2, 1, d, "fp16", 9, times=60.0, cap=200.0, mask="causal", slopes=True)


@pytest.mark.parametrize("cap", [2.0 ** 60, 2.0 ** -60])
def test_the_widest_and_the_narrowest_cap(run, cap):
    """Scores as they are, and scores that are all but equal."""
    run([140, 3, 290], 2, 2, 64, "bf16", 11, cap=cap)
    run([300], 2, 1, 128, "bf16", 13, cap=cap, mask="causal")


# Documents of 192 tokens and more on average run two tiles of rows a block at
# d = 128; a group of 32 x 32 scores that all lie within 0.7 caps takes the
# polynomial in the backward, which N(0,1) scores do at a cap of 30 and hardly
# ever at 2.5.
SHAPES = {"one tile": [140, 3, 290], "two tiles": [300, 1, 77, 513], "long": [1030]}
MASKS = ["full", "causal", "prefix"]


def _mask(lengths, mask):
    if mask != "prefix":
        return {"mask": mask}
    return {"mask": mask, "prefix_len": [(5 * n + 3) // 7 + (i % 2) * 200 for i, n in enumerate(lengths)]}


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("d", [64, 128])
def test_usual_caps_and_small_scores(run, d, shape, mask):
    n = SHAPES[shape]
    run(n, 2, 2, d, "bf16", 15, cap=30.0, **_mask(n, mask))
    run(n, 2, 1, d, "fp16", 17, cap=30.0, **_mask(n, mask))


@pytest.mark.parametrize("cap", [30.0, 10.0, 2.5])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("d", [64, 128])
def test_caps_that_scores_reach(run, d, shape, cap):
    """Queries four times as large: few scores beyond 0.7 caps, many, nearly all."""
    run(SHAPES[shape], 2, 1, d, "bf16", 19, times=4.0, cap=cap)
    run(SHAPES[shape], 2, 2, d, "fp16", 21, times=4.0, cap=cap, mask="causal")


@pytest.mark.parametrize("cap", [0.0, 2.5, 30.0])
@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("d", [64, 128])
def test_caps_with_a_distance_bias(run, d, shape, mask, cap):
    n = SHAPES[shape]
    run(n, 4, 2, d, "bf16", 23, cap=cap, slopes=True, **_mask(n, mask))
    hidden = [max(0, x - 40) if i % 2 else x for i, x in enumerate(n)]
    run(n, 2, 2, d, "fp16", 25, cap=cap, slopes=True, key_len=hidden, **_mask(n, mask))
