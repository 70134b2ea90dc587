"""Host side of the operators on rows of hidden states and of the cross entropy:
calls that their contract rules out are refused before any CUDA call, and the
oracle's generator is the published one."""
import inspect

import pytest
import torch

import maxsim_scoring_02_gb300 as m
from maxsim_scoring_02_gb300 import build as mbuild
from tests import _fake_cuda as fake
from tests import _layer_ref as ref

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return m.load_library()


def _v(at=0x100000, stride=256):
    return m._Rows(at, stride)


# ------------------------------------------------------------ the generator

@pytest.mark.parametrize("counter,key,words", [
    # the authors' known answers for philox4x32-10
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))])
def test_generator_known_answers(counter, key, words):
    assert tuple(ref.philox_words(counter, key)) == words


def test_lots_are_the_generators_halves():
    seed, call, d = (5 << 40) + 77, (9 << 33) + 4, 19
    got = ref.lots(3, d, seed, call, first=100)
    for r in range(3):
        for j in range(d):
            w = ref.philox_words((j // 8, 100 + r, call & 0xffffffff, call >> 32), (seed & 0xffffffff, seed >> 32))
            assert got[r, j] == (w[j % 8 // 2] >> (16 * (j % 2))) & 0xffff


# ---------------------------------------------------------------- the C calls

def _dropout(lib, x=None, res=None, T=10, d=64, p=0.1, rng=0x2000, dt=0, out=None):
    return lib.maxsim_dropout(x or _v(), res, T, d, p, rng, dt, out or _v(0x900000), None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(d=0), dict(dt=7), dict(p=-0.1), dict(p=1.0), dict(p=0.999999), dict(p=float("nan")),
    dict(rng=None), dict(rng=0x2004), dict(x=_v(0)), dict(x=_v(0x100001)), dict(x=_v(stride=-1)), dict(out=_v(0x900000, 63)),
    dict(out=_v(0x900000, 0)), dict(res=_v(0)), dict(dt=2, x=_v(0x100002))])
def test_dropout_refusals(lib, kw):
    assert _dropout(lib, **kw) == INVALID


def test_dropout_of_nothing_and_of_too_much(lib):
    assert _dropout(lib, T=0) == 0
    assert _dropout(lib, T=2 ** 31) == UNSUPPORTED


# (out's address, its stride) beside x at 0x100000 with 10 rows of 64 bf16, 512 bytes apart
OVERLAPS = [(0x100002, 256), (0x100000, 128), (0x100000 + 126, 256), (0x100000 - 2, 256), (0x100000 + 512 - 126, 256),
            (0x100000 + 512 * 9 + 126, 64), (0x100000 - 128 * 9, 64), (0x100040, 264)]


@pytest.mark.parametrize("at,stride", OVERLAPS)
def test_results_that_overlap_an_input_otherwise_are_refused(lib, at, stride):
    bad = _v(at, stride)
    assert _dropout(lib, out=bad) == INVALID
    assert _dropout(lib, x=_v(0x900000), res=_v(), out=bad) == INVALID
    assert _norm(lib, out=bad) == INVALID
    assert _norm(lib, sum=bad) == INVALID
    assert _norm_bwd(lib, dx=bad, dy=_v()) == INVALID and _norm_bwd(lib, dres=bad, h=_v()) == INVALID


def _spec(**change):
    v = dict(T=10, d=64, dtype=0, weight_dtype=2, format=0, eps=1e-6, p=0.1, rng=0x2000, weight=0x3000)
    v.update(change)
    return m._NormSpec(*v.values())


def _norm(lib, x=None, res=None, sum=None, out=None, scale=None, **change):
    return lib.maxsim_rms_norm(_spec(**change), x or _v(), res, sum, out or _v(0x900000), scale, None)


def _norm_bwd(lib, dy=None, h=None, dsum=None, dx=None, dres=None, dw=None, ws=None, n=0, **change):
    return lib.maxsim_rms_norm_backward(_spec(**change), dy or _v(0x500000), h or _v(0x600000), dsum, dx, dres, dw, ws, n, None)


@pytest.mark.parametrize("change,status", [
    ({"T": -1}, 1), ({"d": 0}, 1), ({"dtype": 3}, 1), ({"weight_dtype": 1}, 1), ({"weight": 0x3002}, 1), ({"format": 3}, 1),
    ({"eps": 0.0}, 1), ({"eps": -1.0}, 1), ({"eps": float("nan")}, 1), ({"eps": float("inf")}, 1), ({"eps": 1e-30}, 1),
    ({"p": 1.0}, 1), ({"rng": None}, 1), ({"rng": 0x2001}, 1), ({"d": 16385}, 2), ({"T": 2 ** 31}, 2)])
def test_norm_spec_refusals(lib, change, status):
    assert _norm(lib, **change) == status and _norm_bwd(lib, **change) == status
    assert lib.maxsim_rms_norm_backward_workspace_size(_spec(**change)) == 0


def test_norm_refusals(lib):
    assert _norm(lib, T=0) == 0 and _norm_bwd(lib, T=0) == 0
    for kw in (dict(x=_v(0)), dict(x=_v(0x100001)), dict(res=_v(0)), dict(out=_v(0x900000, 32)), dict(sum=_v(0x900000)),
               dict(sum=_v(0x800000, 10)), dict(format=1), dict(format=2, scale=0x3002),
               dict(format=1, scale=0x4000, out=_v()),              # bytes over the rows they come from
               dict(format=1, scale=0x4000, out=_v(0x100000, 512))):
        assert _norm(lib, **kw) == INVALID, kw


def test_norm_backward_refusals(lib):
    need = m.load_library().maxsim_rms_norm_backward_workspace_size(_spec())
    assert need >= 10 * 64 * 4
    out = _v(0x900000)
    for ws, n in ((None, BIG), (0x1008, BIG), (0x1000, need - 1)):
        assert _norm_bwd(lib, dx=out, dw=0x7000, ws=ws, n=n) == WORKSPACE
    for kw in (dict(dx=out, dres=out), dict(dw=0x7000, weight=None), dict(dw=0x7002, ws=0x1000, n=BIG), dict(dx=_v(0x900000, 8)),
               dict(dsum=_v(0)), dict(format=1), dict(h=_v(0))):
        assert _norm_bwd(lib, **kw) == INVALID, kw


def _loss(**change):
    v = dict(T=10, V=100, d=64, dtype=0, scale=1.0, targets=0x2000)
    v.update(change)
    return m._LossSpec(*v.values())


def _forward(lib, x=None, w=None, loss=0x3000, lse=0x4000, ws=0x10000, n=BIG, **change):
    return lib.maxsim_cross_entropy(_loss(**change), x or _v(), w or _v(0x900000), loss, lse, ws, n, None)


def _backward(lib, x=None, w=None, dloss=0x3000, lse=0x4000, dx=None, dw=None, ws=0x10000, n=BIG, **change):
    return lib.maxsim_cross_entropy_backward(_loss(**change), dloss, x or _v(), w or _v(0x900000), lse, dx or _v(0x1100000),
                                             dw or _v(0x1900000), ws, n, None)


@pytest.mark.parametrize("change,status", [
    ({"T": -1}, 1), ({"V": 0}, 1), ({"d": 0}, 1), ({"dtype": 5}, 1), ({"scale": 0.0}, 1), ({"scale": -1.0}, 1),
    ({"scale": float("nan")}, 1), ({"scale": float("inf")}, 1), ({"targets": None}, 1), ({"targets": 0x2004}, 1),
    ({"dtype": 2}, 2), ({"d": 60}, 2), ({"d": 70000}, 2), ({"T": 2 ** 31}, 2), ({"V": 2 ** 31}, 2), ({"scale": 2.0 ** 61}, 2),
    ({"scale": 2.0 ** -61}, 2)])
def test_loss_spec_refusals(lib, change, status):
    assert _forward(lib, **change) == status and _backward(lib, **change) == status
    assert lib.maxsim_cross_entropy_workspace_size(_loss(**change)) == 0
    assert lib.maxsim_cross_entropy_backward_workspace_size(_loss(**change)) == 0


def test_rows_of_numbers_overlap_nothing_that_is_written(lib):
    """x at 0x100000 has 10 rows of 64 bf16, 512 bytes apart: its last byte is 0x10127F."""
    for kw in (dict(format=1, scale=0x900010), dict(format=1, scale=0x10127C), dict(format=1, scale=0x300000, res=_v(0x300000)),
               dict(format=1, scale=0x300020, sum=_v(0x300000)), dict(weight=0x900040), dict(weight=0x300000, sum=_v(0x300000))):
        assert _norm(lib, **kw) == INVALID, kw
    out = _v(0x900000)
    for kw in (dict(dx=out, weight=0x900000), dict(dres=out, weight=0x900000), dict(dx=out, dw=0x900040, ws=0x1000, n=BIG),
               dict(dres=out, dw=0x900040, ws=0x1000, n=BIG)):
        assert _norm_bwd(lib, **kw) == INVALID, kw
    for kw in (dict(loss=0x4000), dict(loss=0x4024), dict(lse=0x100000), dict(loss=0x10127C), dict(lse=0x900000), dict(loss=0x2048)):
        assert _forward(lib, **kw) == INVALID, kw
    for kw in (dict(dx=_v(0x3000)), dict(dw=_v(0x4000)), dict(dx=_v(0x4000)), dict(dw=_v(0x2000, 64))):
        assert _backward(lib, **kw) == INVALID, kw


@pytest.mark.parametrize("bad", [_v(0), _v(0x100008), _v(stride=100), _v(stride=0), _v(stride=-64), _v(stride=56)])
def test_loss_view_refusals(lib, bad):
    assert _forward(lib, x=bad) == INVALID and _forward(lib, w=bad) == INVALID
    for name in ("x", "w", "dx", "dw"):
        assert _backward(lib, **{name: bad}) == INVALID, name


def test_loss_overlaps_and_workspaces(lib):
    for kw in (dict(dx=_v()), dict(dw=_v(0x900000)), dict(dx=_v(0x100010)), dict(dx=_v(0x1900000)), dict(dloss=None),
               dict(lse=None), dict(lse=0x4001)):
        assert _backward(lib, **kw) == INVALID, kw
    for kw in (dict(loss=None), dict(lse=None), dict(loss=0x3002)):
        assert _forward(lib, **kw) == INVALID, kw
    need = lib.maxsim_cross_entropy_workspace_size(_loss())
    assert need >= 10 * 8
    for ws, n in ((None, BIG), (0x10008, BIG), (0x10000, need - 1)):
        assert _forward(lib, ws=ws, n=n) == WORKSPACE
    need = lib.maxsim_cross_entropy_backward_workspace_size(_loss())
    assert need >= 10 * 100 * 2
    for ws, n in ((None, BIG), (0x10010, BIG), (0x10000, need - 1)):
        assert _backward(lib, ws=ws, n=n) == WORKSPACE
    assert _forward(lib, T=0) == 0


def test_the_backwards_workspace_is_bounded(lib):
    """A piece of dz, whatever the vocabulary; sums of dx where it has several pieces."""
    for T, V in ((8192, 1 << 20), (100, 1 << 24), (1 << 20, 300)):
        need = lib.maxsim_cross_entropy_backward_workspace_size(_loss(T=T, V=V))
        assert need <= (256 << 20) + 4 * T * 256 + 64 * T * 64 * 4 + 4 * T + 4096


# --------------------------------------------------- what the binding makes, where

BF, F32, I64, U8 = torch.bfloat16, torch.float32, torch.int64, torch.uint8


@pytest.fixture
def cuda(monkeypatch):
    return fake.Cuda(monkeypatch, m)


def _calls(cuda, index=0):
    t = lambda shape, dtype: cuda.tensor(shape, dtype, index)  # noqa: E731
    x, h, w, rng = t((6, 64), BF), t((6, 64), BF), t((64,), F32), t((2,), I64)
    W, y, row = t((9, 64), BF), t((6,), I64), t((6,), F32)
    return {
        "dropout": (lambda **kw: m.encoder_dropout(x, 0.1, rng, residual=h, **kw), 1),
        "rms_norm": (lambda **kw: m.encoder_rms_norm(x, w, residual=h, p=0.1, rng=rng, fmt="int8", want_sum=True, **kw), 3),
        "rms_norm_backward": (lambda **kw: m.encoder_rms_norm_backward(x, h, w, p=0.1, rng=rng, **kw), 4),
        "cross_entropy": (lambda **kw: m.encoder_cross_entropy(x, W, y, **kw), 3),
        "cross_entropy_backward": (lambda **kw: m.encoder_cross_entropy_backward(row, x, W, y, row, **kw), 3),
    }


ENTRIES = ["dropout", "rms_norm", "rms_norm_backward", "cross_entropy", "cross_entropy_backward"]


@pytest.mark.parametrize("name", ENTRIES)
def test_a_call_on_another_stream_makes_its_memory_there(cuda, name):
    call, count = _calls(cuda)[name]
    other, outer = fake.Stream(0, 0x77), cuda.streams[0]
    result = call(stream=other)
    result = result if isinstance(result, tuple) else (result,)
    assert len(cuda.made) == count and all(t.pool is other for t in cuda.made)
    for t in cuda.made:
        assert (outer in t.users) == any(t is r for r in result)
    assert len(cuda.lib.calls) == 1 and 0x77 in [getattr(a, "value", a) for a in cuda.lib.calls[0][2]]
    assert cuda.streams[0] is outer


@pytest.mark.parametrize("name", ENTRIES)
def test_a_call_runs_on_its_tensors_device(cuda, name):
    call, count = _calls(cuda, 1)[name]
    call()
    assert [device for _, device, _ in cuda.lib.calls] == [1] and cuda.device == 0
    assert len(cuda.made) == count and all(t.index == 1 and t.pool is cuda.streams[1] for t in cuda.made)
    with pytest.raises(ValueError):
        call(stream=fake.Stream(0, 0x77))
    assert len(cuda.lib.calls) == 1


ROW, MAT = (6,), (6, 64)
ARGUMENTS = {
    "encoder_dropout": dict(x=(MAT, BF), rng=((2,), I64), residual=(MAT, BF), out=(MAT, BF)),
    "encoder_rms_norm": dict(x=(MAT, BF), weight=((64,), F32), residual=(MAT, BF), rng=((2,), I64),
                             out=(MAT, torch.int8), sum_out=(MAT, BF), scale=(ROW, F32)),
    "encoder_rms_norm_backward": dict(dy=(MAT, BF), h=(MAT, BF), weight=((64,), F32), dsum=(MAT, BF), rng=((2,), I64),
                                      dx=(MAT, BF), dresidual=(MAT, BF), dweight=((64,), F32), workspace=((64,), U8)),
    "encoder_cross_entropy": dict(x=(MAT, BF), weight=((9, 64), BF), targets=(ROW, I64), loss=(ROW, F32), lse=(ROW, F32),
                                  workspace=((64,), U8)),
    "encoder_cross_entropy_backward": dict(dloss=(ROW, F32), x=(MAT, BF), weight=((9, 64), BF), targets=(ROW, I64),
                                           lse=(ROW, F32), dx=(MAT, BF), dweight=((9, 64), BF), workspace=((64,), U8)),
}
OTHERS = {"encoder_dropout": {"p": 0.5}, "encoder_rms_norm": {"fmt": "int8", "p": 0.5}, "encoder_rms_norm_backward": {"p": 0.5}}


@pytest.mark.parametrize("name", ARGUMENTS)
def test_tensors_of_two_devices_or_of_other_types_and_sizes_are_refused(cuda, name):
    f, shapes, how = getattr(m, name), ARGUMENTS[name], OTHERS.get(name, {})
    every = lambda odd, index=0, shape=None, dtype=None: {  # noqa: E731
        k: cuda.tensor(shape or v[0] if k == odd else v[0], dtype or v[1] if k == odd else v[1], index if k == odd else 1)
        for k, v in shapes.items()}
    f(**every(None), **how)
    assert len(cuda.lib.calls) == 1
    for odd, (shape, dtype) in shapes.items():
        with pytest.raises(ValueError):
            f(**every(odd), **how)
        with pytest.raises(TypeError):
            f(**every(odd, 1, dtype=torch.float64), **how)
        if odd != "workspace":
            with pytest.raises(ValueError):
                f(**every(odd, 1, shape=shape[:-1] + (shape[-1] + 1,)), **how)
    assert len(cuda.lib.calls) == 1


def test_other_refusals_of_the_binding(cuda):
    x, rng = cuda.tensor(MAT, BF), cuda.tensor((2,), I64)
    with pytest.raises(ValueError):
        m.encoder_dropout(x, 0.1, None)
    with pytest.raises(ValueError):
        m.encoder_dropout(cuda.tensor((2, 3, 64), BF), 0.1, rng)
    with pytest.raises(ValueError):
        m.encoder_dropout(x.t(), 0.1, rng)
    with pytest.raises(ValueError):
        m.encoder_rms_norm(x, fmt="fp4")
    with pytest.raises(ValueError):
        m.encoder_rms_norm(x, scale=cuda.tensor(ROW, F32))
    with pytest.raises(TypeError):
        m.encoder_rms_norm(x, cuda.tensor((64,), torch.float16))
    with pytest.raises(ValueError):
        m.encoder_rms_norm_backward(x, x, dweight=cuda.tensor((64,), BF))
    with pytest.raises(TypeError):
        m.encoder_cross_entropy(cuda.tensor(MAT, F32), cuda.tensor((9, 64), F32), cuda.tensor(ROW, I64))
    assert not cuda.lib.calls


def test_every_encoder_entry_point_with_a_stream_is_covered():
    with_stream = {n[len("encoder_"):] for n in dir(m) if n.startswith("encoder_")
                   and "stream" in inspect.signature(getattr(m, n)).parameters}
    assert with_stream == set(ENTRIES)
