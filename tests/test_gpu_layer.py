"""GPU: dropout, norm and cross entropy together, as a training step uses them:
one after another, captured into a graph, on other streams, and when a wait
runs out."""
import importlib.util
import os

import pytest
import torch

import workloads
from tests import _layer_ref as ref
from tests.test_gpu_dropout import _rng, rows
from tests.test_gpu_streams import _freed_but_pending

pytestmark = pytest.mark.gpu
m = pytest.importorskip("maxsim_scoring_02_gb300")
DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lib = m.load_library()
    yield lib
    assert lib.maxsim_debug_set_faults(0, 0) == 0


class Step:
    """x -> dropout -> h = res + dropout -> norm -> cross entropy, and back."""

    def __init__(self, T, V, d, seed=1):
        self.x, self.res = rows(T, d, seed, torch.bfloat16), rows(T, d, seed + 1, torch.bfloat16)
        self.w = 1 + 0.2 * workloads.normal((d,), seed=seed + 2, device=DEV)
        self.W = (workloads.normal((V, d), seed=seed + 3, device=DEV) * 2 / d ** 0.5).bfloat16()
        g = torch.Generator().manual_seed(seed)
        t = torch.randint(0, V, (T,), generator=g)
        t[torch.rand(T, generator=g) < 0.3] = -100
        self.t, self.dloss = t.to(DEV), torch.full((T,), 1.0 / T, device=DEV)
        self.rng = _rng(11, 3)

    def run(self, **kw):
        x1 = m.encoder_dropout(self.x, 0.2, self.rng, **kw)
        y, h = m.encoder_rms_norm(x1, self.w, residual=self.res, p=0.1, rng=self.rng, want_sum=True, **kw)
        loss, lse = m.encoder_cross_entropy(y, self.W, self.t, **kw)
        dy, dW = m.encoder_cross_entropy_backward(self.dloss, y, self.W, self.t, lse, **kw)
        dx1, dres, dw = m.encoder_rms_norm_backward(dy, h, self.w, p=0.1, rng=self.rng, **kw)
        dx = m.encoder_dropout(dx1, 0.2, self.rng, **kw)
        return x1, y, h, loss, lse, dy, dW, dx1, dres, dw, dx


def test_a_step_stage_by_stage():
    """Each stage against fp64 from what the stage before it gave."""
    s = Step(333, 1500, 264)
    x1, y, h, loss, lse, dy, dW, dx1, dres, dw, dx = s.run()
    u = 2.0 ** -8
    ref.within(x1, *ref.dropout(s.x, 0.2, s.rng))
    ref.within(h, *ref.dropout(x1, 0.1, s.rng, s.res))
    want, _ = ref.norm(h, s.w, 1e-6)
    ref.within(y, want, (u + ref.ROW) * want.abs())
    ce = ref.cross_entropy(y, s.W, s.t, 1.0, s.dloss)
    for got, name in ((loss, "loss"), (lse, "lse"), (dy, "dx"), (dW, "dw")):
        ref.within(got, ce[name], ce[name + "_tol"], name)
    back, tol, dw64, size = ref.norm_backward(dy, h, s.w, 1e-6)
    ref.within(dres, back, tol + u * back.abs())
    keep, f = ref.kept(333, 264, 0.1, s.rng, DEV)
    ref.within(dx1, torch.where(keep, back * f, 0.0), (tol + (u + 2.0 ** -23) * back.abs()) * f)
    ref.within(dw, dw64, (ref.ROW + 70 * 2.0 ** -24) * size)
    ref.within(dx, *ref.dropout(dx1, 0.2, s.rng))


def test_a_captured_step_draws_anew_and_takes_new_inputs():
    s, other = Step(200, 900, 128), Step(200, 900, 128, seed=50)
    s.run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = s.run()
        s.rng[1] += 1
    first = None
    for i in range(3):
        number = s.rng.clone()
        g.replay()
        torch.cuda.synchronize()
        live = Step(200, 900, 128) if i < 2 else other
        live.rng = number
        assert all(torch.equal(a, b) for a, b in zip(got, live.run()))
        assert s.rng[1] == number[1] + 1
        if i == 0:
            first = got[1].clone()
        elif i == 1:                                  # new inputs in the same places
            assert not torch.equal(first, got[1])
            for a, b in ((s.x, other.x), (s.res, other.res), (s.w, other.w), (s.W, other.W), (s.t, other.t)):
                a.copy_(b)
    assert m.maxsim_device_status() == (0, 0)


def test_two_graphs_with_one_workspace():
    """Two captured steps that share their workspace, replayed in turn, while calls of the same kind run between them."""
    s = [Step(150, 700 + 300 * i, 128, seed=9 * i) for i in range(2)]
    size = max(m.encoder_cross_entropy_backward_workspace_size(q.x, q.W, q.t) for q in s)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    graphs, outs = [], []
    for q in s:
        q.lse = m.encoder_cross_entropy(q.x, q.W, q.t)[1]   # what a graph reads has to live as long as it
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(m.encoder_cross_entropy_backward(q.dloss, q.x, q.W, q.t, q.lse, workspace=ws))
        graphs.append(g)
        q.want = m.encoder_cross_entropy_backward(q.dloss, q.x, q.W, q.t, q.lse)
    for i in (0, 1, 1, 0, 1, 0):
        graphs[i].replay()
        s[1 - i].run()
        assert all(torch.equal(a, b) for a, b in zip(outs[i], s[i].want))


CALLS = ["dropout", "norm", "norm_8", "norm_backward", "loss", "loss_backward"]


def _call(name):
    s = Step(300, 700, 136)
    loss, lse = m.encoder_cross_entropy(s.x, s.W, s.t)
    return {
        "dropout": lambda **kw: m.encoder_dropout(s.x, 0.3, s.rng, residual=s.res, **kw),
        "norm": lambda **kw: m.encoder_rms_norm(s.x, s.w, residual=s.res, p=0.1, rng=s.rng, want_sum=True, **kw),
        "norm_8": lambda **kw: m.encoder_rms_norm(s.x, s.w, fmt="int8", **kw),
        "norm_backward": lambda **kw: m.encoder_rms_norm_backward(s.res, s.x, s.w, p=0.1, rng=s.rng, **kw),
        "loss": lambda **kw: m.encoder_cross_entropy(s.x, s.W, s.t, **kw),
        "loss_backward": lambda **kw: m.encoder_cross_entropy_backward(s.dloss, s.x, s.W, s.t, lse, **kw),
    }[name]


@pytest.mark.parametrize("name", CALLS)
def test_pending_writes_of_the_current_stream_reach_no_call_on_another(name):
    call = _call(name)
    want = call()
    want = [t.clone() for t in (want if isinstance(want, tuple) else (want,))]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(stream=s)
    for _ in range(3):
        torch.cuda.synchronize()
        _freed_but_pending()
        got = call(stream=s)
        got = got if isinstance(got, tuple) else (got,)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert m.maxsim_device_status() == (0, 0)


def test_two_streams_at_once():
    """Steps on two streams, with nothing between them, give what each gives alone."""
    s = [Step(400, 3000, 256, seed=3), Step(250, 5000, 128, seed=7)]
    want = [q.run() for q in s]
    streams = [torch.cuda.Stream() for _ in s]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [q.run(stream=st) for q, st in zip(s, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("direction", ["forward", "backward"])
def test_waits_that_run_out_are_reported_and_the_next_call_is_right(_lib, direction):
    s = Step(300, 2000, 256)
    loss, lse = m.encoder_cross_entropy(s.x, s.W, s.t)
    if direction == "forward":
        call = lambda: m.encoder_cross_entropy(s.x, s.W, s.t)  # noqa: E731
    else:
        call = lambda: m.encoder_cross_entropy_backward(s.dloss, s.x, s.W, s.t, lse)  # noqa: E731
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    assert m.maxsim_device_status() == (0, 0)
    assert _lib.maxsim_debug_set_faults(m.DEBUG_STALL_FWD_LOADER, 50_000_000) == 0
    try:
        call()
        st, flags = m.maxsim_device_status()
        assert st == 4 and flags & m.DEVERR_TIMEOUT
    finally:
        assert _lib.maxsim_debug_set_faults(0, 0) == 0
    got = call()
    torch.cuda.synchronize()
    assert m.maxsim_device_status() == (0, 0)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("pretrain_encoder", os.path.join(ROOT, "examples", "pretrain_encoder.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_the_example_runs(example):
    losses = example.train(steps=4, n=16, longest=40, vocab=700, width=128, heads=2)
    assert len(losses) == 4 and all(l == l and abs(l) < 1e3 for l in losses)
    tokens, _, offsets = example.batch(5, 40, 700, seed=3)
    e = example.Encoder(700, 128, 2, 64, seed=1)
    number = torch.zeros((), dtype=torch.int64, device=DEV)
    rows8, scale = e.embeddings(tokens, offsets, number)
    scores = m.maxsim_score_i8(rows8[:9].contiguous(), scale[:9].contiguous(), rows8, scale, offsets)
    # unit vectors: nine tokens score at most nine, up to the codes' rounding; text 0 has tokens 0 .. of its own
    assert (scores.view(-1) <= 9.1).all()


def test_the_examples_gradient_is_the_losses(example):
    """Along each weight's gradient, with the dropout fixed: a step of s * g / |g|
    changes the loss by about s * |g| (to 25 %: the forward rounds to bf16, and
    curvature is left out). s moves no row by more than a twentieth of its length:
    most of the table's gradient is the mask token's row, and as a normed row it
    turns by s / |row|, so that a step of a part of the whole table's length (50 rows'
    worth of it) turns that one row around and says nothing of the derivative."""
    data = example.batch(48, 64, 600, seed=5)
    e = example.Encoder(600, 128, 2, 64, seed=2)
    number = torch.full((), 7, dtype=torch.int64, device=DEV)
    _, grads = e.loss(*data, number)
    for name, g in zip(e.names, grads):
        w, norm, ends = getattr(e, name), g.norm().item(), []
        of_row = lambda t: t.reshape(t.shape[0], -1).norm(dim=1)  # noqa: E731
        s = 0.05 * (of_row(w) / (of_row(g) / norm).clamp_min(1e-9)).min().item()
        for sign in (1, -1):
            setattr(e, name, w + sign * s * g / norm)
            ends.append(e.loss(*data, number, backward=False)[0].item())
        setattr(e, name, w)
        assert abs((ends[0] - ends[1]) / (2 * s * norm) - 1) <= 0.25, (name, ends, norm)
