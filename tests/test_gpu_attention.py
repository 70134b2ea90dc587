"""GPU: packed attention, forward and backward, against the fp64 plain form
within the bounds derived in tests/_encoder_ref.py."""
import math

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


def _offsets(lengths):
    return workloads.csr_offsets(torch.tensor(lengths, dtype=torch.int64)).to(DEV)


def _inputs(T, H, G, d, dtype, seed):
    """q, k, v as views of one projection output, and dO."""
    x = workloads.normal((T, H + 2 * G, d), seed=seed, device=DEV).to(DT[dtype])
    dO = workloads.normal((T, H, d), seed=seed + 1, device=DEV).to(DT[dtype])
    return x[:, :H], x[:, H:H + G], x[:, H + G:], dO


def _run(lengths, H, G, d, dtype, seed=1, key_len=None, prefix_len=None, slopes=False, backward=True, **how):
    T = sum(lengths)
    q, k, v, dO = _inputs(T, H, G, d, dtype, seed)
    off = _offsets(lengths)
    kw = dict(how)
    if key_len is not None:
        kw["key_len"] = torch.tensor(key_len, dtype=torch.int32, device=DEV)
    if prefix_len is not None:
        kw["prefix_len"] = torch.tensor(prefix_len, dtype=torch.int32, device=DEV)
    if slopes:
        kw["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device=DEV)
    out, lse = m.maxsim_attention(q, k, v, off, want_lse=True, **kw)
    r = ref.attention(q, k, v, lengths, dO=dO if backward else None, **kw)
    got = {"out": out}
    if backward:
        got["dq"], got["dk"], got["dv"] = m.maxsim_attention_backward(dO, q, k, v, out, lse, off, **kw)
    torch.cuda.synchronize()
    assert m.maxsim_device_status() == (0, 0)
    for name, x in got.items():
        ref.check(x, r, name)
    empty = torch.isinf(r["lse"])
    assert torch.equal(torch.isinf(lse), empty) and (lse[empty] < 0).all()
    # an lse is off by its scores' error at most (half of FP), and its own roundings
    assert ((lse.double() - r["lse"])[~empty].abs() <= ref.FP / 2 + 2.0 ** -21 * r["lse"][~empty].abs()).all()
    assert torch.equal(m.maxsim_attention(q, k, v, off, **kw), out)  # the same without lse, and again
    return got


LENGTHS = {
    "one token": [1],
    "tiny": [1, 2, 3, 0, 5, 8, 1, 0, 0, 17],
    "tile edges": [127, 128, 129, 0, 64, 65, 63],
    "ragged": [300, 1, 77, 513],
    "long": [2051],
    "many short": [(7 * i) % 53 for i in range(90)],
}


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_full_mask(lengths, d, dtype):
    _run(LENGTHS[lengths], 2, 2, d, dtype, seed=10)


@pytest.mark.parametrize("d", [8, 16, 40, 72, 96, 120])
def test_head_sizes(d):
    _run([130, 5, 64], 3, 3, d, "bf16", seed=20)
    _run([130, 5, 64], 3, 3, d, "fp16", seed=21, mask="causal")


@pytest.mark.parametrize("heads,kv_heads", [(8, 1), (6, 2), (12, 4), (5, 5)])
@pytest.mark.parametrize("d", [64, 128])
def test_shared_heads(heads, kv_heads, d):
    _run([200, 33, 150], heads, kv_heads, d, "bf16", seed=30)


@pytest.mark.parametrize("mask", ["full", "causal", "prefix"])
@pytest.mark.parametrize("lengths", ["tiny", "tile edges", "ragged", "long"])
def test_masks_and_hidden_keys(mask, lengths):
    n = LENGTHS[lengths]
    kw = {}
    if mask == "prefix":
        kw["prefix_len"] = [(5 * x + 3) // 7 + (i % 2) * 200 for i, x in enumerate(n)]
    _run(n, 2, 1, 64, "bf16", seed=40, mask=mask, **kw)
    hidden = [0 if i % 3 == 1 else x // 2 if i % 3 == 2 else max(0, x - 1) for i, x in enumerate(n)]
    _run(n, 2, 2, 128, "bf16", seed=41, mask=mask, key_len=hidden, **kw)


@pytest.mark.parametrize("mask", ["full", "causal"])
@pytest.mark.parametrize("d", [64, 128])
def test_cap_and_distance_bias(mask, d):
    n = [140, 3, 290]
    _run(n, 2, 2, d, "bf16", seed=50, mask=mask, cap=2.5)
    _run(n, 4, 2, d, "fp16", seed=51, mask=mask, slopes=True)
    _run(n, 2, 1, d, "bf16", seed=52, mask=mask, cap=1.0, slopes=True, scale=0.3, key_len=[100, 0, 290])


def test_rows_that_see_nothing_are_zero():
    n = [70, 128, 200]
    got = _run(n, 2, 2, 64, "bf16", seed=60, key_len=[0, 128, 0])
    for name in ("out", "dq", "dk", "dv"):
        assert (got[name][:70] == 0).all() and (got[name][198:] == 0).all(), name


@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
@pytest.mark.parametrize("d", [64, 128])
def test_hidden_values_never_reach_a_row(poison, d):
    """Hidden keys and values of one document, and every value of another, are
    not numbers: the rest is as if they were."""
    n, hide = [90, 150, 40, 300], [60, 150, 40, 170]
    q, k, v, dO = _inputs(sum(n), 2, 2, d, "bf16", 70)
    off, kl = _offsets(n), torch.tensor(hide, dtype=torch.int32, device=DEV)
    out, lse = m.maxsim_attention(q, k, v, off, key_len=kl, want_lse=True)
    grads = m.maxsim_attention_backward(dO, q, k, v, out, lse, off, key_len=kl)
    k2, v2, q2, dO2 = k.clone(), v.clone(), q.clone(), dO.clone()
    for t in (k2, v2):
        t[60:90] = poison
        t[280 + 170:] = poison
    for t in (k2, v2, q2, dO2):
        t[240:280] = poison
    out2, lse2 = m.maxsim_attention(q2, k2, v2, off, key_len=kl, want_lse=True)
    grads2 = m.maxsim_attention_backward(dO2, q2, k2, v2, out2, lse2, off, key_len=kl)
    rows = torch.ones(sum(n), dtype=torch.bool, device=DEV)
    rows[240:280] = False
    assert torch.equal(out2[rows], out[rows]) and torch.equal(lse2[:, rows], lse[:, rows])
    for a, b in zip(grads2, grads):
        assert torch.equal(a[rows], b[rows])


def test_large_scores_stay_finite():
    """Scores of thousands: the softmax is a selection, nothing overflows."""
    n = [200]
    q, k, v, dO = _inputs(200, 1, 1, 64, "bf16", 80)
    off = _offsets(n)
    q, k = q * 30, k * 30
    out, lse = m.maxsim_attention(q, k, v, off, want_lse=True)
    grads = m.maxsim_attention_backward(dO, q, k, v, out, lse, off)
    for t in (out, lse, *grads):
        assert torch.isfinite(t).all()
    r = ref.attention(q, k, v, n)
    # scores of up to 5e4 are off by 900 times what N(0,1) inputs allow: 0.13 of a weight
    assert ((out.double() - r["out"]).abs() <= r["out_tol"] + 0.26 * v.double().abs().max()).all()
    assert ((lse.double() - r["lse"]).abs() <= 0.13 + 2.0 ** -21 * r["lse"].abs()).all()


def test_gradients_against_differences():
    """<grad, x> in random directions against central differences of the fp64
    forward; the gradient may be off by its bound in every element."""
    n, H, G, d = [37, 5, 20], 2, 1, 16
    q, k, v, dO = _inputs(sum(n), H, G, d, "bf16", 90)
    off = _offsets(n)
    kw = dict(mask="causal", cap=3.0, slopes=torch.tensor([0.1, 0.02], device=DEV))
    out, lse = m.maxsim_attention(q, k, v, off, want_lse=True, **kw)
    grads = m.maxsim_attention_backward(dO, q, k, v, out, lse, off, **kw)
    r = ref.attention(q, k, v, n, dO=dO, **kw)

    def loss(a, b, c):
        total = 0.0
        s = 0
        for x in n:
            for h in range(H):
                z, _, i, j = ref.scores(a[s:s + x, h], b[s:s + x, 0], 1 / math.sqrt(d), 3.0, kw["slopes"][h].double(), x)
                p = torch.softmax(torch.where(j <= i, z, -math.inf), 1)
                total = total + (p @ c[s:s + x, 0] * dO[s:s + x, h].double()).sum()
            s += x
        return total.item()

    base = [t.double() for t in (q, k, v)]
    for which, name in enumerate(("dq", "dk", "dv")):
        for seed in range(3):
            w = workloads.normal(base[which].shape, seed=200 + seed, device=DEV).double()
            h = 1e-5
            up, dn = list(base), list(base)
            up[which], dn[which] = base[which] + h * w, base[which] - h * w
            slope = (loss(*up) - loss(*dn)) / (2 * h)
            mine = (grads[which].double() * w).sum().item()
            assert abs(mine - slope) <= (r[name + "_tol"] * w.abs()).sum().item() + 1e-6 * abs(slope), name


def test_gradients_land_in_views_of_one_buffer():
    n, H, G, d = [150, 31], 4, 2, 64
    q, k, v, dO = _inputs(181, H, G, d, "bf16", 95)
    off = _offsets(n)
    out, lse = m.maxsim_attention(q, k, v, off, want_lse=True)
    dq, dk, dv = m.maxsim_attention_backward(dO, q, k, v, out, lse, off)
    buf = torch.full((181, H + 2 * G + 1, d), 7.0, dtype=torch.bfloat16, device=DEV)
    m.maxsim_attention_backward(dO, q, k, v, out, lse, off, dq=buf[:, :H], dk=buf[:, H:H + G],
                                dv=buf[:, H + G:H + 2 * G])
    assert torch.equal(buf[:, :H], dq) and torch.equal(buf[:, H:H + G], dk) and torch.equal(buf[:, H + G:-1], dv)
    assert (buf[:, -1] == 7).all()


def test_offsets_beyond_32_bits():
    """Tokens 2^22 elements apart: the last ones lie beyond 2^32 elements."""
    n, H, d, stride = [1000, 90], 2, 64, 1 << 22
    T = sum(n)
    q, k, v, dO = _inputs(T, H, H, d, "bf16", 97)
    buf = torch.empty(T * stride, dtype=torch.bfloat16, device=DEV)
    views = [torch.as_strided(buf, (T, H, d), (stride, d, 1), i * H * d) for i in range(8)]
    for t, w in zip((q, k, v, dO), views):
        w.copy_(t)
    off = _offsets(n)
    out, lse = m.maxsim_attention(q, k, v, off, want_lse=True)
    out2, lse2 = m.maxsim_attention(*views[:3], off, out=views[4], want_lse=True)
    assert torch.equal(out2, out) and torch.equal(lse2, lse)
    a = m.maxsim_attention_backward(dO, q, k, v, out, lse, off)
    b = m.maxsim_attention_backward(views[3], *views[:3], out2, lse2, off, dq=views[5], dk=views[6], dv=views[7])
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_another_stream_and_repeats():
    n = [500, 20]
    q, k, v, dO = _inputs(520, 4, 2, 128, "bf16", 98)
    off = _offsets(n)
    out, lse = m.maxsim_attention(q, k, v, off, want_lse=True)
    grads = m.maxsim_attention_backward(dO, q, k, v, out, lse, off)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(3):
            o2, l2 = m.maxsim_attention(q, k, v, off, want_lse=True)
            g2 = m.maxsim_attention_backward(dO, q, k, v, o2, l2, off)
    s.synchronize()
    assert torch.equal(o2, out) and torch.equal(l2, lse) and all(torch.equal(a, b) for a, b in zip(g2, grads))
    torch.cuda.synchronize()
    o3, l3 = m.maxsim_attention(q, k, v, off, want_lse=True, stream=s)      # the stream as an argument
    g3 = m.maxsim_attention_backward(dO, q, k, v, o3, l3, off, stream=s)
    junk = torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV)       # may not be the workspace's memory
    s.synchronize()
    assert torch.equal(o3, out) and all(torch.equal(a, b) for a, b in zip(g3, grads)) and (junk == 255).all()


@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("d", [64, 128])
def test_what_ran_before_changes_no_bit(cap, d):
    """Scores whose maximum grows along the keys, documents that end inside a tile:
    neither what other calls leave on the chip nor their order shows in a result."""
    for n in ([300, 1, 77, 513], [40, 17, 90, 9, 33, 64, 21] * 6):
        q, k, v, dO = _inputs(sum(n), 3, 3, d, "bf16", 103)
        q = q * 6
        off = _offsets(n)

        def run():
            out, lse = m.maxsim_attention(q, k, v, off, cap=cap, want_lse=True)
            return (out, lse) + tuple(m.maxsim_attention_backward(dO, q, k, v, out, lse, off, cap=cap))

        first = run()
        for seed in range(4):
            a, b, c, e = _inputs(2000, 4, 4, 128, "bf16", 200 + seed)
            o, l = m.maxsim_attention(a * 30, b, c, _offsets([2000]), want_lse=True)
            m.maxsim_attention_backward(e, a * 30, b, c, o, l, _offsets([2000]))
            assert all(torch.equal(x, y) for x, y in zip(run(), first))


def test_capture_in_a_graph():
    n = [128, 60]
    q, k, v, _ = _inputs(188, 2, 2, 64, "fp16", 99)
    off = _offsets(n)
    want = m.maxsim_attention(q, k, v, off)
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.maxsim_attention(q, k, v, off, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_inconsistent_documents_are_reported_and_skipped():
    q, k, v, dO = _inputs(100, 1, 1, 64, "bf16", 100)
    good = m.maxsim_attention(q[:40], k[:40], v[:40], _offsets([40]))
    for off in ([0, 40, 30, 100], [0, 40, 101], [0, 40, -5, 100]):
        out = m.maxsim_attention(q, k, v, torch.tensor(off, dtype=torch.int64, device=DEV))
        st, flags = m.maxsim_device_status()
        assert st == 1 and flags & m.DEVERR_BAD_INPUT
        assert torch.equal(out[:40], good)
    m.maxsim_attention(q, k, v, _offsets([40, 60]), key_len=torch.tensor([41, 60], dtype=torch.int32, device=DEV))
    assert m.maxsim_device_status()[0] == 1
    assert m.maxsim_device_status() == (0, 0)


@pytest.mark.parametrize("d,n", [(64, [60, 20, 33]), (64, [400]), (128, [60, 20, 33]), (128, [400])])
def test_waits_that_run_out_are_reported(d, n):
    """The loaders bring nothing (a test-only switch): every wait gives up after
    its bound, the call reports it, and the next one is as if nothing had been."""
    lib = m.load_library()
    q, k, v, dO = _inputs(sum(n), 2, 1, d, "bf16", 104)
    off = _offsets(n)
    out, lse = m.maxsim_attention(q, k, v, off, want_lse=True)
    grads = m.maxsim_attention_backward(dO, q, k, v, out, lse, off)
    torch.cuda.synchronize()
    assert lib.maxsim_debug_set_faults(1, 50_000_000) == 0
    try:
        m.maxsim_attention(q, k, v, off)
        forward = m.maxsim_device_status()
        m.maxsim_attention_backward(dO, q, k, v, out, lse, off)
        backward = m.maxsim_device_status()
    finally:
        assert lib.maxsim_debug_set_faults(0, 0) == 0
    assert forward[0] == backward[0] == 4
    o2, l2 = m.maxsim_attention(q, k, v, off, want_lse=True)
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    assert all(torch.equal(a, b) for a, b in zip(m.maxsim_attention_backward(dO, q, k, v, out, lse, off), grads))
    assert m.maxsim_device_status() == (0, 0)


def test_nothing_to_do():
    q, k, v, dO = _inputs(0, 2, 2, 64, "bf16", 101)
    out, lse = m.maxsim_attention(q, k, v, _offsets([0, 0]), want_lse=True)
    assert out.shape == (0, 2, 64) and lse.shape == (2, 0)
    assert [tuple(t.shape) for t in m.maxsim_attention_backward(dO, q, k, v, out, lse, _offsets([0, 0]))] == [(0, 2, 64)] * 3


def test_refusals():
    q, k, v, dO = _inputs(64, 4, 2, 64, "bf16", 102)
    off = _offsets([64])
    with pytest.raises(TypeError):
        m.maxsim_attention(q, k.half(), v, off)
    with pytest.raises(ValueError):
        m.maxsim_attention(q, k, v[:, :1], off)
    with pytest.raises(ValueError):
        m.maxsim_attention(q, k, v, off, mask="window")
    with pytest.raises(ValueError):
        m.maxsim_attention(q, k, v, off, mask="prefix")
    with pytest.raises(ValueError):
        m.maxsim_attention(q.cpu(), k, v, off)
    with pytest.raises(TypeError):
        m.maxsim_attention(q, k, v, off.int())
    with pytest.raises(m.MaxSimError) as e:     # fp32 has no kernel
        m.maxsim_attention(q.float(), k.float(), v.float(), off)
    assert e.value.status == 2
    with pytest.raises(m.MaxSimError) as e:     # heads not a multiple of kv_heads
        m.maxsim_attention(q[:, :3], k, v, off)
    assert e.value.status == 1
    with pytest.raises(m.MaxSimError) as e:     # a view that starts off a 16-byte boundary
        m.maxsim_attention(q[..., 4:60], k[..., 8:], v[..., 8:], off)
    assert e.value.status in (1, 2)
    with pytest.raises(m.MaxSimError) as e:
        m.maxsim_attention(q, k, v, off, scale=0.0)
    assert e.value.status == 1
    out, lse = m.maxsim_attention(q, k, v, off, want_lse=True)
    with pytest.raises(m.MaxSimError) as e:
        m.maxsim_attention_backward(dO, q, k, v, out, lse, off,
                                    workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == 5
