"""Sampling against the definition in 64 bits: tokens and numbers of words left exactly, shares to fp32.

Tolerance.  A weight is good to 2^-29 of itself (an error of its own for every logit) and rounded to a multiple of q = 2^-44
of the largest (a larger power of two above 2^18 words).  Both are of either sign: the errors of a sum are at most some
2^-30 sqrt(sum w^2) and 0.29 q sqrt(V) in deviations, so eight of both are 2^-27 sqrt(sum w^2) + 2.4 q sqrt(V).  A row in
which a decision lies nearer than that to its border says nothing about the others and is not compared: at most one in a
hundred, which is asserted.  A share is a float's weight over such a sum: good to two roundings, 2^-23 of itself."""
import numpy as np
import pytest

import sample_ref as ref
from gpu_util import device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return device()


def _run(dev, x, u, t=None, k=None, p=None, m=None, stride=None, offset=0, want_all=True, stream=None):
    import torch

    from weight_streaming_gemv_gb300 import qlin

    R, V = x.shape
    stride = V if stride is None else stride
    buf = torch.full((R * stride + offset + 8,), float("nan"), device=dev)
    rows = buf[offset: offset + R * stride].view(R, stride)
    rows[:, :V] = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dev)
    up = lambda a, d: None if a is None else torch.from_numpy(np.ascontiguousarray(np.broadcast_to(a, R), d)).to(dev)
    tok = torch.full((R + 1,), 77, dtype=torch.int32, device=dev)
    probs = torch.full((R + 1,), 7.5, device=dev) if want_all else None
    kept = torch.full((R + 1,), 77, dtype=torch.int32, device=dev) if want_all else None
    qlin.qlin_sample(rows, stride, up(u, np.float32), up(t, np.float32), up(k, np.int32), up(p, np.float32),
                     up(m, np.float32), R, V, tok, probs, kept, stream)
    torch.cuda.synchronize()
    assert tok[R] == 77
    if not want_all:
        return tok.cpu().numpy()[:R], None, None
    assert probs[R] == 7.5 and kept[R] == 77
    return tok.cpu().numpy()[:R], probs.cpu().numpy()[:R], kept.cpu().numpy()[:R]


def _compare(x, u, t, k, p, m, got, most=0.01):
    R = len(x)
    at = lambda a, i, d: d if a is None else np.broadcast_to(a, R)[i].item()
    tok, probs, kept = got
    V = x.shape[1]
    skipped, rounding = 0, 2.4 * V ** 0.5 * 2.0 ** (max(18, (V - 1).bit_length()) - 62)
    for i in range(R):
        f32 = lambda v: float(np.float32(v))
        w = ref.draw(np.float32(x[i]), f32(np.broadcast_to(u, R)[i]), f32(at(t, i, 1.0)), int(at(k, i, 0)),
                     f32(at(p, i, 1.0)), f32(at(m, i, 0.0)))
        if 1e-15 < w[3] < 2.0 ** -27 * w[4] + rounding:  # (a border met exactly is no accident: equal weights)
            skipped += 1
            continue
        assert (int(tok[i]), int(kept[i])) == (w[0], w[2]), (i, (tok[i], kept[i]), w)
        assert abs(float(probs[i]) - w[1]) <= 2.0 ** -23 * w[1], (i, probs[i], w)
    assert skipped <= max(1, most * R), f"{skipped} of {R} rows too near a border"


SETTINGS = {
    "free": dict(),
    "cold": dict(t=0.3),
    "hot": dict(t=3.0),
    "greedy": dict(t=0.0),
    "k1": dict(t=0.8, k=1),
    "k50": dict(t=0.8, k=50),
    "k5000": dict(t=1.1, k=5000),
    "k_most": dict(t=1.0, k=10 ** 9),
    "p": dict(p=0.9),
    "p_small": dict(p=1e-6),
    "p_none": dict(p=0.0),
    "p_most": dict(t=1.2, p=0.9999),
    "m": dict(m=0.05),
    "m_all": dict(m=1.0),
    "k_p": dict(t=0.8, k=64, p=0.95),
    "k_p_wide": dict(t=1.5, k=4000, p=0.7),
    "all": dict(t=0.9, k=300, p=0.9, m=0.02),
    "all_wide": dict(t=1.3, k=9000, p=0.97, m=0.0005),
    "p_m": dict(t=1.0, p=0.95, m=0.001),
}


@pytest.mark.parametrize("name", list(SETTINGS))
@pytest.mark.parametrize("V", [1, 2, 5, 100, 513, 2048, 16385, 32000, 70001, 262144])
def test_settings(dev, name, V):
    rng = np.random.default_rng(V)
    R = 24 if V < 100000 else 8
    x = rng.standard_normal((R, V)) * 3
    if V > 5:
        x[:, 3] = -np.inf
        x[1] *= 3  # a row with a clear favourite
        x[2, V // 2:] = -np.inf
    s = SETTINGS[name]
    a = [s.get(n) for n in ("t", "k", "p", "m")]
    u = rng.random(R)
    _compare(x, u, *a, _run(dev, x, u, *a))


def test_rows_of_their_own_settings(dev):
    rng = np.random.default_rng(7)
    R, V = 300, 20011
    x = rng.standard_normal((R, V)) * rng.choice([0.5, 2, 4, 10], (R, 1))
    t = rng.choice([0.0, 0.1, 0.7, 1.0, 2.5], R)
    k = rng.choice([0, 1, 2, 40, 1000, 1535, 1536, 1537, 15000, V - 1, V, -3], R)
    p = rng.choice([1.0, 0.01, 0.5, 0.9, 0.99, 2.0], R)
    m = rng.choice([0.0, 0.0, 0.001, 0.2, 5.0], R)
    u = rng.random(R)
    _compare(x, u, t, k, p, m, _run(dev, x, u, t, k, p, m))


@pytest.mark.parametrize("V", [2100, 60000])
def test_lists_of_any_length(dev, V):
    """words left by top-k about the numbers at which a list, and a sort of it, is full"""
    rng = np.random.default_rng(V)
    k = np.array([127, 128, 129, 900, 1023, 1024, 1025, 1500, 1990, 2030, 2047, 2048, 2049, 2060, 2099, 2100, 3000] * 2)
    R = len(k)
    x, u = rng.standard_normal((R, V)) * rng.choice([1.0, 3.0], (R, 1)), rng.random(R)
    p, m = rng.choice([1.0, 0.9, 0.99], R), rng.choice([0.0, 0.0, 1e-3], R)
    t = rng.choice([0.8, 1.5], R)
    _compare(x, u, t, k, p, m, _run(dev, x, u, t, k, p, m))


@pytest.mark.parametrize("V", [500, 30000, 262144])
def test_min_p_next_to_top_p(dev, V):
    """min-p's border well before top-p's, well behind it, and next to it"""
    rng = np.random.default_rng(V)
    R = 60 if V < 100000 else 16
    x, u = rng.standard_normal((R, V)) * 3, rng.random(R)
    t, p = rng.uniform(0.5, 2.0, R), rng.uniform(0.3, 1.0, R)
    m = np.exp(rng.uniform(np.log(1e-6), 0.0, R))
    for i in range(0, R, 3):  # as much as the last word that top-p keeps weighs, and a little more or less
        w = np.sort(np.exp((np.float32(x[i]).astype(np.float64) - np.float32(x[i]).max()) / np.float32(t[i])))[::-1]
        at = min(V - 1, int(np.searchsorted(np.cumsum(w), np.float32(p[i]) * w.sum())))
        m[i] = w[at] * rng.choice([1.0 - 1e-3, 1.0 - 1e-6, 1.0 + 1e-6, 1.0 + 1e-3, 1.02, 0.98])
    _compare(x, u, t, None, p, m, _run(dev, x, u, t, None, p, m), most=0.05)


def test_min_p_just_behind_top_p(dev):
    """min-p's border one word or a few behind top-p's, where 6000 equal words are half of the sum: what a histogram says of
    their weight is off by as much for each"""
    rng = np.random.default_rng(11)
    R, V, n = 36, 131072, 6000
    for _ in range(8):
        x = -np.log(rng.uniform(np.exp(6.0), np.exp(10.0), (R, V)))  # as much weight in every part of the range
        x[:, :n] = np.log(np.exp(x[:, n:]).sum(1, keepdims=True) / n) + rng.uniform(0.0, 0.05, (R, 1))
        x[:, n] = x[:, 0] + rng.uniform(0.2, 0.4, R)
        x = x[:, rng.permutation(V)]
        u, p, m = rng.random(R), rng.uniform(0.53, 0.7, R), np.zeros(R)
        for i in range(R):
            w = np.sort(np.exp(np.float32(x[i]).astype(np.float64) - np.float32(x[i]).max()))[::-1]
            m[i] = w[int(np.searchsorted(np.cumsum(w), np.float32(p[i]) * w.sum())) + 1 + i % 3]
        _compare(x, u, None, None, p, m, _run(dev, x, u, None, None, p, m), most=0.03)


@pytest.mark.parametrize("V", [7, 3000, 50000, 262144])
@pytest.mark.parametrize("levels", [1, 2, 5])
def test_equal_logits(dev, V, levels):
    """few different logits, every cut inside many equal words; at one level the weights are 1 and every border is met"""
    rng = np.random.default_rng(levels)
    R = 10
    x = rng.integers(0, levels, (R, V)).astype(np.float64) * 0.75 - 1.0
    x[:, -1] = 0.75 * (levels - 1) - 1.0
    u = np.array([0.0, 0.25, 0.5, 0.999, rng.random(), rng.random(), rng.random(), rng.random(), 0.75, 0.125])
    k = np.array([0, 0, 1, V // 2, max(1, V - 1), V // 3 + 1, 0, 5, 2, 0])
    p = np.array([1.0, 0.5, 0.25, 1.0, 1.0, 0.75, 0.125, 0.5, 1.0, 0.9])
    _compare(x, u, None, k, p, None, _run(dev, x, u, None, k, p, None), most=0.3)


def test_zeros_of_either_sign_are_equal(dev):
    x = np.full((2, 4000), -0.0)
    x[0, ::2] = 0.0
    x[:, 0] = -5.0
    u = np.array([0.0, 0.999])
    got = _run(dev, x, u, 1.0, 3)
    assert got[0].tolist() == [1, 3] and got[2].tolist() == [3, 3]


@pytest.mark.parametrize("V", [60, 9000])
def test_close_logits(dev, V):
    """logits that differ in their last bits, of every size: bins that hold many words, cuts among neighbours"""
    rng = np.random.default_rng(V)
    R = 40
    base = np.float32(10.0) ** rng.integers(-30, 30, (R, 1)).astype(np.float32) * np.float32(1.2345)
    x = (base.view(np.int32) + rng.integers(0, 3000, (R, V))).astype(np.int32).view(np.float32).astype(np.float64)
    x *= rng.choice([-1, 1], (R, 1))
    u, k = rng.random(R), rng.integers(1, V, R)
    k[::3] = 0
    p = rng.choice([1.0, 0.4, 0.8], R)
    t = np.where(rng.random(R) < 0.5, 1.0, np.abs(x).max(1) / 1e4 + 1e-30)
    _compare(x, u, t, k, p, None, _run(dev, x, u, t, k, p, None), most=0.2)


def test_low_values_count_as_they_are(dev):
    """a mask of the type's lowest value instead of minus infinity: words that are left, but weigh nothing"""
    rng = np.random.default_rng(3)
    V = 30000
    x = np.full((6, V), np.finfo(np.float32).min, np.float64)
    x[:, rng.permutation(V)[:40]] = rng.standard_normal(40) * 2
    u = rng.random(6)
    k, p = np.array([0, 10, 100, 5000, 0, 100]), np.array([1.0, 1.0, 1.0, 1.0, 0.9, 0.9])
    _compare(x, u, 0.7, k, p, None, _run(dev, x, u, 0.7, k, p, None))


@pytest.mark.parametrize("V", [7, 3000, 50000])
@pytest.mark.parametrize("k,p,m", [(None, None, None), (4, None, None), (2500, 0.7, None), (None, 0.8, None), (None, 0.9, 0.3),
                                   (None, None, 1.0)])
def test_logits_and_temperatures_next_to_the_types_range(dev, V, k, p, m):
    """logits whose differences fp32 does not hold, and temperatures as large: their weights are those of the definition"""
    rng = np.random.default_rng(V)
    big = float(np.finfo(np.float32).max)
    t = np.array([1e38, 3e38, 2e37, 1e38, big, 1e30, 1.0, 1e-20, 3e31, 1e38, 1e33, np.inf])
    R = len(t)
    x = rng.uniform(-1, 1, (R, V)) * big
    x[3] = rng.choice([-big, big], V)
    x[3, 1] = big
    x[5] = 1e31 * rng.standard_normal(V) + 3e38  # beside one another, far from 0
    x[7] = np.float32(2e30) + 1e24 * rng.integers(0, 1 << 20, V)
    x[8] = 1e31 * rng.standard_normal(V)
    x[9] = -1e-40  # the largest's share of the temperature is nothing
    x[9, ::2] = -big
    x[10] = 5.0 * rng.standard_normal(V)
    u = rng.random(R)
    got = _run(dev, x, u, t, k, p, m)
    if m == 1.0:
        # at a finite temperature only the words of the largest logit weigh 1: exp(-1e-33), below it, is 1 in 64 bits, so
        # that the definition's cut has to be made by the logits here (row 10)
        f = np.float32(x)
        x = np.where(np.isfinite(t)[:, None] & (f < f.max(1, keepdims=True)), -np.inf, x)
        m = None
    _compare(x, u, t, k, p, m, got, most=0.2)


def test_temperatures(dev):
    rng = np.random.default_rng(9)
    t = np.array([1e-45, 1e-38, 1e-6, 0.01, 1e3, 1e30, np.inf, np.nan, -1.0, -0.0, 3e38, 1e-3])
    x = rng.standard_normal((len(t), 5000)) * 3
    u = rng.random(len(t))
    for k, p, m in ((None, None, None), (37, None, None), (None, 0.6, None), (3000, 0.5, 0.2)):
        _compare(x, u, t, k, p, m, _run(dev, x, u, t, k, p, m))


@pytest.mark.parametrize("V", [3, 3000, 70001, 262144])
@pytest.mark.parametrize("k,m", [(None, None), (40, None), (2500, None), (None, 0.3), (40, 0.01), (None, float("nan"))])
def test_top_p_of_zero_and_less(dev, V, k, m):
    """a top_p of 0 or less leaves the first word alone, whatever stands beside it; a NaN is no bound"""
    rng = np.random.default_rng(V)
    p = np.array([-1.0, -np.inf, -1e-30, -0.0, 0.0, -3e38, np.nan, np.nan, -1.0, 0.9])
    R = len(p)
    x, u = rng.standard_normal((R, V)) * 3, rng.random(R)
    x[8] = 1.5  # all alike
    got = _run(dev, x, u, 0.8, k, p, m)
    for i in (0, 1, 2, 3, 4, 5, 8):
        assert (got[0][i], got[1][i], got[2][i]) == (np.float32(x[i]).argmax(), 1.0, 1), i
    _compare(x, u, 0.8, k, p, m, got, most=0.1)


def test_rows_that_hold_no_answer(dev):
    x = np.random.default_rng(1).standard_normal((6, 40000))
    x[0, 39999] = np.nan
    x[1, 0] = np.inf
    x[2] = -np.inf
    x[3, 5] = np.nan
    x[4, :] = -np.inf
    x[4, 31234] = -3e38
    for t in (None, 0.0):
        tok, probs, kept = _run(dev, x, 0.5, t)
        assert tok[:5].tolist() == [-1, -1, -1, -1, 31234] and probs[:5].tolist() == [0, 0, 0, 0, 1]
        assert kept[:5].tolist() == [0, 0, 0, 0, 1] and tok[5] >= 0


def test_u_at_the_ends(dev):
    x = np.zeros((5, 6))
    x[:, 5] = -200.0  # weighs nothing
    x[:, 0] = -np.inf
    tok, probs, kept = _run(dev, x, np.array([0.0, 1.0, 2.0, -1.0, np.nan]))
    assert tok.tolist() == [1, 4, 4, 1, 1] and (probs == 0.25).all() and (kept == 5).all()


@pytest.mark.parametrize("V,stride,offset", [(1000, 1001, 0), (1000, 1004, 4), (999, 1000, 1), (33001, 33003, 3), (262143, 262144, 0)])
def test_strides_and_alignment(dev, V, stride, offset):
    rng = np.random.default_rng(stride)
    R = 5
    x, u = rng.standard_normal((R, V)) * 3, rng.random(R)
    for k, p in ((None, None), (20, 0.9), (None, 0.8)):
        _compare(x, u, 0.9, k, p, None, _run(dev, x, u, 0.9, k, p, None, stride=stride, offset=offset))


@pytest.mark.parametrize("V", [900001, 1 << 21])
def test_large_vocabularies(dev, V):
    """more words than the shared memory of a cluster holds, and fewer bits to a weight"""
    rng = np.random.default_rng(V)
    x, u = rng.standard_normal((4, V)) * 3, rng.random(4)
    x[3] = np.round(x[3])
    for t, k, p in ((1.0, None, None), (0.7, 100, 0.9), (1.0, None, 0.9), (1.5, 700000, 0.99)):
        _compare(x, u, t, k, p, None, _run(dev, x, u, t, k, p, None), most=0.5)


def test_many_rows_and_no_outputs(dev):
    rng = np.random.default_rng(2)
    x, u = rng.standard_normal((2000, 130)), rng.random(2000)
    full = _run(dev, x, u, 0.9, 20, 0.9)
    _compare(x, u, 0.9, 20, 0.9, None, full)
    tok, _, _ = _run(dev, x, u, 0.9, 20, 0.9, want_all=False)
    assert np.array_equal(tok, full[0])


def test_frequencies(dev):
    """what is drawn follows the weights: 40000 draws from eight words, every count within five deviations"""
    n, w = 40000, np.array([1, 2, 3, 4, 5, 6, 7, 12]) / 40
    x = np.tile(np.log(w), (n, 1))
    tok, _, _ = _run(dev, x, np.random.default_rng(0).random(n))
    c = np.bincount(tok, minlength=8)
    assert (np.abs(c - n * w) <= 5 * np.sqrt(n * w * (1 - w))).all(), c


def test_graph_and_streams(dev):
    """captured and replayed with other inputs; two calls at once on two streams"""
    import torch

    from weight_streaming_gemv_gb300 import qlin

    rng = np.random.default_rng(4)
    R, V = 6, 50000
    xs = [rng.standard_normal((R, V)).astype(np.float32) * 3 for _ in range(3)]
    us = [rng.random(R).astype(np.float32) for _ in range(3)]
    want = [_run(dev, x, u, None, None, 0.9)[0] for x, u in zip(xs, us)]
    up = lambda a: torch.from_numpy(a).to(dev)
    p = torch.full((R,), 0.9, device=dev)
    x, u, tok = up(xs[0]).clone(), up(us[0]).clone(), torch.zeros(R, dtype=torch.int32, device=dev)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qlin.qlin_sample(x, V, u, None, None, p, None, R, V, tok)
    for i in (1, 2, 0):
        x.copy_(up(xs[i])), u.copy_(up(us[i]))
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(tok.cpu().numpy(), want[i])
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    dx, du = [up(v) for v in xs], [up(v) for v in us]
    toks = [torch.zeros(R, dtype=torch.int32, device=dev) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, i in ((a, 0), (b, 1)):
            qlin.qlin_sample(dx[i], V, du[i], None, None, p, None, R, V, toks[i], stream=s)
    torch.cuda.synchronize()
    assert all(np.array_equal(toks[i].cpu().numpy(), want[i]) for i in (0, 1))
