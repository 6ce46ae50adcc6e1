"""GPU parity of beam search's selection and of the caches' reordering.

Selection against the definition in 64 bits: parents and tokens equal, scores
within fp32's rounding of the result (half a step, 2^-24 relative) plus the
sum's error: each exponential has a relative error of about 2^-22 and their
sum no more, so lse is off by at most 2^-22 absolutely, 3e-7 with the
rounding of a score near 1; 1e-6 + 2^-23 |score| leaves a factor 3.  The
random inputs' neighbouring candidates are checked to lie further apart than
twice that.  Reordering: equal bytes."""
import numpy as np
import pytest

from gpu_util import device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return device()


def _select(dev, logits, scores, n_out, finished=None, eos=0, pad=0, offset=0):
    """logits [G][B][V] and the rest as numpy; pad: floats between rows, offset: floats before the first"""
    import torch

    from weight_streaming_gemv_gb300 import qlin

    G, B, V = logits.shape
    buf = torch.full((offset + G * B * (V + pad),), float("nan"), device=dev)
    x = buf[offset:].view(G * B, V + pad)
    x[:, :V] = torch.from_numpy(np.ascontiguousarray(logits, np.float32)).view(G * B, V).to(dev)
    sc = torch.from_numpy(np.ascontiguousarray(scores, np.float32)).to(dev)
    fin = None if finished is None else torch.from_numpy(np.ascontiguousarray(finished, np.uint8)).to(dev)
    out = torch.empty((G, n_out), device=dev)
    par, tok = (torch.empty((G, n_out), dtype=torch.int32, device=dev) for _ in range(2))
    nb = qlin.qlin_beam_select_workspace_size(G, B, V, n_out)
    ws = torch.randint(0, 255, (nb,), dtype=torch.uint8, device=dev)
    qlin.qlin_beam_select(x, V + pad, sc, fin, eos, G, B, V, n_out, out, par, tok, ws, nb)
    torch.cuda.synchronize()
    return out.cpu().numpy(), par.cpu().numpy(), tok.cpu().numpy()


def _ref(logits, scores, n_out, finished=None, eos=0):
    G, B, V = logits.shape
    S = np.full((G, n_out), -np.inf)
    P, T = np.full((G, n_out), -1), np.full((G, n_out), -1)
    gap = np.inf
    for g in range(G):
        c = np.full((B, V), -np.inf)
        for b in range(B):
            base = float(scores[g, b])
            if finished is not None and finished[g, b]:
                c[b, eos] = base
            elif base > -np.inf:
                x = logits[g, b].astype(np.float64)
                if np.isnan(x).any() or (x == np.inf).any() or (x == -np.inf).all():
                    continue
                m = x.max()
                with np.errstate(over="ignore", under="ignore"):
                    c[b] = base + ((x - m) - np.log(np.exp(x - m).sum()))
        flat = c.reshape(-1)
        order = np.argsort(-flat, kind="stable")[: n_out + 1]
        order = order[flat[order] > -np.inf]
        d = -np.diff(flat[order])
        d = d[d > 0]
        gap = min(gap, d.min()) if d.size else gap
        order = order[:n_out]
        S[g, : order.size], P[g, : order.size], T[g, : order.size] = flat[order], order // V, order % V
    return S, P, T, gap


def _check(dev, logits, scores, n_out, finished=None, eos=0, need_gap=True, **kw):
    s, p, t = _select(dev, logits, scores, n_out, finished, eos, **kw)
    S, P, T, gap = _ref(logits, scores, n_out, finished, eos)
    if need_gap:
        assert gap > 2e-8, "two candidates too close to be told apart: another seed"
    np.testing.assert_array_equal(p, P)
    np.testing.assert_array_equal(t, T)
    fin = np.isfinite(S)
    np.testing.assert_array_equal(np.isfinite(s), fin)
    assert (s[~fin] == -np.inf).all()
    assert (np.abs(s[fin] - S[fin]) <= 1e-6 + np.abs(S[fin]) * 2.0 ** -23).all()


@pytest.mark.parametrize("G,B,V,n", [(1, 1, 1, 1), (1, 1, 1, 4), (1, 2, 3, 5), (2, 4, 512, 4), (1, 3, 1023, 6),
                                     (3, 5, 1025, 10), (1, 4, 262144, 4), (2, 8, 100003, 16), (1, 64, 5000, 128),
                                     (7, 1, 32000, 2), (40, 3, 777, 6), (1, 64, 40001, 64), (1, 1, 200, 128)])
def test_sizes(dev, G, B, V, n):
    rng = np.random.default_rng(V + B)
    _check(dev, rng.normal(0, 3, (G, B, V)).astype(np.float32), -rng.random((G, B)).astype(np.float32) * 8, n)


@pytest.mark.parametrize("pad,offset", [(0, 0), (1, 0), (4, 0), (3, 2), (0, 1)])
def test_strides_and_alignment(dev, pad, offset):
    rng = np.random.default_rng(5)
    _check(dev, rng.normal(0, 3, (2, 3, 4100)).astype(np.float32), -rng.random((2, 3)).astype(np.float32), 6, pad=pad,
           offset=offset)


def test_first_step_dead_and_finished_beams(dev):
    rng = np.random.default_rng(6)
    x = rng.normal(0, 3, (3, 4, 3000)).astype(np.float32)
    x[1] = x[1, 0]  # the beams are still one
    s = -rng.random((3, 4)).astype(np.float32)
    s[1] = [0, -np.inf, -np.inf, -np.inf]
    fin = np.zeros((3, 4), np.uint8)
    fin[0, 2], fin[2] = 1, 255
    s[0, 2] = -0.01
    _check(dev, x, s, 8, fin, 17)
    # every beam dead; a finished beam with a score of minus infinity
    s[:] = -np.inf
    _check(dev, x, s, 8, fin, 2999)


def test_words_that_are_not_allowed(dev):
    rng = np.random.default_rng(7)
    x = rng.normal(0, 3, (2, 3, 2500)).astype(np.float32)
    x[:, :, 40:] = -np.inf
    x[0, 1] = -np.inf           # a beam with no word left
    x[1, 2, 3:] = -np.inf       # a beam with three
    s = -rng.random((2, 3)).astype(np.float32)
    _check(dev, x, s, 100)
    x[x == -np.inf] = np.finfo(np.float32).min  # masks of the type's lowest value
    x[0, 1] = -1.0
    x[0, 1, 5:9] = np.finfo(np.float32).min
    _check(dev, x, s, 20, need_gap=False)


def test_beam_of_lowest_values_only(dev):
    x = np.full((1, 2, 1000), np.finfo(np.float32).min, np.float32)
    x[0, 1] = 3e38
    s = np.float32([[-1.0, -2.0]])
    out, par, tok = _select(dev, x, s, 5)
    # every word of a beam is equally likely: the first beam's first words
    np.testing.assert_array_equal(par, [[0] * 5])
    np.testing.assert_array_equal(tok, [[0, 1, 2, 3, 4]])
    np.testing.assert_allclose(out, np.full((1, 5), -1 - np.log(1000)), rtol=1e-6)


def test_logarithm_of_every_count(dev):
    # Group g: g + 1 equally likely words against a finished beam whose score is fp32's nearest to their offer.  The
    # sum is exact, so which comes first tells the logarithm's error.  Its series leaves out less than 1e-11; behind w
    # (|w| <= 1/5, kept in two floats) the rest, at most 2 w^3 / 3 (1 + ...) < 6e-3, is rounded some six times at
    # 2^-24 each: 2.2e-9.
    G = 1500
    x = np.full((G, 2, G), -np.inf, np.float32)
    for g in range(G):
        x[g, 0, : g + 1] = 0
    lse = np.log(np.arange(1, G + 1, dtype=np.float64))
    score = (-lse).astype(np.float32)
    s = np.zeros((G, 2), np.float32)
    s[:, 1] = score
    fin = np.zeros((G, 2), np.uint8)
    fin[:, 1] = 1
    out, par, tok = _select(dev, x, s, 1, fin, 7)
    gap = score.astype(np.float64) + lse
    sure = np.abs(gap) > 3e-9
    assert sure.mean() > 0.8
    np.testing.assert_array_equal(par[sure, 0], gap[sure] > 0)
    assert par[0, 0] == 0  # a tie
    np.testing.assert_allclose(out[:, 0], score, rtol=2.0 ** -23)


@pytest.mark.parametrize("levels", [1, 2])
def test_sums_of_equal_logits(dev, levels):
    # So many rows that each is one slice, of equal words (or of two levels, 4 apart): every term rounds the same way.
    # An offer is score - log V (with two levels log(V / 2 (1 + e^-4)) for the upper half's words).  Its error: 8 roundings
    # of a tile's sum, the exponential's 2^-22, an argument's 2^-24 of at most 6, and the result's own, 2^-24 of 12:
    # 2^-21 + 2^-22 + 2^-21.4 + 2^-20.4 = 1.8e-6.
    import torch

    from weight_streaming_gemv_gb300 import qlin

    G, V = 460, 100000
    x = torch.linspace(-3, 3, G, device=dev)[:, None].repeat(1, V)
    if levels == 2:
        x[:, 1::2] -= 4
    sc, out = torch.zeros((G, 1), device=dev), torch.empty((G, 2), device=dev)
    par, tok = (torch.empty((G, 2), dtype=torch.int32, device=dev) for _ in range(2))
    nb = qlin.qlin_beam_select_workspace_size(G, 1, V, 2)
    ws = torch.empty(nb, dtype=torch.uint8, device=dev)
    qlin.qlin_beam_select(x, V, sc, None, 0, G, 1, V, 2, out, par, tok, ws, nb)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(par.cpu().numpy(), np.zeros((G, 2)))
    np.testing.assert_array_equal(tok.cpu().numpy(), np.tile([0, levels], (G, 1)))
    d = x.double()
    want = -(torch.log(torch.exp(d - d[:, :1]).sum(1))).cpu().numpy()
    assert np.abs(out.cpu().numpy() - want[:, None]).max() <= 1.8e-6


def test_large_scores_and_logits(dev):
    rng = np.random.default_rng(12)
    # a beam's score swallows its words' differences: the words in the order of their logits
    x = rng.normal(0, 3, (1, 3, 5000)).astype(np.float32)
    for big in (np.float32(3e34), np.float32(np.inf)):
        s, p, t = _select(dev, x, np.float32([[-1, big, -2]]), 6)
        assert (p == 1).all() and (s == big).all()
        np.testing.assert_array_equal(t[0], np.argsort(-x[0, 1], kind="stable")[:6])
    # logits beyond 2^24: the sum is taken relative to the largest
    x = (3e7 + 2 * np.stack([rng.permutation(4000) for _ in range(2)])).astype(np.float32)[None]
    x[0, 1] -= 2e7
    _check(dev, x, np.float32([[-0.5, -1.25]]), 9)
    x[0, 0] = -x[0, 0]
    _check(dev, x, np.float32([[-0.5, -1.25]]), 9)


def test_logits_beyond_the_scales_range(dev):
    # Finite logits of any size: behind 2^24 the sum is taken relative to the largest, and a whole-number scale has no
    # room for them from 7e7 on.  The beams' scores make the large one win.
    rng = np.random.default_rng(13)
    V = 40000  # (several slices)
    s = np.float32([[-0.5, -1.25]])
    small = rng.normal(0, 3, V).astype(np.float32)
    for big, step in ((7e7, 8), (1e8, 8), (-1e8, 8), (-7e7, 8), (2e12, 131072)):  # (steps are fp32's there)
        x = np.stack([(big + step * rng.permutation(V)).astype(np.float32), small])[None]
        _check(dev, x, s, 9)
    for big in (6.9e7, 7e7, 1e8, 3e38, np.finfo(np.float32).max, np.finfo(np.float32).min):
        x = np.stack([np.full(V, big, np.float32), small])[None]
        _check(dev, x, s, 20, need_gap=False)        # all of its words are equal
        x[0, 0] = small
        x[0, 0, [7, 11, 30000]] = big                # in slices of ordinary ones, and beside slices without
        _check(dev, x, s, 6, need_gap=False)
        for bad in (np.nan, np.inf):                 # in the slice of the large ones, and in another
            for at in (8, 39000):
                y = x.copy()
                y[0, 0, at] = bad
                _check(dev, y, s, 6, need_gap=False)


def test_nan_and_infinity(dev):
    rng = np.random.default_rng(8)
    x = rng.normal(0, 3, (1, 4, 9000)).astype(np.float32)
    x[0, 1, 8500], x[0, 2, 3] = np.nan, np.inf
    _check(dev, x, np.float32([[-9, 0, 0, -8]]), 8)
    s, p, t = _select(dev, x, np.float32([[np.nan, 0, 0, -np.inf]]), 3)
    assert (p == -1).all() and (t == -1).all() and (s == -np.inf).all()


@pytest.mark.parametrize("V", [300, 5000, 70000])
def test_ties_go_to_the_lowest_beam_then_word(dev, V):
    x = np.zeros((1, 3, V), np.float32)
    _check(dev, x, np.zeros((1, 3), np.float32), 128, need_gap=False)          # everything equal
    x[0, 1, V // 2:] = 1.0
    x[0, 2] = x[0, 1]                                                          # two equal beams
    _check(dev, x, np.zeros((1, 3), np.float32), 70, need_gap=False)
    x = np.round(np.random.default_rng(9).normal(0, 1, (2, 2, V))).astype(np.float32)  # many equal values
    _check(dev, x, np.float32([[0, -1], [-1, -1]]), 100, need_gap=False)


def test_zeros_of_either_sign_are_equal(dev):
    x = np.full((1, 2, 4000), -1, np.float32)
    x[:, :, 100:1900:3] = 0.0
    x[:, :, 101:1900:3] = -0.0
    _check(dev, x, np.zeros((1, 2), np.float32), 12, need_gap=False)
    _check(dev, x, np.float32([[0, -1]]), 128, need_gap=False)


def test_sorted_logits(dev):
    x = np.linspace(-5, 5, 60000, dtype=np.float32)[None, None]
    _check(dev, np.concatenate([x, x[:, :, ::-1]], 1), np.float32([[0, -1e-3]]), 64)


def test_select_captured(dev):
    import torch

    from weight_streaming_gemv_gb300 import qlin

    G, B, V, n = 2, 4, 20000, 8
    rng = np.random.default_rng(10)
    x = torch.empty((G * B, V), device=dev)
    sc, out = torch.zeros((G, B), device=dev), torch.empty((G, n), device=dev)
    par, tok = (torch.empty((G, n), dtype=torch.int32, device=dev) for _ in range(2))
    nb = qlin.qlin_beam_select_workspace_size(G, B, V, n)
    ws = torch.empty(nb, dtype=torch.uint8, device=dev)
    call = lambda: qlin.qlin_beam_select(x, V, sc, None, 0, G, B, V, n, out, par, tok, ws, nb)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        h, s = rng.normal(0, 3, (G, B, V)).astype(np.float32), -rng.random((G, B)).astype(np.float32)
        x.copy_(torch.from_numpy(h).view(G * B, V))
        sc.copy_(torch.from_numpy(s))
        graph.replay()
        torch.cuda.synchronize()
        S, P, T, _ = _ref(h, s, n)
        np.testing.assert_array_equal(par.cpu().numpy(), P)
        np.testing.assert_array_equal(tok.cpu().numpy(), T)


# ------------------------------------------------------------------ reordering
def _reorder(dev, x, parents, rows=None, plane_major=False):
    import torch

    from weight_streaming_gemv_gb300 import qlin

    par = torch.as_tensor(np.ascontiguousarray(parents, np.int32)).to(dev)
    G, B = par.shape
    r = None if rows is None else torch.as_tensor(np.ascontiguousarray(rows, np.int32)).to(dev)
    e = x.element_size()
    sd, pd = (1, 0) if plane_major else (0, 1)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    qlin.qlin_beam_reorder(x, x.stride(sd) * e, x.stride(pd) * e, x.shape[pd], x.stride(2) * e, x.shape[2], par, r, G, B,
                           st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0


def _expect(x, parents, rows, plane_major):
    y = x.copy()
    G, B = np.shape(parents)
    for g in range(G):
        n = x.shape[2] if rows is None else min(max(rows[g], 0), x.shape[2])
        for b in range(B):
            p = parents[g][b]
            if 0 <= p < B:
                a, c = g * B + b, g * B + p
                if plane_major:
                    y[:, a, :n] = x[:, c, :n]
                else:
                    y[a, :, :n] = x[c, :, :n]
    return y


def _parents(rng, G, B):
    p = rng.integers(0, B, (G, B))
    p[rng.random((G, B)) < 0.2] = -1
    return p


@pytest.mark.parametrize("plane_major", [False, True])
@pytest.mark.parametrize("G,B,planes,R,row", [(1, 2, 1, 1, 4), (1, 4, 52, 40, 256), (3, 5, 6, 17, 36), (2, 64, 3, 9, 64),
                                              (5, 16, 2, 300, 128), (1, 3, 2, 5000, 64), (200, 2, 1, 1, 4),
                                              (1, 1, 4, 4, 16)])
def test_reorder(dev, G, B, planes, R, row, plane_major):
    import torch

    rng = np.random.default_rng(B)
    shape = (planes, G * B, R, row) if plane_major else (G * B, planes, R, row)
    x = rng.normal(size=shape).astype(np.float32)
    rows = rng.integers(-1, R + 2, G)
    rows[0] = R
    for par, rw in ((_parents(rng, G, B), rows), (np.stack([rng.permutation(B) for _ in range(G)]), None),
                    (np.zeros((G, B), int), rows), (np.tile(np.arange(B), (G, 1)), None),
                    (np.full((G, B), 2147483647), None)):
        t = torch.from_numpy(x).to(dev)
        _reorder(dev, t, par, rw, plane_major)
        np.testing.assert_array_equal(t.cpu().numpy(), _expect(x, par, rw, plane_major))


def test_reorder_rotates_in_place_and_replays(dev):
    # a rotation of every beam, captured and replayed: after B replays everything is back
    import torch

    from weight_streaming_gemv_gb300 import qlin

    B = 12
    x = torch.randn((B, 4, 1000, 64), device=dev)
    first = x.clone()
    par = torch.as_tensor(np.int32([(b + 5) % B for b in range(B)])).to(dev)
    n = torch.as_tensor(np.int32([900])).to(dev)
    call = lambda: qlin.qlin_beam_reorder(x, x.stride(0) * 4, x.stride(1) * 4, 4, 256, 1000, par, n, 1, B)
    call()
    torch.cuda.synchronize()
    assert torch.equal(x[:, :, :900], first[par.long(), :, :900]) and torch.equal(x[:, :, 900:], first[:, :, 900:])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(B - 1):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(x, first)


def test_reorder_past_32_bits(dev):
    # beams 3 GB apart, rows of a plane that is longer than 2^31 bytes
    import torch

    from weight_streaming_gemv_gb300 import qlin

    x = torch.empty((3, 3 << 27, 8), dtype=torch.bfloat16, device=dev)  # 3 beams of one plane of 6 GB
    for b in range(3):
        x[b, :5], x[b, -5:] = b + 1, b + 11
    par = torch.as_tensor(np.int32([2, 0, 0])).to(dev)
    st = x.stride(0) * 2
    qlin.qlin_beam_reorder(x, st, st, 1, 16, x.shape[1], par, None, 1, 3)
    torch.cuda.synchronize()
    assert [float(x[b, 0, 0]) for b in range(3)] == [3, 1, 1]
    assert [float(x[b, -1, 7]) for b in range(3)] == [13, 11, 11]
