"""The attention over lanes on the tensor cores, for work that is mostly too
little for it: the caches have more rows than the kernel for little work takes,
or the lanes are given over and over, and each test asks the library which way
its calls go.

References and the tolerance of random inputs are those of test_gpu_many; a
test with other inputs derives its own."""
import numpy as np
import pytest

from gpu_util import device
from test_gpu_many import Call, _close, _i32, _ref

pytestmark = pytest.mark.gpu

ROWS = {"f32": 33000, "bf16": 66000}  # of a sequence: more than 1024 blocks of 32 or 64 keys


@pytest.fixture(scope="module")
def dev():
    return device()


class Long:
    """caches [n_seqs][2][ROWS][kv_dim], the first `used` rows random, the others NaN"""

    def __init__(self, dev, kind, n_seqs, used, n_kv, hd, seed=0):
        import torch

        from weight_streaming_gemv_gb300 import qlin

        g = torch.Generator(device=dev).manual_seed(seed)
        self.t = torch.full((n_seqs, 2, ROWS[kind], n_kv * hd), float("nan"), device=dev,
                            dtype=torch.float32 if kind == "f32" else torch.bfloat16)
        self.t[:, :, :used] = torch.randn((n_seqs, 2, used, n_kv * hd), generator=g, device=dev).to(self.t.dtype)
        self.n_kv, self.hd, self.used = n_kv, hd, used
        self.k, self.v = self.t[:, 0], self.t[:, 1]
        self.c = qlin.kv_cache(self.k, self.v)

    def host(self, s):
        f = lambda x: x[s, : self.used].float().cpu().numpy().reshape(self.used, self.n_kv, self.hd)
        return f(self.k), f(self.v)


def _goes(kv, n, H, n_kv, hd, window=0, sinks=0, prefix=None):
    from weight_streaming_gemv_gb300 import qlin

    return qlin.qlin_attention_on_tensor_cores(prefix and prefix.c, kv.c, n, H, n_kv, hd, window, sinks)


def _on_tensor_cores(c, kv, window=0, sinks=0, prefix=None):
    assert _goes(kv, c.n, c.H, c.n_kv, c.hd, window, sinks, prefix)


def _often(dev, kv, n, H, n_kv, hd, window, sinks):
    """A call of n lanes as often as it takes (without a window once: the caches' rows are too many)."""
    times = next(t for t in range(1, 4096 // n + 1) if _goes(kv, n * t, H, n_kv, hd, window, sinks))
    c = Call(dev, n * times, H, n_kv, hd)
    c.q.copy_(c.q[:n].repeat(times, 1, 1))
    return c, lambda x: np.tile(x, (times,) + (1,) * (np.ndim(x) - 1))


# rows of a tile: 1 (one warpgroup), 24 (two), 48 or 32 (all), several tiles, several lanes to a tile
HEADS = [(1, 1, 64), (24, 1, 64), (48, 1, 128), (4, 1, 256), (6, 2, 80), (96, 2, 16), (10, 1, 240), (5, 1, 48)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("H,n_kv,hd", HEADS)
@pytest.mark.parametrize("window,sinks", [(100, 3), (700, 130), (0, 0)])
def test_unseen_rows_never_reach_the_outputs(dev, kind, H, n_kv, hd, window, sinks):
    # one token, a token that sees few rows, a chunk, lanes of one sequence far apart (a tile whose rows share little),
    # a long stretch, all of it behind rows that no lane sees or only some do
    used = 1500
    pos = [170, 20] + list(range(900, 940)) + [100, 1300, 150, 1200] + [1400]
    seqs = [0, 1] + [2] * 40 + [3] * 4 + [4]
    clean = Long(dev, kind, 5, used, n_kv, hd, 3)
    host = [clean.host(s) for s in range(5)]
    c, often = _often(dev, clean, len(pos), H, n_kv, hd, window, sinks)
    q = c.q.cpu().numpy()
    want = np.stack([_ref(q[i], *host[s], p, window, sinks, n_kv) for i, (p, s) in enumerate(zip(pos, seqs))])
    sees = lambda s, j: any(t == s and j <= p and (j > p - (window or used) or j < sinks) for p, t in zip(pos, seqs))
    hidden = [[j for j in range(used) if not sees(s, j)] for s in range(5)]
    assert all(len(h) > 50 for h in hidden)
    for bad in (float("nan"), float("inf"), -float("inf"), 3.3e38):
        kv = Long(dev, kind, 5, used, n_kv, hd, 3)
        for s in range(5):
            kv.t[s, :, hidden[s]] = bad
            kv.t[s, :, used:] = bad
        c.lanes(kv, _i32(often(pos), dev), _i32(often(seqs), dev), window, sinks)
        _close(c.result(), often(want))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("H,n_kv,hd", HEADS)
@pytest.mark.parametrize("window,sinks", [(100, 3), (700, 130), (0, 0)])
def test_not_finite_rows_that_some_lanes_see(dev, kind, H, n_kv, hd, window, sinks):
    # a value or key that is not finite makes outputs NaN for the lanes that see it, of the KV head it belongs to, and
    # for no others: at the ends and in the middle of 64 rows, in first rows, in every head's last dim
    used = 1500
    pos = list(range(700, 790)) + [1400, 40, 1000]
    seqs = [0] * 90 + [1, 1, 1]
    clean = Long(dev, kind, 2, used, n_kv, hd, 5)
    host = [clean.host(s) for s in range(2)]
    c, often = _often(dev, clean, len(pos), H, n_kv, hd, window, sinks)
    q = c.q.cpu().numpy()
    want = np.stack([_ref(q[i], *host[s], p, window, sinks, n_kv) for i, (p, s) in enumerate(zip(pos, seqs))])
    g = n_kv - 1  # the KV head, and its query heads
    mine = slice(g * (H // n_kv), H)
    for s, row, dim, which, bad in [(0, 704, hd - 1, 1, "nan"), (0, 720, 0, 1, "inf"), (0, 767, hd // 2, 1, "-inf"),
                                    (0, 768, hd - 1, 0, "nan"), (1, 2, hd - 1, 1, "inf"), (1, 990, 1, 1, "nan"),
                                    (1, 1000, hd - 1, 1, "-inf"), (1, 39, 5, 0, "nan")]:
        kv = Long(dev, kind, 2, used, n_kv, hd, 5)
        kv.t[s, which, row, g * hd + dim] = float(bad)
        c.lanes(kv, _i32(often(pos), dev), _i32(often(seqs), dev), window, sinks)
        got, ref = c.result(), often(want)
        sees = often([t == s and row <= p and (row > p - (window or used) or row < sinks) for p, t in zip(pos, seqs)])
        _close(got[~sees], ref[~sees])
        if g > 0:
            _close(got[sees][:, : mine.start], ref[sees][:, : mine.start])
        assert not np.isfinite(got[sees][:, mine]).all(axis=-1).any(), (row, which, bad)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("lanes", [40, 90])
def test_rising_and_falling_scores(dev, kind, lanes):
    # Scores that rise (or fall) by 13 over every 128 keys: the running maximum is passed by 2^8 and more at every 128,
    # in runs of ten of them to a block and more (20 to 45 pairs of lanes, four KV heads, 17 times 128 keys on average).
    #
    # Tolerance: a score, up to smax = 0.1 * 3199, is rounded to fp32 once when its terms are added (2^-24 smax: a key's
    # 64 products are equal), its weight exp of it less the same maximum for all, and the largest scores' errors enter
    # the sum too: 2 * 2^-24 smax, and once more for exp2 (2^-22) and the constants: 4 * 2^-24 smax.  An output left
    # unscaled by a risen maximum is off by 2^8 and more.
    import torch

    used, n_kv, hd = 3200, 4, 64
    kv = Long(dev, kind, 2, used, n_kv, hd, 6)
    ramp = (torch.arange(used, device=dev, dtype=torch.float32) / 320)[:, None].expand(used, n_kv * hd)
    kv.k[0, :used] = ramp.to(kv.t.dtype)
    kv.k[1, :used] = ramp.flip(0).to(kv.t.dtype)
    c = Call(dev, lanes, n_kv, n_kv, hd)
    _on_tensor_cores(c, kv)
    c.q[:] = 4.0
    c.q[1::4] = -4.0
    rng = np.random.default_rng(7)
    pos = rng.integers(0, used, lanes)
    pos[:4] = used - 1
    seqs = np.arange(lanes) // 2 % 2
    c.lanes(kv, _i32(pos, dev), _i32(seqs, dev))
    got, q, host = c.result(), c.q.cpu().numpy(), [kv.host(0), kv.host(1)]
    ref = np.stack([_ref(q[i], *host[s], p, 0, 0, n_kv) for i, (s, p) in enumerate(zip(seqs, pos))])
    e = np.linalg.norm(got - ref, axis=-1) / np.linalg.norm(ref, axis=-1)
    assert e.max() <= 4 * 2.0 ** -24 * 320, e.max()


def _replayed(dev, kind, c, call, ref):
    """call(pos) captured twice in a row on one workspace, replayed with other positions"""
    import torch

    pos = torch.zeros(c.n, dtype=torch.int32, device=dev)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        call(pos, st)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(pos, None)
        call(pos, None)
    rng = np.random.default_rng(8)
    for _ in range(3):
        ps = rng.integers(-1, 500, c.n)
        pos.copy_(_i32(ps, dev))
        c.ws.random_(0, 255)
        graph.replay()
        _close(c.result(), np.stack([ref(i, p) if p >= 0 else np.zeros((c.H, c.hd)) for i, p in enumerate(ps)]))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("lanes", [4, 64, 65, 130])  # (planned by every block, and by one for all)
def test_captured_and_on_another_stream(dev, kind, lanes):
    kv = Long(dev, kind, 4, 500, 1, 128, 11)
    c = Call(dev, lanes, 4, 1, 128)
    _on_tensor_cores(c, kv)
    s = np.arange(lanes) // 3 % 4
    seqs, q, host = _i32(s, dev), c.q.cpu().numpy(), [kv.host(i) for i in range(4)]
    _replayed(dev, kind, c, lambda pos, st: c.lanes(kv, pos, seqs, stream=st),
              lambda i, p: _ref(q[i], *host[s[i]], p, 0, 0, 1))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("lanes", [9, 70])
def test_prefix_captured(dev, kind, lanes):
    P = 210
    pre, kv = Long(dev, kind, 1, P, 2, 64, 12), Long(dev, kind, lanes, 300, 2, 64, 13)
    c = Call(dev, lanes, 6, 2, 64)
    _on_tensor_cores(c, kv, prefix=pre)
    seqs, plen, q = _i32(np.arange(lanes), dev), _i32([P], dev), c.q.cpu().numpy()
    both = [[np.concatenate([a, b]) for a, b in zip(pre.host(0), kv.host(i))] for i in range(lanes)]
    _replayed(dev, kind, c, lambda pos, st: c.prefix(pre, plen, None, kv, pos, seqs, stream=st),
              lambda i, p: _ref(q[i], *both[i], p, 0, 0, 2))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_two_calls_at_once(dev, kind):
    # two streams, each with a workspace of its own, over the same caches
    import torch

    kv = Long(dev, kind, 3, 900, 1, 128, 14)
    calls = [Call(dev, n, 4, 1, 128, seed) for n, seed in ((30, 1), (100, 2))]
    at = [(_i32(np.arange(c.n) * 7 % 900, dev), _i32(np.arange(c.n) % 3, dev)) for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, (pos, seqs), st in zip(calls, at, streams):
            _on_tensor_cores(c, kv)
            c.lanes(kv, pos, seqs, stream=st)
    host = [kv.host(s) for s in range(3)]
    for c in calls:
        got, q = c.result(), c.q.cpu().numpy()
        _close(got, np.stack([_ref(q[i], *host[i % 3], i * 7 % 900, 0, 0, 1) for i in range(c.n)]))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_offsets_past_32_bits(dev, kind):
    # the second sequence starts more than 2^31 elements behind the first
    import torch

    from weight_streaming_gemv_gb300 import qlin

    rows, used, kvd, stride = ROWS[kind], 300, 64, (1 << 31) + 4096
    buf = torch.empty(stride + 2 * rows * kvd, dtype=torch.float32 if kind == "f32" else torch.bfloat16, device=dev)
    view = lambda off: buf.as_strided((2, rows, kvd), (stride, kvd, 1), off)
    k, v = view(0), view(rows * kvd)
    for s in range(2):
        for t in (k, v):
            t[s, :used] = torch.randn((used, kvd), device=dev).to(buf.dtype)
    kv = type("K", (), {"c": qlin.kv_cache(k, v)})
    c = Call(dev, 2, 2, 1, 64)
    _on_tensor_cores(c, kv)
    c.lanes(kv, _i32([299, 150], dev), _i32([1, 0], dev))
    got, q = c.result(), c.q.cpu().numpy()
    f = lambda t, s: t[s, :used].float().cpu().numpy().reshape(used, 1, 64)
    _close(got, np.stack([_ref(q[i], f(k, s), f(v, s), p, 0, 0, 1) for i, (p, s) in enumerate([(299, 1), (150, 0)])]))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("lanes", [8, 100])
def test_same_inputs_same_bits(dev, kind, lanes):
    kv = Long(dev, kind, 8, 3000, 2, 128, 12)
    c = Call(dev, lanes, 8, 2, 128)
    _on_tensor_cores(c, kv)
    pos, seqs = _i32(np.arange(lanes) * 997 % 3000, dev), _i32(np.arange(lanes) % 8, dev)
    c.lanes(kv, pos, seqs)
    first = c.result().copy()
    for _ in range(5):
        c.ws.random_(0, 255)
        c.out[: c.n] = 1.0
        c.lanes(kv, pos, seqs)
        np.testing.assert_array_equal(c.result(), first)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("lanes", [3, 80])
def test_scores_of_any_size(dev, kind, lanes):
    # Finite scores far below those of real models: equal ones give the mean of the values, a larger one takes all, in
    # whole and in split tiles.  (Equal scores are equal bits: what is left is the mean's error, a few 2^-24 of the values'
    # 2-norm, within TOL.)
    import torch

    used, H, hd = 1000, 2, 64
    kv = Long(dev, kind, 3, used, 1, hd, 15)
    kv.k[0, :used] = -1e16
    kv.k[1, :used] = -1e17
    kv.k[1, 400] = 0.0
    kv.k[2, :used] = -2e17
    kv.k[2, 300:302] = -1e17
    c = Call(dev, lanes, H, 1, hd)
    _on_tensor_cores(c, kv)
    c.q[:] = 1e16
    c.q[:, 1] = 3e18
    seqs = np.arange(lanes) % 3
    c.lanes(kv, _i32([used - 1] * lanes, dev), _i32(seqs, dev))
    got, host = c.result(), [kv.host(s)[1][:, 0].astype(np.float64) for s in range(3)]
    want = [host[0].mean(0), host[1][400], host[2][300:302].mean(0)]
    _close(got, np.stack([np.broadcast_to(want[s], (H, hd)) for s in seqs]))


@pytest.mark.parametrize("pattern", [0x3F80FFFF, 0x3F80C0FF, 0x3F80BF80, 0x3F817FFF])
def test_products_of_an_fp32_cache(dev, pattern):
    # Products that all have one sign and lose the most where operands are cut into bf16 terms: keys whose every value
    # has the pattern's mantissa against keys of bf16 values, which lose nothing, in scores of about 32 and 46.
    #
    # Tolerance: what is left out of a product, 2 * mid * lo with mid < 2^-7 and lo <= 2^-16 of the leading bit (where mid
    # is rounded to nearest), is at most 2^-22: 46 * 2^-22 = 1.1e-5 in the difference of two scores.  Each score is
    # rounded to fp32 once when its terms are added, 46 * 2^-24 = 2.8e-6 at most, twice.  exp2 has 2^-22 for each key.
    # An output here is (a e^x - b) / (a e^x + b), x the difference's error: half of it.  (1.1e-5 + 5.6e-6 + 4.8e-7) / 2
    # = 8.6e-6; where mid is 2^-7 (the first pattern) lo is 2^-23 and the first part is nothing: 3.1e-6.
    import torch

    used, hd = 900, 256
    kv = Long(dev, "f32", 1, used, 1, hd, 16)
    x = torch.tensor([pattern], dtype=torch.int32, device=dev).view(torch.float32)
    kv.k[0, :used] = 1.015625
    kv.k[0, 1:used:2] = x
    kv.v[0, :used] = -1.0
    kv.v[0, 1:used:2] = 1.0
    c = Call(dev, 1, 2, 1, hd)
    _on_tensor_cores(c, kv)
    c.q[0, 0] = 2 * x
    c.q[0, 1] = (x.double() * (16 / np.log2(np.e) / 4)).float()  # (with the softmax's scale in it: the pattern again)
    c.lanes(kv, _i32([used - 1], dev), _i32([0], dev))
    got, q = c.result(), c.q.cpu().numpy()
    ref = _ref(q[0], *kv.host(0), used - 1, 0, 0, 1)
    e = np.abs(got[0] - ref).max(-1)
    assert (e <= (3.2e-6 if pattern == 0x3F80FFFF else 8.6e-6)).all(), e
