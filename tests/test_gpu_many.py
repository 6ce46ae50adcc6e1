"""GPU parity of the attention over lanes (windows, first tokens, shared
prompts) against the definition in 64 bits, lane by lane.

Tolerance.  A score is a sum of up to 256 products of 24-bit factors in fp32:
with half a step (2^-24) lost per term, random in sign, the error is about
sqrt(3 * 256) * 2^-24 of the running sum, whose size here stays below about 8
(scores of standard deviation 2): 1.3e-5 in the worst key, and the weights
have that relative error.  A row's outputs are weighted means, so their
2-norm is off by at most that much relatively; 2e-5 leaves a factor 1.5.  A
wrongly seen or unseen key among n moves a row by about 1/sqrt(n), 3e-2 at
n = 1000."""
import numpy as np
import pytest

from gpu_util import device

pytestmark = pytest.mark.gpu
TOL = 2e-5


@pytest.fixture(scope="module")
def dev():
    return device()


def _ref(q, keys, vals, p, window, sinks, n_kv):
    """one lane in 64 bits: q [H][hd]; keys, vals [>= p + 1][n_kv][hd], by position"""
    H, hd = q.shape
    j = np.arange(p + 1)
    seen = (j > p - window) | (j < sinks) if window else np.ones(p + 1, bool)
    k, v = keys[: p + 1][seen].astype(np.float64), vals[: p + 1][seen].astype(np.float64)
    out = np.zeros((H, hd))
    for h in range(H):
        g = h // (H // n_kv)
        s = k[:, g] @ q[h].astype(np.float64) / np.sqrt(hd)
        w = np.exp(s - s.max())
        out[h] = (w / w.sum()) @ v[:, g]
    return out


def _close(got, ref):
    """every row of every lane and head by its own 2-norm"""
    e = np.linalg.norm(got - ref, axis=-1) / np.maximum(np.linalg.norm(ref, axis=-1), 1e-30)
    assert np.isfinite(got).all()
    assert e.max() <= TOL, f"worst row {np.unravel_index(e.argmax(), e.shape)}: {e.max()}"


class Caches:
    """caches [n_seqs][layers][2][rows][kv_dim], the last layer's the ones used"""

    def __init__(self, dev, kind, n_seqs, rows, n_kv, hd, seed=0, layers=2, fill=None):
        import torch

        from weight_streaming_gemv_gb300 import qlin

        g = torch.Generator(device=dev).manual_seed(seed)
        t = torch.randn((n_seqs, layers, 2, rows, n_kv * hd), generator=g, device=dev)
        self.t = t.to(torch.bfloat16 if kind == "bf16" else torch.float32)
        self.n_kv, self.hd, self.rows = n_kv, hd, rows
        self.k, self.v = self.t[:, -1, 0], self.t[:, -1, 1]
        self.c = qlin.kv_cache(self.k, self.v)

    def host(self, s):
        f = lambda x: x[s].float().cpu().numpy().reshape(self.rows, self.n_kv, self.hd)
        return f(self.k), f(self.v)


def _i32(x, dev):
    import torch

    return torch.as_tensor(np.ascontiguousarray(x, np.int32)).to(dev)


class Call:
    """One set of buffers around the two entry points."""

    def __init__(self, dev, n_lanes, H, n_kv, hd, seed=1, extra=3):
        import torch

        from weight_streaming_gemv_gb300 import qlin

        g = torch.Generator(device=dev).manual_seed(seed)
        self.n, self.H, self.n_kv, self.hd = n_lanes, H, n_kv, hd
        self.q = torch.randn((n_lanes, H, hd), generator=g, device=dev) * 2
        self.out = torch.full((n_lanes + extra, H, hd), 7.5, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.bytes = qlin.qlin_attention_lanes_workspace_size(n_lanes, H, n_kv, hd)
        self.ws = torch.randint(0, 255, (self.bytes,), dtype=torch.uint8, device=dev)

    def lanes(self, kv, pos, seqs, window=0, sinks=0, stream=None):
        from weight_streaming_gemv_gb300 import qlin

        qlin.qlin_attention_lanes(self.q, kv.c, pos, seqs, self.n, self.H, self.n_kv, self.hd, window, sinks,
                                  self.out, self.status, self.ws, self.bytes, stream)

    def prefix(self, pre, plen, pof, kv, pos, seqs, window=0, sinks=0, stream=None):
        from weight_streaming_gemv_gb300 import qlin

        qlin.qlin_attention_prefix(self.q, pre.c, plen, pof, kv.c, pos, seqs, self.n, self.H, self.n_kv, self.hd,
                                   window, sinks, self.out, self.status, self.ws, self.bytes, stream)

    def result(self, status=0):
        import torch

        torch.cuda.synchronize()
        assert int(self.status.item()) == status
        got = self.out.cpu().numpy()
        assert (got[self.n:] == 7.5).all(), "rows behind the last lane were written"
        return got[: self.n]


def _times(kind, n, rows, H, n_kv, hd, window, sinks):
    """How often n lanes have to be given for the call to be too much work for the kernel of little work (by the
    multiply-adds that it goes by, 300 M at most)."""
    keys = min(rows, window + sinks) if window else rows
    per = 32 if kind == "f32" else 64
    gh = 1 if H == n_kv else 2 if H <= 2 * n_kv else 4 if H <= 4 * n_kv else 8
    fma = -(-keys // per) * per * n * n_kv * -(-(H // n_kv) // gh) * gh * hd * 2
    return min(int(300e6 // fma) + 1, 4096 // n)


def _check_lanes(dev, kind, n_seqs, rows, H, n_kv, hd, pos, seqs, window, sinks, seed=0, status=0):
    """The lanes once, and given over and over until the other kernel takes them (as many as there can be)."""
    kv = Caches(dev, kind, n_seqs, rows, n_kv, hd, seed)
    n, ref = len(pos), None
    for times in sorted({1, _times(kind, n, rows, H, n_kv, hd, window, sinks)}):
        c = Call(dev, n * times, H, n_kv, hd, seed + 1)
        c.q.copy_(c.q[:n].repeat(times, 1, 1))
        c.lanes(kv, _i32(np.tile(np.int64(pos), times), dev), _i32(np.tile(np.int64(seqs), times), dev), window, sinks)
        got, q = c.result(status), c.q.cpu().numpy()
        if ref is None:
            ref = np.zeros((n, H, hd))
            for i, (p, s) in enumerate(zip(pos, seqs)):
                if 0 <= p < rows and 0 <= s < n_seqs:
                    ref[i] = _ref(q[i], *kv.host(s), p, window, sinks, n_kv)
        _close(got, np.tile(ref, (times, 1, 1)))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("p", [0, 1, 63, 64, 127, 128, 129, 255, 300, 1000])
def test_one_token(dev, kind, p):
    _check_lanes(dev, kind, 1, p + 1, 4, 1, 256, [p], [0], 0, 0, seed=p)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("H,n_kv,hd", [(4, 1, 256), (1, 1, 16), (2, 2, 32), (3, 1, 64), (16, 2, 128), (10, 2, 80),
                                       (8, 8, 64), (6, 2, 192), (71, 1, 64), (130, 2, 48), (8, 1, 240)])
def test_head_layouts(dev, kind, H, n_kv, hd):
    # one token each, at positions around a block of 128 rows
    pos, seqs = [0, 5, 127, 128, 260, 399], [3, 1, 0, 4, 2, 5]
    _check_lanes(dev, kind, 6, 400, H, n_kv, hd, pos, seqs, 0, 0, seed=H)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (64, 4), (128, 0), (129, 130), (200, 4), (511, 1),
                                          (4000, 4), (2147483647, 2147483647), (1, 2147483647)])
def test_windows(dev, kind, window, sinks):
    # single tokens of many users at mixed positions, two of them in one sequence
    pos = [0, 1, 63, 127, 128, 200, 511, 640, 699, 350]
    seqs = [0, 1, 2, 3, 4, 0, 1, 2, 3, 3]
    _check_lanes(dev, kind, 5, 700, 4, 2, 64, pos, seqs, window, sinks, seed=window % 97)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (33, 0), (100, 4), (1, 2)])
@pytest.mark.parametrize("H,n_kv,hd", [(4, 1, 256), (6, 2, 64), (40, 1, 32)])
def test_prompt_chunks(dev, kind, window, sinks, H, n_kv, hd):
    # two prompts' chunks, a token between them, padding, and a chunk listed backwards
    pos = list(range(90, 90 + 131)) + [40] + [-1] * 3 + list(range(0, 70)) + [-1] + list(range(39, -1, -1))
    seqs = [1] * 131 + [3] + [0] * 3 + [2] * 70 + [2] + [0] * 40
    _check_lanes(dev, kind, 4, 256, H, n_kv, hd, pos, seqs, window, sinks, seed=window)


def test_many_lanes_of_short_sequences(dev):
    # more lanes than SMs by far, each with a handful of keys
    pos = [i % 5 for i in range(4096)]
    seqs = [i % 64 for i in range(4096)]
    _check_lanes(dev, "f32", 64, 8, 2, 2, 16, pos, seqs, 3, 1)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_long_context(dev, kind):
    _check_lanes(dev, kind, 2, 40000, 8, 2, 128, [39999, 17], [1, 0], 0, 0)
    _check_lanes(dev, kind, 2, 40000, 8, 2, 128, [39998, 39999], [1, 1], 20000, 130)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_runs_of_lanes_past_a_thousand(dev, kind):
    # one prompt's chunk of 2100 lanes, and lanes of few sequences that return to each of them (a sample is compared)
    S, R, H, n_kv, hd = 7, 2200, 4, 1, 64
    kv = Caches(dev, kind, S, R, n_kv, hd, 14, layers=1)
    rng = np.random.default_rng(15)
    runs = rng.integers(0, S, 4000)
    for pos, seqs in ((list(range(60, 2160)), [3] * 2100),
                      (rng.integers(-1, R, 4000).tolist(), np.repeat(runs, rng.integers(1, 5, 4000))[:4000].tolist())):
        c = Call(dev, len(pos), H, n_kv, hd)
        c.lanes(kv, _i32(pos, dev), _i32(seqs, dev), 300, 5)
        got, q = c.result(), c.q.cpu().numpy()
        host = [kv.host(s) for s in range(S)]
        for i in list(range(1000, 1060)) + list(range(2030, 2060)) + rng.integers(0, len(pos), 60).tolist():
            if pos[i] >= 0:
                _close(got[i], _ref(q[i], *host[seqs[i]], pos[i], 300, 5, n_kv))
            else:
                assert (got[i] == 0).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("H,n_kv,hd", [(2, 2, 64), (4, 1, 256), (96, 2, 64)])
def test_many_blocks_per_sm(dev, kind, H, n_kv, hd):
    # each SM runs through many blocks of keys and several tiles: single tokens of 40 users at long contexts
    # together with a chunk of a prompt (a sample of the lanes is compared)
    S, R = 41, 8000
    kv = Caches(dev, kind, S, R, n_kv, hd, 13, layers=1)
    pos = [R - 1 - 37 * i for i in range(40)] + list(range(3000, 3300))
    seqs = list(range(40)) + [40] * 300
    for window, sinks in ((0, 0), (1500, 200)):
        c = Call(dev, len(pos), H, n_kv, hd)
        c.lanes(kv, _i32(pos, dev), _i32(seqs, dev), window, sinks)
        got, q = c.result(), c.q.cpu().numpy()
        for i in [0, 1, 17, 39, 40, 41, 100, 200, 338, 339]:
            k, v = kv.host(seqs[i])
            _close(got[i], _ref(q[i], k, v, pos[i], window, sinks, n_kv))


@pytest.mark.parametrize("times", [1, 40])  # (40: too much work for the kernel of little work)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_unseen_rows_never_reach_the_outputs(dev, kind, times):
    import torch

    S, R, H, n_kv, hd, W, sinks = 3, 300, 4, 2, 64, 50, 3
    pos = ([170, 20] + list(range(100, 164))) * times
    seqs = ([0, 1] + [2] * 64) * times
    for bad in (float("nan"), float("inf"), -float("inf"), 3.4e38):
        kv = Caches(dev, kind, S, R, n_kv, hd, 3)
        clean = [kv.host(s) for s in range(S)]
        for t in (kv.k, kv.v):
            t[0, 171:] = bad
            t[0, 3:121] = bad
            t[1, 21:] = bad
            t[2, 164:] = bad
            t[2, 3:51] = bad
        c = Call(dev, len(pos), H, n_kv, hd)
        c.lanes(kv, _i32(pos, dev), _i32(seqs, dev), W, sinks)
        got, q = c.result(), c.q.cpu().numpy()
        if bad != bad:
            want = np.stack([_ref(q[i], *clean[s], p, W, sinks, n_kv) for i, (p, s) in enumerate(zip(pos, seqs))])
        _close(got, want)
    # a row that some lanes of a chunk see and others do not: NaN for those that see it, and only those
    clean_ref = [_ref(q[i], *clean[s], p, W, sinks, n_kv) for i, (p, s) in enumerate(zip(pos, seqs))]
    for which in range(2):
        kv = Caches(dev, kind, S, R, n_kv, hd, 3)
        (kv.k, kv.v)[which][2, 130, :hd] = float("nan")  # KV head 0 alone
        c = Call(dev, len(pos), H, n_kv, hd)
        c.lanes(kv, _i32(pos, dev), _i32(seqs, dev), W, sinks)
        torch.cuda.synchronize()
        got, q = c.out.cpu().numpy()[: len(pos)], c.q.cpu().numpy()
        for i, (p, s) in enumerate(zip(pos, seqs)):
            sees = s == 2 and 130 <= p < 130 + W
            ref = clean_ref[i]
            _close(got[i, H // 2:], ref[H // 2:])
            if sees:
                assert np.isnan(got[i, : H // 2]).all(axis=-1 if which == 0 else None).all() or which == 1
                assert np.isnan(got[i, : H // 2]).any(axis=-1).all()
            else:
                _close(got[i, : H // 2], ref[: H // 2])


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_lanes_out_of_range(dev, kind):
    # position and sequence out of range: zeros and the status bit; padding alone: zeros, no status
    _check_lanes(dev, kind, 3, 40, 2, 1, 64, [39, 40, 5, -1, 5, 2147483647, 7], [0, 1, 3, 0, -1, 2, 2], 0, 0, status=1)
    _check_lanes(dev, kind, 3, 40, 2, 1, 64, [-1, -5, -2147483648], [0, 99, -1], 0, 0)
    c = Call(dev, 2, 2, 1, 64)
    pre, kv = Caches(dev, kind, 2, 16, 1, 64), Caches(dev, kind, 2, 16, 1, 64)
    for plen, pof, pos in [([17, 3], [0, 1], [4, 4]), ([-1, 3], [0, 1], [4, 4]), ([5, 3], [2, 1], [4, 4]),
                           ([5, 3], [-1, 1], [4, 4]), ([5, 3], [0, 1], [21, 4])]:
        c.status.zero_()
        c.prefix(pre, _i32(plen, dev), _i32(pof, dev), kv, _i32(pos, dev), _i32([0, 1], dev))
        got, q = c.result(1), c.q.cpu().numpy()
        assert (got[0] == 0).all()
        (pk, pv), (k, v) = pre.host(1), kv.host(1)
        _close(got[1], _ref(q[1], np.concatenate([pk[:3], k]), np.concatenate([pv[:3], v]), 4, 0, 0, 1))


def test_large_scores_and_equal_scores(dev):
    # a running maximum that keeps rising, and rows whose weights are all equal
    import torch

    kv = Caches(dev, "f32", 2, 900, 1, 64, 5)
    ramp = torch.arange(900, device=dev, dtype=torch.float32)[:, None] / 40.0
    kv.k[0] = ramp * torch.ones((1, 64), device=dev) / 8.0
    kv.k[1] = 0.0
    c = Call(dev, 3, 1, 1, 64)
    c.q[0] = 4.0
    c.q[1] = -4.0
    c.lanes(kv, _i32([899, 899, 899], dev), _i32([0, 0, 1], dev))
    got, q = c.result(), c.q.cpu().numpy()
    # scores up to 90 (all 64 products of one sign): half a step of 90 is 2^-18
    ref = np.stack([_ref(q[i], *kv.host(s), 899, 0, 0, 1) for i, s in enumerate([0, 0, 1])])
    e = np.linalg.norm(got - ref, axis=-1) / np.linalg.norm(ref, axis=-1)
    assert e.max() <= 8 * 64 * 2.0 ** -24 * 90, e


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,n_kv,hd", [(1, 4, 1, 256), (4, 4, 1, 256), (16, 8, 2, 128), (64, 4, 1, 64), (5, 3, 3, 80)])
@pytest.mark.parametrize("P", [0, 1, 127, 128, 700])
def test_shared_prompt(dev, kind, B, H, n_kv, hd, P):
    R = 40
    pre, kv = Caches(dev, kind, 1, max(P, 1), n_kv, hd, 7), Caches(dev, kind, B, R, n_kv, hd, 8)
    own = [(7 * i) % R for i in range(B)]  # own rows - 1
    pos = [P + o for o in own]
    if P > 5:
        pos[0] = P - 5  # a lane that is still inside the prompt
    pk, pv = pre.host(0)
    ref = None
    for times in sorted({1, _times(kind, B, max(P, 1) + R, H, n_kv, hd, 0, 0)}):
        c = Call(dev, B * times, H, n_kv, hd)
        c.q.copy_(c.q[:B].repeat(times, 1, 1))
        c.prefix(pre, _i32([P], dev), None, kv, _i32(np.tile(pos, times), dev), _i32(np.tile(np.arange(B), times), dev))
        got, q = c.result(), c.q.cpu().numpy()
        if ref is None:
            ref = []
            for i in range(B):
                k, v = kv.host(i)
                ref.append(_ref(q[i], np.concatenate([pk[:P], k]), np.concatenate([pv[:P], v]), pos[i], 0, 0, n_kv))
        _close(got, np.tile(np.stack(ref), (times, 1, 1)))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (30, 0), (30, 4), (200, 3), (150, 170), (1, 0)])
def test_several_prompts(dev, kind, window, sinks):
    # prompts of several lengths (one empty), lanes of one prompt beside each other and apart, chunks of
    # one sequence behind a prompt, windows that end inside the prompt or behind it
    plens = [160, 0, 37, 129]
    pre, kv = Caches(dev, kind, 4, 160, 2, 64, 9), Caches(dev, kind, 9, 64, 2, 64, 10)
    pof = [0, 0, 0, 3, 3, 1, 1, 2, 0, 2] + [3] * 30
    seqs = [0, 1, 2, 3, 4, 5, 6, 7, 8, 7] + [4] * 30
    own = [0, 9, 63, 40, 5, 3, 63, 20, 33, 21] + list(range(6, 36))
    pos = [plens[f] + o for f, o in zip(pof, own)]
    N, ref = len(pos), None
    for times in sorted({1, _times(kind, N, 160 + 64, 6, 2, 64, window, sinks)}):
        tile = lambda x: _i32(np.tile(x, times), dev)
        c = Call(dev, N * times, 6, 2, 64)
        c.q.copy_(c.q[:N].repeat(times, 1, 1))
        c.prefix(pre, _i32(plens, dev), tile(pof), kv, tile(pos), tile(seqs), window, sinks)
        got, q = c.result(), c.q.cpu().numpy()
        if ref is None:
            ref = []
            for i, (f, s, p) in enumerate(zip(pof, seqs, pos)):
                (pk, pv), (k, v) = pre.host(f), kv.host(s)
                n = plens[f]
                ref.append(_ref(q[i], np.concatenate([pk[:n], k]), np.concatenate([pv[:n], v]), p, window, sinks, 2))
        _close(got, np.tile(np.stack(ref), (times, 1, 1)))


def test_offsets_past_32_bits(dev):
    # the second sequence starts more than 2^31 elements (2^32 bytes) behind the first
    import torch

    from weight_streaming_gemv_gb300 import qlin

    rows, kvd, stride = 300, 64, (1 << 31) + 4096
    buf = torch.empty(stride + 2 * rows * kvd, dtype=torch.bfloat16, device=dev)
    view = lambda off: buf.as_strided((2, rows, kvd), (stride, kvd, 1), off)
    k, v = view(0), view(rows * kvd)
    for s in range(2):
        k[s] = torch.randn((rows, kvd), device=dev).to(torch.bfloat16)
        v[s] = torch.randn((rows, kvd), device=dev).to(torch.bfloat16)
    c = Call(dev, 2, 2, 1, 64)
    kv = type("K", (), {"c": qlin.kv_cache(k, v)})
    c.lanes(kv, _i32([299, 150], dev), _i32([1, 0], dev))
    got, q = c.result(), c.q.cpu().numpy()
    f = lambda t, s: t[s].float().cpu().numpy().reshape(rows, 1, 64)
    _close(got, np.stack([_ref(q[i], f(k, s), f(v, s), p, 0, 0, 1) for i, (p, s) in enumerate([(299, 1), (150, 0)])]))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("H,n_kv,hd", [(4, 1, 256), (3, 3, 16), (10, 1, 64), (2, 1, 80)])
@pytest.mark.parametrize("rows", [33, 65, 100, 300, 516, 640, 641, 1000, 1281])
def test_little_work_in_any_number_of_pieces(dev, kind, rows, H, n_kv, hd):
    # 1 to 41 pieces of a lane's keys: alone, as clusters of 2 to 16, with a merging launch; a short lane leaves most
    # of its pieces empty, a padding lane all
    kv = Caches(dev, kind, 2, rows, n_kv, hd, rows)
    pos, seqs = [rows - 1, 0, rows // 2, -1], [0, 1, 1, 0]
    c = Call(dev, 4, H, n_kv, hd, rows)
    c.lanes(kv, _i32(pos, dev), _i32(seqs, dev))
    got, q = c.result(), c.q.cpu().numpy()
    for i in range(3):
        _close(got[i], _ref(q[i], *kv.host(seqs[i]), pos[i], 0, 0, n_kv))
    assert (got[3] == 0).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [30, 100, 600, 2000])  # alone, a cluster, and pieces that a second kernel joins
def test_scores_below_the_types_range(dev, kind, rows):
    # The first fifth of the keys have scores that fp32 cannot hold (-8e40): no weight.  The others' are equal, and far
    # below zero: the mean of their values.
    import torch

    H, hd, n = 2, 64, rows // 5
    kv = Caches(dev, kind, 2, rows, 1, hd, 31)
    kv.k[0] = -3e-19
    kv.k[0, :n] = -1e20
    c = Call(dev, 2, H, 1, hd)
    c.q[:] = 1e20
    c.q[1] = 0.0
    c.lanes(kv, _i32([rows - 1, rows - 1], dev), _i32([0, 1], dev))
    got = c.result()
    v, w = kv.host(0)[1].astype(np.float64), kv.host(1)[1].astype(np.float64)
    _close(got[0], np.broadcast_to(v[n:, 0].mean(0), (H, hd)))
    _close(got[1], np.broadcast_to(w[:, 0].mean(0), (H, hd)))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("n", [6, 640])
def test_sequences_inside_rows(dev, kind, n):
    # row r of every sequence side by side: seq_stride below row_stride, and k and v interleaved (640 lanes are too
    # much for the kernel of little work)
    import torch

    from weight_streaming_gemv_gb300 import qlin

    S, R, H, n_kv, hd = 5, 700, 4, 2, 128
    g = torch.Generator(device=dev).manual_seed(21)
    t = torch.randn((R, S, 2, n_kv * hd), generator=g, device=dev).to(torch.float32 if kind == "f32" else torch.bfloat16)
    k, v = t[:, :, 0].permute(1, 0, 2), t[:, :, 1].permute(1, 0, 2)

    class View:
        c = qlin.kv_cache(k, v)

    rng = np.random.default_rng(22)
    pos, seqs = rng.integers(0, R, n), np.sort(rng.integers(0, S, n))
    c = Call(dev, n, H, n_kv, hd)
    c.lanes(View, _i32(pos, dev), _i32(seqs, dev), 300, 3)
    got, q = c.result(), c.q.cpu().numpy()
    f = lambda x: x.float().cpu().numpy().reshape(R, n_kv, hd)
    host = [(f(k[s]), f(v[s])) for s in range(S)]
    for i in list(range(6)) + rng.integers(0, n, 40).tolist():
        _close(got[i], _ref(q[i], *host[seqs[i]], pos[i], 300, 3, n_kv))


def test_captured_and_on_another_stream(dev):
    import torch

    kv = Caches(dev, "bf16", 4, 500, 1, 128, 11)
    c = Call(dev, 4, 4, 1, 128)
    pos, seqs = _i32([0, 0, 0, 0], dev), _i32([0, 1, 2, 3], dev)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        c.lanes(kv, pos, seqs, 100, 2, st)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.lanes(kv, pos, seqs, 100, 2)
        c.lanes(kv, pos, seqs, 100, 2)  # the same workspace twice in a row
    q = c.q.cpu().numpy()
    for ps in ([499, 3, 128, 250], [5, 499, 0, 127], [-1, 100, 101, 102]):
        pos.copy_(_i32(ps, dev))
        graph.replay()
        got = c.result()
        ref = np.stack([_ref(q[i], *kv.host(i), p, 100, 2, 1) if p >= 0 else np.zeros((4, 128)) for i, p in enumerate(ps)])
        _close(got, ref)


def test_same_inputs_same_bits(dev):
    kv = Caches(dev, "f32", 8, 3000, 2, 128, 12)
    c = Call(dev, 8, 8, 2, 128)
    pos, seqs = _i32([2999, 100, 2000, 1500, 3, 2998, 640, 1], dev), _i32(np.arange(8), dev)
    c.lanes(kv, pos, seqs)
    first = c.result().copy()
    for _ in range(3):
        c.ws.random_(0, 255)
        c.lanes(kv, pos, seqs)
        np.testing.assert_array_equal(c.result(), first)
