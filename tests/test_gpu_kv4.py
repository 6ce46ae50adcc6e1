"""GPU parity of the paged 4-bit cache: appending (codes, scales and rotated queries bit for bit), reading back, and the
attention over it against the definition in 64 bits, lane by lane.

Tolerance of the attention.  The cache's values are exact on both sides.  A score is a sum of up to 256 products in fp32,
of queries that keep 22 bits or more: with half a step (2^-24, or 2^-23 of a query) lost per term, random in sign, the
error is about sqrt(3 * 256) * 2^-24 of the running sum, whose size here stays below about 8 (scores of standard
deviation 2): 1.3e-5 in the worst key, and the weights have that relative error.  A row's outputs are weighted means, so
their 2-norm is off by at most that much relatively; 2e-5 leaves a factor 1.5.  A wrongly seen or unseen key among n moves
a row by about 1/sqrt(n), 1e-2 at n = 10000."""
import numpy as np
import pytest

import kv4_ref as ref
from gpu_util import device
from kv4_util import Pool, i32

pytestmark = pytest.mark.gpu
TOL = 2e-5


@pytest.fixture(scope="module")
def dev():
    return device()


# ------------------------------------------------------------------ appending and reading
class Rows:
    """the lanes' q, k and v as parts of one row, with floats between the rows that nobody reads"""

    def __init__(self, dev, n, H, G, hd, seed=1, gap=8, scale=1.0):
        import torch

        rng = np.random.default_rng(seed)
        self.n, self.H, self.G, self.hd = n, H, G, hd
        self.x = (rng.standard_normal((n, (H + 2 * G) * hd + gap)) * scale).astype(np.float32)
        self.dev = dev
        self.upload()

    def upload(self):
        import torch

        self.d = torch.from_numpy(self.x).to(self.dev)

    def part(self, what, t=None):
        H, G, hd = self.H, self.G, self.hd
        a, b = {"q": (0, H * hd), "k": (H * hd, (H + G) * hd), "v": ((H + G) * hd, (H + 2 * G) * hd)}[what]
        return (self.x if t is None else t)[:, a:b]

    def heads(self, what):
        return self.part(what).reshape(self.n, -1, self.hd)


def _rope(dev, rows, hd):
    import torch

    from weight_streaming_gemv_gb300 import qlin

    c = torch.empty((rows, hd // 2), device=dev)
    s = torch.empty((rows, hd // 2), device=dev)
    qlin.t158_rope_table(c, s, rows, hd, 10000.0)
    return c, s


def _append(pool, r, pos, seqs, rope=None, rope_rows=0, q=True, status=None, q_out=None):
    import torch

    from weight_streaming_gemv_gb300 import qlin

    out = torch.full((r.n + 1, r.H, r.hd), 7.5, device=r.dev) if q_out is None else q_out
    c, s = rope if rope else (None, None)
    stride = r.d.stride(0)
    qlin.qlin_kv4_append(pool.c, r.part("k", r.d), r.part("v", r.d), stride, r.part("q", r.d) if q else None, stride,
                         out if q else None, c, s, rope_rows, i32(pos, r.dev), i32(seqs, r.dev), r.n, r.H, r.G, r.hd,
                         status)
    torch.cuda.synchronize()
    return out


def _expect(pool, r, pos, seqs, rope, live):
    """the pool's bytes after the call, and the rotated queries"""
    codes, scales = pool.codes.copy(), pool.scales.copy()
    q, k, v = (r.heads(w).copy() for w in "qkv")
    if rope:
        c, s = (t.cpu().numpy() for t in rope)
        at = np.clip(pos, 0, len(c) - 1)
        q, k = (ref.rotate(x, c[at][:, None], s[at][:, None]) for x in (q, k))
    q[~live] = 0
    page = pool.table[np.where(live, seqs, 0), np.where(live, pos, 0) // pool.page]
    for i, x in ((0, k), (1, v)):
        code, b = ref.quantise(x[live])
        codes[i][page[live], :, pos[live] % pool.page] = ref.pack(code)
        scales[i][page[live], :, pos[live] % pool.page] = b
    return codes, scales, q


@pytest.mark.parametrize("H,G,hd,page", [(4, 1, 256, 64), (8, 2, 128, 16), (3, 3, 64, 32), (1, 1, 64, 256), (16, 4, 256, 128)])
@pytest.mark.parametrize("rotate", [True, False])
@pytest.mark.parametrize("lanes", [1, 7, 600])
def test_append_bit_exact(dev, H, G, hd, page, rotate, lanes):
    import torch

    rng = np.random.default_rng(lanes)
    S = min(lanes, 5)
    rows = -(-lanes // S) + 40
    pool = Pool(dev, S, rows, G, hd, page)
    seqs = np.arange(lanes) % S
    pos = rng.permutation(pool.rows)[: -(-lanes // S)][np.arange(lanes) // S]  # no place twice
    pos[rng.random(lanes) < 0.1] = -1
    r = Rows(dev, lanes, H, G, hd, scale=10.0 ** rng.integers(-4, 4))
    rope = _rope(dev, pool.rows, hd) if rotate else None
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    out = _append(pool, r, pos, seqs, rope, pool.rows, status=status).cpu().numpy()
    codes, scales, q = _expect(pool, r, pos, seqs, rope, pos >= 0)
    assert int(status) == 0
    assert np.array_equal(pool.d_scales.cpu().numpy(), scales)
    assert np.array_equal(pool.d_codes.cpu().numpy(), codes)
    assert np.array_equal(out[:lanes], q) and (out[lanes] == 7.5).all()


@pytest.mark.parametrize("H,G,hd,page", [(5, 1, 64, 16), (8, 2, 128, 32), (16, 4, 256, 64), (1, 1, 64, 256), (13, 13, 64, 16),
                                         (4, 1, 256, 16)])
@pytest.mark.parametrize("q", [True, False])
def test_append_many_lanes(dev, H, G, hd, page, q):
    """so many lanes that a thread takes several rows, numbers of rows that do not divide, padding, values that are not
    finite, a position behind the tables"""
    import torch

    lanes, S = 1301, 7
    rng = np.random.default_rng(H)
    pool = Pool(dev, S, 260, G, hd, page)
    seqs = np.arange(lanes) % S
    pos = rng.permutation(250)[np.arange(lanes) // S]
    pos[rng.random(lanes) < 0.1] = -1
    r = Rows(dev, lanes, H, G, hd)
    rope = _rope(dev, 249, hd)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    out = _append(pool, r, pos, seqs, rope, 249, q=q, status=status).cpu().numpy()
    live = (pos >= 0) & (pos < 249)
    codes, scales, want = _expect(pool, r, pos, seqs, rope, live)
    assert int(status) == int((pos == 249).any())
    assert np.array_equal(pool.d_scales.cpu().numpy(), scales)
    assert np.array_equal(pool.d_codes.cpu().numpy(), codes)
    if q:
        assert np.array_equal(out[:lanes], want) and (out[lanes] == 7.5).all()
    # a value of a key of the last lane that is not finite: its group's others are as without it
    at = int(np.flatnonzero(live)[-1])
    r.part("k")[at, (G - 1) * hd + 5] = np.inf
    r.upload()
    status.zero_()
    _append(pool, r, np.where(np.arange(lanes) == at, pos, -1), seqs, None, 0, q=q, status=status)
    assert int(status) == 4


@pytest.mark.parametrize("hd", [64, 256])
def test_append_every_scale_and_ties(dev, hd):
    """rows whose largest value walks over every scale, its neighbours included, and values half-way between codes"""
    import torch

    up = np.nextafter(ref.SCALES.astype(np.float32) * np.float32(7), np.float32(np.inf))
    tops = np.concatenate((ref.SCALES * 7, up, np.nextafter(up, np.float32(0)), [0.0, 1e-30, 3e-7, 1e5, 3e38])).astype(np.float32)
    n, G = len(tops), 1
    r = Rows(dev, n, 1, G, hd)
    k = np.tile((np.arange(hd) % 29 - 14) / 2, (n, 1))  # halves of -14 .. 14 steps: ties where the scale fits
    r.part("k")[:] = k * (tops / 7)[:, None]
    r.part("k")[:, 0] = tops
    r.part("v")[:] = -r.part("k")
    r.upload()
    pool = Pool(dev, 1, n, G, hd, 16)
    pos, seqs = np.arange(n), np.zeros(n, int)
    _append(pool, r, pos, seqs, q=False)
    codes, scales, _ = _expect(pool, r, pos, seqs, None, pos >= 0)
    assert np.array_equal(pool.d_scales.cpu().numpy(), scales)
    assert np.array_equal(pool.d_codes.cpu().numpy(), codes)


def test_append_not_finite(dev):
    import torch

    r = Rows(dev, 4, 2, 2, 128)
    r.part("k")[0, 5] = np.nan
    r.part("v")[1, 40] = np.inf
    r.part("v")[2, 130] = -np.inf
    r.part("k")[3, :32] = np.nan
    r.upload()
    pool = Pool(dev, 1, 16, 2, 128, 16)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    pos, seqs = np.arange(4), np.zeros(4, int)
    _append(pool, r, pos, seqs, status=status)
    codes, scales, _ = _expect(pool, r, pos, seqs, None, pos >= 0)
    assert int(status) == 4
    assert np.array_equal(pool.d_scales.cpu().numpy(), scales) and np.array_equal(pool.d_codes.cpu().numpy(), codes)
    # a query that is not finite is nobody else's
    status.zero_()
    r = Rows(dev, 1, 2, 2, 128)
    r.part("q")[0, 3] = np.nan
    r.upload()
    _append(pool, r, np.array([9]), np.array([0]), status=status)
    assert int(status) == 0


def test_append_out_of_range_and_padding(dev):
    import torch

    pool = Pool(dev, 3, 64, 1, 64, 16, spare=2)
    t = pool.table.copy()
    t[1, 2] = -1
    t[2, 1] = pool.codes.shape[1]
    pool.set_table(t)
    #                 ok  pad  seq  seq  past  page  page  rope ok
    pos = np.array([3, -1, 0, 0, pool.rows, 40, 17, 50, 5])
    seqs = np.array([0, 7, 3, -1, 0, 1, 2, 0, 2])
    live = np.array([1, 0, 0, 0, 0, 0, 0, 0, 1], bool)
    r = Rows(dev, 9, 2, 1, 64)
    rope = _rope(dev, 48, 64)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    out = _append(pool, r, pos, seqs, rope, 48, status=status).cpu().numpy()
    codes, scales, q = _expect(pool, r, pos, seqs, rope, live)
    assert int(status) == 1
    assert np.array_equal(pool.d_codes.cpu().numpy(), codes) and np.array_equal(pool.d_scales.cpu().numpy(), scales)
    assert np.array_equal(out[:9], q)
    status.zero_()
    _append(pool, Rows(dev, 2, 2, 1, 64), np.array([-1, -5]), np.array([0, 99]), status=status)
    assert int(status) == 0


def test_append_in_place(dev):
    import torch

    pool, n = Pool(dev, 1, 64, 2, 128, 32), 40
    r = Rows(dev, n, 4, 2, 128)
    rope = _rope(dev, 64, 128)
    want = _append(pool, r, np.arange(n), np.zeros(n, int), rope, 64)[:n]
    from weight_streaming_gemv_gb300 import qlin

    q = r.part("q", r.d).contiguous().view(n, 4, 128)
    qlin.qlin_kv4_append(pool.c, r.part("k", r.d), r.part("v", r.d), r.d.stride(0), q, 512, q, rope[0], rope[1], 64,
                         i32(np.arange(n), dev), i32(np.zeros(n), dev), n, 4, 2, 128)
    torch.cuda.synchronize()
    assert torch.equal(q, want)


@pytest.mark.parametrize("hd,page", [(64, 16), (128, 256), (256, 32)])
def test_read(dev, hd, page):
    import torch

    from weight_streaming_gemv_gb300 import qlin

    G, S = 3, 4
    pool = Pool(dev, S, 100, G, hd, page)
    t = pool.table.copy()
    t[3, -1] = -4
    pool.set_table(t)
    rng = np.random.default_rng(3)
    n = 333
    pos, seqs = rng.integers(-2, pool.rows, n), rng.integers(0, S, n)
    pos[:3], seqs[:3] = (pool.rows, 0, 5), (0, S, -1)
    k = torch.full((n + 1, G, hd), 7.5, device=dev)
    v, k2 = torch.full_like(k, 7.5), torch.full_like(k, 7.5)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    qlin.qlin_kv4_read(pool.c, i32(pos, dev), i32(seqs, dev), n, G, hd, k, v, status)
    qlin.qlin_kv4_read(pool.c, i32(pos, dev), i32(seqs, dev), n, G, hd, k2, None, None)
    want = np.zeros((2, n, G, hd))
    for s in range(S):
        a, b, there = pool.host(s)
        for i in np.nonzero((seqs == s) & (pos >= 0) & (pos < pool.rows))[0]:
            if there[pos[i]]:
                want[0, i], want[1, i] = a[pos[i]], b[pos[i]]
    assert int(status) == 1
    assert np.array_equal(k.cpu().numpy()[:n], want[0]) and np.array_equal(v.cpu().numpy()[:n], want[1])
    assert torch.equal(k, k2) and (k[n] == 7.5).all()
    qlin.qlin_kv4_read(pool.c, i32(pos, dev), i32(seqs, dev), n, G, hd, None, None, None)  # (checks the lanes only)


# ------------------------------------------------------------------ attention
class Call:
    def __init__(self, dev, n_lanes, H, n_kv, hd, seed=1, extra=3, scale=2.0):
        import torch

        from weight_streaming_gemv_gb300 import qlin

        g = torch.Generator(device=dev).manual_seed(seed)
        self.n, self.H, self.n_kv, self.hd, self.dev = n_lanes, H, n_kv, hd, dev
        self.q = torch.randn((n_lanes, H, hd), generator=g, device=dev) * scale
        self.out = torch.full((n_lanes + extra, H, hd), 7.5, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.bytes = qlin.qlin_attention_kv4_workspace_size(n_lanes, H, n_kv, hd)
        self.ws = torch.randint(0, 255, (self.bytes,), dtype=torch.uint8, device=dev)

    def go(self, pool, pos, seqs, window=0, sinks=0, stream=None):
        from weight_streaming_gemv_gb300 import qlin

        qlin.qlin_attention_kv4(self.q, pool.c, pos, seqs, self.n, self.H, self.n_kv, self.hd, window, sinks, self.out,
                                self.status, self.ws, self.bytes, stream)

    def result(self, status=0):
        import torch

        torch.cuda.synchronize()
        assert int(self.status.item()) == status
        got = self.out.cpu().numpy()
        assert (got[self.n:] == 7.5).all(), "rows behind the last lane were written"
        return got[: self.n]


def _lanes(pool, H, hd, pos, seqs, window, sinks, tensor):
    """the lanes so often that the call goes the way asked for: (positions, sequences)"""
    from weight_streaming_gemv_gb300 import qlin

    on = lambda n: qlin.qlin_attention_kv4_on_tensor_cores(pool.c, n, H, pool.n_kv, hd, window, sinks)
    if not tensor:
        if on(len(pos)):
            pytest.skip("too much work for the kernel of little work")
        return pos, seqs
    times = 1
    while not on(times * len(pos)):
        times *= 2
        if times * len(pos) > 4096:
            pytest.skip("too little work for the tensor cores")
    return np.tile(pos, times), np.tile(seqs, times)


def _check(pool, call, pos, seqs, window, sinks, status=0, lanes=None):
    got = call.result(status)
    q = call.q.cpu().numpy()
    host = {}
    for i in range(call.n) if lanes is None else lanes:
        s, p = int(seqs[i]), int(pos[i])
        if p < 0 or s < 0 or s >= pool.n_seqs or p >= pool.rows:
            assert (got[i] == 0).all(), i
            continue
        if s not in host:
            host[s] = pool.host(s)
        want = ref.attend(q[i], host[s][0], host[s][1], p, window, sinks, call.n_kv, host[s][2])
        e = np.linalg.norm(got[i] - want, axis=-1) / np.maximum(np.linalg.norm(want, axis=-1), 1e-30)
        assert np.isfinite(got[i]).all() and e.max() <= TOL, f"lane {i} (sequence {s}, position {p}): {e}"
    return got


SHAPES = [(4, 1, 256), (1, 1, 64), (8, 2, 128), (6, 3, 64), (16, 2, 256), (12, 1, 128), (40, 1, 64), (3, 3, 256)]


@pytest.mark.parametrize("H,G,hd", SHAPES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (100, 4), (64, 70)])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("tensor", [False, True])
def test_users(dev, H, G, hd, window, sinks, page, tensor):
    """single tokens of sequences of every length around the borders of pages and tiles"""
    pos = np.array([0, 1, 2, 15, 16, 17, 63, 64, 65, 126, 127, 128, 129, 255, 256, 257, 300, 383, 384, 511, 520, -1])
    pool = Pool(dev, len(pos), 521, G, hd, page)
    n = len(pos)
    pos, seqs = _lanes(pool, H, hd, pos, np.arange(n), window, sinks, tensor)
    call = Call(dev, len(pos), H, G, hd)
    call.go(pool, i32(pos, dev), i32(seqs, dev), window, sinks)
    _check(pool, call, pos, seqs, window, sinks, lanes=list(range(n)) + list(range(n, len(pos), 37)))


@pytest.mark.parametrize("H,G,hd", [(4, 1, 256), (8, 2, 128), (3, 3, 64), (5, 1, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
@pytest.mark.parametrize("order", ["along", "against", "mixed"])
@pytest.mark.parametrize("tensor", [False, True])
def test_chunks(dev, H, G, hd, window, sinks, order, tensor):
    """chunks of prompts, their lanes in any order, padding between them"""
    rng = np.random.default_rng(5)
    pool = Pool(dev, 3, 700, G, hd, 32)
    pos = np.concatenate((np.arange(150), np.arange(400, 500), np.full(20, -1), np.arange(690, 700)))
    seqs = np.concatenate((np.zeros(150, int), np.ones(100, int), np.zeros(20, int), np.full(10, 2)))
    idx = {"along": np.arange(len(pos)), "against": np.arange(len(pos))[::-1], "mixed": rng.permutation(len(pos))}[order]
    n = len(pos)
    pos, seqs = _lanes(pool, H, hd, pos[idx], seqs[idx], window, sinks, tensor)
    call = Call(dev, len(pos), H, G, hd)
    call.go(pool, i32(pos, dev), i32(seqs, dev), window, sinks)
    _check(pool, call, pos, seqs, window, sinks, lanes=list(range(0, n, 3)) + list(range(n, len(pos), 31)))


@pytest.mark.parametrize("H,G,hd,page,n,rows", [(4, 1, 256, 64, 3, 9000), (8, 2, 128, 128, 2, 20000), (2, 1, 64, 16, 5, 5000),
                                                (4, 1, 256, 64, 64, 1500), (16, 1, 128, 32, 1, 33000)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (4000, 4)])
def test_long(dev, H, G, hd, page, n, rows, window, sinks):
    rng = np.random.default_rng(n)
    pool = Pool(dev, n, rows, G, hd, page)
    pos = rng.integers(rows // 2, rows, n)
    pos[0] = rows - 1
    seqs = rng.permutation(n)
    call = Call(dev, n, H, G, hd)
    call.go(pool, i32(pos, dev), i32(seqs, dev), window, sinks)
    _check(pool, call, pos, seqs, window, sinks, lanes=range(0, n, max(1, n // 6)))


@pytest.mark.parametrize("times", [1, 200])
def test_pages_out_of_range(dev, times):
    """keys on missing pages count as not seen; entries that no lane needs are not looked at"""
    pool = Pool(dev, 4, 640, 2, 128, 32)
    t = pool.table.copy()
    t[0, 3] = -1           # inside what lane 0 sees
    t[1, :10] = -9         # before lane 1's window, but for its first tokens
    t[1, 19:] = 1 << 30    # behind its last page
    t[2, :] = -1           # everything
    t[3, 18] = pool.codes.shape[1]
    pool.set_table(t)
    pos, seqs = np.tile([500, 600, 300, 639], times), np.tile([0, 1, 2, 3], times)
    call = Call(dev, len(pos), 4, 2, 128)
    call.go(pool, i32(pos, dev), i32(seqs, dev), 200, 0)
    got = _check(pool, call, pos, seqs, 200, 0, status=1, lanes=[*range(4), *range(4 * times - 4, 4 * times)])
    assert (got[2::4] == 0).all()
    # the lanes that need no missing page raise nothing
    call.status.zero_()
    pos = np.where(seqs == 1, 600, -1)
    call.go(pool, i32(pos, dev), i32(seqs, dev), 200, 0)
    _check(pool, call, pos, seqs, 200, 0, status=0, lanes=range(4))


@pytest.mark.parametrize("times", [1, 100])
def test_lanes_out_of_range(dev, times):
    pool = Pool(dev, 2, 200, 1, 256, 64)
    pos = np.tile([10, pool.rows, 5, 7, -3, 199], times)
    seqs = np.tile([0, 0, 2, -1, 9, 1], times)
    call = Call(dev, len(pos), 4, 1, 256)
    call.go(pool, i32(pos, dev), i32(seqs, dev))
    _check(pool, call, pos, seqs, 0, 0, status=1)


def test_shared_pages(dev):
    """a prompt's pages stand in several sequences' tables"""
    pool = Pool(dev, 6, 400, 1, 256, 64)
    t = pool.table.copy()
    t[:, :4] = t[0, :4]
    pool.set_table(t)
    pos, seqs = np.array([399, 300, 256, 255, 100, 399]), np.arange(6)
    call = Call(dev, 6, 4, 1, 256)
    call.go(pool, i32(pos, dev), i32(seqs, dev))
    _check(pool, call, pos, seqs, 0, 0)


@pytest.mark.parametrize("tensor", [False, True])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("case", ["rising", "falling", "spikes", "large", "tiny", "flat"])
def test_scores_of_any_kind(dev, tensor, hd, case):
    """maxima that rise or fall along a sequence, single large scores, scores far apart and values near the least scale"""
    import torch

    from weight_streaming_gemv_gb300 import qlin

    H, G, n, rows = 4, 1, 3, 1500
    pool = Pool(dev, n, rows, G, hd, 64)
    call = Call(dev, n, H, G, hd)
    rng = np.random.default_rng(hd)
    x = rng.standard_normal((2, n * pool.per, G, 64, hd), np.float32)
    along = (np.arange(pool.rows) / pool.rows).astype(np.float32)
    q = call.q.cpu().numpy()
    if case in ("rising", "falling"):  # scores from -20 to 20 along a common direction of the queries
        q = np.broadcast_to(q[:1, :1], q.shape).copy()
        way = q[0, 0] / np.linalg.norm(q[0, 0]) ** 2 * np.sqrt(hd)
        t = (40 * along - 20) * (1 if case == "rising" else -1)
        x[0] = 0.1 * x[0] + t.reshape(1, -1, 1, 64, 1).repeat(n, 0).reshape(n * pool.per, 1, 64, 1) * way
    elif case == "spikes":
        x[0] *= np.where(rng.random(x[0].shape[:3]) < 0.01, 6, 0.2)[..., None]
    elif case == "large":
        q *= 300.0
    elif case == "tiny":
        x *= 3e-6
        q *= 1e4
    else:
        x[0] = 0.0
    call.q.copy_(torch.from_numpy(q))
    code, b = ref.quantise(x)
    own = pool.table.reshape(-1)
    pool.codes[:, own], pool.scales[:, own] = ref.pack(code), b
    pool.d_codes.copy_(torch.from_numpy(pool.codes)), pool.d_scales.copy_(torch.from_numpy(pool.scales))
    pos, seqs = _lanes(pool, H, hd, np.array([rows - 1, 700, 130]), np.arange(n), 0, 0, tensor)
    big = Call(dev, len(pos), H, G, hd)
    big.q.copy_(call.q.repeat(len(pos) // n, 1, 1))
    big.go(pool, i32(pos, dev), i32(seqs, dev))
    if case != "large":
        _check(pool, big, pos, seqs, 0, 0, lanes=list(range(n)) + [len(pos) - 1])
        return
    # scores of some hundreds: an error of 2^-22 of the score is an error of the weights; a factor 300 over the others
    got, k = big.result(), [pool.host(s) for s in range(n)]
    for i in range(n):
        want = ref.attend(q[i], k[i][0], k[i][1], int(pos[i]), 0, 0, G)
        e = np.linalg.norm(got[i] - want, axis=-1) / np.linalg.norm(want, axis=-1)
        assert e.max() <= 300 * TOL, e


@pytest.mark.parametrize("tensor", [False, True])
def test_queries_that_are_not_finite(dev, tensor):
    """a NaN or an infinity in a query stays with its lane and head's outputs; rows of zeros and of huge values are right"""
    pool = Pool(dev, 4, 900, 2, 128, 32)
    pos, seqs = _lanes(pool, 4, 128, np.array([899, 899, 500, 10]), np.arange(4), 0, 0, tensor)
    call = Call(dev, len(pos), 4, 2, 128)
    call.q[0, 1, 5] = float("nan")
    call.q[1, 3, 7] = float("inf")
    call.q[2, 0] = 0.0
    call.q[3, 2] = 1e-30
    call.go(pool, i32(pos, dev), i32(seqs, dev))
    got, q = call.result(), call.q.cpu().numpy()
    assert np.isnan(got[0, 1]).all() and np.isnan(got[1, 3]).any()
    for i in range(4):
        k, v, _ = pool.host(i)
        heads = [h for h in range(4) if np.isfinite(q[i, h]).all()]
        want = ref.attend(np.where(np.isfinite(q[i]), q[i], 0), k, v, int(pos[i]), 0, 0, 2)
        e = np.linalg.norm(got[i] - want, axis=-1) / np.linalg.norm(want, axis=-1)
        assert e[heads].max() <= TOL


@pytest.mark.parametrize("case", ["few", "users", "chunk", "long"])
def test_scores_past_the_types_range(dev, case):
    """finite queries whose scores fp32 does not hold: NaN for their lane and head, never a number; the others are right"""
    import torch

    from weight_streaming_gemv_gb300 import qlin

    H, G, hd = 4, 1, 256
    pool = Pool(dev, 3, 20000 if case == "long" else 700, G, hd, 64)
    pos, seqs = {"few": ([100, 699, 5], [0, 1, 2]), "users": (list(range(0, 700, 2)) * 3, [0] * 350 + [1] * 350 + [2] * 350),
                 "chunk": (list(range(100)) * 12, ([0] * 100 + [1] * 100) * 6), "long": ([19999, 15000, 700], [2, 0, 1])}[case]
    assert qlin.qlin_attention_kv4_on_tensor_cores(pool.c, len(pos), H, G, hd, 0, 0) == (case != "few")
    call = Call(dev, len(pos), H, G, hd)
    # along a key that the lane sees: its score is some 3e38 * 20, the others' may be anything
    hot = [i for i in range(len(pos)) if i % 7 == 0]
    host = [pool.host(s)[0] for s in range(3)]
    q = call.q.cpu().numpy()
    for i in hot:
        q[i, i % H] = np.sign(host[seqs[i]][pos[i] // 2, 0]) * 3e38
    call.q.copy_(torch.from_numpy(q))
    call.go(pool, i32(pos, dev), i32(seqs, dev))
    got = call.result()
    for i in hot:
        assert np.isnan(got[i, i % H]).all(), (i, pos[i])
    full = [pool.host(s) for s in range(3)]
    for i in list(range(min(24, len(pos)))) + list(range(0, len(pos), 61)):
        heads = [h for h in range(H) if i not in hot or h != i % H]
        want = ref.attend(np.where(np.abs(q[i]) > 1e30, 0, q[i]), full[seqs[i]][0], full[seqs[i]][1], pos[i], 0, 0, G)
        e = np.linalg.norm(got[i] - want, axis=-1) / np.linalg.norm(want, axis=-1)
        assert e[heads].max() <= TOL, (i, e)


@pytest.mark.parametrize("tensor", [False, True])
def test_same_bits_whatever_else_runs(dev, tensor):
    """the same call twice, in a graph replayed with other positions, and beside another call on another stream"""
    import torch

    H, G, hd, n = 8, 2, 128, 6
    pool = Pool(dev, n, 1200, G, hd, 16)
    pos, seqs = _lanes(pool, H, hd, np.array([1199, 5, 640, 700, -1, 127]), np.arange(n), 0, 0, tensor)
    d_pos, d_seqs = i32(pos, dev), i32(seqs, dev)
    call, other = Call(dev, len(pos), H, G, hd), Call(dev, len(pos), H, G, hd, seed=9)
    call.go(pool, d_pos, d_seqs)
    want = call.result().copy()
    other.go(pool, d_pos, d_seqs)
    want2 = other.result().copy()
    call.out.fill_(7.5)
    call.go(pool, d_pos, d_seqs)
    assert np.array_equal(call.result(), want)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    live = d_pos.clone()
    with torch.cuda.graph(g):
        call.go(pool, live, d_seqs)
    live.copy_(i32(np.where(pos > 0, pos // 2, pos), dev))
    g.replay()
    torch.cuda.synchronize()
    _check(pool, call, np.where(pos > 0, pos // 2, pos), seqs, 0, 0, lanes=range(n))
    live.copy_(d_pos)
    g.replay()
    assert np.array_equal(call.result(), want)
    torch.cuda.synchronize()
    for _ in range(10):
        call.go(pool, d_pos, d_seqs)
        other.go(pool, d_pos, d_seqs, stream=s)
    assert np.array_equal(call.result(), want) and np.array_equal(other.result(), want2)


@pytest.mark.parametrize("tensor", [False, True])
def test_pools_past_32_bits(dev, tensor):
    """pages whose codes lie more than 2^32 bytes into the pool"""
    import torch

    from weight_streaming_gemv_gb300 import qlin

    hd, G, page = 256, 1, 256
    n_pages = (1 << 32) // (page * hd // 2) + 40
    small = Pool(dev, 2, 1500, G, hd, page)
    own = torch.from_numpy(small.table.reshape(-1).astype(np.int64)).to(dev)
    codes = [torch.empty((n_pages, G, page, hd // 2), dtype=torch.uint8, device=dev) for _ in range(2)]
    scales = [torch.empty((n_pages, G, page, hd // 32), dtype=torch.uint8, device=dev) for _ in range(2)]
    at = torch.arange(n_pages - 1, n_pages - 1 - own.numel(), -1, device=dev)
    for i in (0, 1):
        codes[i][at], scales[i][at] = small.d_codes[i][own], small.d_scales[i][own]
    table = at.int().view(2, -1).contiguous()
    big = type("Big", (), dict(c=qlin.kv4_cache(codes[0], codes[1], scales[0], scales[1], table), n_kv=G))
    pos, seqs = _lanes(big, 4, hd, np.array([1499, 800]), np.arange(2), 0, 0, tensor)
    call = Call(dev, len(pos), 4, G, hd)
    call.go(big, i32(pos, dev), i32(seqs, dev))
    _check(small, call, pos, seqs, 0, 0, lanes=range(2))
    # appending there and reading back
    r = Rows(dev, 2, 4, G, hd)
    big.codes, big.scales = None, None
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    _append(big, r, np.array([1400, 3]), np.array([1, 0]), status=status)
    back = torch.empty((2, G, hd), device=dev)
    qlin.qlin_kv4_read(big.c, i32([1400, 3], dev), i32([1, 0], dev), 2, G, hd, back, None, status)
    code, b = ref.quantise(r.heads("k"))
    assert int(status) == 0
    assert np.array_equal(back.cpu().numpy(), ref.values(ref.pack(code), b).astype(np.float32))


def test_append_graph_and_streams(dev):
    """a captured append replayed with other rows and positions; two appends at once to different sequences"""
    import torch

    pool = Pool(dev, 2, 128, 2, 128, 32)
    rope = _rope(dev, 128, 128)
    from weight_streaming_gemv_gb300 import qlin

    rows = [Rows(dev, 5, 4, 2, 128, seed=s) for s in range(3)]
    live = rows[0].d.clone()
    pos, seqs = i32(np.arange(5), dev), i32(np.zeros(5), dev)
    out = torch.empty((5, 4, 128), device=dev)
    go = lambda x, p, s, o, stream=None: qlin.qlin_kv4_append(
        pool.c, rows[0].part("k", x), rows[0].part("v", x), x.stride(0), rows[0].part("q", x), x.stride(0), o, rope[0], rope[1],
        128, p, s, 5, 4, 2, 128, None, stream)
    go(live, pos, seqs, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go(live, pos, seqs, out)
    for k in (1, 2):
        live.copy_(rows[k].d), pos.copy_(i32(np.arange(5) + 7 * k, dev))
        pool.refresh()
        g.replay()
        torch.cuda.synchronize()
        codes, scales, q = _expect(pool, rows[k], np.arange(5) + 7 * k, np.zeros(5, int), rope, np.ones(5, bool))
        assert np.array_equal(pool.d_codes.cpu().numpy(), codes) and np.array_equal(pool.d_scales.cpu().numpy(), scales)
        assert np.array_equal(out.cpu().numpy(), q)
    s = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(out) for _ in range(2)]
    p2 = i32(np.arange(5) + 90, dev)
    torch.cuda.synchronize()
    for i in (0, 1):
        go(rows[i].d, p2, i32(np.full(5, i), dev), outs[i], s[i])
    torch.cuda.synchronize()
    for i in (0, 1):
        at = np.arange(5) + 90
        k, v, _ = (pool.refresh(), pool.host(i))[1]
        code, b = ref.quantise(rows[i].heads("v"))
        assert np.array_equal(v[at], ref.values(ref.pack(code), b))
