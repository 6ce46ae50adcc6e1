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
