"""Refusals of the operators for many sequences (no GPU: every call fails, or
sizes its workspace, on the host before anything is launched)."""
import ctypes

import pytest

qlin = pytest.importorskip("weight_streaming_gemv_gb300.qlin")


@pytest.fixture(scope="module", autouse=True)
def built():
    from weight_streaming_gemv_gb300 import build

    build.build()


def _kv(**kw):
    c = qlin.QlinKvC()
    c.k, c.v, c.seq_stride, c.row_stride, c.n_seqs, c.rows, c.type = 4096, 8192, 64 * 256, 256, 2, 64, 0
    for n, v in kw.items():
        setattr(c, n, v)
    return c


def _attend(prefix=None, **kw):
    a = dict(q=16, kv=_kv(), positions=32, seqs=48, n_lanes=2, n_heads=4, n_kv=1, head_dim=256, window=0, sinks=0,
             out=64, status=None, ws=80, bytes=1 << 40)
    a.update(kw)
    kv = ctypes.byref(a["kv"]) if a["kv"] is not None else None
    head = (a["q"],)
    if prefix is not None:
        head += (ctypes.byref(prefix), a.get("prefix_len", 96), a.get("prefix_of"))
    fn = qlin.lib().qlin_attention_lanes if prefix is None else qlin.lib().qlin_attention_prefix
    return fn(*head, kv, a["positions"], a["seqs"], a["n_lanes"], a["n_heads"], a["n_kv"], a["head_dim"], a["window"],
              a["sinks"], a["out"], a["status"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("prefix", [None, _kv(row_stride=512)])
@pytest.mark.parametrize("bad,status", [
    (dict(q=None), 1), (dict(kv=None), 1), (dict(positions=None), 1), (dict(seqs=None), 1), (dict(out=None), 1),
    (dict(ws=None), 1), (dict(bytes=16), 1), (dict(q=24), 1), (dict(out=72), 1), (dict(ws=88), 1),
    (dict(positions=33), 1), (dict(seqs=49), 1), (dict(status=50), 1),
    (dict(n_lanes=0), 1), (dict(n_lanes=4097), 2), (dict(n_heads=3, n_kv=2), 1), (dict(n_kv=0), 1),
    (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(head_dim=24), 2), (dict(head_dim=272, kv=_kv(row_stride=512)), 2),
    (dict(head_dim=8), 2), (dict(kv=_kv(k=None)), 1), (dict(kv=_kv(v=None)), 1), (dict(kv=_kv(k=8)), 1),
    (dict(kv=_kv(row_stride=252)), 1), (dict(kv=_kv(row_stride=258)), 1), (dict(kv=_kv(seq_stride=2)), 1),
    (dict(kv=_kv(seq_stride=-256)), 1), (dict(kv=_kv(n_seqs=0)), 1), (dict(kv=_kv(rows=0)), 1),
    (dict(kv=_kv(type=2)), 2), (dict(kv=_kv(row_stride=1 << 40)), 2),
    (dict(kv=_kv(type=1, row_stride=260)), 1),
])
def test_attention_refuses(prefix, bad, status):
    assert _attend(prefix, **bad) == status
    assert qlin.lib().qlin_last_error().decode().startswith("qlin_attention_")


def test_prefix_refuses():
    assert _attend(_kv(k=None)) == 1
    assert _attend(_kv(type=1)) == 1  # types differ
    assert _attend(_kv(), prefix_len=None) == 1
    assert _attend(_kv(), prefix_len=98) == 1
    assert _attend(_kv(), prefix_of=3) == 1
    assert "not 4-byte aligned" in qlin.lib().qlin_last_error().decode()


def test_attention_on_tensor_cores():
    f = lambda kv, *a, prefix=None: qlin.qlin_attention_on_tensor_cores(prefix, kv, *a)
    assert not f(_kv(), 2, 4, 1, 256, 0, 0)
    assert not f(_kv(rows=30000), 2, 4, 1, 256, 500, 4)
    for t in (0, 1):  # (more rows than the kernel for little work takes, whatever the lanes)
        assert f(_kv(rows=66000, type=t), 1, 1, 1, 16, 0, 0)
        assert f(_kv(rows=8, type=t), 1, 1, 1, 16, 0, 0, prefix=_kv(rows=66000, type=t))
        assert f(_kv(rows=4096, n_seqs=64, type=t), 4096, 4, 1, 256, 0, 0)
    for a, status in [((0, 4, 1, 256, 0, 0), 1), ((4097, 4, 1, 256, 0, 0), 2), ((2, 3, 2, 64, 0, 0), 1),
                      ((2, 4, 1, 24, 0, 0), 2), ((2, 4, 1, 256, -1, 0), 1), ((2, 4, 1, 256, 0, -1), 1)]:
        with pytest.raises(qlin.QlinError) as e:
            f(_kv(), *a)
        assert e.value.status == status
    for kv, prefix in ((_kv(k=None), None), (_kv(rows=0), None), (_kv(), _kv(row_stride=252)), (_kv(), _kv(type=1))):
        with pytest.raises(qlin.QlinError) as e:
            f(kv, 2, 4, 1, 256, 0, 0, prefix=prefix)
        assert e.value.status == 1
    assert qlin.lib().qlin_attention_on_tensor_cores(None, None, 2, 4, 1, 256, 0, 0) == -1


def test_attention_workspace_size():
    f = qlin.qlin_attention_lanes_workspace_size
    assert f(1, 4, 1, 256) > 0 and f(4096, 4, 1, 256) >= f(64, 4, 1, 256) >= f(1, 4, 1, 256)
    for bad in [(0, 4, 1, 256), (4097, 4, 1, 256), (1, 3, 2, 256), (1, 4, 0, 256), (1, 4, 1, 8), (1, 4, 1, 264)]:
        assert f(*bad) == 0


def _select(**kw):
    a = dict(logits=16, row_stride=1000, scores=32, finished=None, eos=0, n_groups=2, beams=4, vocab=1000, n_out=4,
             out_scores=48, parents=64, tokens=80, ws=96, bytes=1 << 30)
    a.update(kw)
    return qlin.lib().qlin_beam_select(*a.values(), None)


@pytest.mark.parametrize("bad,status", [
    (dict(logits=None), 1), (dict(scores=None), 1), (dict(out_scores=None), 1), (dict(parents=None), 1),
    (dict(tokens=None), 1), (dict(ws=None), 1), (dict(bytes=100), 1), (dict(row_stride=999), 1), (dict(beams=0), 1),
    (dict(beams=65), 2), (dict(n_out=129), 2), (dict(n_out=0), 1), (dict(vocab=0), 1), (dict(n_groups=0), 1),
    (dict(vocab=(1 << 24) + 1, row_stride=1 << 25), 2), (dict(n_groups=1 << 15), 2), (dict(logits=18), 1),
    (dict(scores=33), 1), (dict(ws=100), 1), (dict(finished=8, eos=1000), 1), (dict(finished=8, eos=-1), 1),
])
def test_select_refuses(bad, status):
    assert _select(**bad) == status
    assert qlin.lib().qlin_last_error().decode().startswith("qlin_beam_select")


def test_select_workspace_size():
    f = qlin.qlin_beam_select_workspace_size
    assert f(1, 4, 262144, 4) > 0
    assert f(1, 65, 1000, 4) == f(1, 4, 1000, 129) == f(0, 4, 1000, 4) == f(1, 4, (1 << 24) + 1, 4) == 0


def _reorder(**kw):
    a = dict(cache=4096, seq_stride=52 * 64 * 1024, plane_stride=64 * 1024, n_planes=52, row_bytes=1024, max_rows=64,
             parents=16, n_rows=None, n_groups=2, beams=4, status=None)
    a.update(kw)
    return qlin.lib().qlin_beam_reorder(*a.values(), None)


@pytest.mark.parametrize("bad,status", [
    (dict(cache=None), 1), (dict(parents=None), 1), (dict(cache=8), 1), (dict(row_bytes=1000), 1), (dict(row_bytes=0), 1),
    (dict(seq_stride=52 * 64 * 1024 + 8), 1), (dict(plane_stride=64 * 1024 + 8), 1), (dict(n_planes=0), 1),
    (dict(max_rows=0), 1), (dict(n_groups=0), 1), (dict(beams=0), 1), (dict(beams=65), 2), (dict(parents=18), 1),
    (dict(n_rows=18), 1), (dict(status=2), 1),
    (dict(plane_stride=63 * 1024), 1),          # planes overlap
    (dict(seq_stride=51 * 64 * 1024), 1),       # sequences overlap
    (dict(seq_stride=-16), 1), (dict(row_bytes=1 << 41), 1),
    (dict(max_rows=2 ** 31 - 1), 1),            # rows past the plane's stride
])
def test_reorder_refuses(bad, status):
    assert _reorder(**bad) == status
    assert qlin.lib().qlin_last_error().decode().startswith("qlin_beam_reorder")


def test_kv_cache_describes_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros((3, 5, 2, 7, 32), dtype=torch.bfloat16)
    c = qlin.kv_cache(x[:, 4, 0], x[:, 4, 1])
    assert (c.seq_stride, c.row_stride, c.n_seqs, c.rows, c.type) == (5 * 2 * 7 * 32, 32, 3, 7, qlin.KV_BF16)
    assert c.v - c.k == 7 * 32 * 2
    with pytest.raises(ValueError):
        qlin.kv_cache(x[:, 0, 0], x[:, 0, 1].float())
    with pytest.raises(ValueError):
        qlin.kv_cache(x[0, 0, 0], x[0, 0, 1])
    with pytest.raises(ValueError):
        qlin.kv_cache(x[:, 0, 0].half(), x[:, 0, 1].half())


def test_prefix_step_refuses():
    import ctypes as ct

    L, m, n = qlin.lib(), qlin.T158ModelC(), ct.c_size_t()
    assert L.decode_lanes_t158_prefix_workspace_size(ct.byref(m), 4, ct.byref(n)) == 1  # an empty model
    m.n_layers, m.dim, m.n_heads, m.n_kv_heads, m.head_dim = 1, 64, 2, 1, 32
    m.ffn, m.vocab, m.max_pos = 96, 100, 64
    for j in range(qlin.T158_NMAT):
        m.w[j], m.pitch[j] = 4096, 32
    for f in ("scales", "g_attn", "g_ffn", "g_final", "emb", "rope_cos", "rope_sin"):
        setattr(m, f, 4096)
    assert L.decode_lanes_t158_prefix_workspace_size(ct.byref(m), 4, ct.byref(n)) == 0 and n.value > 0
    assert L.decode_lanes_t158_prefix_workspace_size(ct.byref(m), 0, ct.byref(n)) == 1
    p = qlin.T158PromptsC()

    def call(**kw):
        for k, v in dict(kv=4096, len=4096, n_prompts=1, rows=64).items():
            setattr(p, k, kw.pop(k, v))
        a = dict(of=None, kvs=4096, own=8, n_seqs=2, n_lanes=2, tok=16, pos=16, seq=16, lg=None, nx=16, ws=4096,
                 wsb=n.value, mx=4)
        a.update(kw)
        return L.decode_lanes_t158_prefix(ct.byref(m), ct.byref(p), *a.values(), None)

    assert call(kv=None) == 1 and call(len=None) == 1 and call(n_prompts=0) == 1 and call(rows=0) == 1
    assert call(own=0) == 1 and call(kv=8) == 1 and call(len=6) == 1 and call(of=2) == 1 and call(kvs=None) == 1
    assert call(rows=2 ** 30 + 1) == 2 and call(own=2 ** 30 + 1) == 2  # (more than the attention takes)
    assert call(wsb=64) == 1 and call(n_lanes=5) == 1 and call(ws=8) == 1
    assert "decode_lanes_t158" in L.qlin_last_error().decode()
