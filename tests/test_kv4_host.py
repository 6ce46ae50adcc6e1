"""Refusals of the paged 4-bit cache's operators (no GPU: every call fails, or sizes its workspace, on the host before
anything is launched), and the numpy form of the cache that the GPU tests go by."""
import ctypes

import numpy as np
import pytest

import kv4_ref as ref

qlin = pytest.importorskip("weight_streaming_gemv_gb300.qlin")


@pytest.fixture(scope="module", autouse=True)
def built():
    from weight_streaming_gemv_gb300 import build

    build.build()


def _kv(**kw):
    c = qlin.QlinKv4C()
    c.k, c.v, c.k_scale, c.v_scale, c.table = 4096, 8192, 16384, 32768, 64
    c.table_stride, c.n_pages, c.page_rows, c.n_seqs, c.max_pages = 8, 16, 64, 2, 8
    for n, v in kw.items():
        setattr(c, n, v)
    return c


BAD_KV = [
    (dict(k=None), 1), (dict(v=None), 1), (dict(k_scale=None), 1), (dict(v_scale=None), 1), (dict(table=None), 1),
    (dict(k=4112), 1), (dict(v=8208), 1), (dict(k_scale=16392), 1), (dict(v_scale=32776), 1), (dict(table=66), 1),
    (dict(n_pages=0), 1), (dict(n_seqs=0), 1), (dict(max_pages=0), 1), (dict(table_stride=7), 1),
    (dict(page_rows=8), 2), (dict(page_rows=48), 2), (dict(page_rows=512), 2), (dict(page_rows=0), 2),
    (dict(n_pages=1 << 30), 2), (dict(max_pages=1 << 28, table_stride=1 << 28), 2),
]


def _append(**kw):
    a = dict(kv=_kv(), k=16, v=32, kv_stride=256, q=48, q_stride=1024, q_out=64, cos=80, sin=96, rope_rows=128,
             positions=4, seqs=8, n_lanes=2, n_heads=4, n_kv=1, head_dim=256, status=None)
    a.update(kw)
    kv = ctypes.byref(a["kv"]) if a["kv"] is not None else None
    return qlin.lib().qlin_kv4_append(kv, a["k"], a["v"], a["kv_stride"], a["q"], a["q_stride"], a["q_out"], a["cos"],
                                      a["sin"], a["rope_rows"], a["positions"], a["seqs"], a["n_lanes"], a["n_heads"],
                                      a["n_kv"], a["head_dim"], a["status"], None)


@pytest.mark.parametrize("bad,status", [(dict(kv=_kv(**b)), s) for b, s in BAD_KV] + [
    (dict(kv=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(q=None), 1), (dict(q_out=None), 1),
    (dict(cos=None), 1), (dict(sin=None), 1), (dict(positions=None), 1), (dict(seqs=None), 1),
    (dict(k=20), 1), (dict(v=40), 1), (dict(q=52), 1), (dict(q_out=72), 1), (dict(cos=88), 1), (dict(sin=100), 1),
    (dict(positions=6), 1), (dict(seqs=9), 1), (dict(status=3), 1),
    (dict(n_lanes=0), 1), (dict(n_lanes=65537), 2), (dict(n_heads=0), 1), (dict(n_kv=0), 1), (dict(rope_rows=0), 1),
    (dict(kv_stride=252), 1), (dict(kv_stride=258), 1), (dict(q_stride=1020), 1), (dict(q_stride=1026), 1),
    (dict(q_out=48, q_stride=1028), 1), (dict(head_dim=32), 2), (dict(head_dim=96), 2), (dict(head_dim=512), 2),
])
def test_append_refuses(bad, status):
    assert _append(**bad) == status
    assert qlin.lib().qlin_last_error().decode().startswith("qlin_kv4_append")


def _read(**kw):
    a = dict(kv=_kv(), positions=4, seqs=8, n_lanes=2, n_kv=1, head_dim=256, k=16, v=32, status=None)
    a.update(kw)
    kv = ctypes.byref(a["kv"]) if a["kv"] is not None else None
    return qlin.lib().qlin_kv4_read(kv, a["positions"], a["seqs"], a["n_lanes"], a["n_kv"], a["head_dim"], a["k"], a["v"],
                                    a["status"], None)


@pytest.mark.parametrize("bad,status", [(dict(kv=_kv(**b)), s) for b, s in BAD_KV] + [
    (dict(kv=None), 1), (dict(positions=None), 1), (dict(seqs=None), 1), (dict(k=20), 1), (dict(v=40), 1),
    (dict(positions=6), 1), (dict(seqs=9), 1), (dict(status=3), 1), (dict(n_lanes=0), 1),
    (dict(n_lanes=(1 << 20) + 1), 2), (dict(n_kv=0), 1), (dict(head_dim=16), 2),
])
def test_read_refuses(bad, status):
    assert _read(**bad) == status
    assert qlin.lib().qlin_last_error().decode().startswith("qlin_kv4_read")


def _attend(**kw):
    a = dict(q=16, kv=_kv(), positions=32, seqs=48, n_lanes=2, n_heads=4, n_kv=1, head_dim=256, window=0, sinks=0,
             out=64, status=None, ws=80, bytes=1 << 40)
    a.update(kw)
    kv = ctypes.byref(a["kv"]) if a["kv"] is not None else None
    return qlin.lib().qlin_attention_kv4(a["q"], kv, a["positions"], a["seqs"], a["n_lanes"], a["n_heads"], a["n_kv"],
                                         a["head_dim"], a["window"], a["sinks"], a["out"], a["status"], a["ws"],
                                         a["bytes"], None)


@pytest.mark.parametrize("bad,status", [(dict(kv=_kv(**b)), s) for b, s in BAD_KV] + [
    (dict(q=None), 1), (dict(kv=None), 1), (dict(positions=None), 1), (dict(seqs=None), 1), (dict(out=None), 1),
    (dict(ws=None), 1), (dict(bytes=16), 1), (dict(q=24), 1), (dict(out=72), 1), (dict(ws=88), 1),
    (dict(positions=33), 1), (dict(seqs=49), 1), (dict(status=50), 1),
    (dict(n_lanes=0), 1), (dict(n_lanes=4097), 2), (dict(n_heads=3, n_kv=2), 1), (dict(n_kv=0), 1), (dict(n_heads=0), 1),
    (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(head_dim=32), 2), (dict(head_dim=512), 2),
])
def test_attention_refuses(bad, status):
    assert _attend(**bad) == status
    assert qlin.lib().qlin_last_error().decode().startswith("qlin_attention_kv4")


def test_which_way():
    """little work goes to the CUDA cores, more of any kind to the tensor cores"""
    on = qlin.qlin_attention_kv4_on_tensor_cores
    kv = _kv(max_pages=512, table_stride=512)
    assert not on(kv, 1, 4, 1, 256, 512, 4) and on(kv, 64, 4, 1, 256, 0, 0) and on(kv, 512, 4, 1, 256, 512, 0)
    with pytest.raises(qlin.QlinError):
        on(kv, 0, 4, 1, 256, 0, 0)
    with pytest.raises(qlin.QlinError):
        on(_kv(page_rows=24), 1, 4, 1, 256, 0, 0)


def test_workspace_sizes():
    size = qlin.qlin_attention_kv4_workspace_size
    assert size(1, 4, 1, 256) > 0 and size(4096, 32, 4, 128) > 0
    for bad in ((0, 4, 1, 256), (4097, 4, 1, 256), (1, 3, 2, 256), (1, 4, 0, 256), (1, 4, 1, 48), (1, 0, 1, 64)):
        assert size(*bad) == 0


def test_binding_checks_tensors():
    torch = pytest.importorskip("torch")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    k, sc, t = u8(3, 2, 16, 64), u8(3, 2, 16, 4), torch.zeros((5, 2), dtype=torch.int32)
    c = qlin.kv4_cache(k, k.clone(), sc, sc.clone(), t)
    assert (c.n_pages, c.page_rows, c.n_seqs, c.max_pages, c.table_stride) == (3, 16, 5, 2, 2)
    assert qlin.kv4_cache(k, k, sc, sc, torch.zeros((5, 8), dtype=torch.int32)[:, :2]).table_stride == 8
    for bad in ((k, k, sc, u8(3, 2, 16, 2), t), (k, u8(3, 2, 16, 32), sc, sc, t), (k, k, u8(3, 1, 16, 4), sc, t),
                (k, k, sc, sc, t.long()), (k, k, sc, sc, t[0]), (k[:, :, ::2], k, sc, sc, t), (k.float(), k, sc, sc, t),
                (k, k, sc, sc, torch.zeros((2, 5), dtype=torch.int32).t())):
        with pytest.raises(ValueError):
            qlin.kv4_cache(*bad)


def test_binding_checks_the_tables_rows():
    """rows of a table that lie in one another (an expanded one among them) would be read beyond its end"""
    torch = pytest.importorskip("torch")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    k, sc, flat = u8(3, 2, 16, 64), u8(3, 2, 16, 4), torch.zeros(64, dtype=torch.int32)
    for shape, stride in (((5, 8), (0, 1)), ((5, 8), (7, 1)), ((2, 8), (1, 1))):
        with pytest.raises(ValueError):
            qlin.kv4_cache(k, k, sc, sc, flat.as_strided(shape, stride))
    for shape, stride, want in (((1, 8), (0, 1), 8), ((1, 8), (3, 1), 8), ((5, 8), (8, 1), 8), ((5, 8), (11, 1), 11),
                                ((5, 1), (1, 0), 1)):
        assert qlin.kv4_cache(k, k, sc, sc, flat.as_strided(shape, stride)).table_stride == want


def test_binding_checks_devices():
    """the five tensors of a cache lie on one device"""
    torch = pytest.importorskip("torch")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    k, sc, t = u8(3, 2, 16, 64), u8(3, 2, 16, 4), torch.zeros((5, 2), dtype=torch.int32)
    for i in range(5):
        a = [k, k, sc, sc, t]
        a[i] = a[i].to("meta")
        with pytest.raises(ValueError):
            qlin.kv4_cache(*a)


def test_reference_format():
    """the numpy cache: every byte's scale, rounding, packing there and back"""
    assert SCALE_BITS(np.arange(256)).tolist() == ref.SCALES.tolist()
    x = np.zeros((1, 64), np.float32)
    x[0, :32] = np.linspace(-7, 7, 32)
    x[0, 40] = 7 * 1.0625  # between the scales 1 and 1.125
    code, b = ref.quantise(x)
    assert ref.SCALES[b].tolist() == [[1.0, 1.125]] and code[0, 40] == round(7 * 1.0625 / 1.125)
    assert code[0, 0] == -7 and code[0, 31] == 7 and (code[0, 32:40] == 0).all()
    rng = np.random.default_rng(0)
    c = rng.integers(-8, 8, (5, 128))
    s = rng.integers(0, 256, (5, 4)).astype(np.uint8)
    assert np.array_equal(ref.values(ref.pack(c), s), c * np.repeat(ref.SCALES[s], 32, -1))
    assert ref.pack(np.array([[-8, -8, 7] + [-8] * 5])).tolist() == [[0xF0, 0, 0, 0]]


def SCALE_BITS(b):
    """an fp32 number's exponent and first three bits of mantissa, less a bias"""
    return ((b + (106 << 3)) << 20).astype(np.uint32).view(np.float32).astype(np.float64)


def _sample(**kw):
    a = dict(logits=16, stride=100, u=4, t=8, k=12, p=20, m=24, rows=2, vocab=100, tokens=28, probs=32, kept=36)
    a.update(kw)
    return qlin.lib().qlin_sample(a["logits"], a["stride"], a["u"], a["t"], a["k"], a["p"], a["m"], a["rows"], a["vocab"],
                                  a["tokens"], a["probs"], a["kept"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(logits=None), 1), (dict(u=None), 1), (dict(tokens=None), 1), (dict(rows=0), 1), (dict(vocab=0), 1),
    (dict(stride=99), 1), (dict(rows=65536), 2), (dict(vocab=(1 << 24) + 1, stride=1 << 25), 2), (dict(stride=1 << 40), 2),
    (dict(logits=18), 1), (dict(u=5), 1), (dict(t=9), 1), (dict(k=13), 1), (dict(p=21), 1), (dict(m=26), 1),
    (dict(tokens=29), 1), (dict(probs=33), 1), (dict(kept=37), 1),
])
def test_sample_refuses(bad, status):
    assert _sample(**bad) == status
    assert qlin.lib().qlin_last_error().decode().startswith("qlin_sample")


def _step(n_layers, code_bytes, scale_bytes):
    """decode_lanes_t158_kv4 without its tokens, which it asks for last of all: 16 pages of 64 rows, 2 KV heads of 64"""
    m = qlin.T158ModelC()
    m.n_layers, m.dim, m.n_heads, m.n_kv_heads, m.head_dim, m.ffn, m.vocab, m.max_pos = n_layers, 64, 4, 2, 64, 64, 16, 128
    for j in range(len(m.w)):
        m.w[j], m.pitch[j] = 4096, 64
    for name in ("scales", "g_attn", "g_ffn", "g_final", "emb", "rope_cos", "rope_sin"):
        setattr(m, name, 4096)
    c = qlin.T158Kv4C()
    c.kv, c.code_bytes, c.scale_bytes = _kv(), code_bytes, scale_bytes
    st = qlin.lib().decode_lanes_t158_kv4(ctypes.byref(m), ctypes.byref(c), 1, None, 4, 8, None, 12, 16, 1 << 30, 1, None)
    return st, qlin.lib().qlin_last_error().decode()


def test_step_refuses_layers_in_one_another():
    codes, scales = 16 * 2 * 64 * 32, 16 * 2 * 64 * 2
    for layers, a, b in ((2, codes - 32, scales), (2, codes, scales - 16), (2, 0, 0), (7, codes, 0), (3, codes + 16, scales),
                         (3, codes, scales + 8), (1, -32, 0)):
        st, said = _step(layers, a, b)
        assert st == 1 and "code_bytes" in said, (layers, a, b, said)
    for layers, a, b in ((2, codes, scales), (1, 0, 0), (5, 2 * codes, 2 * scales), (2, codes + 32, scales + 16)):
        st, said = _step(layers, a, b)
        assert st == 1 and "null pointer" in said, (layers, a, b, said)


@pytest.mark.parametrize("name", ["attention_kv4.cu", "attention_lanes.cu"])
def test_every_bounded_wait_is_heard(name):
    """a wait that gives up has to be reported: no kernel drops the answer of one (but of those behind which it only
    leaves), and the status is raised whoever saw it"""
    import os
    import re

    here = os.path.dirname(os.path.abspath(qlin.__file__))
    with open(os.path.join(here, "csrc", name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    dropped = re.findall(r"(?:^|[;{})])\s*((?:al_wait|al_wait_at|kv_wait_all)\([^;]*\);)", text, re.M)
    assert not dropped, dropped
    # the weights' role, which may be the only one to see it, and the end of the kernel
    weights = text[text.rindex("setmaxnreg.inc"):]
    for m in re.finditer(r"al_wait\(&S\.pv_done", weights):
        assert "S.abort = 1" in weights[m.start(): m.end() + 150]
    assert re.search(r"__syncthreads\(\);\s*if \(tid == 0 && S\.abort\) raise_status\(A\.status, kStatusTimeout\);", weights)
