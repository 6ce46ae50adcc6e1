"""T158Decoder's pages and the arguments of its sampling, without a GPU: the library's calls are stand-ins."""
import types

import pytest

torch = pytest.importorskip("torch")
qlin = pytest.importorskip("weight_streaming_gemv_gb300.qlin")
decoder = pytest.importorskip("weight_streaming_gemv_gb300.decoder")


@pytest.fixture(scope="module", autouse=True)
def built():
    from weight_streaming_gemv_gb300 import build

    build.build()


@pytest.fixture
def paged(monkeypatch):
    monkeypatch.setattr(qlin, "decode_lanes_t158_kv4_workspace_size", lambda m, n: 64)
    d = decoder.T158Decoder.__new__(decoder.T158Decoder)
    d.cfg = types.SimpleNamespace(n_layers=3, n_kv_heads=2, head_dim=64, max_pos=100, vocab=11)
    d.emb, d.model = torch.zeros(1), None
    d.prepare_paged(n_seqs=3, n_pages=9, max_lanes=4, page_rows=16)
    return d


def test_layout(paged):
    c = paged.paged
    assert (c.kv.n_pages, c.kv.page_rows, c.kv.n_seqs, c.kv.max_pages) == (9, 16, 3, 7)
    assert c.code_bytes == 9 * 2 * 16 * 32 and c.scale_bytes == 9 * 2 * 16 * 2
    assert c.kv.v - c.kv.k == 3 * c.code_bytes and c.kv.v_scale - c.kv.k_scale == 3 * c.scale_bytes


def test_pages_are_given_and_taken_back(paged):
    d = paged
    d.paged_room(0, 17)
    d.paged_room(1, 64)
    d.paged_room(0, 17)  # (has them)
    d.paged_room(0, 32)
    t = d.page_table
    assert (t[0] >= 0).sum() == 2 and (t[1] >= 0).sum() == 4 and (t[2] == -1).all()
    used = t[t >= 0].tolist()
    assert len(set(used)) == 6 and len(d.pages_free) == 3 and not set(used) & set(d.pages_free)
    with pytest.raises(MemoryError):
        d.paged_room(2, 49)
    assert len(d.pages_free) == 3 and (t[2] == -1).all()
    d.paged_release(1)
    assert (t[1] == -1).all() and len(d.pages_free) == 7
    d.paged_room(2, 100)
    assert (t[2] >= 0).all() and not d.pages_free and set(t[t >= 0].tolist()) == set(range(9))
    for rows in (-1, 101):
        with pytest.raises(ValueError):
            d.paged_room(0, rows)


def test_sequences_out_of_range(paged):
    """a number below 0 is no sequence: it neither takes the last one's pages nor gives it any"""
    d = paged
    d.paged_room(2, 40)
    table, free = d.page_table.clone(), list(d.pages_free)
    for seq in (-1, -3, 3):
        with pytest.raises(IndexError):
            d.paged_room(seq, 100)
        with pytest.raises(IndexError):
            d.paged_release(seq)
    assert torch.equal(table, d.page_table) and free == d.pages_free and [len(p) for p in d.pages_of] == [0, 0, 3]


def test_sample_checks_its_tensors(paged, monkeypatch):
    calls = []
    monkeypatch.setattr(qlin, "qlin_sample", lambda *a: calls.append(a))
    f, i = lambda n: torch.zeros(n), lambda n: torch.zeros(n, dtype=torch.int32)
    lg = torch.zeros((4, 16))[:, :11]
    paged.sample(lg, f(4), i(4), temperature=f(4), top_k=i(4), top_p=f(4), min_p=f(4), probs=f(4), kept=i(4))
    assert calls[0][1] == 16 and calls[0][7:9] == (4, 11)
    paged.sample(lg[:1].expand(1, 11), f(1), i(1))
    assert calls[1][1] == 11
    for bad in (dict(u=f(3)), dict(u=f(4).double()), dict(tokens=f(4)), dict(top_k=f(4)), dict(kept=f(4)),
                dict(temperature=i(4)), dict(min_p=torch.zeros((4, 2))[:, 0]), dict(logits=lg.double()),
                dict(logits=torch.zeros((11, 4)).t())):
        a = dict(logits=lg, u=f(4), tokens=i(4))
        a.update(bad)
        with pytest.raises(ValueError):
            paged.sample(**a)
    assert len(calls) == 2


def test_sample_wants_the_decoders_device(paged, monkeypatch):
    monkeypatch.setattr(qlin, "qlin_sample", lambda *a: None)
    f, i = torch.zeros(4), torch.zeros(4, dtype=torch.int32)
    paged.sample(torch.zeros((4, 11)), f, i)
    paged.emb = torch.zeros(1, device="meta")  # the weights elsewhere
    with pytest.raises(ValueError):
        paged.sample(torch.zeros((4, 11)), f, i)
