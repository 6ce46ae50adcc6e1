"""T158Decoder's beam search without a GPU: the library's calls are stand-ins
that note their arguments and report what a test has them report."""
import types

import pytest

torch = pytest.importorskip("torch")
qlin = pytest.importorskip("weight_streaming_gemv_gb300.qlin")
decoder = pytest.importorskip("weight_streaming_gemv_gb300.decoder")

N_SEQS, BEAMS, OWN, VOCAB, MAX_POS = 2, 3, 4, 11, 16


@pytest.fixture(scope="module", autouse=True)
def built():
    from weight_streaming_gemv_gb300 import build

    build.build()


@pytest.fixture
def search(monkeypatch):
    """a decoder on the CPU, its caches and the calls made; calls["reorder_bits"] is what the reordering reports"""
    calls = {"reorder_bits": 0, "reorder": 0, "steps": 0, "selects": 0}

    def reorder(cache, ss, ps, planes, row_bytes, max_rows, parents, n_rows, groups, beams, status_word=None, stream=None):
        calls["reorder"] += 1
        if status_word is not None:
            status_word |= calls["reorder_bits"]

    def select(*a):
        calls["selects"] += 1
        a[11].zero_(), a[10].zero_()  # tokens and parents

    def step(*a):
        calls["steps"] += 1

    monkeypatch.setattr(qlin, "qlin_beam_reorder", reorder)
    monkeypatch.setattr(qlin, "qlin_beam_select", select)
    monkeypatch.setattr(qlin, "decode_lanes_t158_prefix", step)
    monkeypatch.setattr(qlin, "decode_lanes_t158_status", lambda ws, stream=None: None)
    monkeypatch.setattr(qlin, "decode_lanes_t158_prefix_workspace_size", lambda m, n: 64)
    d = decoder.T158Decoder.__new__(decoder.T158Decoder)
    d.cfg = types.SimpleNamespace(n_layers=2, kv_dim=4, vocab=VOCAB, max_pos=MAX_POS)
    d.emb, d.model, d.n_seqs = torch.zeros(1), None, N_SEQS
    d.kv_lanes = torch.zeros((N_SEQS, 2, 2, MAX_POS, 4))
    d.prepare_beams(BEAMS, OWN)
    return d, calls


def test_the_reorderings_status_is_kept_and_raised(search):
    d, calls = search
    d.start_beams([3, 5], torch.zeros((N_SEQS, VOCAB)))
    d.check_beams_status()
    calls["reorder_bits"] = 2
    d.step_beams()
    calls["reorder_bits"] = 0
    d.step_beams()  # (what a call reported stays until it is asked for)
    with pytest.raises(qlin.QlinError) as e:
        d.check_beams_status()
    assert e.value.status == 5 and "qlin_beam_reorder" in str(e.value)
    d.check_beams_status()
    assert calls["reorder"] == 6 and calls["steps"] == 2 and calls["selects"] == 3


def test_steps_past_the_models_positions_are_refused(search):
    d, calls = search
    d.start_beams([3, MAX_POS - 2], torch.zeros((N_SEQS, VOCAB)))
    d.step_beams()  # positions 3 and 14: the first token's
    d.step_beams()  # 4 and 15, the last there is
    with pytest.raises(ValueError):
        d.step_beams()
    assert calls["steps"] == 2 and d.beam_t == 3
    d.start_beams(torch.tensor([3, 5]), torch.zeros((N_SEQS, VOCAB)))  # (another search: as long as its caches are)
    for _ in range(OWN):
        d.step_beams()
    with pytest.raises(ValueError):
        d.step_beams()
    for bad in ([3, MAX_POS + 1], [-1, 3]):
        with pytest.raises(ValueError):
            d.start_beams(bad, torch.zeros((N_SEQS, VOCAB)))
    d.start_beams([3, MAX_POS], torch.zeros((N_SEQS, VOCAB)))  # (the first tokens need no position behind the prompt)
    with pytest.raises(ValueError):
        d.step_beams()
