"""A beam search over shared prompts: T158Decoder.step_beams runs the lanes'
step behind prompts kept once, the selection and the reordering together.

Every step is checked from the state before it: the logits of every beam
against the oracle run over the beam's whole token history in one cache, the
selection against the definition in 64 bits on the GPU's own logits, the
histories and caches against the parents.

Tolerance of the logits.  The attention over a shared prompt is the oracle's
to fp32 accuracy (1e-6), not bit for bit, so an int8 activation code can fall
to the other side of a half: at 127 codes a change of 1e-6 does that to about
one code in ten thousand, a few per step here.  One flipped code moves an
output by absmax / 127 of one of K >= 32 inputs, (3 / 127) / sqrt(K) = 4e-3 of
the outputs' size; 2e-2 allows several.  A row too many or too few in one
beam's attention, or another beam's cache, moves its logits by tenths."""
import numpy as np
import pytest

import oracle
import synth
from gpu_util import device, host, max_abs_rel
from test_gpu_beam import _ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return device()


def _oracle_logits(orc, cfg, tokens):
    kvs = np.zeros((1, cfg.n_layers, 2, cfg.max_pos, cfg.kv_dim), np.float32)
    n = len(tokens)
    _, lg = orc.lanes(kvs, np.int32(tokens), np.arange(n, dtype=np.int32), np.zeros(n, np.int32), want_logits=True)
    return lg[-1], kvs[0]


SHAPES = [dict(synth.TINY),
          dict(n_layers=2, dim=128, n_heads=4, n_kv_heads=2, head_dim=64, ffn=160, vocab=512, eps=1e-6, rope_base=10000.0)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("lens,beams,eos", [([9], 1, None), ([9], 4, None), ([7, 150], 3, 5), ([33, 1, 12], 5, None)])
def test_beam_search(dev, shape, lens, beams, eos):
    import torch

    from weight_streaming_gemv_gb300.decoder import T158Decoder

    cfg = synth.DecoderConfig(max_pos=192, **shape)
    w = synth.decoder_weights(cfg, seed=5)
    gpu, orc = T158Decoder(cfg, w, device=dev), oracle.Decoder(cfg, w)
    G, B, own, V = len(lens), beams, 6, cfg.vocab
    prompts = [synth.prompt_ids(20 + g, n, V) for g, n in enumerate(lens)]
    gpu.prepare_lanes(n_seqs=G, max_lanes=max(lens))
    last = torch.empty((G, V), device=dev)
    for g, p in enumerate(prompts):  # the prompts, read in as lanes
        n = len(p)
        gpu.lane_tokens[:n].copy_(torch.as_tensor(np.int32(p)))
        gpu.lane_pos[:n].copy_(torch.arange(n, dtype=torch.int32))
        gpu.lane_seq[:n].fill_(g)
        lg = torch.empty((n, V), device=dev)
        gpu.step_lanes(n, logits=lg)
        last[g] = lg[-1]
    gpu.check_lanes_status()
    gpu.prepare_beams(B, own, eos)
    gpu.start_beams(lens, last)
    hist = [[list(prompts[g]) for _ in range(B)] for g in range(G)]
    scores = np.full((G, B), -np.inf, np.float32)
    scores[:, 0] = 0
    done = np.zeros((G, B), np.uint8)
    for t in range(own + 1):
        if t > 0:
            gpu.step_beams()
        gpu.check_beams_status()
        lg = host(gpu.beam_logits).reshape(G, B, V)
        for g in range(G):
            for b in range(B):
                if scores[g, b] > -np.inf and not done[g, b]:
                    assert max_abs_rel(lg[g, b], _oracle_logits(orc, cfg, hist[g][b])[0]) <= 2e-2, (t, g, b)
        S, P, T, gap = _ref(lg, scores, B, done if eos is not None else None, eos or 0)
        assert gap > 2e-8
        got_t, got_s = gpu.beam_results()
        got_t, got_s = host(got_t), host(got_s)
        np.testing.assert_array_equal(host(gpu.beam_parents), P)
        np.testing.assert_array_equal(got_t[:, :, -1], np.maximum(T, 0))
        assert (np.abs(got_s - S) <= 1e-6 + np.abs(S) * 2.0 ** -23).all()
        hist = [[hist[g][P[g, b]] + [int(T[g, b])] for b in range(B)] for g in range(G)]
        done = np.take_along_axis(done, np.maximum(P, 0), 1) | (T == (eos if eos is not None else -2))
        scores = got_s.copy()
        for g in range(G):
            for b in range(B):
                assert list(got_t[g, b]) == hist[g][b][lens[g]:]
    # the caches followed: the last beams' rows are those of their histories (k of the first layer depends on the
    # token and its position alone, up to nothing but the rotation's rounding)
    kv = host(gpu.kv_beams)
    for g in range(G):
        for b in range(B):
            ref = _oracle_logits(orc, cfg, hist[g][b][:-1])[1]
            np.testing.assert_allclose(kv[g * B + b, 0, 0, :own], ref[0, 0, lens[g]:lens[g] + own], rtol=1e-5, atol=1e-6)


def test_prefix_step_matches_whole_caches(dev):
    # the same lanes with the prompt in every lane's own cache, and behind a prompt kept once
    import torch

    from weight_streaming_gemv_gb300 import qlin
    from weight_streaming_gemv_gb300.decoder import T158Decoder

    cfg = synth.DecoderConfig(max_pos=400, n_layers=3, dim=256, n_heads=4, n_kv_heads=1, head_dim=256, ffn=320, vocab=700,
                              eps=1e-6, rope_base=10000.0)
    w = synth.decoder_weights(cfg, seed=7)
    gpu = T158Decoder(cfg, w, device=dev)
    n, P, own = 20, 300, 16
    gpu.prepare_lanes(n_seqs=n, max_lanes=n)
    gpu.kv_lanes.copy_((torch.randn(gpu.kv_lanes.shape[1:], device=dev) * 0.5).expand_as(gpu.kv_lanes))
    pos = np.int32([P + i % 3 for i in range(n)])
    gpu.lane_tokens.copy_(torch.as_tensor(np.int32(np.arange(n) * 31 % 700)))
    gpu.lane_pos.copy_(torch.as_tensor(pos))
    gpu.lane_seq.copy_(torch.arange(n, dtype=torch.int32))
    prompt = gpu.kv_lanes[0].clone()
    a, b = (torch.empty((n, cfg.vocab), device=dev) for _ in range(2))
    own_kv = torch.zeros((n, cfg.n_layers, 2, own, cfg.kv_dim), device=dev)
    own_kv[:, :, :, :3] = gpu.kv_lanes[:, :, :, P:P + 3]
    gpu.step_lanes(n, logits=a)
    gpu.check_lanes_status()
    nb = qlin.decode_lanes_t158_prefix_workspace_size(gpu.model, n)
    ws = torch.zeros(nb, dtype=torch.uint8, device=dev)
    length = torch.tensor([P], dtype=torch.int32, device=dev)
    pr = qlin.T158PromptsC()
    pr.kv, pr.len, pr.n_prompts, pr.rows = prompt.data_ptr(), length.data_ptr(), 1, cfg.max_pos
    before = prompt.clone()
    qlin.decode_lanes_t158_prefix(gpu.model, pr, None, own_kv, own, n, n, gpu.lane_tokens, gpu.lane_pos, gpu.lane_seq, b,
                                  gpu.lane_next, ws, nb, n)
    qlin.decode_lanes_t158_status(ws)
    assert max_abs_rel(host(b), host(a)) <= 2e-2
    assert torch.equal(prompt, before)
    # a lane that would write into the prompt, one behind its rows, one of no prompt: refused by status, nothing written
    for bad_pos, bad_pre in ((P - 1, 0), (P + own, 0), (P, 1), (P, -1)):
        gpu.lane_pos[3] = bad_pos
        of = torch.zeros(n, dtype=torch.int32, device=dev)
        of[3] = bad_pre
        keep = own_kv[3].clone()
        qlin.decode_lanes_t158_prefix(gpu.model, pr, of, own_kv, own, n, n, gpu.lane_tokens, gpu.lane_pos, gpu.lane_seq,
                                      b, gpu.lane_next, ws, nb, n)
        with pytest.raises(qlin.QlinError) as e:
            qlin.decode_lanes_t158_status(ws)
        assert e.value.status == 1
        assert torch.equal(own_kv[3], keep) and torch.equal(prompt, before)


def test_own_rows_run_out(dev):
    from weight_streaming_gemv_gb300.decoder import T158Decoder
    import torch

    cfg = synth.DecoderConfig(max_pos=32, **synth.TINY)
    gpu = T158Decoder(cfg, synth.decoder_weights(cfg, seed=5), device=dev)
    gpu.prepare_lanes(n_seqs=1, max_lanes=2)
    gpu.prepare_beams(2, 2)
    gpu.start_beams([4], torch.randn((1, cfg.vocab), device=dev))
    gpu.step_beams()
    gpu.step_beams()
    with pytest.raises(ValueError):
        gpu.step_beams()
