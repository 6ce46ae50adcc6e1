"""The lanes' step over a paged cache of 4 bits a value, and answers drawn from it: T158Decoder.prepare_paged, paged_room,
step_paged and sample together.

The step is checked against the same step put together from the library's single calls, layer by layer.  Every one of them
has a test of its own, their order of operations is the step's, and the same kernels see the same numbers: the cache's
bytes, the logits and the tokens are equal bit for bit."""
import numpy as np
import pytest

import sample_ref
import synth
from gpu_util import device

pytestmark = pytest.mark.gpu

SHAPE = dict(n_layers=2, dim=128, n_heads=4, n_kv_heads=2, head_dim=64, ffn=160, vocab=512, eps=1e-6, rope_base=10000.0)


@pytest.fixture(scope="module")
def dev():
    return device()


def _decoder(dev, **kw):
    from weight_streaming_gemv_gb300.decoder import T158Decoder

    cfg = synth.DecoderConfig(max_pos=192, **dict(SHAPE, **kw))
    return cfg, T158Decoder(cfg, synth.decoder_weights(cfg, seed=5), device=dev)


def _by_calls(d, codes, scales, tokens, pos, seqs):
    """one step over lanes from single calls; returns the logits and greedy tokens"""
    import torch

    from weight_streaming_gemv_gb300 import qlin
    from weight_streaming_gemv_gb300.decoder import MATRIX_ORDER

    cfg, dev, M = d.cfg, d.emb.device, tokens.numel()
    dims = {name: (n, k) for name, n, k in cfg.matrices()}
    sc = d.scales.cpu().numpy()

    def lin(l, name, x):
        j = MATRIX_ORDER.index(name)
        n, k = dims[name]
        xq, xs, y = torch.empty((M, k), dtype=torch.int8, device=dev), torch.empty(M, device=dev), torch.empty((M, n), device=dev)
        qlin.qlin_quant_i8(x, xq, xs, M, k)
        ws = torch.empty(max(1, qlin.qlin_t158_i8_workspace_size(M, k)), dtype=torch.uint8, device=dev)
        qlin.qlin_t158_i8_ws(xq, xs, d.w[j][l], d.pitch[j], sc[l, j], y, None, M, n, k, ws, ws.numel())
        return y

    def norm(x, g):
        o = torch.empty_like(x)
        qlin.qlin_rmsnorm(x, g, o, M, cfg.dim, cfg.eps)
        return o

    h = (d.emb[tokens.long()].int() << 16).view(torch.float32)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    H, G, hd = cfg.n_heads, cfg.n_kv_heads, cfg.head_dim
    n_ws = qlin.qlin_attention_kv4_workspace_size(M, H, G, hd)
    ws = torch.empty(n_ws, dtype=torch.uint8, device=dev)
    for l in range(cfg.n_layers):
        x = norm(h, d.g_attn[l])
        q, k, v = (lin(l, n, x) for n in ("wq", "wk", "wv"))
        kv = qlin.kv4_cache(codes[0, l], codes[1, l], scales[0, l], scales[1, l], d.page_table)
        qlin.qlin_kv4_append(kv, k, v, G * hd, q, H * hd, q, d.rope_cos, d.rope_sin, cfg.max_pos, pos, seqs, M, H, G, hd,
                             status)
        att = torch.empty_like(q)
        qlin.qlin_attention_kv4(q, kv, pos, seqs, M, H, G, hd, 0, 0, att, status, ws, n_ws)
        h = h + lin(l, "wo", att)
        x = norm(h, d.g_ffn[l])
        g, u = lin(l, "wg", x), lin(l, "wu", x)
        a = torch.empty_like(g)
        qlin.qlin_geglu(g, u, a, g.numel())
        h = h + lin(l, "wd", a)
    x = norm(h, d.g_final)
    lg = torch.empty((M, cfg.vocab), device=dev)
    nxt = torch.empty(M, dtype=torch.int32, device=dev)
    n_lm = qlin.qlin_lm_head_lanes_workspace_size(cfg.vocab, cfg.dim)
    lm = torch.zeros(n_lm, dtype=torch.uint8, device=dev)
    qlin.qlin_lm_head_lanes(d.emb, x, cfg.vocab, cfg.dim, M, lg, nxt, lm, n_lm)
    assert int(status) == 0
    return lg, nxt


@pytest.mark.parametrize("hd,G", [(64, 2), (128, 1), (256, 1)])
@pytest.mark.parametrize("page", [16, 64])
def test_step_is_its_calls(dev, hd, G, page):
    """prompts of three sequences as chunks, then single tokens of them, one of them out of the pool in between"""
    import torch

    cfg, d = _decoder(dev, head_dim=hd, n_kv_heads=G)
    d.prepare_paged(n_seqs=3, n_pages=3 * (-(-192 // page)), max_lanes=64, page_rows=page)
    codes, scales = d.page_codes.clone(), d.page_scales.clone()
    rng = np.random.default_rng(hd)
    lens = [37, 1, 20]

    def step(tokens, pos, seqs):
        n = len(tokens)
        for t, x in ((d.paged_tokens, tokens), (d.paged_pos, pos), (d.paged_seq, seqs)):
            t[:n].copy_(torch.as_tensor(np.int32(x)))
        lg = torch.empty((n, cfg.vocab), device=dev)
        d.step_paged(n, logits=lg)
        d.check_paged_status()
        want, nxt = _by_calls(d, codes, scales, d.paged_tokens[:n], d.paged_pos[:n], d.paged_seq[:n])
        assert torch.equal(codes, d.page_codes) and torch.equal(scales, d.page_scales)
        assert torch.equal(lg, want) and torch.equal(d.paged_next[:n], nxt)

    for s, n in enumerate(lens):
        d.paged_room(s, n)
    step(rng.integers(0, cfg.vocab, sum(lens)), np.concatenate([np.arange(n) for n in lens]), np.repeat(np.arange(3), lens))
    for k in range(3):
        for s in range(3):
            d.paged_room(s, lens[s] + 1)
        step(rng.integers(0, cfg.vocab, 3), lens, [0, 1, 2])
        lens = [n + 1 for n in lens]
        if k == 1:
            d.paged_release(1)
            d.paged_room(1, 1)
            lens[1] = 0


@pytest.mark.parametrize("hd,G,page", [(256, 1, 64), (128, 2, 256), (64, 4, 16)])
def test_step_on_the_tensor_cores(dev, hd, G, page):
    """steps whose attention goes to the tensor cores: chunks of three prompts in more than 64 lanes, then 70 users' single
    tokens, over two layers' pools"""
    import torch

    from weight_streaming_gemv_gb300 import qlin
    from weight_streaming_gemv_gb300.decoder import T158Decoder

    cfg = synth.DecoderConfig(max_pos=4096, **dict(SHAPE, head_dim=hd, n_kv_heads=G))
    d = T158Decoder(cfg, synth.decoder_weights(cfg, seed=5), device=dev)
    S = 70
    pages = 3 * (-(-600 // page)) + S * (-(-40 // page))
    d.prepare_paged(n_seqs=S, n_pages=pages, max_lanes=640, page_rows=page)
    codes, scales = d.page_codes.clone(), d.page_scales.clone()
    rng = np.random.default_rng(hd)
    lens = np.zeros(S, int)

    def step(counts):
        """counts[s] more tokens of every sequence"""
        for s in np.nonzero(counts)[0]:
            d.paged_room(int(s), int(lens[s] + counts[s]))
        pos = np.concatenate([lens[s] + np.arange(counts[s]) for s in range(S)])
        seqs = np.repeat(np.arange(S), counts)
        n = len(pos)
        assert qlin.qlin_attention_kv4_on_tensor_cores(d.paged.kv, n, 4, G, hd, 0, 0)
        for t, x in ((d.paged_tokens, rng.integers(0, cfg.vocab, n)), (d.paged_pos, pos), (d.paged_seq, seqs)):
            t[:n].copy_(torch.as_tensor(x.astype(np.int32)))
        lg = torch.empty((n, cfg.vocab), device=dev)
        d.step_paged(n, logits=lg)
        d.check_paged_status()
        want, nxt = _by_calls(d, codes, scales, d.paged_tokens[:n], d.paged_pos[:n], d.paged_seq[:n])
        assert torch.equal(codes, d.page_codes) and torch.equal(scales, d.page_scales)
        assert torch.equal(lg, want) and torch.equal(d.paged_next[:n], nxt)
        lens[:] = lens + counts

    first = np.zeros(S, int)
    first[[0, 33, 69]] = 300, 1, 137
    step(first)
    step(np.where(np.arange(S) == 33, 400, rng.integers(0, 4, S)))
    for _ in range(2):
        step(np.ones(S, int))


def test_status_and_padding(dev):
    import torch

    from weight_streaming_gemv_gb300 import qlin

    cfg, d = _decoder(dev)
    d.prepare_paged(n_seqs=2, n_pages=4, max_lanes=8, page_rows=16)
    d.paged_room(0, 16)
    before = d.page_codes.clone()
    d.paged_pos[:2].copy_(torch.tensor([-1, -1]))
    d.step_paged(2)
    d.check_paged_status()
    assert torch.equal(before, d.page_codes)
    for pos, seq in ((16, 0), (0, 1), (0, 5), (192, 0)):  # no page, no page, no sequence, no position
        d.paged_pos[:2].copy_(torch.tensor([pos, -1])), d.paged_seq[:2].copy_(torch.tensor([seq, 0]))
        d.step_paged(2)
        with pytest.raises(qlin.QlinError):
            d.check_paged_status()
        d.check_paged_status()
    assert torch.equal(before, d.page_codes)


def test_drawn_answers(dev):
    """answers to two prompts, drawn with settings of their own, step by step in a graph: every token is what the
    definition draws from the step's logits"""
    import torch

    cfg, d = _decoder(dev)
    d.prepare_paged(n_seqs=2, n_pages=12, max_lanes=32, page_rows=32)
    rng = np.random.default_rng(3)
    lens = [20, 11]
    for s, n in enumerate(lens):
        d.paged_room(s, n + 9)
    n = sum(lens)
    d.paged_tokens[:n].copy_(torch.as_tensor(rng.integers(0, cfg.vocab, n).astype(np.int32)))
    d.paged_pos[:n].copy_(torch.as_tensor(np.concatenate([np.arange(x) for x in lens]).astype(np.int32)))
    d.paged_seq[:n].copy_(torch.as_tensor(np.repeat(np.arange(2), lens).astype(np.int32)))
    lg = torch.empty((n, cfg.vocab), device=dev)
    d.step_paged(n, logits=lg)
    d.check_paged_status()
    last = lg[[lens[0] - 1, n - 1]].contiguous()
    up = lambda a, t=np.float32: torch.as_tensor(np.asarray(a, t)).to(dev)
    settings = dict(temperature=up([0.7, 1.3]), top_k=up([40, 0], np.int32), top_p=up([0.9, 0.8]), min_p=up([0.0, 0.01]))
    u, probs, kept = up([0, 0]), up([0, 0]), up([0, 0], np.int32)

    def check(logits):
        x, got = logits.cpu().numpy(), d.paged_tokens[:2].cpu().numpy()
        for s in range(2):
            a = {k: v[s].item() for k, v in (("t", settings["temperature"]), ("top_k", settings["top_k"]),
                                             ("top_p", settings["top_p"]), ("min_p", settings["min_p"]))}
            w = sample_ref.draw(x[s], float(u[s]), **a)
            assert (int(got[s]), int(kept[s])) == (w[0], w[2])

    u.copy_(up(rng.random(2)))
    d.sample(last, u, d.paged_tokens, probs=probs, kept=kept, **settings)
    check(last)
    d.paged_pos[:2].copy_(up(lens, np.int32)), d.paged_seq[:2].copy_(up([0, 1], np.int32))
    lg2 = torch.empty((2, cfg.vocab), device=dev)
    pos0 = d.paged_pos.clone()
    d.step_paged(2, logits=lg2)  # (the first call outside of the capture; the same rows come again)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d.step_paged(2, logits=lg2)
        d.sample(lg2, u, d.paged_tokens, probs=probs, kept=kept, **settings)
        d.paged_pos.add_(1)
    d.paged_pos.copy_(pos0)
    for _ in range(8):
        u.copy_(up(rng.random(2)))
        g.replay()
        check(lg2)
    d.check_paged_status()
    assert d.paged_pos[:2].tolist() == [x + 8 for x in lens]
