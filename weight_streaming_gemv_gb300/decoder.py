"""Device-resident ternary decoder for ``decode_step_t158``.

Holds the model's device tensors (torch provides the memory), fills the
``t158_model`` descriptor, and owns the KV cache and the workspace.  All
arithmetic happens in libqlin: weights are packed by ``t158_pack`` (host C),
RoPE tables by ``t158_rope_table`` (GPU), and every forward step by
``decode_step_t158``.
"""
from __future__ import annotations

import numpy as np
import torch

from . import qlin

MATRIX_ORDER = ("wq", "wk", "wv", "wo", "wg", "wu", "wd")


class T158Decoder:
    def __init__(self, cfg, weights, device="cuda"):
        """cfg: object with n_layers, dim, n_heads, n_kv_heads, head_dim, ffn, vocab, max_pos, eps,
        rope_base and matrices() -> [(name, rows, cols)]; weights: dict of numpy arrays with
        per-layer int8 trit matrices, scales [L][7], g_attn/g_ffn [L][dim], g_final [dim],
        emb bf16 bits [vocab][dim]."""
        self.cfg = cfg
        dev = torch.device(device)
        L = cfg.n_layers
        dims = {name: (n, k) for name, n, k in cfg.matrices()}
        self.w = []
        self.pitch = []
        for name in MATRIX_ORDER:
            n, k = dims[name]
            pitch = qlin.t158_pitch(k)
            host = np.empty((L, n, pitch), np.uint8)
            for l in range(L):
                host[l] = qlin.t158_pack(weights["layers"][l][name], pitch)
            self.w.append(torch.from_numpy(host).to(dev))
            self.pitch.append(pitch)
        f32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(dev)
        self.scales = f32(weights["scales"])
        self.g_attn = f32(weights["g_attn"])
        self.g_ffn = f32(weights["g_ffn"])
        self.g_final = f32(weights["g_final"])
        self.emb = torch.from_numpy(np.ascontiguousarray(weights["emb"]).view(np.int16)).to(dev)
        half = cfg.head_dim // 2
        self.rope_cos = torch.empty((cfg.max_pos, half), dtype=torch.float32, device=dev)
        self.rope_sin = torch.empty((cfg.max_pos, half), dtype=torch.float32, device=dev)
        qlin.t158_rope_table(self.rope_cos, self.rope_sin, cfg.max_pos, cfg.head_dim, cfg.rope_base)

        m = qlin.T158ModelC()
        m.n_layers, m.dim, m.n_heads, m.n_kv_heads = L, cfg.dim, cfg.n_heads, cfg.n_kv_heads
        m.head_dim, m.ffn, m.vocab, m.max_pos = cfg.head_dim, cfg.ffn, cfg.vocab, cfg.max_pos
        m.eps = cfg.eps
        for j in range(len(MATRIX_ORDER)):
            m.w[j] = self.w[j].data_ptr()
            m.pitch[j] = self.pitch[j]
        m.scales, m.g_attn, m.g_ffn = self.scales.data_ptr(), self.g_attn.data_ptr(), self.g_ffn.data_ptr()
        m.g_final, m.emb = self.g_final.data_ptr(), self.emb.data_ptr()
        m.rope_cos, m.rope_sin = self.rope_cos.data_ptr(), self.rope_sin.data_ptr()
        self.model = m
        self.ws_bytes = qlin.decode_step_t158_workspace_size(m)
        self.workspace = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=dev)
        self.kv = torch.zeros((L, 2, cfg.max_pos, cfg.kv_dim), dtype=torch.float32, device=dev)
        self.token = torch.zeros(1, dtype=torch.int32, device=dev)
        self.logits = torch.empty(cfg.vocab, dtype=torch.float32, device=dev)

    def weight_bytes(self) -> int:
        """Packed bytes at the canonical ceil(K/5) pitch, as the roofline counts them."""
        total = 0
        for name, n, k in self.cfg.matrices():
            total += self.cfg.n_layers * n * ((k + 4) // 5)
        return total

    def step(self, pos: int, token=None, logits: bool = True, stream=None):
        """One forward step at `pos` for the token in self.token (or `token`, a device int32 tensor);
        the greedy token is written back to self.token (so steps chain on the device)."""
        tok = self.token if token is None else token
        qlin.decode_step_t158(self.model, self.kv, self.workspace, self.ws_bytes, tok, pos,
                              self.logits if logits else None, self.token, stream)

    def check_status(self, stream=None):
        qlin.decode_step_t158_status(self.workspace, stream)

    # ---------------------------------------------------------------- sketch head
    def prepare_sketch(self, k: int = 32, n_cand: int = 1024, stream=None):
        """Tables of the sketch head over the tied table, ordered by the final norm gain,
        and the workspace of ``step_sketch``."""
        cfg, dev = self.cfg, self.emb.device
        self.sk_emb_t = torch.empty((cfg.dim, qlin.qlin_sketch_emb_t_pitch(cfg.vocab)), dtype=torch.int16,
                                    device=dev)
        self.sk_signs = torch.empty(qlin.qlin_sketch_signs_bytes(cfg.vocab, cfg.dim) // 8, dtype=torch.int64,
                                    device=dev)
        self.sk_perm = torch.empty(cfg.dim, dtype=torch.int32, device=dev)
        self.sk_ce = torch.zeros(1, dtype=torch.float32, device=dev)
        qlin.qlin_sketch_prepare(self.emb, cfg.vocab, cfg.dim, self.g_final, self.sk_emb_t, self.sk_signs,
                                 self.sk_perm, self.sk_ce, stream)
        sk = qlin.T158SketchC()
        sk.emb_t, sk.signs = self.sk_emb_t.data_ptr(), self.sk_signs.data_ptr()
        sk.perm, sk.c_e = self.sk_perm.data_ptr(), self.sk_ce.data_ptr()
        sk.k, sk.n_cand = k, n_cand
        self.sketch = sk
        self.sk_ws_bytes = qlin.decode_step_t158_sketch_workspace_size(self.model, sk)
        self.sk_workspace = torch.zeros(self.sk_ws_bytes, dtype=torch.uint8, device=dev)

    def step_sketch(self, pos: int, token=None, stream=None):
        """One forward step whose next token comes from the sketch head (two launches)."""
        tok = self.token if token is None else token
        qlin.decode_step_t158_sketch(self.model, self.sketch, self.kv, self.sk_workspace, self.sk_ws_bytes, tok, pos,
                                     self.token, stream)

    def check_sketch_status(self, stream=None):
        qlin.decode_step_t158_sketch_status(self.model, self.sketch, self.sk_workspace, stream)

    # ---------------------------------------------------------------- lanes
    def prepare_lanes(self, n_seqs: int, max_lanes: int):
        """KV caches for n_seqs sequences and the workspace of ``step_lanes``."""
        cfg, dev = self.cfg, self.emb.device
        self.n_seqs, self.max_lanes = n_seqs, max_lanes
        self.kv_lanes = torch.zeros((n_seqs, cfg.n_layers, 2, cfg.max_pos, cfg.kv_dim), dtype=torch.float32,
                                    device=dev)
        self.lanes_ws_bytes = qlin.decode_lanes_t158_workspace_size(self.model, max_lanes)
        self.lanes_workspace = torch.zeros(self.lanes_ws_bytes, dtype=torch.uint8, device=dev)
        self.lane_tokens = torch.zeros(max_lanes, dtype=torch.int32, device=dev)
        self.lane_pos = torch.zeros(max_lanes, dtype=torch.int32, device=dev)
        self.lane_seq = torch.zeros(max_lanes, dtype=torch.int32, device=dev)
        self.lane_next = torch.zeros(max_lanes, dtype=torch.int32, device=dev)

    def step_lanes(self, n_lanes: int, logits=None, stream=None):
        """One step over lanes 0..n_lanes-1 of lane_tokens / lane_pos / lane_seq; the greedy tokens go to
        lane_next (and the logits [n_lanes][vocab] to ``logits`` if given)."""
        qlin.decode_lanes_t158(self.model, self.kv_lanes, self.n_seqs, n_lanes, self.lane_tokens, self.lane_pos,
                               self.lane_seq, logits, self.lane_next, self.lanes_workspace, self.lanes_ws_bytes,
                               self.max_lanes, stream)

    def check_lanes_status(self, stream=None):
        qlin.decode_lanes_t158_status(self.lanes_workspace, stream)

    # ---------------------------------------------------------------- beam search
    def prepare_beams(self, beams: int, own_rows: int, eos: int | None = None):
        """A search over ``beams`` beams for each of the ``n_seqs`` prompts of ``prepare_lanes``, whose caches hold the
        prompts (read in by ``step_lanes``, the last token included); every beam's cache holds the ``own_rows`` rows
        that follow, so a search goes up to own_rows + 1 tokens.  eos: the token that ends a beam (None: none does).
        The calls of a search run on torch's current stream."""
        cfg, dev = self.cfg, self.emb.device
        G, B = self.n_seqs, beams
        i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=dev)
        self.beams, self.own_rows, self.eos = B, own_rows, eos
        self.kv_beams = torch.zeros((G * B, cfg.n_layers, 2, own_rows, cfg.kv_dim), dtype=torch.float32, device=dev)
        self.prompt_len, self.beam_rows = i32(G), i32(G)
        self.beam_prompt = torch.arange(G, dtype=torch.int32, device=dev).repeat_interleave(B)
        self.beam_seq = torch.arange(G * B, dtype=torch.int32, device=dev)
        self.beam_pos, self.beam_next = i32(G * B), i32(G * B)
        self.beam_tokens, self.beam_parents = i32(G, B), i32(G, B)
        # a beam's tokens so far, rows of 16-byte multiples: they follow the selection as the caches do
        self.beam_history = i32(G * B, 1, 1, (own_rows + 4) // 4 * 4)
        self.beam_scores = torch.empty((2, G, B), dtype=torch.float32, device=dev)
        self.beam_done = torch.zeros((G, B), dtype=torch.uint8, device=dev)
        self.beam_status = i32(1)  # of the reordering
        self.beam_logits = torch.empty((G * B, cfg.vocab), dtype=torch.float32, device=dev)
        self.select_ws_bytes = qlin.qlin_beam_select_workspace_size(G, B, cfg.vocab, B)
        self.select_ws = torch.empty(self.select_ws_bytes, dtype=torch.uint8, device=dev)
        self.beams_ws_bytes = qlin.decode_lanes_t158_prefix_workspace_size(self.model, G * B)
        self.beams_ws = torch.zeros(self.beams_ws_bytes, dtype=torch.uint8, device=dev)
        p = qlin.T158PromptsC()
        p.kv, p.len = self.kv_lanes.data_ptr(), self.prompt_len.data_ptr()
        p.n_prompts, p.rows = G, cfg.max_pos
        self.prompts = p

    def start_beams(self, prompt_len, logits):
        """The beams' first tokens: ``logits`` [n_seqs][vocab] are those of each prompt's last token, ``prompt_len``
        (int32 tensor or list) the prompts' lengths.  Lengths on the host are checked, and step_beams refuses a step past
        the model's max_pos; where they are on the device, check_beams_status tells."""
        G, B, V = self.n_seqs, self.beams, self.cfg.vocab
        lens = torch.as_tensor(prompt_len, dtype=torch.int32)
        self.longest = 0 if lens.is_cuda else int(lens.max())
        if self.longest > self.cfg.max_pos or (not lens.is_cuda and int(lens.min()) < 0):
            raise ValueError(f"start_beams: prompts of {lens.tolist()} positions, caches of {self.cfg.max_pos}")
        self.prompt_len.copy_(lens)
        self.beam_rows.zero_()
        self.beam_done.zero_()
        self.beam_t = 0
        self.beam_scores[0].fill_(float("-inf"))  # the beams are still one: only the first counts
        self.beam_scores[0][:, 0] = 0.0
        self.beam_logits.view(G, B, V)[:, 0].copy_(logits)
        self._select()

    def step_beams(self):
        """One token further: a forward step of every beam, the selection, and the beams' caches after it."""
        G, B = self.n_seqs, self.beams
        if self.beam_t > self.own_rows:
            raise ValueError(f"step_beams: the beams' caches hold {self.own_rows} rows")
        if self.longest + self.beam_t > self.cfg.max_pos:
            raise ValueError(f"step_beams: {self.beam_t} tokens behind a prompt of {self.longest}, and the model has "
                             f"{self.cfg.max_pos} positions")
        torch.add(self.prompt_len[self.beam_prompt], self.beam_t - 1, out=self.beam_pos)
        qlin.decode_lanes_t158_prefix(self.model, self.prompts, self.beam_prompt, self.kv_beams, self.own_rows, G * B,
                                      G * B, self.beam_tokens, self.beam_pos, self.beam_seq, self.beam_logits,
                                      self.beam_next, self.beams_ws, self.beams_ws_bytes, G * B)
        self._select()

    def _select(self):
        G, B, V = self.n_seqs, self.beams, self.cfg.vocab
        a, b = self.beam_t & 1, 1 - (self.beam_t & 1)
        done, eos = (None, 0) if self.eos is None else (self.beam_done, self.eos)
        qlin.qlin_beam_select(self.beam_logits, V, self.beam_scores[a], done, eos, G, B, V, B, self.beam_scores[b],
                              self.beam_parents, self.beam_tokens, self.select_ws, self.select_ws_bytes)
        self.beam_rows.fill_(self.beam_t)  # rows of the caches in use: the first tokens came from the prompt
        x, h = self.kv_beams, self.beam_history
        qlin.qlin_beam_reorder(x, x.stride(0) * 4, x.stride(2) * 4, 2 * self.cfg.n_layers, self.cfg.kv_dim * 4,
                               self.own_rows, self.beam_parents, self.beam_rows, G, B, self.beam_status)
        qlin.qlin_beam_reorder(h, h.stride(0) * 4, h.stride(0) * 4, 1, h.stride(0) * 4, 1, self.beam_parents, None, G, B,
                               self.beam_status)
        if self.eos is not None:
            parents = self.beam_parents.long().clamp_min(0)
            self.beam_done.copy_(torch.gather(self.beam_done, 1, parents) | (self.beam_tokens == self.eos))
        # (a place that found no candidate goes on with word 0 and a score of minus infinity)
        self.beam_tokens.clamp_(min=0)
        h[:, 0, 0, self.beam_t] = self.beam_tokens.view(-1)
        self.beam_t += 1

    def beam_results(self):
        """(tokens [n_seqs][beams][steps], scores [n_seqs][beams]), the best beam of a prompt first."""
        return (self.beam_history[:, 0, 0, : self.beam_t].view(self.n_seqs, self.beams, -1),
                self.beam_scores[self.beam_t & 1])

    def check_beams_status(self, stream=None):
        """Raises what the forward steps or the reordering reported since the last check (a wait that gave up there
        leaves some of the beams' states moved and others not), and clears it."""
        qlin.decode_lanes_t158_status(self.beams_ws, stream)
        if self.beam_status.item():
            self.beam_status.zero_()
            raise qlin.QlinError("qlin_beam_reorder", qlin.ERR_TIMEOUT, "a bounded wait gave up: the beams' states are "
                                 "partly moved")

    # ---------------------------------------------------------------- a paged cache of 4 bits a value, sampling
    def prepare_paged(self, n_seqs: int, n_pages: int, max_lanes: int, page_rows: int = 64):
        """A pool of n_pages pages of ``page_rows`` positions, 4 bits a value, that n_seqs sequences draw from (each up to
        the model's max_pos), and the workspace of ``step_paged``.  ``paged_room`` gives a sequence pages before its
        positions are written, ``paged_release`` takes them back; both write the table on torch's current stream."""
        cfg, dev = self.cfg, self.emb.device
        L, G, hd = cfg.n_layers, cfg.n_kv_heads, cfg.head_dim
        u8 = lambda *shape: torch.zeros(shape, dtype=torch.uint8, device=dev)
        i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=dev)
        self.paged_max_lanes = max_lanes
        # k and v, layer by layer
        self.page_codes = u8(2, L, n_pages, G, page_rows, hd // 2)
        self.page_scales = u8(2, L, n_pages, G, page_rows, hd // 32)
        self.page_table = torch.full((n_seqs, -(-cfg.max_pos // page_rows)), -1, dtype=torch.int32, device=dev)
        self.page_rows, self.pages_free, self.pages_of = page_rows, list(range(n_pages))[::-1], [[] for _ in range(n_seqs)]
        c = qlin.T158Kv4C()
        c.kv = qlin.kv4_cache(self.page_codes[0, 0], self.page_codes[1, 0], self.page_scales[0, 0], self.page_scales[1, 0],
                              self.page_table)
        c.code_bytes, c.scale_bytes = self.page_codes.stride(1), self.page_scales.stride(1)
        self.paged = c
        self.paged_ws_bytes = qlin.decode_lanes_t158_kv4_workspace_size(self.model, max_lanes)
        self.paged_workspace = torch.zeros(self.paged_ws_bytes, dtype=torch.uint8, device=dev)
        self.paged_tokens, self.paged_pos, self.paged_seq, self.paged_next = (i32(max_lanes) for _ in range(4))

    def _paged_pages(self, seq: int):
        if not 0 <= seq < len(self.pages_of):
            raise IndexError(f"sequence {seq} of {len(self.pages_of)}")
        return self.pages_of[seq]

    def paged_room(self, seq: int, rows: int):
        """Pages for the first ``rows`` positions of sequence ``seq``; raises MemoryError, and takes none, where the pool has
        too few."""
        if not 0 <= rows <= self.cfg.max_pos:
            raise ValueError(f"paged_room: {rows} positions, and the model has {self.cfg.max_pos}")
        have = self._paged_pages(seq)
        need = -(-rows // self.page_rows) - len(have)
        if need > len(self.pages_free):
            raise MemoryError(f"paged_room: {need} pages for sequence {seq}, {len(self.pages_free)} are free")
        if need > 0:
            new = [self.pages_free.pop() for _ in range(need)]
            self.page_table[seq, len(have): len(have) + need] = torch.tensor(new, dtype=torch.int32).to(self.page_table.device)
            have.extend(new)

    def paged_release(self, seq: int):
        """The sequence's pages go back to the pool."""
        self.pages_free.extend(reversed(self._paged_pages(seq)))
        self.pages_of[seq] = []
        self.page_table[seq].fill_(-1)

    def step_paged(self, n_lanes: int, logits=None, stream=None):
        """``step_lanes`` over the paged cache: lanes 0..n_lanes-1 of paged_tokens / paged_pos / paged_seq (a negative
        position is padding); the greedy tokens go to paged_next, the logits [n_lanes][vocab] to ``logits`` if given."""
        qlin.decode_lanes_t158_kv4(self.model, self.paged, n_lanes, self.paged_tokens, self.paged_pos, self.paged_seq, logits,
                                   self.paged_next, self.paged_workspace, self.paged_ws_bytes, self.paged_max_lanes, stream)

    def check_paged_status(self, stream=None):
        qlin.decode_lanes_t158_status(self.paged_workspace, stream)

    def sample(self, logits, u, tokens, temperature=None, top_k=None, top_p=None, min_p=None, probs=None, kept=None,
               stream=None):
        """Draws a token for every row of ``logits`` [rows][vocab] (fp32, any stride between rows) into ``tokens`` (int32)
        from the random numbers ``u`` [rows] in [0, 1); see qlin_sample for the bounds, tensors of one number per row."""
        rows, vocab = logits.shape
        if logits.dtype != torch.float32 or (vocab > 1 and logits.stride(1) != 1):
            raise ValueError("sample: logits are fp32, a row's contiguous")
        if logits.device != self.emb.device:
            raise ValueError(f"sample: logits on {logits.device}, the decoder is on {self.emb.device}")
        wants = ((u, torch.float32), (tokens, torch.int32), (temperature, torch.float32), (top_k, torch.int32),
                 (top_p, torch.float32), (min_p, torch.float32), (probs, torch.float32), (kept, torch.int32))
        for t, kind in wants:
            if t is not None and (t.dtype != kind or t.numel() < rows or not t.is_contiguous() or t.device != logits.device):
                raise ValueError(f"sample: a tensor of {t.dtype} {tuple(t.shape)} on {t.device} for {rows} rows of {kind}")
        qlin.qlin_sample(logits, logits.stride(0) if rows > 1 else vocab, u, temperature, top_k, top_p, min_p, rows, vocab,
                         tokens, probs, kept, stream)
