"""Measured cases of the operators that serve long conversations from a small cache.

A lane is one token of one sequence at one position.  Three operators, and the
reading of what the first one wrote:

  append  the lanes' queries and keys are rotated to their positions; keys and
          values go into a paged cache of 4 bits a value, and the rows come
          back as the cache holds them
  attend  attention over lanes that reads the paged cache, with a sliding
          window and a few first tokens that stay visible
  sample  the next tokens, drawn with temperature, top-k, top-p and min-p from
          given random numbers, the drawn words' shares and how many words the
          bounds left

The cache: 32 values x of a row share a scale s, a number (8 + m) 2^(e - 24)
in the byte 8 e + m, the least that is at least max|x| / 7; a value is the
code rint(x / s) in -7 .. 7, held as code + 8 in four bits.

``run`` is one call: with ``own`` the library's, without it the plain form in
torch operations.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one user's next token (latency)
        dict(name="append-1-token", op="append", seqs=1, lanes=1, heads=4, kv_heads=1, head_dim=256, page=64,
             context=1024, rotate=True),
        # 64 users' next tokens
        dict(name="append-64-users", op="append", seqs=64, lanes=1, heads=4, kv_heads=1, head_dim=256, page=64,
             context=8192, rotate=True),
        # chunks of two prompts, the second shorter (padding lanes behind it)
        dict(name="append-prompts", op="append", seqs=2, lanes=2048, heads=8, kv_heads=2, head_dim=128, page=32,
             context=4096, rotate=True),
        # one user's next token in a conversation of a thousand (latency)
        dict(name="attend-1-token", op="attend", seqs=1, lanes=1, heads=4, kv_heads=1, head_dim=256, page=64,
             context=1024, window=0, sinks=0),
        # 64 users' next tokens, everything visible
        dict(name="attend-64-users", op="attend", seqs=64, lanes=1, heads=4, kv_heads=1, head_dim=256, page=64,
             context=8192, window=0, sinks=0),
        # 64 users whose layer sees a window and four first tokens
        dict(name="attend-64-window", op="attend", seqs=64, lanes=1, heads=4, kv_heads=1, head_dim=256, page=16,
             context=8192, window=1024, sinks=4),
        # 16 users in long documents
        dict(name="attend-16-long", op="attend", seqs=16, lanes=1, heads=16, kv_heads=2, head_dim=128, page=128,
             context=32768, window=0, sinks=0),
        # chunks of two prompts, the second shorter
        dict(name="attend-prompts", op="attend", seqs=2, lanes=1024, heads=4, kv_heads=1, head_dim=256, page=64,
             context=4096, window=1024, sinks=4),
        # one user's next token, the usual settings of a chat
        dict(name="sample-1-row", op="sample", rows=1, vocab=262144, kind="chat"),
        # 64 users with settings of their own: some greedy, some with every bound, some with none
        dict(name="sample-64-mixed", op="sample", rows=64, vocab=262144, kind="mixed"),
        # 64 users with a bound on the mass alone
        dict(name="sample-64-top-p", op="sample", rows=64, vocab=262144, kind="top_p"),
        # many short answers drawn freely from a smaller vocabulary
        dict(name="sample-256-free", op="sample", rows=256, vocab=32000, kind="free"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("append", "attend", "attend", "sample", "sample"))
    if op == "sample":
        vocab = _log_int(rng, 100, 262144)
        rows = _log_int(rng, 1, min(256, (64 << 18) // vocab))
        return dict(op=op, rows=rows, vocab=vocab, kind=rng.choice(("chat", "mixed", "mixed", "top_p", "free")))
    kv_heads = rng.choice((1, 1, 2, 3, 4))
    heads, hd = kv_heads * rng.choice((1, 2, 3, 4, 8)), rng.choice((64, 128, 256, 256))
    page = rng.choice((16, 32, 64, 128))
    lanes = 1 if rng.random() < 0.6 else _log_int(rng, 2, 2048)
    if op == "append":
        seqs = _log_int(rng, 1, 256) if lanes == 1 else _log_int(rng, 1, max(1, min(8, 4096 // lanes)))
        context = _log_int(rng, lanes, max(lanes, min(8192, (1 << 27) // (seqs * kv_heads * hd))))
        return dict(op=op, seqs=seqs, lanes=lanes, heads=heads, kv_heads=kv_heads, head_dim=hd, page=page,
                    context=context, rotate=rng.random() < 0.8)
    seqs = _log_int(rng, 1, 64) if lanes == 1 else _log_int(rng, 1, max(1, min(8, 2048 // lanes)))
    room = (1 << 27) // (seqs * kv_heads * hd)  # rows of a sequence: at most 2^27 values in all k rows
    if lanes > 1:
        room = min(room, (1 << 25) // (seqs * lanes * heads))
    context = max(lanes, _log_int(rng, max(1, min(lanes, room)), max(lanes, min(room, 32768))))
    window = 0 if rng.random() < 0.5 else _log_int(rng, 1, context)
    return dict(op=op, seqs=seqs, lanes=lanes, heads=heads, kv_heads=kv_heads, head_dim=hd, page=page,
                context=context, window=window, sinks=rng.choice((0, 1, 4, 7)) if window else 0)


# ------------------------------------------------------------------ inputs
def _ints(seed, stream):
    return torch.Generator().manual_seed(1000003 * seed + stream)


def _normal(shape, gen, scale=1.0):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).mul_(scale)


def _positions(c, seed):
    """[seqs][lanes] (-1: padding): a sequence's lanes are its last tokens"""
    S, T, ctx = c["seqs"], c["lanes"], c["context"]
    gen = _ints(seed, 1)
    ends = torch.randint(max(T, ctx // 2, 1), ctx + 1, (S,), generator=gen)  # lengths, the lanes included
    count = torch.randint(max(1, T // 2), T + 1, (S,), generator=gen)
    ends[0], count[0] = ctx, T
    j = torch.arange(T)[None, :]
    return torch.where(j < count[:, None], ends[:, None] - count[:, None] + j, -1).to(torch.int32)


def _table(c, seed):
    """[seqs][pages of a sequence]: the pool's pages in an order of no kind"""
    per = -(-c["context"] // c["page"])
    return torch.randperm(c["seqs"] * per, generator=_ints(seed, 2)).view(c["seqs"], per).to(torch.int32)


def _settings(c, seed):
    """per row: temperature, top_k (0: none), top_p (1: none), min_p (0: none)"""
    n, gen = c["rows"], _ints(seed, 3)
    t, k = torch.full((n,), 0.8), torch.zeros(n, dtype=torch.int32)
    p, m = torch.ones(n), torch.zeros(n)
    if c["kind"] == "chat":
        k[:], p[:] = 64, 0.95
    elif c["kind"] == "top_p":
        t[:], p[:] = 1.0, 0.9
    elif c["kind"] == "mixed":
        some = lambda share: torch.rand(n, generator=gen) < share
        t = 0.25 + 1.25 * torch.rand(n, generator=gen)
        k = torch.where(some(0.5), torch.randint(1, 1000, (n,), generator=gen), 0).to(torch.int32)
        p = torch.where(some(0.5), 0.5 + 0.5 * torch.rand(n, generator=gen), 1.0)
        m = torch.where(some(0.3), 0.1 * torch.rand(n, generator=gen), 0.0)
        t = torch.where(some(0.15), 0.0, t)  # greedy
    return t, k, p, m


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = {"c": c}
    if c["op"] == "sample":
        R, V = c["rows"], c["vocab"]
        s["logits"] = _normal((R, V), gen, 3.0)
        s["logits"][:, 5] = -math.inf  # a word that is not allowed
        s["u"] = torch.rand(R, generator=gen, device=DEV)
        s["temperature"], s["top_k"], s["top_p"], s["min_p"] = (x.to(DEV) for x in _settings(c, seed))
        s["tokens"] = torch.empty(R, dtype=torch.int32, device=DEV)
        s["probs"] = torch.empty(R, device=DEV)
        s["kept"] = torch.empty(R, dtype=torch.int32, device=DEV)
        return s
    H, G, hd, S = c["heads"], c["kv_heads"], c["head_dim"], c["seqs"]
    pos, table = _positions(c, seed), _table(c, seed)
    n, pages = pos.numel(), table.numel()
    s["pos"], s["table"] = pos.reshape(-1).to(DEV), table.to(DEV)
    s["seqs"] = torch.arange(S, dtype=torch.int32).repeat_interleave(c["lanes"]).to(DEV)
    # codes [page][kv head][row][hd / 2] and scales [page][kv head][row][hd / 32], k then v
    shape = (pages, G, c["page"])
    s["codes"] = torch.full((2, *shape, hd // 2), 0x88, dtype=torch.uint8, device=DEV)
    s["scales"] = torch.zeros((2, *shape, hd // 32), dtype=torch.uint8, device=DEV)
    s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    if c["op"] == "append":
        s["qkv"] = _normal((n, (H + 2 * G) * hd), gen)  # as one product gives them
        s["q"], s["k"], s["v"] = s["qkv"].split((H * hd, G * hd, G * hd), 1)
        s["rope"] = None, None
        if c["rotate"]:
            turn = torch.arange(c["context"], device=DEV, dtype=torch.float64)[:, None] * 10000.0 ** (
                -torch.arange(0, hd, 2, device=DEV, dtype=torch.float64) / hd)
            s["rope"] = torch.cos(turn).float(), torch.sin(turn).float()
        s["q_out"] = torch.empty((n, H, hd), device=DEV)
        s["k_out"] = torch.empty((n, G, hd), device=DEV)
        s["v_out"] = torch.empty((n, G, hd), device=DEV)
    else:
        for i in (0, 1):  # some 2^26 values at a time
            for at in range(0, pages, step := max(1, (1 << 26) // (G * c["page"] * hd))):
                part = slice(at, min(pages, at + step))
                s["codes"][i, part], s["scales"][i, part] = _encode(
                    _normal((part.stop - at, G, c["page"], hd), gen))
        s["q"] = _normal((n, H, hd), gen, 2.0)  # scores of standard deviation 2
        s["out"] = torch.empty_like(s["q"])
    if own:
        from weight_streaming_gemv_gb300 import qlin

        s["kv"] = qlin.kv4_cache(s["codes"][0], s["codes"][1], s["scales"][0], s["scales"][1], s["table"])
        if c["op"] == "attend":
            s["bytes"] = qlin.qlin_attention_kv4_workspace_size(n, H, G, hd)
            s["work"] = torch.empty(s["bytes"], dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["c"]
    if own:
        from weight_streaming_gemv_gb300 import qlin

        if c["op"] == "sample":
            qlin.qlin_sample(s["logits"], c["vocab"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"],
                             c["rows"], c["vocab"], s["tokens"], s["probs"], s["kept"])
            return {"tokens": s["tokens"], "probs": s["probs"], "kept": s["kept"]}
        n, H, G, hd = s["pos"].numel(), c["heads"], c["kv_heads"], c["head_dim"]
        if c["op"] == "append":
            row = s["qkv"].stride(0)
            qlin.qlin_kv4_append(s["kv"], s["k"], s["v"], row, s["q"], row, s["q_out"], s["rope"][0], s["rope"][1],
                                 c["context"], s["pos"], s["seqs"], n, H, G, hd, s["status"])
            qlin.qlin_kv4_read(s["kv"], s["pos"], s["seqs"], n, G, hd, s["k_out"], s["v_out"], s["status"])
            return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
        qlin.qlin_attention_kv4(s["q"], s["kv"], s["pos"], s["seqs"], n, H, G, hd, c["window"], c["sinks"], s["out"],
                                s["status"], s["work"], s["bytes"])
        return s["out"]
    return {"append": _plain_append, "attend": _plain_attend, "sample": _plain_sample}[c["op"]](s)


def _encode(x):
    """[..., hd] as codes [..., hd / 2] and scales [..., hd / 32].  Eight values are a little-endian word of 32 bits:
    value 2 i in its bits 4 i on, value 2 i + 1 in its bits 16 + 4 i on."""
    g = x.unflatten(-1, (-1, 32))
    need = g.abs().amax(-1, keepdim=True) / 7.0
    b = (((need.view(torch.int32) + 0xFFFFF) >> 20) - (106 << 3)).clamp(0, 255)
    code = torch.round(g / _scale(b)).clamp(-7, 7).to(torch.int32) + 8
    w = code.flatten(-2).unflatten(-1, (-1, 4, 2)).transpose(-1, -2).flatten(-2).unflatten(-1, (-1, 2))
    return (w[..., 0] | w[..., 1] << 4).flatten(-2).to(torch.uint8), b[..., 0].to(torch.uint8)


def _scale(b):
    """(8 + m) 2^(e - 24) of the byte 8 e + m: an fp32 number's exponent and first three bits"""
    return ((b.to(torch.int32) + (106 << 3)) << 20).view(torch.float32)


def _decode(codes, scales):
    w = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).unflatten(-1, (-1, 2, 4)).transpose(-1, -2).flatten(-3)
    x = (w.float() - 8.0).unflatten(-1, (-1, 32)) * _scale(scales)[..., None]
    return x.flatten(-2)


def _rotate(x, pos, rope):
    """[n, heads, hd] with dims i and i + hd / 2 turned by the position's angles, products rounded, then added"""
    cos, sin = (t[pos.long()][:, None] for t in rope)
    a, b = x.chunk(2, -1)
    return torch.cat((a * cos - b * sin, a * sin + b * cos), -1)


def _plain_append(s):
    c, live = s["c"], s["pos"] >= 0
    H, G, hd = c["heads"], c["kv_heads"], c["head_dim"]
    at = s["pos"].clamp_min(0)
    q, k, v = s["q"].unflatten(1, (H, hd)), s["k"].unflatten(1, (G, hd)), s["v"].unflatten(1, (G, hd))
    if c["rotate"]:
        q, k = _rotate(q, at, s["rope"]), _rotate(k, at, s["rope"])
    page = s["table"][s["seqs"].long(), at.long() // c["page"]].long()[live]
    row = (at.long() % c["page"])[live]
    zero = live[:, None, None]
    back = []
    for i, x in ((0, k), (1, v)):
        s["codes"][i][page, :, row], s["scales"][i][page, :, row] = _encode(x[live])
        rows = torch.zeros_like(x)
        rows[live] = _decode(s["codes"][i][page, :, row], s["scales"][i][page, :, row])
        back.append(rows)
    return {"q": torch.where(zero, q, 0.0), "k": back[0], "v": back[1]}


def _rows(s, i):
    """[seqs][kv heads][rows][hd] of the keys (0) or values (1)"""
    t = s["table"].long()
    x = _decode(s["codes"][i][t], s["scales"][i][t])  # [seqs][pages][kv heads][page][hd]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attend(s):
    c = s["c"]
    S, T, H, G, hd = c["seqs"], c["lanes"], c["heads"], c["kv_heads"], c["head_dim"]
    g = H // G
    k, v = _rows(s, 0), _rows(s, 1)
    q = s["q"].view(S, T, G, g, hd).permute(0, 2, 1, 3, 4).reshape(S, G, T * g, hd)
    p = s["pos"].view(S, 1, T, 1).expand(S, 1, T, g).reshape(S, 1, T * g, 1)
    j = torch.arange(k.shape[2], device=DEV)
    seen = j <= p
    if c["window"]:
        seen = seen & ((j > p - c["window"]) | (j < c["sinks"]))
    x = torch.where(seen, torch.matmul(q, k.transpose(2, 3)) / math.sqrt(hd), -math.inf)
    m = x.amax(-1, keepdim=True)
    w = torch.exp(x - torch.where(torch.isfinite(m), m, 0.0))
    w = w / w.sum(-1, keepdim=True).clamp_min(1e-38)
    return torch.matmul(w, v).view(S, G, T, g, hd).permute(0, 2, 1, 3, 4).reshape(S * T, H, hd)


def _plain_sample(s):
    """in 64 bits: the sums decide between neighbouring words"""
    x, t = s["logits"].double(), s["temperature"].double()[:, None]
    greedy = t <= 0.0
    w = torch.exp((x - x.amax(1, keepdim=True)) / torch.where(greedy, 1.0, t))
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    sw = torch.gather(w, 1, order)
    place = torch.arange(x.shape[1], device=DEV)[None]
    k = s["top_k"].long()[:, None]
    keep = (k <= 0) | (place < k)
    sw = torch.where(keep, sw, 0.0)
    cum = torch.cumsum(sw, 1)
    need = s["top_p"].double()[:, None] * cum[:, -1:]
    keep = keep & ((s["top_p"][:, None] >= 1.0) | (cum - sw < need) | (place == 0))
    keep = keep & (sw >= s["min_p"].double()[:, None])
    keep = torch.where(greedy, place == 0, keep) & (torch.gather(x, 1, order) > -math.inf)
    kept = torch.zeros_like(w).scatter_(1, order, torch.where(keep, sw, 0.0))
    cum = torch.cumsum(kept, 1)
    token = (cum <= s["u"].double()[:, None] * cum[:, -1:]).sum(1, keepdim=True)
    return {"tokens": token[:, 0].int(), "probs": (torch.gather(kept, 1, token) / cum[:, -1:])[:, 0].float(),
            "kept": keep.sum(1).int()}


# ------------------------------------------------------------------ what a pass cannot do without
def _seen(pos, window, sinks):
    """how many positions the tokens at positions pos (a run of consecutive ones) see between them, and in all"""
    pos = [p for p in pos if p >= 0]
    if not pos:
        return 0, 0
    first = lambda p: max(0, p - window + 1) if window else 0
    return (max(pos) + 1 - first(min(pos)) + min(sinks, first(min(pos))),
            sum(p + 1 - first(p) + min(sinks, first(p)) for p in pos))


def work(case):
    c = case
    if c["op"] == "sample":
        return {"bytes": c["rows"] * (4 * c["vocab"] + 32), "flops": 3 * c["rows"] * c["vocab"]}
    H, G, hd = c["heads"], c["kv_heads"], c["head_dim"]
    row = 2 * G * (hd // 2 + hd // 32)  # k and v of one position
    pos = _positions(c, 1).tolist()
    live = sum(p >= 0 for ps in pos for p in ps)
    if c["op"] == "append":
        lanes = c["seqs"] * c["lanes"]
        rope = len({p for ps in pos for p in ps if p >= 0}) * hd * 4 if c["rotate"] else 0
        return {"bytes": live * (4 * hd * (H + 2 * G) + 2 * row) + 4 * hd * lanes * (H + 2 * G) + rope,
                "flops": live * hd * (3 * H * c["rotate"] + 10 * G)}
    seen = [_seen(p, c["window"], c["sinks"]) for p in pos]
    return {"bytes": sum(n for n, _ in seen) * row + 2 * c["seqs"] * c["lanes"] * H * hd * 4,
            "flops": 4 * sum(n for _, n in seen) * H * hd}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "sample":
        return _exact_sample(c, s)
    return _exact_append(c, s) if c["op"] == "append" else _exact_attend(c, s)


def _exact_append(c, s):
    """The queries in 64 bits; keys and values as the numbers next to the 32-bit ones on the cache's grid."""
    H, G, hd = c["heads"], c["kv_heads"], c["head_dim"]
    n, half, pos = s["pos"].numel(), hd // 2, s["pos"].long()
    live = pos >= 0
    x = s["qkv"].view(n, H + 2 * G, hd).double()
    if c["rotate"]:
        cos, sin = (t.double()[pos.clamp_min(0)][:, None] for t in s["rope"])
        lo, hi = x[:, : H + G, :half].clone(), x[:, : H + G, half:].clone()
        near = lambda t: t.float().double()  # the cache's keys are rotated in 32 bits, every product rounded
        x[:, :H, :half] = lo[:, :H] * cos - hi[:, :H] * sin
        x[:, :H, half:] = hi[:, :H] * cos + lo[:, :H] * sin
        x[:, H: H + G, :half] = near(near(lo[:, H:] * cos) - near(hi[:, H:] * sin))
        x[:, H: H + G, half:] = near(near(hi[:, H:] * cos) + near(lo[:, H:] * sin))
    x[~live] = 0.0
    grid = torch.tensor(sorted({(8 + m) * 2.0 ** (e - 24) for m in range(8) for e in range(32)}), dtype=torch.float64,
                        device=DEV)
    g = x[:, H:].reshape(n, 2 * G, hd // 32, 32)
    top = (g.abs().max(-1).values / 7.0).float().double()
    step = grid[torch.searchsorted(grid, top).clamp_max(255)][..., None]
    kv = (torch.round((g / step).float().double()).clamp(-7.0, 7.0) * step).reshape(n, 2 * G, hd)
    return {"q": x[:, :H], "k": kv[:, :G], "v": kv[:, G:]}


def _exact_attend(c, s):
    """sequence by sequence, the pages in their order, exp(score) over its sum for the keys that are seen"""
    H, G, hd, T, B = c["heads"], c["kv_heads"], c["head_dim"], c["lanes"], c["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    pos, table = s["pos"].view(-1, T), s["table"].tolist()
    place = torch.tensor([4 * (i // 2) + 16 * (i % 2) for i in range(8)], device=DEV)  # of a word's values
    for q in range(c["seqs"]):
        rows = torch.nonzero(pos[q] >= 0)[:, 0]
        if not rows.numel():
            continue
        at = pos[q][rows].long()[:, None]
        last = int(at.max())
        kv = []
        for i in (0, 1):
            ids = table[q][: last // B + 1]
            word = torch.cat([s["codes"][i, p] for p in ids], 1).view(torch.int32).long()  # [G][rows][hd / 8]
            step = torch.cat([s["scales"][i, p] for p in ids], 1).double()
            step = (8.0 + step % 8) * torch.exp2(torch.floor(step / 8) - 24.0)
            code = ((word[..., None] >> place) & 15).double().flatten(-2) - 8.0
            kv.append((code * step.repeat_interleave(32, -1))[:, : last + 1])
        j = torch.arange(last + 1, device=DEV)[None]
        hidden = j > at
        if c["window"]:
            hidden |= (at - j >= c["window"]) & (j >= c["sinks"])
        for h in range(H):
            k, v = (x[h // (H // G)] for x in kv)
            for a in range(0, len(rows), 512):
                part = rows[a: a + 512] + q * T
                z = s["q"][part, h].double() @ k.T * hd ** -0.5
                z.masked_fill_(hidden[a: a + 512], -math.inf)
                e = torch.exp(z - z.max(dim=1, keepdim=True).values)
                out[part, h] = (e @ v) / e.sum(1, keepdim=True)
    return out


def _exact_sample(c, s):
    """row by row: the words from the largest logit on, those that the three bounds leave, and the drawn one's share"""
    probs = torch.empty(c["rows"], dtype=torch.float64, device=DEV)
    t, top_k, top_p, min_p, u = (s[n].tolist() for n in ("temperature", "top_k", "top_p", "min_p", "u"))
    for r in range(c["rows"]):
        if t[r] <= 0.0:
            probs[r] = 1.0
            continue
        x = s["logits"][r].double()
        val, at = torch.sort(x, descending=True, stable=True)
        e = torch.exp((val - val[0]) / t[r])
        n = min(top_k[r], c["vocab"]) if top_k[r] > 0 else c["vocab"]
        if top_p[r] < 1.0:
            run = torch.cumsum(e[:n], 0)
            n = min(n, 1 + int((run < top_p[r] * run[-1]).sum()))
        n = max(1, min(n, int((e >= min_p[r]).sum())))
        ids, order = torch.sort(at[:n])
        e = e[:n][order]
        run = torch.cumsum(e, 0)
        probs[r] = e[min(n - 1, int((run <= u[r] * run[-1]).sum()))] / run[-1]
    return {"tokens": None, "probs": probs, "kept": None}
