"""Measured cases of the operators that serve many sequences at once.

Four operators over the caches of lanes (a lane is one token of one sequence
at one position):

  window   attention over lanes with a sliding window and a few first tokens
           that stay visible: single tokens of many users, prompt chunks
  prefix   attention of lanes that share a prompt kept once: its keys and
           values are read once for all lanes, each lane's own rows follow
  select   beam search's selection over beams and vocabulary, from the logits
  reorder  the beams' caches follow the selection, in place

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
        # one user's next token: a local layer that sees 512 positions and 4 first tokens (latency)
        dict(name="window-1-token", op="window", seqs=1, lanes=1, heads=4, kv_heads=1, head_dim=256, kv="float32",
             context=1024, window=512, sinks=4),
        # 64 users' next tokens, half-precision caches, a wide window
        dict(name="window-64-users", op="window", seqs=64, lanes=1, heads=4, kv_heads=1, head_dim=256, kv="bfloat16",
             context=8192, window=4096, sinks=4),
        # 16 users at long contexts with everything visible
        dict(name="window-16-long", op="window", seqs=16, lanes=1, heads=16, kv_heads=2, head_dim=128, kv="float32",
             context=32768, window=0, sinks=0),
        # chunks of two prompts, the second shorter (padding lanes behind it)
        dict(name="window-prompts", op="window", seqs=2, lanes=2048, heads=4, kv_heads=1, head_dim=256,
             kv="bfloat16", context=4096, window=1024, sinks=4),
        # one user's beam search over four beams, a few tokens in (latency)
        dict(name="prefix-4-beams", op="prefix", prompts=1, beams=4, heads=4, kv_heads=1, head_dim=256, kv="float32",
             prompt=1000, suffix=24, window=0, sinks=0),
        # eight users with eight beams each
        dict(name="prefix-8x8-beams", op="prefix", prompts=8, beams=8, heads=8, kv_heads=2, head_dim=128,
             kv="bfloat16", prompt=4096, suffix=64, window=0, sinks=0),
        # 64 answers drawn from one long document
        dict(name="prefix-64-answers", op="prefix", prompts=1, beams=64, heads=4, kv_heads=1, head_dim=256,
             kv="bfloat16", prompt=131072, suffix=256, window=0, sinks=0),
        # the selection behind prefix-4-beams
        dict(name="select-4-beams", op="select", groups=1, beams=4, vocab=262144, n_out=4, first=False, done=0),
        # the selection behind prefix-8x8-beams: twice the beams come out, so that finished ones can be set aside
        dict(name="select-8x8-beams", op="select", groups=8, beams=8, vocab=262144, n_out=16, first=False, done=1),
        # the caches of four beams after a step, one beam staying where it is
        dict(name="reorder-4-beams", op="reorder", groups=1, beams=4, planes=52, max_rows=64, rows=40, row=256,
             kv="float32", kept=1, sources=2),
        # many beams with long answers
        dict(name="reorder-64-beams", op="reorder", groups=4, beams=16, planes=52, max_rows=256, rows=250, row=256,
             kv="float32", kept=2, sources=9),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _heads(rng):
    kv_heads = rng.choice((1, 1, 2, 3, 4))
    return kv_heads * rng.choice((1, 2, 3, 4, 8)), kv_heads, rng.choice((64, 128, 256, 256))


def draw(rng):
    op = rng.choice(("window", "window", "prefix", "prefix", "select", "reorder"))
    kv = rng.choice(("float32", "bfloat16"))
    if op == "window":
        heads, kv_heads, hd = _heads(rng)
        lanes = 1 if rng.random() < 0.6 else _log_int(rng, 2, 2048)
        seqs = _log_int(rng, 1, 64) if lanes == 1 else _log_int(rng, 1, max(1, min(8, 2048 // lanes)))
        room = (1 << 27) // (seqs * kv_heads * hd)  # rows of a sequence: at most 2^27 values in all k rows
        if lanes > 1:
            room = min(room, (1 << 25) // (seqs * lanes * heads))
        context = max(lanes, _log_int(rng, max(1, min(lanes, room)), max(lanes, min(room, 32768))))
        window = 0 if rng.random() < 0.3 else _log_int(rng, 1, context)
        return dict(op=op, seqs=seqs, lanes=lanes, heads=heads, kv_heads=kv_heads, head_dim=hd, kv=kv,
                    context=context, window=window, sinks=rng.choice((0, 1, 4, 7)) if window else 0)
    if op == "prefix":
        heads, kv_heads, hd = _heads(rng)
        prompts = _log_int(rng, 1, 8)
        beams = _log_int(rng, 1, 64 // prompts)
        suffix = _log_int(rng, 1, 256)
        room = (1 << 25) // (prompts * kv_heads * hd)
        room = min(room, (1 << 28) // (prompts * beams * heads * 8))
        prompt = _log_int(rng, 1, max(1, min(room, 131072)))
        window = 0 if rng.random() < 0.8 else _log_int(rng, 1, prompt + suffix)
        return dict(op=op, prompts=prompts, beams=beams, heads=heads, kv_heads=kv_heads, head_dim=hd, kv=kv,
                    prompt=prompt, suffix=suffix, window=window, sinks=rng.choice((0, 4)) if window else 0)
    if op == "select":
        groups = _log_int(rng, 1, 8)
        beams = _log_int(rng, 1, 64 // groups)
        vocab = _log_int(rng, 300, 262144)
        first = rng.random() < 0.2
        return dict(op=op, groups=groups, beams=beams, vocab=vocab, n_out=beams * rng.choice((1, 2)), first=first,
                    done=0 if first else rng.randint(0, max(0, beams // 3)))
    groups = _log_int(rng, 1, 8)
    beams = _log_int(rng, 2, 64 // groups)
    kept = rng.randint(0, beams // 2)
    max_rows = _log_int(rng, 1, 256)
    return dict(op=op, groups=groups, beams=beams, planes=2 * _log_int(rng, 1, 26), max_rows=max_rows,
                rows=rng.randint(1, max_rows), row=rng.choice((16, 64, 256, 512)), kv=kv, kept=kept,
                sources=rng.randint(2, max(2, beams - kept)))


# ------------------------------------------------------------------ inputs
def _ints(seed, stream):
    return torch.Generator().manual_seed(1000003 * seed + stream)


def _randint(lo, hi, n, gen):
    """n whole numbers in [lo, hi]"""
    return torch.randint(lo, hi + 1, (n,), generator=gen)


def _normal(shape, gen, dtype="float32", scale=1.0):
    x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)
    return (x if scale == 1.0 else x.mul_(scale)).to(getattr(torch, dtype))


def _window_lanes(c, seed):
    """positions [seqs][lanes] (-1: padding): a sequence's lanes are its last tokens"""
    S, T, ctx = c["seqs"], c["lanes"], c["context"]
    gen = _ints(seed, 1)
    ends = _randint(max(T, ctx // 2, 1), ctx, S, gen)  # the sequences' lengths, their lanes included
    count = _randint(max(1, T // 2), T, S, gen)
    ends[0], count[0] = ctx, T
    j = torch.arange(T)[None, :]
    pos = ends[:, None] - count[:, None] + j
    return torch.where(j < count[:, None], pos, -1).to(torch.int32)


def _prefix_lanes(c, seed):
    """the prompts' lengths and the lanes' positions, lane i of prompt i // beams"""
    gen = _ints(seed, 2)
    length = _randint(max(1, c["prompt"] // 2), c["prompt"], c["prompts"], gen)
    length[0] = c["prompt"]
    own_rows = _randint(1, c["suffix"], c["prompts"] * c["beams"], gen)
    return length.to(torch.int32), (length.repeat_interleave(c["beams"]) + own_rows - 1).to(torch.int32)


def _parents(c, seed):
    """[groups][beams]: `kept` beams stay, the others take the place of one of `sources` beams, none its own"""
    gen = _ints(seed, 3)
    out = []
    for _ in range(c["groups"]):
        order = torch.randperm(c["beams"], generator=gen).tolist()
        moved = order[c["kept"]:]
        src = torch.randperm(c["beams"], generator=gen).tolist()[: min(c["sources"], c["beams"])]
        par = list(range(c["beams"]))
        for n, b in enumerate(moved):
            s = src[n % len(src)]
            par[b] = s if s != b else src[(n + 1) % len(src)]
        out.append(par)
    return torch.tensor(out, dtype=torch.int32)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = {"c": c}
    if c["op"] in ("window", "prefix"):
        H, G, hd = c["heads"], c["kv_heads"], c["head_dim"]
        if c["op"] == "window":
            n_seqs, rows = c["seqs"], c["context"]
            pos = _window_lanes(c, seed)
            seqs = torch.arange(n_seqs, dtype=torch.int32)[:, None].expand(pos.shape).reshape(-1)
        else:
            n_seqs, rows = c["prompts"] * c["beams"], c["suffix"]
            length, pos = _prefix_lanes(c, seed)
            seqs = torch.arange(n_seqs, dtype=torch.int32)
            s["prefix"] = _normal((c["prompts"], 2, c["prompt"], G * hd), gen, c["kv"])
            s["prefix_len"] = length.to(DEV)
            s["prefix_of"] = (seqs // c["beams"]).to(torch.int32).to(DEV)
        s["cache"] = _normal((n_seqs, 2, rows, G * hd), gen, c["kv"])  # k then v, as the decoder lays its caches out
        s["pos"] = pos.reshape(-1).to(DEV)
        s["seqs"] = seqs.to(DEV).contiguous()
        n = s["pos"].numel()
        s["q"] = _normal((n, H, hd), gen, scale=2.0)  # scores of standard deviation 2
        s["out"] = torch.empty_like(s["q"])
        if own:
            from weight_streaming_gemv_gb300 import qlin

            s["kv"] = qlin.kv_cache(s["cache"][:, 0], s["cache"][:, 1])
            if c["op"] == "prefix":
                s["prefix_kv"] = qlin.kv_cache(s["prefix"][:, 0], s["prefix"][:, 1])
            s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
            s["bytes"] = qlin.qlin_attention_lanes_workspace_size(n, H, G, hd)
            s["work"] = torch.empty(s["bytes"], dtype=torch.uint8, device=DEV)
    elif c["op"] == "select":
        Gr, B, V = c["groups"], c["beams"], c["vocab"]
        s["logits"] = _normal((Gr * B, V), gen, scale=3.0)
        s["logits"][:, 5] = -math.inf  # a token that is not allowed
        s["scores"] = torch.rand((Gr, B), generator=gen, device=DEV) * -8.0 - 4.0
        if c["first"]:  # the beams are still one: only the first of each group counts
            s["scores"][:] = -math.inf
            s["scores"][:, 0] = 0.0
        done = torch.zeros((Gr, B), dtype=torch.uint8)
        done[:, B - c["done"]:] = 1
        s["done"], s["eos"] = done.to(DEV), 1
        s["out_scores"] = torch.empty((Gr, c["n_out"]), device=DEV)
        s["parents"] = torch.empty((Gr, c["n_out"]), dtype=torch.int32, device=DEV)
        s["tokens"] = torch.empty((Gr, c["n_out"]), dtype=torch.int32, device=DEV)
        if own:
            from weight_streaming_gemv_gb300 import qlin

            s["bytes"] = qlin.qlin_beam_select_workspace_size(Gr, B, V, c["n_out"])
            s["work"] = torch.empty(s["bytes"], dtype=torch.uint8, device=DEV)
    else:
        s["cache"] = _normal((c["groups"] * c["beams"], c["planes"], c["max_rows"], c["row"]), gen, c["kv"])
        s["parents"] = _parents(c, seed).to(DEV)
        s["rows"] = torch.full((c["groups"],), c["rows"], dtype=torch.int32, device=DEV)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["c"]
    if own:
        from weight_streaming_gemv_gb300 import qlin

        if c["op"] == "window":
            qlin.qlin_attention_lanes(s["q"], s["kv"], s["pos"], s["seqs"], s["q"].shape[0], c["heads"],
                                      c["kv_heads"], c["head_dim"], c["window"], c["sinks"], s["out"], s["status"],
                                      s["work"], s["bytes"])
            return s["out"]
        if c["op"] == "prefix":
            qlin.qlin_attention_prefix(s["q"], s["prefix_kv"], s["prefix_len"], s["prefix_of"], s["kv"], s["pos"],
                                       s["seqs"], s["q"].shape[0], c["heads"], c["kv_heads"], c["head_dim"],
                                       c["window"], c["sinks"], s["out"], s["status"], s["work"], s["bytes"])
            return s["out"]
        if c["op"] == "select":
            qlin.qlin_beam_select(s["logits"], c["vocab"], s["scores"], s["done"], s["eos"], c["groups"], c["beams"],
                                  c["vocab"], c["n_out"], s["out_scores"], s["parents"], s["tokens"], s["work"],
                                  s["bytes"])
            return {"scores": s["out_scores"], "parents": s["parents"], "tokens": s["tokens"]}
        x = s["cache"]
        plane = x.stride(1) * x.element_size()
        qlin.qlin_beam_reorder(x, x.stride(0) * x.element_size(), plane, c["planes"], c["row"] * x.element_size(),
                               c["max_rows"], s["parents"], s["rows"], c["groups"], c["beams"])
        return x
    return {"window": _plain_window, "prefix": _plain_prefix, "select": _plain_select,
            "reorder": _plain_reorder}[c["op"]](s)


def _softmax(x, seen):
    """softmax over the last axis of the seen places; zeros in a row that sees none"""
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(x - torch.where(torch.isfinite(m), m, 0.0)), 0.0)
    return p / p.sum(-1, keepdim=True).clamp_min(1e-38)


def _seen(p, j, window, sinks):
    """which keys, at positions j, a token at position p sees"""
    ok = j <= p
    if window:
        ok = ok & ((j > p - window) | (j < sinks))
    return ok


def _plain_window(s):
    c = s["c"]
    S, T, H, G, hd, R = c["seqs"], c["lanes"], c["heads"], c["kv_heads"], c["head_dim"], c["context"]
    g = H // G
    k, v = (s["cache"][:, i].float().view(S, R, G, hd).transpose(1, 2) for i in (0, 1))  # [S][G][R][hd]
    q = s["q"].view(S, T, G, g, hd).permute(0, 2, 1, 3, 4).reshape(S, G, T * g, hd)
    p = s["pos"].view(S, 1, T, 1).expand(S, 1, T, g).reshape(S, 1, T * g, 1)
    seen = _seen(p, torch.arange(R, device=DEV), c["window"], c["sinks"])
    w = _softmax(torch.matmul(q, k.transpose(2, 3)) / math.sqrt(hd), seen)
    return torch.matmul(w, v).view(S, G, T, g, hd).permute(0, 2, 1, 3, 4).reshape(S * T, H, hd)


def _plain_prefix(s):
    c = s["c"]
    F, B, H, G, hd, P, R = c["prompts"], c["beams"], c["heads"], c["kv_heads"], c["head_dim"], c["prompt"], c["suffix"]
    g = H // G
    pk, pv = (s["prefix"][:, i].float().view(F, P, G, hd).transpose(1, 2) for i in (0, 1))  # [F][G][P][hd]
    k, v = (s["cache"][:, i].float().view(F * B, R, G, hd).transpose(1, 2) for i in (0, 1))  # [F B][G][R][hd]
    q = s["q"].view(F, B, G, g, hd)
    qp = q.permute(0, 2, 1, 3, 4).reshape(F, G, B * g, hd)
    x = torch.matmul(qp, pk.transpose(2, 3)).view(F, G, B, g, P)
    y = torch.matmul(q.reshape(F * B, G, g, hd), k.transpose(2, 3)).view(F, B, G, g, R).transpose(1, 2)
    p = s["pos"].view(F, 1, B, 1, 1)
    n = s["prefix_len"].view(F, 1, 1, 1, 1)
    j, r = torch.arange(P, device=DEV), n + torch.arange(R, device=DEV)
    seen = torch.cat([(j < n) & _seen(p, j, c["window"], c["sinks"]), _seen(p, r, c["window"], c["sinks"])], -1)
    w = _softmax(torch.cat([x, y], -1) / math.sqrt(hd), seen)
    o = torch.matmul(w[..., :P].reshape(F, G, B * g, P), pv).view(F, G, B, g, hd).transpose(1, 2)
    u = torch.matmul(w[..., P:].transpose(1, 2).reshape(F * B, G, g, R), v).view(F, B, G, g, hd)
    return (o + u).reshape(F * B, H, hd)


def _plain_select(s):
    c = s["c"]
    Gr, B, V, n = c["groups"], c["beams"], c["vocab"], c["n_out"]
    x = s["logits"].double().view(Gr, B, V)  # two beams' candidates can be nearer than 32 bits tell apart
    m = x.amax(-1, keepdim=True)
    x = x - (m + torch.log(torch.exp(x - m).sum(-1, keepdim=True)))
    base = s["scores"].double().view(Gr, B, 1)
    done = s["done"].view(Gr, B, 1) != 0
    only = torch.where(torch.arange(V, device=DEV) == s["eos"], base, -math.inf)
    x = torch.where(done, only, base + x).view(Gr, B * V)
    top, at = torch.sort(x, dim=-1, descending=True, stable=True)
    top, at = top[:, :n], at[:, :n]
    none = top == -math.inf
    return {"scores": top.float(), "parents": torch.where(none, -1, at // V).int(),
            "tokens": torch.where(none, -1, at % V).int()}


def _plain_reorder(s):
    c, x = s["c"], s["cache"]
    first = torch.arange(c["groups"], device=DEV)[:, None] * c["beams"]
    x[:, :, : c["rows"]] = x[(first + s["parents"]).view(-1), :, : c["rows"]]
    return x


# ------------------------------------------------------------------ what a pass cannot do without
def _union(pos, window, sinks):
    """how many positions the tokens at positions pos (a run of consecutive ones) see between them"""
    pos = [p for p in pos if p >= 0]
    if not pos:
        return 0
    lo, hi = min(pos), max(pos)
    start = max(0, lo - window + 1) if window else 0
    return hi + 1 - start + min(sinks, start)


def _pairs(pos, window, sinks):
    n = 0
    for p in pos:
        if p >= 0:
            start = max(0, p - window + 1) if window else 0
            n += p + 1 - start + min(sinks, start)
    return n


def work(case):
    c = case
    e = 4 if c.get("kv") == "float32" else 2
    if c["op"] == "window":
        pos = _window_lanes(c, 1).tolist()
        row = c["kv_heads"] * c["head_dim"] * e
        rows = sum(_union(p, c["window"], c["sinks"]) for p in pos)
        pairs = sum(_pairs(p, c["window"], c["sinks"]) for p in pos)
        lanes = c["seqs"] * c["lanes"]
        return {"bytes": 2 * rows * row + 2 * lanes * c["heads"] * c["head_dim"] * 4,
                "flops": 4 * pairs * c["heads"] * c["head_dim"]}
    if c["op"] == "prefix":
        length, pos = _prefix_lanes(c, 1)
        length, pos = length.tolist(), pos.tolist()
        row, B = c["kv_heads"] * c["head_dim"] * e, c["beams"]
        rows = pairs = 0
        for f, n in enumerate(length):
            first = n  # the first prompt row behind the sinks that a lane of this prompt sees
            for p in pos[f * B:(f + 1) * B]:
                start = max(0, p - c["window"] + 1) if c["window"] else 0
                first = min(first, start)
                rows += p + 1 - max(start, n) + max(0, min(c["sinks"], start) - n)  # its own rows
            rows += n - first + min(c["sinks"], first)
            pairs += _pairs(pos[f * B:(f + 1) * B], c["window"], c["sinks"])
        return {"bytes": 2 * rows * row + 2 * len(pos) * c["heads"] * c["head_dim"] * 4,
                "flops": 4 * pairs * c["heads"] * c["head_dim"]}
    if c["op"] == "select":
        n = c["groups"] * c["beams"] * c["vocab"]
        live = 1 if c["first"] else c["beams"] - c["done"]
        return {"bytes": 4 * c["groups"] * live * c["vocab"] + 12 * c["groups"] * c["n_out"], "flops": 3 * n}
    par = _parents(c, 1).tolist()
    seq = c["planes"] * c["rows"] * c["row"] * e
    moved = sum(p != b for ps in par for b, p in enumerate(ps))
    read = sum(len({p for b, p in enumerate(ps) if p != b}) for ps in par)
    return {"bytes": (moved + read) * seq, "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "window":
        return _exact_lanes(c, s, None)
    if c["op"] == "prefix":
        return _exact_lanes(c, s, s["prefix_len"].tolist())
    if c["op"] == "select":
        return _exact_select(c, s)
    return None  # copies: nothing is computed


def _exact_lanes(c, s, length):
    """lane by lane for single tokens, run by run for the lanes of one sequence: the keys in the order of their
    positions, exp(score) over its sum for those that are seen"""
    H, G, hd = c["heads"], c["kv_heads"], c["head_dim"]
    per = c["lanes"] if length is None else 1
    pos = s["pos"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for first in range(0, len(pos), per):
        run = [i for i in range(first, first + per) if pos[i] >= 0]
        if not run:
            continue
        last = max(pos[i] for i in run)
        mine = s["cache"][first // per]
        if length is None:
            keys, vals = mine[0, : last + 1], mine[1, : last + 1]
        else:
            f = first // c["beams"]
            keys, vals = (torch.cat([s["prefix"][f, i, : length[f]], mine[i, : last + 1 - length[f]]]) for i in (0, 1))
        at = torch.tensor([pos[i] for i in run], device=DEV)[:, None]
        j = torch.arange(keys.shape[0], device=DEV)[None]
        hidden = j > at
        if c["window"]:
            hidden |= (at - j >= c["window"]) & (j >= c["sinks"])
        for h in range(H):
            cols = slice(h // (H // G) * hd, (h // (H // G) + 1) * hd)
            for a in range(0, len(run), 512):
                part = run[a: a + 512]
                z = s["q"][part, h].double() @ keys[:, cols].double().T * hd ** -0.5
                z.masked_fill_(hidden[a: a + 512], -math.inf)
                e = torch.exp(z - z.max(dim=1, keepdim=True).values)
                out[part, h] = (e @ vals[:, cols].double()) / e.sum(1, keepdim=True)
    return out


def _exact_select(c, s):
    scores = torch.empty((c["groups"], c["n_out"]), dtype=torch.float64, device=DEV)
    done = s["done"].tolist()
    for g in range(c["groups"]):
        cand = []
        for b in range(c["beams"]):
            base = float(s["scores"][g, b])
            if done[g][b]:
                cand.append(torch.tensor([base], dtype=torch.float64, device=DEV))
            elif base > -math.inf:
                row = s["logits"][g * c["beams"] + b].double()
                row = row - torch.logsumexp(row, 0)
                cand.append(torch.topk(row, min(c["n_out"], c["vocab"])).values + base)
        best = torch.cat(cand + [torch.full((c["n_out"],), -math.inf, dtype=torch.float64, device=DEV)])
        scores[g] = torch.topk(best, c["n_out"]).values
    return {"scores": scores, "parents": None, "tokens": None}
