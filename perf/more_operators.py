"""Measured cases of a full-attention layer's operators: rotary positions, attention over packed prompts, attention of
decode steps over a paged cache with a shared prefix, and the page operators of that cache.

`own = False` runs each operator in a plain form of elementary torch operations; `own = True` makes the
calls of `gated_deltanet_linear_step_amd.ops` that a serving loop makes (a prepared call, launched every step).
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ES = {"bf16": 2, "f16": 2, "f32": 4}
HALF, INTERLEAVED = 0, 1
VARLEN = "512,1024,2048,4096,8192,6144,3584,4608"


# ---- cases --------------------------------------------------------------------------------------------

def listed():
    return [
        # the next token of 64 sequences, a quarter of each head turned, keys and values to their pages: latency only
        dict(name="rope decode", op="rope", tokens=64, Hq=16, Hkv=2, D=256, rot=64, layout=HALF, dtype="bf16", far=32768,
             ps=16, scaled=False),
        # neighbouring pairs, whole heads in f32 at far positions of a stretched context, in rows of their own
        dict(name="rope far f32", op="rope", tokens=1537, Hq=8, Hkv=4, D=96, rot=96, layout=INTERLEAVED, dtype="f32",
             far=1000000, ps=0, scaled=True),
        # a long prompt's queries and keys
        dict(name="rope prompt", op="rope", tokens=8192, Hq=32, Hkv=8, D=128, rot=128, layout=HALF, dtype="bf16", far=8192,
             ps=64, scaled=False),
        # a few short prompts, lengths of one, zero and an odd tail: latency of the whole call
        dict(name="prompt short", op="prompt", lens="1,77,0,200,64", past="0,0,0,0,0", Hq=4, Hkv=2, D=64, dtype="f16", ps=0),
        # one prompt of 4096 tokens on wide heads, eight queries to a key head
        dict(name="prompt 4096", op="prompt", lens="4096", past="0", Hq=16, Hkv=2, D=256, dtype="bf16", ps=0),
        # eight packed prompts of mixed lengths
        dict(name="prompt varlen", op="prompt", lens=VARLEN, past="0,0,0,0,0,0,0,0", Hq=32, Hkv=8, D=128, dtype="bf16", ps=0),
        # pieces of prompts that go on: a few tokens against many cached ones on pages
        dict(name="prompt cached", op="prompt", lens="128,333", past="16384,4667", Hq=16, Hkv=4, D=128, dtype="f16", ps=16),
        # one user's next token after a long text: the long axis has to be split
        dict(name="step b1", op="step", B=1, T=1, longest=32768, prefix=0, Hq=16, Hkv=2, D=256, dtype="bf16", ps=64),
        # the serving step of 64 sequences of all lengths
        dict(name="step b64", op="step", B=64, T=1, longest=8192, prefix=0, Hq=32, Hkv=8, D=128, dtype="bf16", ps=16),
        # 64 requests behind one long common text, three drafted tokens verified in one call
        dict(name="step prefix", op="step", B=64, T=3, longest=700, prefix=16000, Hq=16, Hkv=4, D=128, dtype="f16", ps=32),
        # parallel samples of four prompts: the last ones' pages go back, new ones fork, and get room for their tokens
        dict(name="pages fork", op="fork", prompts=4, samples=8, longest=1500, grow=100, planes=24, pages=1024, elems=8192,
             ps=16),
        # half of the requests ended: the others' pages move together
        dict(name="pages compact", op="compact", rows=40, longest=1500, planes=24, pages=2048, elems=8192, ps=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    hkv = rng.choice((1, 2, 4, 8))
    return dict(Hkv=hkv, Hq=hkv * rng.choice((1, 2, 3, 4, 5, 8) if hkv < 8 else (1, 2, 4)), D=rng.choice((64, 96, 128, 256)))


def draw(rng):
    op = rng.choice(("rope", "prompt", "prompt", "step", "step", "fork", "compact"))
    if op in ("fork", "compact"):
        ps = rng.choice((16, 32, 64))
        longest = _log(rng, 10, 1500)
        c = dict(op=op, ps=ps, longest=longest, planes=rng.choice((2, 4, 10, 24)), elems=64 * rng.choice((1, 3, 16, 64, 128)))
        if op == "fork":
            c.update(prompts=rng.choice((1, 2, 3, 4)), samples=rng.choice((1, 2, 5, 8)), grow=rng.choice((0, 1, 30, 100)))
            rows = c["prompts"] * c["samples"]
            need = c["prompts"] * (longest // ps + 1) + rows * (c["grow"] // ps + 2)
        else:
            c.update(rows=rng.choice((2, 3, 10, 25, 40)))
            need = c["rows"] * (longest // ps + 1)
        pages = need + rng.choice((1, 17, 100))
        return dict(c, pages=pages, planes=max(1, min(c["planes"], 2 ** 29 // (pages * c["elems"]))))
    c = dict(op=op, **_heads(rng), dtype=rng.choice(("bf16", "f16")))
    if op == "rope":
        d = c["D"]
        return dict(c, dtype=rng.choice(("bf16", "f16", "f32")), tokens=_log(rng, 1, 4096),
                    rot=rng.choice((d, d, d // 2, d // 4, 2 * rng.randrange(1, d // 2 + 1))), layout=rng.choice((HALF, INTERLEAVED)),
                    far=_log(rng, 10, 1000000), ps=rng.choice((0, 16, 64)), scaled=rng.random() < 0.5)
    if op == "prompt":
        n = rng.choice((1, 1, 2, 3, 5, 8))
        # pairs of tokens, heads and elements of the largest listed case, spread over its factors
        total = max(n, _log(rng, 1, min(12288, 12288 * 32 * 128 // (c["Hq"] * c["D"]))))
        parts = [rng.random() for _ in range(n)]
        lens = [int(total * p / sum(parts)) for p in parts]
        if n > 2 and rng.random() < 0.5:
            lens[rng.randrange(n)] = 0
        if not any(lens):
            lens[-1] = 1
        ps = rng.choice((0, 16, 64))
        past = [_log(rng, 1, 8192) - 1 if ps and k < 2048 else 0 for k in lens]
        return dict(c, lens=",".join(map(str, lens)), past=",".join(map(str, past)), ps=ps)
    B = _log(rng, 1, 64)
    longest = _log(rng, 4, 32768)
    longest = max(4, min(longest, 8192 * 64 * 8 * 128 // (B * c["Hkv"] * c["D"])))
    return dict(c, B=B, T=rng.choice((1, 1, 1, 2, 3, 4)), longest=longest,
                prefix=rng.choice((0, 0, _log(rng, 1, 16000))), ps=rng.choice((16, 32, 64, 128)))


def _ints(text):
    return [int(n) for n in text.split(",")]


def _step_lens(case):
    """Tokens of each sequence in its own pages: the longest, and the others spread below it."""
    B, T, top = case["B"], case["T"], case["longest"]
    return [max(T, top - (top - T) * ((i * 37) % B) // B) for i in range(B)]


def _prompt_lens(case):
    """Lengths of the fork's prompts, or of the compaction's rows: odd ones, the first the longest."""
    n = case["prompts"] if case["op"] == "fork" else case["rows"]
    return [max(1, case["longest"] - (case["longest"] * 5 * i) // (8 * n)) for i in range(n)]


def _moved(case):
    """Pages that a compaction moves, from its inputs alone: in use behind the number of pages in use."""
    refs = _fragmented(case, 0)[1]
    used = int((refs > 0).sum())
    return int((refs[used:] > 0).sum())


def work(case):
    if case["op"] == "rope":
        rows = 2 * case["Hq"] + (4 if case["ps"] else 2) * case["Hkv"]
        return dict(bytes=case["tokens"] * (rows * case["D"] * ES[case["dtype"]] + 4) + 4 * case["rot"],
                    flops=3 * case["tokens"] * (case["Hq"] + case["Hkv"]) * case["rot"])
    if case["op"] in ("fork", "compact"):
        if case["op"] == "fork":
            n = case["samples"] * sum(k % case["ps"] != 0 for k in _prompt_lens(case))
        else:
            n = _moved(case)
        return dict(bytes=2 * max(n, 1) * case["planes"] * case["elems"] * 2 + 4 * case["pages"], flops=0)
    es, Hq, Hkv, D = ES[case["dtype"]], case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "prompt":
        lens, past = _ints(case["lens"]), _ints(case["past"])
        pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(lens, past))
        tokens, keys = sum(lens), sum(n + p for n, p in zip(lens, past))
    else:
        lens, T = _step_lens(case), case["T"]
        pairs = sum(T * (n + case["prefix"]) - T * (T - 1) // 2 for n in lens)
        tokens, keys = case["B"] * T, sum(lens) + case["prefix"]
    return dict(bytes=es * D * (2 * tokens * Hq + 2 * keys * Hkv), flops=4 * pairs * Hq * D)


# ---- inputs -------------------------------------------------------------------------------------------

def _frequencies(rot, scaled):
    """Radians a token of each pair, and what multiplies cosine and sine: plain, or stretched from 8192 to 32 times as
    many tokens, where pairs that turn often keep their frequency and slow ones are divided."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    w = 1e6 ** (-2 * i / rot)
    if not scaled:
        return w, 1.0
    turns = 8192 * w / (2 * math.pi)
    keep = ((turns.log() - math.log(1)) / (math.log(32) - math.log(1))).clamp(0, 1)
    return w * (keep + (1 - keep) / 32), 0.1 * math.log(32) + 1


def _attention_inputs(rand, dt, queries, keys, Hq, Hkv, D):
    """Queries and keys of an order of magnitude that leaves some sharp rows, values with a mean of their own a channel."""
    q = (1.5 * rand(queries, Hq, D)).to(dt)
    k = rand(keys, Hkv, D).to(dt)
    v = (rand(keys, Hkv, D) + 0.5 * rand(Hkv, D)).to(dt)
    return q, k, v


def _on_pages(k, v, lens, ps, gen, spare):
    """Rows of sequences (and of what they share) put on shuffled pages [page][head][token][D]; their tables."""
    need = [-(-n // ps) for n in lens]
    pages = sum(need) + spare
    ids = torch.randperm(pages, generator=gen, device=DEV)
    table = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32, device=DEV)
    pools = [torch.zeros(pages, ps, *x.shape[1:], dtype=x.dtype, device=DEV) for x in (k, v)]
    at = row = 0
    for i, (n, m) in enumerate(zip(lens, need)):
        table[i, :m] = ids[at:at + m].to(torch.int32)
        for pool, x in zip(pools, (k, v)):
            pad = torch.zeros(m * ps, *x.shape[1:], dtype=x.dtype, device=DEV)
            pad[:n] = x[row:row + n]
            pool[ids[at:at + m]] = pad.view(m, ps, *x.shape[1:])
        at, row = at + m, row + n
    k_pages, v_pages = (pool.transpose(1, 2).contiguous() for pool in pools)
    return k_pages, v_pages, table


def _fragmented(case, seed):
    """Page tables of many rows filled in turn, so that their pages lie between one another, after every second row has
    ended; the first two rows share their first pages."""
    ps, lens = case["ps"], _prompt_lens(case)
    width = max(-(-n // ps) for n in lens) + 1
    gen = torch.Generator().manual_seed(seed)
    order = torch.randperm(case["pages"], generator=gen).tolist()
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    refs = torch.zeros(case["pages"], dtype=torch.int32)
    for r, n in enumerate(lens):
        if r % 2 == 0:
            for e in range(-(-n // ps)):
                page = int(table[0, e]) if r == 2 and e < 4 and table[0, e] >= 0 else order.pop()
                table[r, e] = page
                refs[page] += 1
    return table, refs


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    s = dict(case=case)
    if case["op"] in ("fork", "compact"):
        s["pool"] = torch.randn(case["planes"], case["pages"], case["elems"], generator=gen, device=DEV, dtype=torch.bfloat16)
        if case["op"] == "compact":
            table, refs = _fragmented(case, seed)
            s.update(table0=table.to(DEV), refs0=refs.to(DEV))
            s.update(table=s["table0"].clone(), refs=s["refs0"].clone())
            s["page_map"] = torch.empty(case["pages"], dtype=torch.int32, device=DEV)
            s["used"] = torch.empty(1, dtype=torch.int32, device=DEV)
        else:
            lens, ps, n = _prompt_lens(case), case["ps"], case["prompts"] * case["samples"]
            width = max(-(-(k + case["grow"]) // ps) for k in lens)
            table = torch.full((case["prompts"] + n, width), -1, dtype=torch.int32)
            refs = torch.zeros(case["pages"], dtype=torch.int32)
            ids = torch.randperm(case["pages"], generator=torch.Generator().manual_seed(seed)).to(torch.int32)
            at = 0
            for r, k in enumerate(lens):
                m = -(-k // ps)
                table[r, :m] = ids[at:at + m]
                refs[ids[at:at + m].long()] = 1
                at += m
            src = torch.arange(case["prompts"]).repeat_interleave(case["samples"])
            tokens = torch.tensor(lens)[src]
            s.update(table=table.to(DEV), refs=refs.to(DEV), src=src.to(DEV, torch.int32),
                     dst=(torch.arange(n) + case["prompts"]).to(DEV, torch.int32), lens=tokens.to(DEV, torch.int32),
                     grown=(tokens + case["grow"]).to(DEV, torch.int32))
            s["status"], s["status2"] = (torch.empty(n, dtype=torch.int32, device=DEV) for _ in range(2))
    elif case["op"] == "rope":
        n, Hq, Hkv, D, dt = case["tokens"], case["Hq"], case["Hkv"], case["D"], DT[case["dtype"]]
        mixed = rand(n, (Hq + 2 * Hkv) * D).to(dt)  # one row per token, as the projection leaves it
        parts = mixed.split([Hq * D, Hkv * D, Hkv * D], 1)
        s.update({name: x.unflatten(1, (-1, D)) for name, x in zip("qkv", parts)})
        w, s["magnitude"] = _frequencies(case["rot"], case["scaled"])
        s["w"] = w.to(DEV)
        s["positions"] = torch.randint(0, case["far"], (n,), generator=gen, device=DEV).to(torch.int32)
        s["q_out"] = torch.empty(n, Hq, D, dtype=dt, device=DEV)
        if case["ps"]:
            ps = case["ps"]
            pages = -(-n // ps) + 3
            s["k_pages"], s["v_pages"] = (torch.zeros(pages, Hkv, ps, D, dtype=dt, device=DEV) for _ in range(2))
            s["slots"] = torch.randperm(pages * ps, generator=gen, device=DEV)[:n].to(torch.int32)
            if n > 64:  # a prompt's tokens fill its pages in order
                at = torch.arange(n, device=DEV)
                s["slots"] = (torch.randperm(pages, generator=gen, device=DEV)[at // ps] * ps + at % ps).to(torch.int32)
        else:
            s["k_out"] = torch.empty(n, Hkv, D, dtype=dt, device=DEV)
    elif case["op"] == "prompt":
        lens, past = _ints(case["lens"]), _ints(case["past"])
        both = [n + p for n, p in zip(lens, past)]
        s["q"], s["k"], s["v"] = _attention_inputs(rand, DT[case["dtype"]], sum(lens), sum(both), case["Hq"], case["Hkv"], case["D"])
        for name, of in (("q", lens), ("k", both)):
            s["cu_%s_host" % name] = torch.tensor([0] + of).cumsum(0).to(torch.int32)
            s["cu_" + name] = s["cu_%s_host" % name].to(DEV)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(sum(lens), case["Hq"], device=DEV) if case["ps"] else None
        if case["ps"]:
            s["k"], s["v"], s["table"] = _on_pages(s["k"], s["v"], both, case["ps"], gen, 3)
    else:
        B, T, lens, prefix = case["B"], case["T"], _step_lens(case), case["prefix"]
        q, k, v = _attention_inputs(rand, DT[case["dtype"]], B * T, sum(lens) + prefix, case["Hq"], case["Hkv"], case["D"])
        s["k"], s["v"], tables = _on_pages(k, v, [prefix] + lens, case["ps"], gen, 3)
        s.update(q=q, out=torch.empty_like(q), lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
        s["table"] = tables[1:, :-(-max(lens) // case["ps"])].contiguous()
        s["prefix"] = tables[0, :-(-prefix // case["ps"])].contiguous() if prefix else None
        s["lse"] = torch.empty(B * T, case["Hq"], device=DEV) if prefix else None
    if own:  # the launcher that a serving loop builds once and keeps; it holds no data beyond these tensors
        s["calls"] = _prepared(s)
    return s


def _prepared(s):
    from gated_deltanet_linear_step_amd import ops
    c = s["case"]
    if c["op"] == "rope":
        to = dict(k_pages=s["k_pages"], v_pages=s["v_pages"], v=s["v"], slots=s["slots"]) if c["ps"] else dict(k_out=s["k_out"])
        return [ops.prepare_rope(s["positions"], s["w"], q=s["q"], q_out=s["q_out"], k=s["k"], magnitude=s["magnitude"],
                                 layout=(ops.ROPE_HALF, ops.ROPE_INTERLEAVED)[c["layout"]], **to)]
    if c["op"] == "prompt":
        need = ops.attention_prefill_workspace_bytes(Hq=c["Hq"], Hkv=c["Hkv"], head_dim=c["D"], num_seqs=len(_ints(c["lens"])),
                                                     total_tokens=sum(_ints(c["lens"])))
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)
        return [ops.prepare_attention_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_q_host"], s["out"], workspace,
                                              cu_k=s["cu_k"], cu_k_host=s["cu_k_host"], table=s.get("table"), lse=s["lse"])]
    if c["op"] == "step":
        need = ops.attention_decode_workspace_bytes(Hq=c["Hq"], Hkv=c["Hkv"], head_dim=c["D"], batch=c["B"],
                                                    tokens_per_seq=c["T"], max_len=c["longest"], prefix_len=c["prefix"])
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)
        return [ops.prepare_attention_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], s["out"], workspace, batch=c["B"],
                                             tokens_per_seq=c["T"], max_len=c["longest"], prefix_table=s["prefix"],
                                             prefix_len=c["prefix"], lse=s["lse"])]
    workspace = torch.empty(max(ops.pages_workspace_bytes(c["pages"]), 256), dtype=torch.uint8, device=DEV)
    if c["op"] == "compact":
        return [ops.prepare_pages_compact(s["pool"], s["table"], s["refs"], s["page_map"], s["used"], workspace)]
    return [ops.prepare_pages_free(s["table"], s["refs"], s["dst"]),
            ops.prepare_pages_fork(s["pool"], s["table"], s["refs"], s["src"], s["dst"], s["lens"], s["status"], workspace,
                                   page_size=c["ps"]),
            ops.prepare_pages_reserve(s["table"], s["refs"], s["dst"], s["grown"], s["status2"], page_size=c["ps"])]


# ---- one pass -----------------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if op == "compact":  # the tables as the program holds them before the pass
        s["table"].copy_(s["table0"])
        s["refs"].copy_(s["refs0"])
    if own:
        for call in s["calls"]:
            call.launch()
    else:
        {"rope": _rope, "prompt": _prompt, "step": _step, "fork": _fork, "compact": _compact}[op](s)
    names = {"rope": ("q_out", "k_out", "k_pages", "v_pages"), "prompt": ("out", "lse"), "step": ("out", "lse"),
             "fork": ("pool", "table", "refs", "status", "status2"), "compact": ("pool", "table", "refs", "page_map", "used")}[op]
    return {name: s[name] for name in names if s.get(name) is not None}


def _pairs(x, rot, layout):
    return (x[..., :rot // 2], x[..., rot // 2:rot]) if layout == HALF else (x[..., :rot:2], x[..., 1:rot:2])


def _rope(s):
    c = s["case"]
    rot, layout = c["rot"], c["layout"]
    angle = s["positions"].double()[:, None, None] * s["w"]
    cos, sin = ((f(angle) * s["magnitude"]).float() for f in (torch.cos, torch.sin))

    def turn(x, to):
        to.copy_(x)
        a, b = (y.float() for y in _pairs(x, rot, layout))
        left, right = _pairs(to, rot, layout)
        left.copy_(a * cos - b * sin)
        right.copy_(b * cos + a * sin)
        return to

    turn(s["q"], s["q_out"])
    if not c["ps"]:
        turn(s["k"], s["k_out"])
        return
    at = s["slots"].long()
    page, token = at // c["ps"], at % c["ps"]
    s["k_pages"][page, :, token] = turn(s["k"], torch.empty_like(s["k"]))
    s["v_pages"][page, :, token] = s["v"]


def _softmax_values(scores, v):
    """softmax(scores) v over the last axis and its log-sum; rows without a key are 0 and -inf."""
    top = scores.amax(-1, keepdim=True).clamp_min(-1e30)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    return (p @ v) / total.clamp_min(1e-30), (top + total.log()).squeeze(-1)


def _prompt(s):
    c = s["case"]
    Hkv, D, G = c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    cu_q, cu_k = s["cu_q_host"].tolist(), s["cu_k_host"].tolist()
    for i in range(len(cu_q) - 1):  # each prompt's own products: a padded batch would compute several times as much
        a, b, n = cu_q[i], cu_q[i + 1], cu_k[i + 1] - cu_k[i]
        if a == b:
            continue
        if c["ps"]:
            at = s["table"][i, :-(-n // c["ps"])].long()
            k, v = (s[x][at].transpose(1, 2).flatten(0, 1)[:n].float() for x in "kv")
        else:
            k, v = (s[x][cu_k[i]:cu_k[i + 1]].float() for x in "kv")
        q = s["q"][a:b].float().view(b - a, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * (b - a), D)
        scores = (q @ k.permute(1, 2, 0)).mul_(D ** -0.5).view(Hkv, G, b - a, n)
        hidden = torch.ones(b - a, n, dtype=torch.bool, device=DEV).triu_(n - (b - a) + 1)
        scores.masked_fill_(hidden, -math.inf)
        o, lse = _softmax_values(scores.view(Hkv, G * (b - a), n), v.transpose(0, 1))
        s["out"][a:b] = o.view(Hkv, G, b - a, D).permute(2, 0, 1, 3).reshape(b - a, -1, D)
        if s["lse"] is not None:
            s["lse"][a:b] = lse.view(Hkv * G, b - a).t()


def _step(s):
    c = s["case"]
    B, T, Hkv, D, G = c["B"], c["T"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    at = s["table"].long().clamp_min(0)
    k, v = (s[x][at].transpose(1, 2).flatten(2, 3).float() for x in "kv")       # [B, Hkv, keys, D]
    q = s["q"].float().view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D) * D ** -0.5
    scores = (q @ k.transpose(2, 3)).view(B, Hkv, T, G, -1)
    seen = s["lens"][:, None] - (T - 1) + torch.arange(T, device=DEV)           # keys that token t sees
    hidden = torch.arange(k.shape[2], device=DEV) >= seen[..., None]            # [B, T, keys]
    scores = scores.masked_fill_(hidden[:, None, :, None], -math.inf).view(B, Hkv, T * G, -1)
    if c["prefix"]:  # its products once for all rows
        shared = s["prefix"].long()
        kp, vp = (s[x][shared].transpose(0, 1).flatten(1, 2)[:, :c["prefix"]].float() for x in "kv")  # [Hkv, prefix, D]
        rows = q.transpose(0, 1).reshape(Hkv, B * T * G, D)
        front = (rows @ kp.transpose(1, 2)).view(Hkv, B, T * G, -1).transpose(0, 1)
        top = torch.maximum(scores.amax(-1, keepdim=True), front.amax(-1, keepdim=True))
        p, pf = (scores - top).exp_(), (front - top).exp_()
        total = p.sum(-1, keepdim=True) + pf.sum(-1, keepdim=True)
        o = pf.transpose(0, 1).reshape(Hkv, B * T * G, -1) @ vp
        o = (p @ v + o.view(Hkv, B, T * G, D).transpose(0, 1)) / total
        lse = (top + total.log()).squeeze(-1)
    else:
        o, lse = _softmax_values(scores, v)
    s["out"].copy_(o.view(B, Hkv, T, G, D).transpose(1, 2).reshape(s["out"].shape))
    if s["lse"] is not None:
        s["lse"].copy_(lse.view(B, Hkv, T, G).transpose(1, 2).reshape(B * T, -1))


def _lowest_free(refs):
    """Pages in the order in which they are handed out: the free ones, the lowest first."""
    return torch.sort((refs > 0).to(torch.int32), stable=True).indices.to(torch.int32)


def _count(refs, pages, by):
    """refs += by at every page of the list that is one (>= 0)."""
    refs.index_add_(0, pages.clamp_min(0).flatten().long(), (pages >= 0).flatten().to(torch.int32) * by)


def _fork(s):
    table, refs, ps = s["table"], s["refs"], s["case"]["ps"]
    src, dst, lens, grown = (s[n].long() for n in ("src", "dst", "lens", "grown"))
    entry = torch.arange(table.shape[1], device=DEV)
    # free: what the rows held goes back
    _count(refs, table[dst], -1)
    table[dst] = -1
    # fork: full pages are shared, one that is filled in part is copied (pages are enough in every case here)
    part = lens % ps != 0
    full = lens // ps
    new = _lowest_free(refs)[(part.cumsum(0) - part.long())]
    rows = torch.where(entry < full[:, None], table[src], -1)
    rows = torch.where(part[:, None] & (entry == full[:, None]), new[:, None], rows)
    last = table[src].gather(1, full.clamp_max(table.shape[1] - 1)[:, None])[:, 0].long()
    first = table[src][:, 0].long()  # copied onto itself where no page is filled in part
    s["pool"][:, torch.where(part, new.long(), first)] = s["pool"][:, torch.where(part, last, first)]
    _count(refs, rows, 1)
    table[dst] = rows
    s["status"].zero_()
    # reserve: pages for the tokens to come
    need = (entry < ((grown + ps - 1) // ps)[:, None]) & (table[dst] < 0)
    order = need.flatten().cumsum(0).view(need.shape) - 1
    rows = torch.where(need, _lowest_free(refs)[order.clamp_min(0)], table[dst])
    _count(refs, torch.where(need, rows, -1), 1)
    table[dst] = rows
    s["status2"].zero_()


def _compact(s):
    table, refs = s["table"], s["refs"]
    pages = refs.shape[0]
    used = refs > 0
    count = used.sum()
    at = torch.arange(pages, device=DEV)
    # the i-th page in use behind the count goes to the i-th free one before it; other pages keep their place
    far = used & (at >= count)
    hole = _lowest_free(refs)  # the first `far.sum()` of them lie before the count
    rank = far.long().cumsum(0) - 1
    to = torch.where(far, hole[rank.clamp_min(0)].long(), at)
    moved = torch.sort(far.to(torch.int32), stable=True, descending=True).indices[:pages // 2]  # at most half of all move
    moved = torch.where(far[moved], moved, moved[0])  # what is left of the list repeats its first page
    s["pool"][:, to[moved]] = s["pool"][:, moved]
    s["page_map"].copy_(to)
    s["used"].copy_(count)
    refs.copy_(torch.where(at < count, torch.zeros_like(refs).index_add_(0, to, refs * used), 0))
    table.copy_(torch.where(table >= 0, to[table.clamp_min(0).long()].to(torch.int32), table))


# ---- the definitions in 64 bits -----------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _rope64, "prompt": _prompt64, "step": _step64, "fork": _fork64, "compact": _compact64}[case["op"]](s)


def _rope64(s):
    c = s["case"]
    half = c["rot"] // 2
    # pairs as complex numbers, times m e^(i p w)
    turn = torch.polar(torch.full_like(s["w"], s["magnitude"]).expand(c["tokens"], -1), s["positions"].double()[:, None] * s["w"])
    got = {}
    for name in "qk":
        x = s[name].double()
        if c["layout"] == HALF:
            z = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * turn[:, None]
            got[name] = torch.cat([z.real, z.imag, x[..., 2 * half:]], -1)
        else:
            z = torch.view_as_complex(x[..., :2 * half].unflatten(-1, (half, 2)).contiguous()) * turn[:, None]
            got[name] = torch.cat([torch.view_as_real(z).flatten(-2), x[..., 2 * half:]], -1)
    if not c["ps"]:
        return dict(q_out=got["q"], k_out=got["k"])
    pools = []
    for x in (got["k"], s["v"].double()):
        flat = torch.zeros(s["k_pages"].shape[0] * c["ps"], c["Hkv"], c["D"], dtype=torch.float64, device=DEV)
        flat[s["slots"].long()] = x
        pools.append(flat.view(-1, c["ps"], c["Hkv"], c["D"]).transpose(1, 2))
    return dict(q_out=got["q"], k_pages=pools[0], v_pages=pools[1])


def _rows64(q, k, v, seen):
    """Attention of the rows q [n, D] over the keys before seen [n], a block of rows at a time."""
    out, lse = [], []
    for i in range(0, len(q), 2048):
        top = int(seen[i:i + 2048].max())
        z = q[i:i + 2048] @ k[:top].t() / math.sqrt(q.shape[1])
        z[torch.arange(top, device=DEV)[None] >= seen[i:i + 2048, None]] = -math.inf
        lse.append(torch.logsumexp(z, 1))
        out.append(torch.exp(z - lse[-1][:, None]) @ v[:top])
    return torch.cat(out), torch.cat(lse)


def _gathered(s, i, n):
    """Keys and values of the first n tokens of table row i (a list of pages where i is one), [n, Hkv, D]."""
    pages = (s["table"][i] if isinstance(i, int) else i).tolist()[:-(-n // s["case"]["ps"])]
    return (torch.cat([s[x][p].transpose(0, 1) for p in pages] or [s[x][0, :, :0].transpose(0, 1)])[:n].double() for x in "kv")


def _prompt64(s):
    c = s["case"]
    cu_q, cu_k, G = s["cu_q"].tolist(), s["cu_k"].tolist(), c["Hq"] // c["Hkv"]
    if work(case=c)["flops"] > 1e13:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    for i in range(len(cu_q) - 1):
        a, b, n = cu_q[i], cu_q[i + 1], cu_k[i + 1] - cu_k[i]
        if a == b:
            continue
        k, v = _gathered(s, i, n) if c["ps"] else (s[x][cu_k[i]:cu_k[i + 1]].double() for x in "kv")
        seen = n - (b - a) + 1 + torch.arange(b - a, device=DEV)
        for h in range(c["Hq"]):
            out[a:b, h], lse[a:b, h] = _rows64(s["q"][a:b, h].double(), k[:, h // G], v[:, h // G], seen)
    return dict(out=out) if s["lse"] is None else dict(out=out, lse=lse)


def _step64(s):
    c = s["case"]
    G, T = c["Hq"] // c["Hkv"], c["T"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    front = tuple(_gathered(s, s["prefix"], c["prefix"])) if c["prefix"] else None
    for b, n in enumerate(s["lens"].tolist()):
        k, v = _gathered(s, b, n)
        if front:
            k, v = torch.cat([front[0], k]), torch.cat([front[1], v])
        seen = len(k) - T + 1 + torch.arange(T, device=DEV)
        for h in range(c["Hkv"]):
            q = s["q"][b * T:(b + 1) * T, h * G:(h + 1) * G].double().flatten(0, 1)
            o, l = _rows64(q, k[:, h], v[:, h], seen.repeat_interleave(G))
            out[b * T:(b + 1) * T, h * G:(h + 1) * G] = o.view(T, G, -1)
            lse[b * T:(b + 1) * T, h * G:(h + 1) * G] = l.view(T, G)
    return dict(out=out) if s["lse"] is None else dict(out=out, lse=lse)


def _fork64(s):
    table, refs, ps = s["table"].tolist(), s["refs"].tolist(), s["case"]["ps"]
    pool = s["pool"].clone()
    for r in s["dst"].tolist():
        for page in table[r]:
            refs[page] -= page >= 0
        table[r] = [-1] * len(table[r])
    jobs = list(zip(*(s[n].tolist() for n in ("src", "dst", "lens", "grown"))))
    for a, b, n, _ in jobs:
        for e in range(-(-n // ps)):
            table[b][e] = table[a][e] if (e + 1) * ps <= n else refs.index(0)
            refs[table[b][e]] += 1
            if (e + 1) * ps > n:
                pool[:, table[b][e]] = pool[:, table[a][e]]
    for _, b, _, n in jobs:
        for e in range(-(-n // ps)):
            if table[b][e] < 0:
                table[b][e] = refs.index(0)
                refs[table[b][e]] = 1
    return dict(pool=pool.double(), table=torch.tensor(table, dtype=torch.int32), refs=torch.tensor(refs, dtype=torch.int32),
                status=torch.zeros(len(jobs), dtype=torch.int32), status2=torch.zeros(len(jobs), dtype=torch.int32))


def _compact64(s):
    table, refs, pool = s["table0"].tolist(), s["refs0"].tolist(), s["pool"].clone()
    count, to = sum(r > 0 for r in refs), list(range(len(refs)))
    for page in range(count, len(refs)):
        if refs[page] > 0:
            to[page] = refs.index(0)
            pool[:, to[page]] = pool[:, page]
            refs[to[page]], refs[page] = refs[page], 0
    table = [[to[page] if page >= 0 else page for page in row] for row in table]
    whole = {name: torch.tensor(x, dtype=torch.int32) for name, x in dict(table=table, refs=refs, page_map=to, used=[count]).items()}
    return dict(pool=pool.double(), **whole)
