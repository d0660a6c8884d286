"""Measured cases of the decayed linear attention (decode and prefill), the RMS norm with residual and 8-bit
output, and the int8 product with token and channel scales.

`own = False` runs each operator in a plain form of elementary torch operations; `own = True` makes the
calls of `gated_deltanet_linear_step_amd.ops` that a serving loop makes (a prepared call, launched every step).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ES = {"bf16": 2, "f16": 2, "f32": 4}
GROUPED, TILED = 0, 1
SHAPES = ((32, 32), (64, 64), (96, 96), (128, 128), (64, 128), (128, 64), (128, 256), (256, 128), (256, 256))
VARLEN = "512,1024,2048,4096,8192,6144,3584,4608"


# ---- cases --------------------------------------------------------------------------------------------

def listed():
    return [
        # one user's next token through one layer of a 48-head model: latency only
        dict(name="decode b1", op="decode", B=1, T=1, Hk=16, Hv=48, dk=128, dv=128, map=TILED, dtype="bf16",
             decay="head", slots=False),
        # the serving step of 64 sequences, fixed decay for each head; every state streams through once
        dict(name="decode b64", op="decode", B=64, T=1, Hk=16, Hv=32, dk=128, dv=128, map=TILED, dtype="bf16",
             decay="head", slots=False),
        # drafted tokens verified in one call, an odd batch out of a slot pool, decay given per token
        dict(name="decode b37 t5 slots", op="decode", B=37, T=5, Hk=8, Hv=16, dk=64, dv=128, map=GROUPED, dtype="f16",
             decay="token", slots=True),
        # a few short prompts in f32, lengths of one, zero and an odd tail: latency of the whole call
        dict(name="prefill short f32", op="prefill", lens="1,77,0,200,64", Hk=2, Hv=4, dk=64, dv=64, map=GROUPED,
             dtype="f32", decay="token"),
        # one prompt of 4096 tokens: few rows, so the long axis has to be split
        dict(name="prefill t4096", op="prefill", lens="4096", Hk=16, Hv=32, dk=128, dv=128, map=GROUPED, dtype="bf16",
             decay="head"),
        # eight packed prompts of mixed lengths, decay per token, states carried in
        dict(name="prefill varlen", op="prefill", lens=VARLEN, Hk=16, Hv=32, dk=128, dv=128, map=TILED, dtype="bf16",
             decay="token"),
        # the norm before a decode step's projections: 64 rows
        dict(name="norm decode", op="norm", rows=64, hidden=2048, dtype="bf16", residual=True, out16=False, q8=True),
        # the same for a prompt, with the 16-bit rows kept too (the small gate projections read them)
        dict(name="norm prompt", op="norm", rows=8192, hidden=4096, dtype="bf16", residual=True, out16=True, q8=True),
        # a width that no vector load divides, no residual, 16-bit rows only
        dict(name="norm odd", op="norm", rows=1537, hidden=5003, dtype="f16", residual=False, out16=True, q8=False),
        # the mixed-row projection of a decode step of 64 sequences: the weights stream through once
        dict(name="matmul decode", op="matmul", M=64, N=8192, K=2048, dtype="bf16"),
        # the output projection of a ragged prompt; no size divides a tile
        dict(name="matmul ragged", op="matmul", M=1001, N=2050, K=4112, dtype="f16"),
        # the mixed-row projection of a long prompt: bound by the matrix units
        dict(name="matmul prompt", op="matmul", M=8192, N=8192, K=2048, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    hk = rng.choice((1, 2, 4, 8, 16))
    return hk, hk * rng.choice((1, 2, 3) if hk == 16 else (1, 2, 3, 4))


def draw(rng):
    op = rng.choice(("decode", "prefill", "norm", "matmul"))
    if op in ("decode", "prefill"):
        hk, hv = _heads(rng)
        dk, dv = rng.choice(SHAPES)
        c = dict(op=op, Hk=hk, Hv=hv, dk=dk, dv=dv, map=rng.choice((GROUPED, TILED)),
                 dtype=rng.choice(("bf16", "bf16", "f16", "f32")), decay=rng.choice(("head", "token")))
        if op == "decode":
            top = max(1, min(96, 64 * 32 * 128 * 128 // (hv * dk * dv)))
            return dict(c, B=_log(rng, 1, top), T=rng.choice((1, 1, 1, 2, 3, 4, 6, 8)), slots=rng.random() < 0.5)
        n = rng.choice((1, 1, 2, 3, 5, 8, 16))
        # 1/16 of the largest listed case in f32 arithmetic on wide heads, the whole of it on narrow ones
        top = max(n, min(30208, 4096 * 32 * 128 * 128 // (hv * dk * dv)))
        total = max(n, _log(rng, 1, top))
        parts = [rng.random() for _ in range(n)]
        lens = [int(total * p / sum(parts)) for p in parts]
        if n > 2 and rng.random() < 0.5:
            lens[rng.randrange(n)] = 0
        if not any(lens):
            lens[-1] = 1
        return dict(c, lens=",".join(map(str, lens)))
    if op == "norm":
        hidden = _log(rng, 64, 8192)
        q8 = rng.random() < 0.7
        return dict(op=op, rows=_log(rng, 1, 4096), hidden=hidden // 16 * 16 if q8 else hidden,
                    dtype=rng.choice(("bf16", "bf16", "f16", "f32")), residual=rng.random() < 0.7,
                    out16=(not q8) or rng.random() < 0.4, q8=q8)
    return dict(op=op, M=_log(rng, 1, 4096), N=_log(rng, 16, 8192), K=16 * _log(rng, 4, 400),
                dtype=rng.choice(("bf16", "bf16", "f16", "f32")))


def _lens(case):
    return [int(n) for n in case["lens"].split(",")]


def work(case):
    es = ES[case["dtype"]]
    if case["op"] in ("decode", "prefill"):
        hk, hv, dk, dv = case["Hk"], case["Hv"], case["dk"], case["dv"]
        lens = [case["T"]] * case["B"] if case["op"] == "decode" else _lens(case)
        tokens = sum(lens)
        g = 4 * hv * (tokens if case["decay"] == "token" else 1)
        moved = tokens * es * (2 * hk * dk + 2 * hv * dv) + g + 8 * sum(n > 0 for n in lens) * hv * dk * dv
        return dict(bytes=moved, flops=4 * tokens * hv * dk * dv)
    if case["op"] == "norm":
        n = case["rows"] * case["hidden"]
        moved = n * es * (1 + 2 * case["residual"] + case["out16"]) + case["q8"] * (n + 4 * case["rows"])
        return dict(bytes=moved + 4 * case["hidden"], flops=(5 + 3 * case["q8"]) * n)
    M, N, K = case["M"], case["N"], case["K"]
    return dict(bytes=M * K + N * K + M * N * es + 4 * (M + N), flops=2 * M * N * K)


# ---- inputs -------------------------------------------------------------------------------------------

def _attention_inputs(case, tokens, slots, rand):
    hk, hv, dk, dv, dt = case["Hk"], case["Hv"], case["dk"], case["dv"], DT[case["dtype"]]
    # one mixed row per token, as a projection or gdn_conv_update leaves it; keys of about unit length
    mixed = rand(tokens, 2 * hk * dk + hv * dv)
    mixed[:, hk * dk:2 * hk * dk] *= dk ** -0.5
    mixed = mixed.to(dt)
    s = dict(case=case, q=mixed[:, :hk * dk], k=mixed[:, hk * dk:2 * hk * dk], v=mixed[:, 2 * hk * dk:],
             state=rand(slots, hv, dv, dk) * 0.1, out=torch.empty(tokens, hv, dv, dtype=dt, device=DEV), g=None, rate=None)
    if case["decay"] == "head":
        # decays 1 - 2^-5 ... 1 - 2^-9 over the heads
        s["rate"] = torch.log1p(-torch.exp2(-5 - 4 * torch.arange(hv, device=DEV, dtype=torch.float32) / max(1, hv - 1)))
        s["rate"] *= 1 + 0.05 * rand(hv).clamp(-1, 1)
    else:
        # a rate for each head times the softplus of a projection
        s["g"] = -0.15 * torch.nn.functional.softplus(rand(tokens, hv) - 1)
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    dt = DT[case["dtype"]]
    if case["op"] == "decode":
        B, T = case["B"], case["T"]
        s = _attention_inputs(case, B * T, B + (5 if case["slots"] else 0), rand)
        s["slots"] = torch.randperm(B + 5, generator=gen, device=DEV)[:B].to(torch.int32) if case["slots"] else None
    elif case["op"] == "prefill":
        lens = _lens(case)
        s = _attention_inputs(case, sum(lens), len(lens), rand)
        s["cu_host"] = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
        s["cu"] = s["cu_host"].to(DEV)
    elif case["op"] == "norm":
        rows, hidden = case["rows"], case["hidden"]
        # a residual stream: some channels much larger than the rest
        channel = torch.exp(0.7 * rand(hidden))
        s = dict(case=case, x=(rand(rows, hidden) * channel).to(dt), weight=1 + 0.1 * rand(hidden),
                 residual=(rand(rows, hidden) * channel).to(dt) if case["residual"] else None)
        s["residual_out"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["out"] = torch.empty_like(s["x"]) if case["out16"] else None
        s["out_q"] = torch.empty(rows, hidden, dtype=torch.int8, device=DEV) if case["q8"] else None
        s["out_scale"] = torch.empty(rows, device=DEV) if case["q8"] else None
        s["values"] = torch.empty(rows, hidden, dtype=torch.bfloat16, device=DEV) if case["q8"] else None
    else:
        M, N, K = case["M"], case["N"], case["K"]

        def rows8(n):  # normal rows in 8 bits, the largest of each at 127
            x = rand(n, K)
            top = x.abs().amax(1, keepdim=True)
            return (x * (127 / top)).round().to(torch.int8), (top / 127).flatten()

        s = dict(case=case, out=torch.empty(M, N, dtype=dt, device=DEV))
        s["a"], s["a_scale"] = rows8(M)
        s["w"], s["w_scale"] = rows8(N)
        s["w_scale"] = s["w_scale"] * K ** -0.5
    if own:  # the launcher that a serving loop builds once and keeps; it holds no data beyond these tensors
        s["call"] = _prepared(s)
    return s


def _prepared(s):
    from gated_deltanet_linear_step_amd import ops
    case = s["case"]
    if case["op"] == "norm":
        return ops.prepare_add_rms_norm(s["x"], s["weight"], residual=s["residual"], residual_out=s["residual_out"],
                                        out=s["out"], out_q=s["out_q"], out_scale=s["out_scale"], eps=1e-6)
    if case["op"] == "matmul":
        return ops.prepare_quant_matmul(s["a"], s["a_scale"], s["w"], s["w_scale"], s["out"])
    heads = dict(Hk=case["Hk"], Hv=case["Hv"], dk=case["dk"], dv=case["dv"], head_map=case["map"])
    heads.update(dict(g=s["g"]) if s["rate"] is None else dict(decay_param=s["rate"], decay=ops.DECAY_NEGATIVE_RATE))
    if case["op"] == "decode":
        return ops.prepare_linattn_decode_step(s["q"], s["k"], s["v"], s["state"], s["out"], batch=case["B"],
                                               tokens_per_seq=case["T"], state_slots=s["slots"], **heads)
    need = ops.linattn_prefill_workspace_bytes(num_seqs=len(_lens(case)), total_tokens=s["q"].shape[0],
                                               Hk=case["Hk"], Hv=case["Hv"], dk=case["dk"], dv=case["dv"])
    workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)
    return ops.prepare_linattn_prefill_chunked(s["q"], s["k"], s["v"], s["state"], s["cu"], s["cu_host"], s["out"],
                                               workspace, **heads)


# ---- one pass -----------------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        s["call"].launch()
        if op == "norm":
            return _norm_outputs(s, s["out_q"], s["out_scale"])
        return dict(out=s["out"]) if op == "matmul" else dict(out=s["out"], state=s["state"])
    return {"decode": _decode, "prefill": _prefill, "norm": _norm, "matmul": _matmul}[op](s)


def _norm_outputs(s, out_q, out_scale):
    """The rows in 8 bits as the values they stand for (bf16 holds as many bits), with the scales: one more
    pass over them on either side."""
    got = dict(out=s["out"], residual=s["residual_out"])
    if out_q is not None:
        got.update(scale=out_scale, q8=torch.mul(out_q, out_scale[:, None], out=s["values"]))
    return {k: v for k, v in got.items() if v is not None}


def _k_head(case, device):
    h = torch.arange(case["Hv"], device=device)
    return h // (case["Hv"] // case["Hk"]) if case["map"] == GROUPED else h % case["Hk"]


def _log_decay(s, tokens):
    return s["g"] if s["rate"] is None else s["rate"].expand(tokens, -1)


def _tokens(s):
    """q, k [tokens, Hv, dk], v [tokens, Hv, dv] in 32 bits and g [tokens, Hv] in 64."""
    c, t = s["case"], s["q"].shape[0]
    at = _k_head(c, DEV)
    q, k = (s[n].reshape(t, c["Hk"], c["dk"])[:, at].float() for n in "qk")
    return q, k, s["v"].reshape(t, c["Hv"], c["dv"]).float(), _log_decay(s, t).double()


def _chunk(q, k, v, g):
    """Chunks [..., C, d] with log decays g [..., C]: the outputs of the chunk's own tokens, the factors of the
    entering state for each token, and what the chunk adds to the state."""
    G = g.cumsum(-1)
    C = g.shape[-1]
    below = torch.ones(C, C, dtype=torch.bool, device=g.device).tril()
    D = torch.where(below, torch.exp(G[..., :, None] - G[..., None, :]), 0.0).float()
    own_out = (q @ k.transpose(-1, -2) * D) @ v
    left = torch.exp(G[..., -1:] - G).float()
    return own_out, torch.exp(G).float(), (v * left[..., None]).transpose(-1, -2) @ k


def _decode(s):
    c = s["case"]
    B, T = c["B"], c["T"]
    q, k, v, g = (x.unflatten(0, (B, T)).transpose(1, 2) for x in _tokens(s))
    at = torch.arange(B, device=DEV) if s["slots"] is None else s["slots"].long()
    S = s["state"][at]
    own_out, enter, add = _chunk(q, k, v, g)
    o = (own_out + enter[..., None] * (q @ S.transpose(-1, -2))) * c["dk"] ** -0.5
    s["out"].copy_(o.transpose(1, 2).reshape(s["out"].shape))
    s["state"][at] = S * enter[..., -1, None, None] + add
    return dict(out=s["out"], state=s["state"])


def _prefill(s, C=64):
    c = s["case"]
    q, k, v, g = _tokens(s)
    cu = s["cu"].long()
    lens = cu[1:] - cu[:-1]
    chunks = (s["cu_host"].long().diff() + C - 1) // C  # on the host: shapes follow from it
    n = int(chunks.sum())
    seq = torch.repeat_interleave(torch.arange(len(lens)), chunks).to(DEV)
    first = (chunks.cumsum(0) - chunks).to(DEV)
    row = (torch.arange(n, device=DEV) - first[seq])[:, None] * C + torch.arange(C, device=DEV)
    there = row < lens[seq][:, None]
    at = torch.where(there, row + cu[seq][:, None], 0)

    def tiles(x):  # [n, Hv, C, ...], zero behind a sequence's end
        x = x[at] * there.reshape(n, C, *[1] * (x.dim() - 1)).to(x.dtype)
        return x.transpose(1, 2)

    q, k, v, g = tiles(q), tiles(k), tiles(v), tiles(g)
    own_out, enter, add = _chunk(q, k, v, g)
    # state at each chunk's start, and at each sequence's end: a product over the sequence's chunks
    total = g.sum(-1)                                        # [n, Hv]
    run_ = total.cumsum(0)
    run0 = run_ - total
    base = torch.cat([run0, torch.zeros_like(run0[:1])])[first.clamp(max=n)]   # before each sequence [N, Hv]
    ends = torch.cat([torch.zeros_like(run_[:1]), run_])[first + chunks.to(DEV)]
    upto = torch.cat([run0, ends])                           # [n + N, Hv]
    whose = torch.cat([seq, torch.arange(len(lens), device=DEV)])
    idx = torch.arange(n, device=DEV)
    limit = torch.cat([idx, first + chunks.to(DEV)])
    see = (whose[:, None] == seq[None]) & (idx[None] < limit[:, None])
    W = torch.where(see[..., None], torch.exp(upto[:, None] - run_[None]), 0.0).float()     # [n + N, n, Hv]
    S = W.permute(2, 0, 1) @ add.transpose(0, 1).reshape(c["Hv"], n, -1)
    S = S.transpose(0, 1).reshape(-1, c["Hv"], c["dv"], c["dk"])
    S += torch.exp(upto - base[whose]).float()[..., None, None] * s["state"][whose]
    o = (own_out + enter[..., None] * (q @ S[:n].transpose(-1, -2))) * c["dk"] ** -0.5
    s["out"].copy_(o.transpose(1, 2)[there])
    s["state"].copy_(S[n:])
    return dict(out=s["out"], state=s["state"])


def _norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
        s["residual_out"].copy_(h)
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * s["weight"]
    if s["out"] is not None:
        s["out"].copy_(y)
    if s["out_q"] is None:
        return _norm_outputs(s, None, None)
    top = y.abs().amax(1, keepdim=True)
    s["out_q"].copy_((y * (127 / top)).round())
    s["out_scale"].copy_(top.flatten() / 127)
    return _norm_outputs(s, s["out_q"], s["out_scale"])


def _matmul(s):
    # sums of 1024 products of 8-bit values stay below 2^24, so each block is exact in 32 bits
    K = s["a"].shape[1]
    pad = -K % 1024
    a, w = (torch.nn.functional.pad(s[n].float(), (0, pad)).unflatten(1, (-1, 1024)).transpose(0, 1) for n in "aw")
    total = (a @ w.transpose(1, 2)).sum(0, dtype=torch.float64)
    s["out"].copy_(total * s["a_scale"][:, None] * s["w_scale"])
    return dict(out=s["out"])


# ---- the definitions in 64 bits -----------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "matmul":
        total = s["a"].double() @ s["w"].double().t()
        return dict(out=total * s["a_scale"].double()[:, None] * s["w_scale"].double())
    if case["op"] == "norm":
        h = s["x"].double() + (s["residual"].double() if case["residual"] else 0)
        y = h / (h.pow(2).mean(1, keepdim=True) + 1e-6).sqrt() * s["weight"].double()
        step = y.abs().amax(1) / 127
        got = dict(out=y if case["out16"] else None, residual=h if case["residual"] else None)
        if case["q8"]:
            got.update(scale=step, q8=(y / step[:, None]).round() * step[:, None])
        return {k: v for k, v in got.items() if v is not None}
    # token after token: S <- exp(g) S + v k^T, o = S q / sqrt(dk)
    hk, hv, dk, dv = case["Hk"], case["Hv"], case["dk"], case["dv"]
    lens = [case["T"]] * case["B"] if case["op"] == "decode" else _lens(case)
    starts = np.concatenate([[0], np.cumsum(lens)])
    heads = [h * hk // hv if case["map"] == GROUPED else h % hk for h in range(hv)]
    q, k = (s[n].double().reshape(-1, hk, dk)[:, heads] for n in "qk")
    v = s["v"].double().reshape(-1, hv, dv)
    g = s["rate"].double().expand(len(q), hv) if case["decay"] == "head" else s["g"].double()
    slots = list(range(len(lens))) if s.get("slots") is None else s["slots"].tolist()
    order = sorted(range(len(lens)), key=lambda i: -lens[i])  # the longest first: those still running are a prefix
    S = s["state"].double()[[slots[i] for i in order]]
    out = torch.zeros(len(q), hv, dv, dtype=torch.float64, device=DEV)
    first = torch.tensor([int(starts[i]) for i in order], device=DEV)
    for t in range(max(lens)):
        n = sum(lens[i] > t for i in order)
        r = first[:n] + t
        live = S[:n]
        live.mul_(g[r].exp()[:, :, None, None]).add_(v[r][..., None] * k[r][..., None, :])
        out[r] = (live @ q[r][..., None])[..., 0] / math.sqrt(dk)
    state = s["state"].double()
    state[[slots[i] for i in order]] = S
    return dict(out=out, state=state)
