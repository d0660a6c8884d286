"""Attention over packed prompts and in decode steps against 64 bits (attn_reference: its bounds)."""
import math

import pytest
import torch

from attn_reference import attention64, causal, near
from gated_deltanet_linear_step_amd import ops

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
B16, F16 = torch.bfloat16, torch.float16
NAN, INF = float("nan"), float("inf")


def rand(gen, *shape):
    return torch.randn(*shape, generator=gen)


def packed(lens, keys, Hq, Hkv, D, dtype, seed):
    """Queries, keys and values as views of wider rows, NaN in what the views leave out."""
    gen = torch.Generator().manual_seed(seed)
    T, n = sum(lens), sum(keys)
    q = torch.full((T, Hq * D + 16), NAN)
    q[:, :Hq * D] = 1.5 * rand(gen, T, Hq * D)
    kv = torch.full((n, 2 * Hkv * D + 8), NAN)
    kv[:, :2 * Hkv * D] = rand(gen, n, 2 * Hkv * D)
    q, kv = q.to(dtype).to(DEV), kv.to(dtype).to(DEV)
    return (q[:, :Hq * D].unflatten(1, (Hq, D)), kv[:, :Hkv * D].unflatten(1, (Hkv, D)),
            kv[:, Hkv * D:2 * Hkv * D].unflatten(1, (Hkv, D)))


def offsets(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32)


def on_pages(k, v, keys, ps, seed, spare=2, fill=NAN):
    """Packed keys and values on shuffled pages; what no key fills is NaN. (k_pages, v_pages, table)"""
    gen = torch.Generator().manual_seed(seed)
    need = [-(-n // ps) for n in keys]
    ids = torch.randperm(sum(need) + spare, generator=gen)
    pools = [torch.full((len(ids), x.shape[1], ps, x.shape[2]), fill, dtype=x.dtype, device=DEV) for x in (k, v)]
    table = torch.full((len(keys), max(need + [1]) + 1), -1, dtype=torch.int32)
    at = row = 0
    for s, n in enumerate(keys):
        for e in range(need[s]):
            page, m = int(ids[at + e]), min(ps, n - e * ps)
            table[s, e] = page
            for pool, x in zip(pools, (k, v)):
                pool[page, :, :m] = x[row + e * ps:row + e * ps + m].transpose(0, 1)
        at, row = at + need[s], row + n
    return pools[0], pools[1], table.to(DEV)


def check_prompts(got, lse, q, k, v, lens, keys, scale):
    a = b = 0
    for T, n in zip(lens, keys):
        want = attention64(q[a:a + T], k[b:b + n], v[b:b + n], causal(T, n, q.device), scale)
        near(got[a:a + T], want[0], want[2])
        if lse is not None:
            near(lse[a:a + T], want[1], want[3])
        a, b = a + T, b + n


HEADS = [(1, 1, 64, B16), (4, 2, 64, F16), (3, 1, 96, B16), (8, 8, 96, F16), (10, 2, 128, F16), (4, 4, 128, B16), (16, 2, 256, B16), (6, 2, 256, F16)]
LENS = [[1], [2], [127], [128], [129], [31, 32, 33], [0, 1, 0, 64, 65, 0, 63, 200, 0], [700]]


@pytest.mark.parametrize("Hq,Hkv,D,dtype", HEADS)
@pytest.mark.parametrize("lens", LENS, ids=lambda x: "-".join(map(str, x)))
def test_prompts(Hq, Hkv, D, dtype, lens):
    q, k, v = packed(lens, lens, Hq, Hkv, D, dtype, sum(lens))
    lse = torch.full((sum(lens), Hq), 7.0, device=DEV)
    out = ops.attention_prefill(q, k, v, offsets(lens), lse=lse)
    check_prompts(out, lse, q, k, v, lens, lens, D ** -0.5)


# keys before the queries, fewer keys than queries, no keys, and lengths that split a row's keys
PAST = [([5], [6]), ([1], [2000]), ([3, 40], [700, 41]), ([20, 9, 3], [4, 0, 3]), ([0, 17, 130], [50, 1017, 130]), ([200], [5000])]


@pytest.mark.parametrize("ps", [0, 16, 32, 64, 256, 1024])
@pytest.mark.parametrize("lens,keys", PAST, ids=lambda x: "-".join(map(str, x)))
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(4, 2, 64, F16), (3, 1, 96, B16), (8, 2, 128, B16), (8, 1, 256, F16)])
def test_queries_at_the_end_of_longer_or_shorter_keys(Hq, Hkv, D, dtype, lens, keys, ps):
    q, k, v = packed(lens, keys, Hq, Hkv, D, dtype, ps + sum(keys))
    lse = torch.full((sum(lens), Hq), 7.0, device=DEV)
    scale = 0.11
    if ps:
        kp, vp, table = on_pages(k, v, keys, ps, 1)
        out = ops.attention_prefill(q, kp, vp, offsets(lens), cu_k=offsets(keys), table=table, lse=lse, scale=scale)
    else:
        out = ops.attention_prefill(q, k, v, offsets(lens), cu_k=offsets(keys).to(DEV), lse=lse, scale=scale)
    check_prompts(out, lse, q, k, v, lens, keys, scale)


def test_many_short_prompts():
    gen = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 6, (1000,), generator=gen).tolist()
    q, k, v = packed(lens, lens, 6, 2, 64, B16, 5)
    out = ops.attention_prefill(q, k, v, offsets(lens).long())
    cu = offsets(lens).tolist()
    whose = torch.repeat_interleave(torch.arange(1000), torch.tensor(lens)).to(DEV)
    at = torch.arange(cu[-1], device=DEV)
    want = attention64(q, k, v, (whose[:, None] == whose) & (at[:, None] >= at), 64 ** -0.5)
    near(out, want[0], want[2])


@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_rows_beside_the_outputs_stay(D):
    lens, Hq, Hkv = [70, 3], 4, 2
    q, k, v = packed(lens, lens, Hq, Hkv, D, B16, D)
    wide = torch.full((sum(lens) + 5, Hq * D + 24), 7.0, dtype=B16, device=DEV)
    out = wide[:sum(lens), 8:8 + Hq * D].unflatten(1, (Hq, D))
    ops.attention_prefill(q, k, v, offsets(lens), out=out)
    check_prompts(out, None, q, k, v, lens, lens, D ** -0.5)
    assert (wide[sum(lens):] == 7).all() and (wide[:, :8] == 7).all() and (wide[:, 8 + Hq * D:] == 7).all()
    # fewer tokens than rows of q and out
    full = torch.full((sum(lens), Hq, D), 7.0, dtype=B16, device=DEV)
    ops.attention_prefill(q, k, v, offsets([70]), out=full)
    check_prompts(full[:70], None, q[:70], k[:70], v[:70], [70], [70], D ** -0.5)
    assert (full[70:] == 7).all()


@pytest.mark.parametrize("D,dtype", [(64, B16), (96, F16), (128, F16), (256, B16)])
@pytest.mark.parametrize("bad", [INF, -INF, NAN])
@pytest.mark.parametrize("where", ["k", "v"])
def test_what_is_not_finite_stays_with_the_queries_that_see_it(D, dtype, bad, where):
    lens, Hq, Hkv = [150, 40], 4, 2
    q, k, v = packed(lens, lens, Hq, Hkv, D, dtype, 3)
    clean_k, clean_v = k.clone(), v.clone()
    (k if where == "k" else v)[100, 1, D // 2] = bad  # key 100 of head 1 of the first prompt
    out = ops.attention_prefill(q, k, v, offsets(lens))
    want = attention64(q[:150], clean_k[:150], clean_v[:150], causal(150, 150, DEV), D ** -0.5)
    sees = torch.zeros(150, Hq, D, dtype=torch.bool, device=DEV)
    sees[100:, 2:, :] = True if where == "k" else False
    if where == "v":
        sees[100:, 2:, D // 2] = True
    near(torch.where(sees, 0, out[:150].double()), torch.where(sees, 0, want[0]), want[2])
    if where == "v" or bad != bad:
        assert not torch.isfinite(out[:150][sees]).any()
    tail = attention64(q[150:], clean_k[150:], clean_v[150:], causal(40, 40, DEV), D ** -0.5)
    near(out[150:], tail[0], tail[2])


def test_scores_that_grow_along_the_keys():
    """Maxima that move by a little and by a lot from tile to tile."""
    n, D = 1000, 128
    for step in (0.01, 0.3, 5.0):
        q = torch.zeros(n, 1, D, device=DEV)
        q[:, 0, 0] = 1
        k = torch.zeros(n, 1, D, device=DEV)
        k[:, 0, 0] = step * torch.arange(n, device=DEV)
        v = torch.randn(n, 1, D, generator=torch.Generator(DEV).manual_seed(1), device=DEV)
        q, k, v = q.to(B16), k.to(B16), v.to(B16)
        for flip in (False, True):
            kk = k.flip(0) if flip else k
            lse = torch.empty(n, 1, device=DEV)
            out = ops.attention_prefill(q, kk, v, offsets([n]), scale=1.0, lse=lse)
            check_prompts(out, lse, q, kk, v, [n], [n], 1.0)


def test_scores_of_minus_infinity_are_no_keys():
    q, k, v = packed([40], [40], 2, 1, 64, B16, 9)
    k = k.clone()
    q = q.abs() + 0.01
    k[:] = -INF
    lse = torch.full((40, 2), 7.0, device=DEV)
    out = ops.attention_prefill(q, k, v, offsets([40]), lse=lse)
    assert (out == 0).all() and (lse == -INF).all()


# ---- decode steps -------------------------------------------------------------------------------------

def decode_inputs(lens, prefix, T, Hq, Hkv, D, dtype, ps, seed):
    keys = [prefix] + [max(n, 0) for n in lens]
    q, k, v = packed([len(lens) * T], keys, Hq, Hkv, D, dtype, seed)
    kp, vp, table = on_pages(k, v, keys, ps, seed)
    return q, k, v, kp, vp, table[1:].contiguous(), table[0].contiguous() if prefix else None


def check_steps(out, lse, q, k, v, lens, prefix, T, scale, max_len=None):
    at = prefix
    for b, n in enumerate(lens):
        own = max(n, 0)
        m = own if max_len is None else min(own, max_len)
        kb, vb = torch.cat([k[:prefix], k[at:at + m]]), torch.cat([v[:prefix], v[at:at + m]])
        j = torch.arange(prefix + m, device=DEV)[None]
        t = torch.arange(T, device=DEV)[:, None]
        sees = (j < prefix) | (j - prefix < m - T + 1 + t)
        rows = slice(b * T, (b + 1) * T)
        want = attention64(q[rows], kb, vb, sees, scale)
        near(out[rows], want[0], want[2])
        if lse is not None:
            near(lse[rows], want[1], want[3])
        at += own


STEPS = [([1], 1), ([17], 1), ([5, 0, 300, 64, 65, 2, -3, 1], 1), ([1, 2, 4, 5, 700, 33], 4), ([1500, 3], 2), ([40, 0, 129], 17)]


@pytest.mark.parametrize("Hq,Hkv,D,dtype", HEADS)
@pytest.mark.parametrize("lens,T", STEPS, ids=str)
@pytest.mark.parametrize("prefix", [0, 1, 333])
def test_steps(Hq, Hkv, D, dtype, lens, T, prefix):
    ps = {64: 16, 96: 64, 128: 32, 256: 128}[D]
    q, k, v, kp, vp, table, front = decode_inputs(lens, prefix, T, Hq, Hkv, D, dtype, ps, prefix + T)
    lse = torch.full((len(lens) * T, Hq), 7.0, device=DEV)
    out = ops.attention_decode(q, kp, vp, table, torch.tensor(lens, dtype=torch.int32, device=DEV), batch=len(lens),
                               tokens_per_seq=T, max_len=max(max(lens), 0), prefix_table=front, prefix_len=prefix, lse=lse)
    check_steps(out, lse, q, k, v, lens, prefix, T, D ** -0.5)


@pytest.mark.parametrize("ps", [16, 32, 64, 128, 512, 1024])
def test_steps_on_pages_of_every_size(ps):
    lens = [1, ps - 1, ps, ps + 1, 2 * ps + 5, 900]
    q, k, v, kp, vp, table, front = decode_inputs(lens, 3 * ps + 7, 1, 8, 2, 128, B16, ps, ps)
    out = ops.attention_decode(q, kp, vp, table, torch.tensor(lens, dtype=torch.int32, device=DEV), batch=6, max_len=max(lens),
                               prefix_table=front, prefix_len=3 * ps + 7)
    check_steps(out, None, q, k, v, lens, 3 * ps + 7, 1, 128 ** -0.5)


@pytest.mark.parametrize("B,longest,Hq,Hkv,D", [(1, 9000, 16, 2, 256), (1, 20001, 1, 1, 64), (3, 5000, 12, 4, 96), (130, 500, 8, 2, 128),
                                                (600, 40, 4, 1, 64)])
def test_steps_of_few_and_many_sequences(B, longest, Hq, Hkv, D):
    lens = [max(1, longest - 37 * i) for i in range(B)]
    q, k, v, kp, vp, table, _ = decode_inputs(lens, 0, 1, Hq, Hkv, D, F16, 64, B)
    lse = torch.empty(B, Hq, device=DEV)
    out = ops.attention_decode(q, kp, vp, table, torch.tensor(lens, dtype=torch.int32, device=DEV), batch=B, max_len=longest, lse=lse)
    check_steps(out, lse, q, k, v, lens, 0, 1, D ** -0.5)


def test_lengths_past_max_len_end_there():
    lens = [300, 100, 50]
    q, k, v, kp, vp, table, _ = decode_inputs(lens, 0, 2, 4, 2, 64, B16, 16, 8)
    out = ops.attention_decode(q, kp, vp, table, torch.tensor(lens, dtype=torch.int32, device=DEV), batch=3, tokens_per_seq=2, max_len=100)
    check_steps(out, None, q, k, v, lens, 0, 2, 64 ** -0.5, max_len=100)


def test_no_keys_at_all():
    q = torch.randn(6, 4, 64, device=DEV).to(B16)
    pool = torch.full((1, 2, 16, 64), NAN, dtype=B16, device=DEV)
    table = torch.full((3, 1), -1, dtype=torch.int32, device=DEV)
    lse = torch.zeros(6, 4, device=DEV)
    for max_len in (0, 16):
        out = ops.attention_decode(q, pool, pool, table, torch.zeros(3, dtype=torch.int32, device=DEV), batch=3, tokens_per_seq=2,
                                   max_len=max_len, lse=lse)
        assert (out == 0).all() and (lse == -INF).all()


@pytest.mark.parametrize("D,dtype", [(64, F16), (128, B16), (256, B16)])
@pytest.mark.parametrize("bad", [-1, -2 ** 31, 10 ** 6, 2 ** 31 - 1])
def test_keys_of_an_entry_that_is_no_page_are_not_seen(D, dtype, bad):
    ps, n, Hq, Hkv = 16, 400, 4, 2
    q, k, v = packed([n], [n], Hq, Hkv, D, dtype, D)
    kp, vp, table = on_pages(k, v, [n], ps, 2)
    for e in (0, 3, 7, 8, 24):
        table[0, e] = bad
    gone = torch.isin(torch.arange(n, device=DEV) // ps, torch.tensor([0, 3, 7, 8, 24], device=DEV))
    sees = causal(n, n, DEV) & ~gone
    out = ops.attention_prefill(q, kp, vp, offsets([n]), table=table)
    want = attention64(q, k, v, sees, D ** -0.5)
    near(out, want[0], want[2])
    # one query of a step, behind a prefix with the same holes
    front = table[0].contiguous()
    own = torch.full((1, 2), bad, dtype=torch.int32, device=DEV)
    own[0, 1] = int(table[0, 1])
    out = ops.attention_decode(q[-1:], kp, vp, own, torch.tensor([30], dtype=torch.int32, device=DEV), batch=1, max_len=30,
                               prefix_table=front, prefix_len=n)
    ks, vs = torch.cat([k, k[ps:2 * ps - 2]]), torch.cat([v, v[ps:2 * ps - 2]])
    keep = torch.cat([~gone, torch.ones(ps - 2, dtype=torch.bool, device=DEV)])
    want = attention64(q[-1:], ks, vs, keep[None], D ** -0.5)
    near(out, want[0], want[2])


@pytest.mark.parametrize("D,dtype", [(64, B16), (128, F16), (256, B16)])
@pytest.mark.parametrize("bad", [INF, NAN])
def test_steps_do_not_see_what_is_not_finite_behind_their_keys(D, dtype, bad):
    """Drafted tokens: an earlier one does not see the keys and values of a later one."""
    T, n, ps = 4, 90, 32
    q, k, v, kp, vp, table, _ = decode_inputs([n], 0, T, 4, 2, D, dtype, ps, 4)
    page, at = int(table[0, (n - 1) // ps]), (n - 1) % ps
    kp[page, :, at] = bad
    vp[page, :, at] = bad
    out = ops.attention_decode(q, kp, vp, table, torch.tensor([n], dtype=torch.int32, device=DEV), batch=1, tokens_per_seq=T, max_len=n)
    check_steps(out[:T - 1], None, q[:T - 1], k[:n - 1], v[:n - 1], [n - 1], 0, T - 1, D ** -0.5)
    assert not torch.isfinite(out[T - 1]).any()


# ---- where and when calls run -------------------------------------------------------------------------

def chain_inputs(seed):
    lens, prefix = [900, 31, 260], 500
    q, k, v, kp, vp, table, front = decode_inputs(lens, prefix, 1, 8, 2, 128, B16, 16, seed)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    qp, kk, vv = packed([130, 9], [130, 9], 8, 2, 128, B16, seed + 1)
    cu, past = offsets([130, 9]), offsets([1000, 60])
    pk, pv, ptable = on_pages(*packed([1], [1000, 60], 8, 2, 128, B16, seed + 2)[1:], [1000, 60], 16, seed)
    return dict(step=(q, kp, vp, table, n, front, prefix), prompt=(qp, kk, vv, cu, cu.to(DEV)),
                more=(qp, pk, pv, cu, cu.to(DEV), past, past.to(DEV), ptable))


def chain(s, stream=None):
    q, kp, vp, table, n, front, prefix = s["step"]
    a = ops.attention_decode(q, kp, vp, table, n, batch=3, max_len=900, prefix_table=front, prefix_len=prefix, stream=stream)
    qp, k, v, cu, cud = s["prompt"]
    b = ops.attention_prefill(qp, k, v, cud, cu_seqlens_host=cu, stream=stream)
    qp, k, v, cu, cud, ck, ckd, table = s["more"]
    c = ops.attention_prefill(qp, k, v, cud, cu_seqlens_host=cu, cu_k=ckd, cu_k_host=ck, table=table, stream=stream)
    return a, b, c


def test_two_streams_at_once_and_replayed_graphs():
    sets = [chain_inputs(s) for s in (1, 2)]
    want = [[t.clone() for t in chain(s)] for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for s, stream in zip(sets, streams):
            got.append(chain(s, stream))
            torch.full((1 << 20,), NAN, device=DEV)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for g, w in zip(got, want) for x, y in zip(g, w))
    graphs = []
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = chain(s)
        graphs.append((graph, outs))
    for turn in range(3):
        for graph, _ in graphs:
            graph.replay()
        chain(sets[0])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for (_, g), w in zip(graphs, want) for x, y in zip(g, w)), turn
    # lengths are read when the graph runs: with a token less the last key is no longer seen
    q, kp, vp, table, n, front, prefix = sets[0]["step"]
    n -= 1
    graphs[0][0].replay()
    torch.cuda.synchronize()
    eager = chain(sets[0])
    assert torch.equal(graphs[0][1][0], eager[0]) and not torch.equal(eager[0], want[0][0])


def test_the_same_call_gives_the_same_bits():
    s = chain_inputs(5)
    first = [t.clone() for t in chain(s)]
    for _ in range(5):
        assert all(torch.equal(x, y) for x, y in zip(chain(s), first))


@pytest.mark.parametrize("paged", [False, True])
def test_offsets_past_32_bits(paged):
    """Keys and values whose byte and element offsets pass 2^31 and 2^32."""
    Hq, Hkv, D, n = 2, 1, 64, 200
    q, k, v = packed([n], [n], Hq, Hkv, D, B16, 3)
    if not paged:
        far = (1 << 24) - 8  # elements from row to row
        buf = torch.empty(n * far, dtype=B16, device=DEV)
        rows = [buf.as_strided((n, Hkv, D), (far, D, 1), at) for at in (0, far // 16 * 8)]
        for row, x in zip(rows, (k, v)):
            row.copy_(x)
        out = ops.attention_prefill(q, rows[0], rows[1], offsets([n]))
        check_prompts(out, None, q, k, v, [n], [n], D ** -0.5)
        return
    stride = 1 << 28
    buf = torch.empty(14 * stride, dtype=B16, device=DEV)
    pools = [buf.as_strided((14, Hkv, 16, D), (stride, 16 * D, D, 1), at) for at in (0, stride // 2)]
    kp, vp, table = on_pages(k, v, [n], 16, 6, spare=1)
    for pool, x in zip(pools, (kp, vp)):
        pool.copy_(x)
    out = ops.attention_prefill(q, *pools, offsets([n]), table=table)
    check_prompts(out, None, q, k, v, [n], [n], D ** -0.5)
    out = ops.attention_decode(q[-1:], *pools, table, torch.tensor([n], dtype=torch.int32, device=DEV), batch=1, max_len=n)
    check_steps(out, None, q[-1:], k, v, [n], 0, 1, D ** -0.5)


# ---- how calls are split -------------------------------------------------------------------------------

@pytest.mark.parametrize("Hq,Hkv,D,tokens", [(8, 1, 256, 6000), (8, 2, 128, 7000)])
def test_prompts_whose_long_blocks_are_cut(Hq, Hkv, D, tokens):
    """Blocks for every CU, of all lengths; a short prompt behind the long one."""
    lens = [tokens, 70]
    q, k, v = packed(lens, lens, Hq, Hkv, D, B16, 3)
    lse = torch.empty(sum(lens), Hq, device=DEV)
    out = ops.attention_prefill(q, k, v, offsets(lens), lse=lse)
    check_prompts(out, lse, q, k, v, lens, lens, D ** -0.5)


@pytest.mark.parametrize("D,dtype", [(64, B16), (96, F16), (128, F16), (256, B16)])
def test_sequences_split_beside_ones_that_are_not(D, dtype):
    """Few queries behind many keys, behind few, behind none, and queries of their own prompt."""
    lens, keys = [1, 3, 0, 64, 5, 200], [6000, 3, 900, 64, 0, 1400]
    q, k, v = packed(lens, keys, 4, 2, D, dtype, D)
    lse = torch.empty(sum(lens), 4, device=DEV)
    kp, vp, table = on_pages(k, v, keys, 16, 3)
    for paged in (False, True):
        out = ops.attention_prefill(q, kp if paged else k, vp if paged else v, offsets(lens), cu_k=offsets(keys), lse=lse,
                                    table=table if paged else None)
        check_prompts(out, lse, q, k, v, lens, keys, D ** -0.5)


@pytest.mark.parametrize("D,dtype", [(64, F16), (96, B16), (128, B16), (256, F16)])
def test_a_bound_far_past_the_lengths(D, dtype):
    """max_len of a whole context, sequences much shorter: most runs are empty, and there are hundreds of them."""
    ps, most = 128, 100000
    for lens, T in (([700], 1), ([1, 0, 300, 2, 40], 2), ([900, 5] * 40, 1)):
        q, k, v, kp, vp, table, front = decode_inputs(lens, 200, T, 4, 2, D, dtype, ps, len(lens))
        wide = torch.full((len(lens), -(-most // ps)), -1, dtype=torch.int32, device=DEV)
        wide[:, :table.shape[1]] = table
        lse = torch.empty(len(lens) * T, 4, device=DEV)
        out = ops.attention_decode(q, kp, vp, wide, torch.tensor(lens, dtype=torch.int32, device=DEV), batch=len(lens), tokens_per_seq=T,
                                   max_len=most, prefix_table=front, prefix_len=200, lse=lse)
        check_steps(out, lse, q, k, v, lens, 200, T, D ** -0.5)


@pytest.mark.parametrize("T,Hq,Hkv,D", [(33, 1, 1, 64), (9, 8, 2, 128), (5, 16, 2, 256), (70, 6, 2, 96), (200, 4, 4, 128)])
def test_steps_of_many_rows(T, Hq, Hkv, D):
    lens = [T, T + 1, 1500, 0, T - 1]
    q, k, v, kp, vp, table, front = decode_inputs(lens, 90, T, Hq, Hkv, D, B16, 16, T)
    lse = torch.empty(len(lens) * T, Hq, device=DEV)
    out = ops.attention_decode(q, kp, vp, table, torch.tensor(lens, dtype=torch.int32, device=DEV), batch=5, tokens_per_seq=T, max_len=1500,
                               prefix_table=front, prefix_len=90, lse=lse)
    check_steps(out, lse, q, k, v, lens, 90, T, D ** -0.5)


def test_tables_and_prefixes_that_share_pages():
    """The same pages in several rows, twice in a row, and in the prefix: keys are only read."""
    ps, n = 16, 64
    q, k, v = packed([3], [n], 4, 2, 128, B16, 8)
    kp, vp, table = on_pages(k, v, [n], ps, 3)
    row = table[0, :4]
    tables = torch.stack([row, row.flip(0), torch.cat([row[:2], row[:2]])]).contiguous()
    order = [torch.arange(n), torch.arange(n).view(4, 16).flip(0).flatten(), torch.cat([torch.arange(32), torch.arange(32)])]
    out = ops.attention_decode(q, kp, vp, tables, torch.tensor([64, 50, 40], dtype=torch.int32, device=DEV), batch=3, max_len=64,
                               prefix_table=row.contiguous(), prefix_len=30)
    for b, m in enumerate((64, 50, 40)):
        at = torch.cat([torch.arange(30), order[b][:m]]).to(DEV)
        want = attention64(q[b:b + 1], k[at], v[at], torch.ones(1, 30 + m, dtype=torch.bool, device=DEV), 128 ** -0.5)
        near(out[b:b + 1], want[0], want[2])


@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_outputs_do_not_depend_on_what_the_workspace_held(D):
    lens, keys = [2, 130], [3000, 700]
    q, k, v = packed(lens, keys, 4, 2, D, B16, 1)
    need = ops.attention_prefill_workspace_bytes(Hq=4, Hkv=2, head_dim=D, num_seqs=2, total_tokens=132)
    outs = []
    for fill in (0, 255, 127):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=DEV)
        outs.append(ops.attention_prefill(q, k, v, offsets(lens), cu_k=offsets(keys), workspace=ws))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    check_prompts(outs[0], None, q, k, v, lens, keys, D ** -0.5)
    n = torch.tensor([5000, 10], dtype=torch.int32, device=DEV)
    q, k, v, kp, vp, table, front = decode_inputs([5000, 10], 100, 1, 4, 2, D, B16, 64, 2)
    need = ops.attention_decode_workspace_bytes(Hq=4, Hkv=2, head_dim=D, batch=2, max_len=5000, prefix_len=100)
    outs = [ops.attention_decode(q, kp, vp, table, n, batch=2, max_len=5000, prefix_table=front, prefix_len=100,
                                 workspace=torch.full((need,), fill, dtype=torch.uint8, device=DEV)) for fill in (0, 255, 127)]
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    check_steps(outs[0], None, q, k, v, [5000, 10], 100, 1, D ** -0.5)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_the_largest_values_stay_finite(D):
    """Values of the order that the documents allow, weights that the running maximum lets grow."""
    n = 300
    q = torch.zeros(n, 1, D, device=DEV)
    q[:, 0, 0] = 1
    k = torch.zeros(n, 1, D, device=DEV)
    k[:, 0, 0] = 0.02 * torch.arange(n, device=DEV)
    v = torch.randn(n, 1, D, generator=torch.Generator(DEV).manual_seed(1), device=DEV) * 2.0 ** 86
    q, k, v = q.to(B16), k.to(B16), v.to(B16)
    out = ops.attention_prefill(q, k, v, offsets([n]), scale=1.0)
    check_prompts(out, None, q, k, v, [n], [n], 1.0)
