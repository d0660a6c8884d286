"""A full-attention layer as a server runs it: pages are reserved, prompts are turned onto them and attended to, samples fork and
decode behind a shared prefix, the cache is compacted, decoding goes on. Every attention output against 64 bits on the keys and
values as they were written (attn_reference), kept here in lists that know nothing of pages."""
import torch
import pytest

from attn_reference import attention64, near
from gated_deltanet_linear_step_amd import ops
from test_rope import turned, close

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
HQ, HKV, D, ROT, PS, B16 = 8, 2, 128, 64, 16, torch.bfloat16


class Server:
    """One layer's cache of 64 pages for up to 10 sequences; row 0 holds the prefix."""

    def __init__(self, seed):
        self.gen = torch.Generator(DEV).manual_seed(seed)
        # a plane of keys and one of values: [2][pages][heads][page size][D]
        self.pool = torch.zeros(2, 64, HKV, PS, D, dtype=B16, device=DEV)
        self.table = torch.full((10, 12), -1, dtype=torch.int32, device=DEV)
        self.refs = torch.zeros(64, dtype=torch.int32, device=DEV)
        self.w = ops.rope_frequencies(ROT, scaling=ops.ROPE_BANDS, factor=4.0, original_length=2048)[0].to(DEV)
        self.written = [[torch.zeros(0, HKV, D, dtype=B16, device=DEV)] * 2 for _ in range(10)]  # turned keys, values

    def put(self, rows, starts, counts, base):
        """Turns counts[i] tokens onto row rows[i] from token starts[i] on; positions from base on. Returns the queries."""
        total = sum(counts)
        mixed = torch.randn(total, (HQ + 2 * HKV) * D, generator=self.gen, device=DEV).to(B16)
        q, k, v = (x.unflatten(1, (-1, D)) for x in mixed.split([HQ * D, HKV * D, HKV * D], 1))
        row = torch.repeat_interleave(torch.tensor(rows), torch.tensor(counts)).to(DEV)
        at = torch.cat([torch.arange(s, s + n) for s, n in zip(starts, counts)]).to(DEV)
        slots = (self.table[row, at // PS] * PS + at % PS).to(torch.int32)
        position = (at + base).to(torch.int32)
        turn = dict(k=k, v=v, k_pages=self.pool[0], v_pages=self.pool[1], slots=slots)
        got = ops.rope(position, self.w, q=q, magnitude=1.1, **turn)
        for x, y in ((q, got), (k, self.pool[0][slots // PS, :, slots % PS])):
            close(y, *turned(x, position, self.w, 1.1, ops.ROPE_HALF))
        first = 0
        for r, n in zip(rows, counts):
            page = slots[first:first + n]
            self.written[r] = [torch.cat([old, pool[page // PS, :, page % PS]]) for old, pool in zip(self.written[r], self.pool)]
            first += n
        return got

    def check(self, out, q, rows, counts, prefix):
        first = 0
        for r, n in zip(rows, counts):
            front = self.written[0] if prefix else [x[:0] for x in self.written[0]]
            k, v = (torch.cat([a, b]) for a, b in zip(front, self.written[r]))
            sees = torch.arange(len(k), device=DEV)[None] <= torch.arange(n, device=DEV)[:, None] + len(k) - n
            want = attention64(q[first:first + n], k, v, sees, D ** -0.5)
            near(out[first:first + n], want[0], want[2])
            first += n


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def test_a_layer_from_prompts_to_forked_decode_steps():
    s = Server(1)
    reserve = lambda rows, lens: ops.pages_reserve(s.table, s.refs, i32(rows), i32(lens), page_size=PS)  # noqa: E731
    # the common prefix, a prompt of its own; then two prompts behind it, on positions from 75 on
    assert reserve([0, 1, 2], [75, 40, 33]).tolist() == [0, 0, 0]
    cu = torch.tensor([0, 75], dtype=torch.int32)
    q = s.put([0], [0], [75], 0)
    s.check(ops.attention_prefill(q, s.pool[0], s.pool[1], cu, table=s.table[:1]), q, [0], [75], False)
    q = s.put([1, 2], [0, 0], [40, 33], 75)
    lens = i32([40, 33])
    # prompts behind a shared prefix: one query a "step", 40 and 33 of them at once by steps of one sequence
    for r, n, at in ((1, 40, 0), (2, 33, 40)):
        out = ops.attention_decode(q[at:at + n], s.pool[0], s.pool[1], s.table[r:r + 1], lens[r - 1:r].contiguous(), batch=1,
                                   tokens_per_seq=n, max_len=64, prefix_table=s.table[0], prefix_len=75)
        s.check(out, q[at:at + n], [r], [n], True)
    # three samples of either, with room for what they decode
    rows = [1, 2, 3, 4, 5, 6]
    assert ops.pages_fork(s.pool, s.table, s.refs, i32([1, 1, 2, 2]), i32([3, 4, 5, 6]), i32([40, 40, 33, 33]), page_size=PS).tolist() == [0] * 4
    s.written[3] = s.written[4] = list(s.written[1])
    s.written[5] = s.written[6] = list(s.written[2])
    have = [40, 33, 40, 40, 33, 33]

    def steps(rows, tokens):
        assert (ops.pages_reserve(s.table, s.refs, i32(rows), i32([have[rows_all.index(r)] + tokens for r in rows]), page_size=PS) == 0).all()
        q = s.put(rows, [have[rows_all.index(r)] for r in rows], [tokens] * len(rows), 75)
        for r in rows:
            have[rows_all.index(r)] += tokens
        out = ops.attention_decode(q, s.pool[0], s.pool[1], s.table[rows].contiguous(), i32([have[rows_all.index(r)] for r in rows]),
                                   batch=len(rows), tokens_per_seq=tokens, max_len=192, prefix_table=s.table[0], prefix_len=75)
        s.check(out, q, rows, [tokens] * len(rows), True)

    rows_all = list(rows)
    for tokens in (1, 1, 3, 1):
        steps(rows, tokens)
    # half of them end, the rest moves together and goes on
    ops.pages_free(s.table, s.refs, i32([1, 4, 6]))
    page_map, used = ops.pages_compact(s.pool, s.table, s.refs)
    torch.cuda.synchronize()
    assert int(s.table.max()) < int(used) == int((s.refs > 0).sum())
    for tokens in (1, 2, 1):
        steps([2, 3, 5], tokens)
    # rejected drafts: entries behind the kept tokens go back
    keep = i32([-(-n // PS) for n in (have[1], have[2], have[4])])
    ops.pages_free(s.table, s.refs, i32([2, 3, 5]), keep=keep)
    steps([2, 3, 5], 1)
    ops.pages_free(s.table, s.refs, i32(list(range(10))))
    assert (s.refs == 0).all() and (s.table == -1).all()


def test_a_captured_decode_step():
    """rope onto pages and the attention of a step as one graph, replayed with other positions, slots and lengths."""
    s = Server(2)
    rows = [1, 2]
    ops.pages_reserve(s.table, s.refs, i32([0, 1, 2]), i32([30, 100, 100]), page_size=PS)
    s.put([0, 1, 2], [0, 0, 0], [30, 60, 17], 0)
    mixed = torch.zeros(2, (HQ + 2 * HKV) * D, dtype=B16, device=DEV)
    q, k, v = (x.unflatten(1, (-1, D)) for x in mixed.split([HQ * D, HKV * D, HKV * D], 1))
    position, slots, lens = i32([0, 0]), i32([-1, -1]), i32([60, 17])
    table = s.table[1:3]

    def step():
        turned_q = ops.rope(position, s.w, q=q, k=k, v=v, k_pages=s.pool[0], v_pages=s.pool[1], slots=slots)
        return turned_q, ops.attention_decode(turned_q, s.pool[0], s.pool[1], table, lens, batch=2, max_len=100,
                                              prefix_table=s.table[0], prefix_len=30)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got_q, got = step()
    have = [60, 17]
    for turn in range(4):
        mixed.copy_(torch.randn(mixed.shape, generator=s.gen, device=DEV))
        at = torch.tensor(have, device=DEV)
        slots.copy_(s.table[torch.tensor(rows, device=DEV), at // PS] * PS + at % PS)
        position.copy_(at + 30)
        lens.copy_(at + 1)
        graph.replay()
        torch.cuda.synchronize()
        want_q, room = turned(q, position, s.w, 1.0, ops.ROPE_HALF)
        close(got_q, want_q, room)
        for i, r in enumerate(rows):
            have[i] += 1
            s.written[r] = [torch.cat([old, pool[slots[i:i + 1] // PS, :, slots[i:i + 1] % PS]]) for old, pool in zip(s.written[r], s.pool)]
        s.check(got, got_q, rows, [1, 1], True)
        eager = ops.attention_decode(got_q, s.pool[0], s.pool[1], table, lens, batch=2, max_len=100, prefix_table=s.table[0], prefix_len=30)
        assert torch.equal(eager, got)
