"""The prefill of the decayed linear attention over sequences that are split into segments: every head shape and type,
weak decays, so that what a segment passes on counts to the end, states between segments against the recurrence,
decays of -inf and numbers that are not finite in each segment, graphs and streams.

Tolerance. As in test_linattn, with u = 2^-24: a term goes through at most 6 u relative error a token that it ages, and 20 u of
constant work; here by age, E <- exp(g) (E + 6 A) + 20 |v| |k|^T beside A <- exp(g) A + |v| |k|^T, which for long
sequences is much less than (6 T + 20) A. A state is off by at most u E, an output by scale u (E |q| + (dk + 2) A |q|)
and its own rounding. (A join of two segments is one factor and one sum in f32, for 64 tokens' age at least.)
"""
import math

import pytest
import torch

from gated_deltanet_linear_step_amd import ops
from test_linattn import SHAPES, make, split_heads, views

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DEV = "cuda:0"
F32 = torch.float32


def recurrence(mixed, S0, g, Hk, dk, dv, head_map, heads=None, keep=0):
    """One sequence in 64 bits on the GPU: outputs, state, their rooms, and the states (with rooms) after every `keep`
    tokens. heads: the v-heads to compute."""
    Hv = S0.shape[0]
    heads = list(range(Hv)) if heads is None else heads
    of = [h // (Hv // Hk) if head_map == ops.MAP_GROUPED else h % Hk for h in heads]
    q, k, v = (x.to(DEV).double() for x in split_heads(mixed, Hk, Hv, dk, dv))
    q, k, v, g = q[:, of], k[:, of], v[:, heads], g.to(DEV).double()[:, heads]
    S = S0[heads].to(DEV).double()
    A, E, after = S.abs(), 20 * S.abs(), {}
    o, room = torch.zeros_like(v), torch.zeros_like(v)
    for t in range(len(q)):
        a = g[t].exp()[:, None, None]
        vk = v[t][..., None] * k[t][:, None]
        E = a * (E + 6 * A) + 20 * vk.abs()
        S, A = a * S + vk, a * A + vk.abs()
        o[t] = (S * q[t][:, None]).sum(-1) / math.sqrt(dk)
        room[t] = ((E + (dk + 2) * A) * q[t].abs()[:, None]).sum(-1) / math.sqrt(dk)
        if keep and (t + 1) % keep == 0:
            after[t + 1] = S, 1.01 * U * E
    return o, S, 1.01 * U * room, 1.01 * U * E, after


def close(got, want, room):
    if got.dtype != F32:
        fin = torch.finfo(got.dtype)
        room = room + fin.eps / 2 * (want.abs() + room) + fin.smallest_normal * fin.eps
    got = got.double()
    assert torch.isfinite(got).all()
    off = (got - want).abs() - room
    assert (off <= 0).all(), f"over the bound by {off.max():.3e}; max |error| {(got - want).abs().max():.3e}"


class Call:
    """The inputs of one call on the GPU, its workspace between guards, and what it left."""

    def __init__(self, c, lens, Hk, Hv, dk, dv, head_map=ops.MAP_GROUPED, decay="token", out_dtype=F32, stream=None):
        self.c, self.lens, self.decay, self.head_map = c, lens, decay, head_map
        self.heads = dict(Hk=Hk, Hv=Hv, dk=dk, dv=dv)
        self.cu = torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32)
        self.mixed, self.start, self.cud = c["mixed"].to(DEV), c["state"].to(DEV), self.cu.to(DEV)
        self.state = self.start.clone()
        n = sum(lens)
        need = ops.linattn_prefill_workspace_bytes(num_seqs=len(lens), total_tokens=n, **self.heads)
        self.room = torch.full((need + 8192,), 77, dtype=torch.uint8, device=DEV)
        self.ws = self.room[4096:4096 + need]
        self.out = torch.empty(n, Hv, dv, dtype=out_dtype, device=DEV)
        self.dec = dict(g=c["g"].to(DEV)) if decay == "token" else \
            dict(decay_param=c["rate"].to(DEV), decay=ops.DECAY_NEGATIVE_RATE)
        self.call = self.prepare(stream)

    def prepare(self, stream=None):
        return ops.prepare_linattn_prefill_chunked(*views(self.mixed, **self.heads), self.state, self.cud, self.cu, self.out,
                                                   self.ws, head_map=self.head_map, stream=stream, **self.dec, **self.heads)

    def run(self):
        self.call.launch()
        torch.cuda.synchronize()
        assert (self.room[:4096] == 77).all() and (self.room[-4096:] == 77).all()
        return self

    def slots(self):
        """The states between segments that the call wrote: [slots][Hv][dv][dk]."""
        Hv, dk, dv = (self.heads[n] for n in ("Hv", "dk", "dv"))
        size = 4 * Hv * dk * dv
        n = 0
        while (n + 1) * size <= len(self.ws) and not (self.ws[n * size:(n + 1) * size] == 77).all():
            n += 1
        return self.ws[:n * size].clone().view(F32).view(n, Hv, dv, dk)

    def log_decays(self, a, b):
        return self.c["g"][a:b] if self.decay == "token" else self.c["rate"].expand(b - a, -1)

    def references(self, heads=None, keep=0):
        refs = []
        for i, n in enumerate(self.lens):
            a, b = int(self.cu[i]), int(self.cu[i + 1])
            refs.append(recurrence(self.c["mixed"][a:b], self.c["state"][i], self.log_decays(a, b), self.heads["Hk"],
                                   self.heads["dk"], self.heads["dv"], self.head_map, heads, keep))
        return refs

    def check(self, refs, heads=None):
        heads = list(range(self.heads["Hv"])) if heads is None else heads
        for i, n in enumerate(self.lens):
            a, b = int(self.cu[i]), int(self.cu[i + 1])
            if n == 0:
                assert torch.equal(self.state[i], self.start[i])
                continue
            o, S, room_o, room_s, _ = refs[i]
            close(self.out[a:b, heads], o, room_o)
            close(self.state[i, heads], S, room_s)


def weakly_decayed(T, Hk, Hv, dk, dv, dtype, seed, slots, factor=0.01):
    c = make(T, Hk, Hv, dk, dv, dtype, seed, slots=slots)
    return dict(c, g=c["g"] * factor, rate=c["rate"] * factor)


@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_every_shape_and_type(dk, dv, dtype):
    Hk, Hv, lens = 1, 2, [520, 5, 0, 390, 0]
    c = weakly_decayed(sum(lens), Hk, Hv, dk, dv, dtype, dk + dv, len(lens))
    for decay, head_map in (("token", ops.MAP_GROUPED), ("rate", ops.MAP_TILED)):
        refs = None
        for out_dtype in dict.fromkeys((F32, dtype, torch.float16)):
            call = Call(c, lens, Hk, Hv, dk, dv, head_map, decay, out_dtype).run()
            slots = len(call.slots())
            assert slots >= 4  # both long sequences have a first, a middle and a last segment
            refs = refs or call.references()
            call.check(refs)


@pytest.mark.parametrize("head_map", [ops.MAP_GROUPED, ops.MAP_TILED])
def test_heads_that_share_a_k_head(head_map):
    Hk, Hv, d, lens = 2, 6, 64, [700, 300]
    c = weakly_decayed(sum(lens), Hk, Hv, d, d, torch.bfloat16, 17, len(lens))
    call = Call(c, lens, Hk, Hv, d, d, head_map, "rate", torch.bfloat16).run()
    assert len(call.slots()) >= 4
    call.check(call.references())


@pytest.mark.parametrize("dtype,dk,dv,lens", [(torch.bfloat16, 128, 128, [1300]), (torch.float16, 64, 64, [900, 40, 500]),
                                              (torch.float32, 96, 96, [640, 0, 1000]), (torch.bfloat16, 256, 256, [700])])
def test_states_between_segments_are_those_of_the_recurrence(dtype, dk, dv, lens):
    """Every state that the call leaves in its workspace is the recurrence's after a multiple of 64 tokens, later and
    later in each sequence in turn."""
    Hk, Hv = 1, 2
    c = weakly_decayed(sum(lens), Hk, Hv, dk, dv, dtype, 3, len(lens))
    call = Call(c, lens, Hk, Hv, dk, dv).run()
    slots = call.slots().double()
    refs = call.references(keep=64)
    call.check(refs)
    points = [(i, t) for i in range(len(lens)) for t in sorted(refs[i][4]) if t < lens[i]]
    at = -1
    for s in slots:
        fits = [n for n in range(at + 1, len(points))
                if ((s - refs[points[n][0]][4][points[n][1]][0]).abs() <= refs[points[n][0]][4][points[n][1]][1]).all()]
        assert len(fits) == 1, f"after {points[at] if at >= 0 else 'the start'}: fits {[points[n] for n in fits]}"
        at = fits[0]
    assert len(slots) >= 2 and {points[n][0] for n in range(at + 1)} >= {i for i, n in enumerate(lens) if n > 600}


def test_more_segments_than_the_card_has_compute_units():
    Hk, Hv, d, n = 4, 8, 128, 20000
    c = weakly_decayed(n, Hk, Hv, d, d, torch.bfloat16, 3, 1, 0.003)
    call = Call(c, [n], Hk, Hv, d, d, out_dtype=torch.bfloat16).run()
    segments = (len(call.slots()) + 1) * Hv
    assert segments > 256
    call.check(call.references(heads=[0, 7]), heads=[0, 7])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_forgetting_in_each_segment(dtype):
    """Decays of -inf, of -1e5 and of 0 in a first, a middle and a last segment and at both ends of a sequence."""
    Hk, Hv, d, lens = 1, 2, 64, [640, 700]
    c = weakly_decayed(sum(lens), Hk, Hv, d, d, dtype, 21, 2)
    for head, at in ((0, 0), (0, 20), (1, 300), (0, 301), (1, 639), (0, 640), (1, 641 + 64), (0, 1000), (1, 1339)):
        c["g"][at, head] = -float("inf")
    c["g"][500:505] = -1e5
    c["g"][1100:1200] = 0
    call = Call(c, lens, Hk, Hv, d, d, out_dtype=dtype).run()
    assert len(call.slots()) >= 4
    call.check(call.references())


@pytest.mark.parametrize("what,bad", [(w, float(b)) for w in ("q", "k", "v", "state") for b in ("nan", "inf")] +
                         [("g", float("nan"))])
@pytest.mark.parametrize("at", [10, 350, 630])
def test_what_is_not_finite_stays_behind_its_token(what, bad, at):
    """In a first, a middle and a last segment: what the formula does not reach stays within its bound, what it does
    reach is not finite."""
    Hk, Hv, d, lens = 2, 2, 64, [640, 600]
    c = weakly_decayed(sum(lens), Hk, Hv, d, d, torch.bfloat16, 5, 2)
    clean = Call(c, lens, Hk, Hv, d, d)
    refs = clean.references()
    if what == "g":
        c["g"][at, 1] = bad
    elif what == "state":
        c["state"][0, 1, 3, 5] = bad
        at = 0
    else:
        dict(zip("qkv", split_heads(c["mixed"], Hk, Hv, d, d)))[what][at, 1, 3] = bad
        q, k, v = views(c["mixed"], Hk, Hv, d, d)
        assert not torch.isfinite(dict(q=q, k=k, v=v)[what][at]).all()
    call = Call(c, lens, Hk, Hv, d, d).run()
    assert len(call.slots()) >= 4
    # the other head, the other sequence and the tokens before
    for i, rows, h in ((0, slice(0, 640), 0), (0, slice(0, at), 1), (1, slice(640, 1240), 0), (1, slice(640, 1240), 1)):
        first = 640 * i
        close(call.out[rows, h], refs[i][0][rows.start - first:rows.stop - first, h], refs[i][2][rows.start - first:rows.stop - first, h])
        if not (i == 0 and h == 1):
            close(call.state[i, h], refs[i][1][h], refs[i][3][h])
    out, state = call.out[:640, 1], call.state[0, 1]
    if what == "q":
        assert not torch.isfinite(out[at]).any()
        close(out[at + 1:], refs[0][0][at + 1:, 1], refs[0][2][at + 1:, 1])
        close(state, refs[0][1][1], refs[0][3][1])
    elif what in ("k", "g"):
        assert not torch.isfinite(out[at:]).any()
        assert not torch.isfinite(state[:, 3] if what == "k" else state).any()
    else:  # one row of the state
        assert not torch.isfinite(out[at:, 3]).any() and not torch.isfinite(state[3, 3 if what == "v" else 5]).any()
        rest = [r for r in range(d) if r != 3]
        close(out[:, rest], refs[0][0][:, 1, rest], refs[0][2][:, 1, rest])
        close(state[rest], refs[0][1][1, rest], refs[0][3][1, rest])


def test_graphs_and_streams_with_states_between_segments():
    """Two calls at once on two streams, each with its workspace, and each as a graph, replayed among eager calls."""
    Hk, Hv, d, lens = 2, 4, 128, [700, 0, 333]
    sets = [weakly_decayed(sum(lens), Hk, Hv, d, d, torch.bfloat16, seed, len(lens)) for seed in (1, 2)]
    kw = dict(head_map=ops.MAP_TILED, decay="rate", out_dtype=torch.bfloat16)
    calls = [Call(c, lens, Hk, Hv, d, d, **kw).run() for c in sets]
    for call in calls:
        assert len(call.slots()) >= 4
        call.check(call.references())
    want = [(call.out.clone(), call.state.clone()) for call in calls]

    def same(call, w):
        assert torch.equal(call.out, w[0]) and torch.equal(call.state, w[1])

    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    both = [Call(c, lens, Hk, Hv, d, d, stream=s, **kw) for c, s in zip(sets, streams)]
    for _ in range(3):
        for call in both:
            call.state.copy_(call.start)
            call.out.zero_()
        torch.cuda.synchronize()
        for call in both:
            call.call.launch()
        torch.cuda.synchronize()
        for call, w in zip(both, want):
            same(call, w)
    graphs = []
    for c in sets:
        graph = torch.cuda.CUDAGraph()
        call = Call(c, lens, Hk, Hv, d, d, **kw)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            call.prepare().launch()
        graphs.append((graph, call))
    for _ in range(3):
        for graph, call in graphs:
            call.state.copy_(call.start)
            call.out.fill_(9)
        torch.cuda.synchronize()
        for graph, call in graphs:
            graph.replay()
        calls[0].call.launch()
        torch.cuda.synchronize()
        for (_, call), w in zip(graphs, want):
            same(call, w)
