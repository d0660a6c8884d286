"""Decayed linear attention (gdn_linattn_decode_step, gdn_linattn_prefill_chunked): refusals on the
CPU, and on the GPU every output and state element against the recurrence in 64 bits.

Tolerance. With u = 2^-24 and the recurrence run on absolute values, A <- exp(g) A + |v| |k|^T, a term
that has aged n tokens went through n steps of at most 6 u relative error each (exp to 2 ulp = 4 u, the
product and the fused add u each); the chunked form applies one factor instead of n and adds at most
20 u of constant work (three 8-bit parts leave nothing of an f32; the products of parts left out are 2^-22 = 4 u of a
product at most, test_linattn_accuracy; its f32 sums are shorter than the recurrence's). So a state element is off by at
most (6 T + 20) u A, and an output by scale * ((6 T + 20) + dk + 2) u (A |q|) plus its own rounding,
eps / 2 of its type (and half its smallest subnormal). Sixteen-bit outputs of the prefill are allowed 3 * 2^-16 of
scale * (A |q|) more here than they need: test_linattn_accuracy holds them to the bound without it.
"""
import ctypes

import pytest
import torch

from gated_deltanet_linear_step_amd import ops

U = 2.0 ** -24
DEV = "cuda:0"
SHAPES = [(32, 32), (64, 64), (96, 96), (128, 128), (64, 128), (128, 64), (128, 256), (256, 128), (256, 256)]
OK, NULL, SHAPE, UNSUPPORTED, OVERFLOW, ALIGN, WORKSPACE = 0, 1, 2, 3, 4, 5, 6


# ---- the recurrence in 64 bits -------------------------------------------------

def reference(q, k, v, S0, g, Hk, head_map, scale):
    """q, k [T][Hk][dk], v [T][Hv][dv], S0 [Hv][dv][dk], g [T][Hv]: (o, S, A |q| scale, A)."""
    Hv = v.shape[1]
    heads = [h // (Hv // Hk) if head_map == ops.MAP_GROUPED else h % Hk for h in range(Hv)]
    q, k, v, g = (x.cpu().double() for x in (q, k, v, g))
    q, k = q[:, heads], k[:, heads]
    S = S0.cpu().double().clone()
    A = S.abs()
    o, oa = torch.zeros_like(v), torch.zeros_like(v)
    for t in range(len(q)):
        a = g[t].exp()[:, None, None]
        S = a * S + v[t][..., None] * k[t][:, None]
        A = a * A + (v[t][..., None] * k[t][:, None]).abs()
        o[t] = scale * (S @ q[t][..., None])[..., 0]
        oa[t] = scale * (A @ q[t].abs()[..., None])[..., 0]
    return o, S, oa, A


def close(got, want, room):
    """got within want +- room element by element, nothing unfinite."""
    got = got.detach().cpu().double()
    assert torch.isfinite(got).all()
    off = (got - want).abs() - room
    assert (off <= 0).all(), f"over the bound by {off.max():.3e}; max |error| {(got - want).abs().max():.3e}"


def check(out, state, ref, T, dk, extra=0.0):
    o, S, oa, A = ref
    n = 6 * T + 20
    fin = torch.finfo(out.dtype)
    room = (n + dk + 2) * U * oa * 1.01 + extra * oa
    close(out, o, room + fin.eps / 2 * (o.abs() + room) + fin.smallest_normal * fin.eps)
    close(state, S, n * U * A * 1.01 + 2.0 ** -149)


def extra16(dtype):
    return 0.0 if dtype == torch.float32 else 3 * 2.0 ** -16


def make(T, Hk, Hv, dk, dv, dtype, seed, pad=0, slots=1):
    """One mixed row per token (pad spare elements at its end), a state pool and log decays."""
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    mixed = rand(T, 2 * Hk * dk + Hv * dv + pad)
    mixed[:, Hk * dk:2 * Hk * dk] *= dk ** -0.5
    mixed = mixed.to(dtype)
    return dict(mixed=mixed, state=rand(slots, Hv, dv, dk), g=-0.3 * rand(T, Hv).abs(),
                rate=-torch.rand(Hv, generator=gen))


def views(mixed, Hk, Hv, dk, dv):
    a, b = Hk * dk, 2 * Hk * dk
    return mixed[:, :a], mixed[:, a:b], mixed[:, b:b + Hv * dv]


def split_heads(mixed, Hk, Hv, dk, dv):
    q, k, v = views(mixed, Hk, Hv, dk, dv)
    T = len(mixed)
    return q.reshape(T, Hk, dk), k.reshape(T, Hk, dk), v.reshape(T, Hv, dv)


# ---- refusals (CPU) ------------------------------------------------------------

_BUF = (ctypes.c_float * 4096)()
P = (ctypes.addressof(_BUF) + 255) // 256 * 256  # never dereferenced: validation fails first


def vp(x):
    return ctypes.c_void_p(x) if x else None


def dims(Hk=2, Hv=4, dk=128, dv=128, head_map=0, flags=0, **kw):
    return ops.make_dims(Hk, Hv, dk, dv, head_map, flags, **kw)


def inputs(**kw):
    given = dict(q=vp(P), k=vp(P), v=vp(P), q_stride=1024, k_stride=1024, v_stride=1024,
                 qkv_dtype=ops.BF16, g=vp(P), decay_param=vp(P))
    given.update(kw)
    return ops.Inputs(**given)


def decode(d=None, inp=None, batch=2, T=1, state=P, slots=0, num_slots=2, out_dtype=0, out=P):
    return ops.load().gdn_linattn_decode_step(ctypes.byref(d or dims()), batch, T, ctypes.byref(inp or inputs()),
                                              vp(state), vp(slots), num_slots, out_dtype, vp(out), None)


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(out=0)), (NULL, dict(state=0)), (NULL, dict(inp=inputs(q=None))), (NULL, dict(inp=inputs(g=None))),
    (NULL, dict(d=dims(flags=ops.HEAD_DECAY), inp=inputs(decay_param=None))),
    (SHAPE, dict(d=dims(Hk=3))), (SHAPE, dict(d=dims(head_map=2))), (SHAPE, dict(d=dims(scale=-1.0))),
    (SHAPE, dict(d=dims(flags=ops.HEAD_DECAY, decay=2))), (SHAPE, dict(T=0)), (SHAPE, dict(batch=-1)),
    (SHAPE, dict(batch=3)), (SHAPE, dict(num_slots=-1)), (SHAPE, dict(inp=inputs(q_stride=100))),
    (UNSUPPORTED, dict(d=dims(dk=96))), (UNSUPPORTED, dict(d=dims(flags=ops.L2NORM_QK))),
    (UNSUPPORTED, dict(d=dims(flags=ops.RAW_GATES))), (UNSUPPORTED, dict(d=dims(flags=ops.GATED_NORM))),
    (UNSUPPORTED, dict(d=dims(flags=32))), (UNSUPPORTED, dict(out_dtype=7)), (UNSUPPORTED, dict(inp=inputs(qkv_dtype=3))),
    (ALIGN, dict(inp=inputs(q=vp(P + 2)))), (ALIGN, dict(inp=inputs(v_stride=1026))), (ALIGN, dict(inp=inputs(g=vp(P + 2)))),
    (ALIGN, dict(d=dims(flags=ops.HEAD_DECAY), inp=inputs(decay_param=vp(P + 1)))), (ALIGN, dict(state=P + 8)),
    (OVERFLOW, dict(batch=2 ** 30, T=4, num_slots=2 ** 30)), (OVERFLOW, dict(batch=2 ** 27, num_slots=2 ** 27)),
    (OVERFLOW, dict(batch=2 ** 20, num_slots=2 ** 20)),
    (OK, dict(batch=0)), (OK, dict(batch=0, inp=inputs(q=None, k=None, v=None), out=0)),
])
def test_decode_refusals(want, kw):
    assert decode(**kw) == want


def prefill(d=None, inp=None, cu=(0, 100, 230), total=230, state=P, out_dtype=0, out=P, ws=P, nbytes=1 << 40, cu_dev=P):
    arr = (ctypes.c_int32 * len(cu))(*cu)
    return ops.load().gdn_linattn_prefill_chunked(ctypes.byref(d or dims()), len(cu) - 1, arr, vp(cu_dev), total,
                                                  ctypes.byref(inp or inputs()), vp(state), out_dtype, vp(out), vp(ws),
                                                  nbytes, None)


@pytest.mark.parametrize("want,kw", [
    (SHAPE, dict(cu=(0, 150, 100), total=100)), (SHAPE, dict(total=231)), (SHAPE, dict(cu=(1, 100, 230))),
    (SHAPE, dict(total=-1)), (NULL, dict(cu_dev=0)), (WORKSPACE, dict(ws=0)), (WORKSPACE, dict(nbytes=0)),
    (ALIGN, dict(ws=P + 128)), (UNSUPPORTED, dict(d=dims(flags=ops.STREAM_STATE))), (NULL, dict(inp=inputs(v=None))),
    (OVERFLOW, dict(d=dims(Hk=2, Hv=2048), cu=(0, 2 ** 21), total=2 ** 21, inp=inputs(v_stride=2048 * 128))),
    (OVERFLOW, dict(cu=(0,) * 2 ** 20 + (5,), total=5)), (WORKSPACE, dict(cu=(0,) * (2 ** 20 - 1) + (5,), total=5, ws=0)),
    (OVERFLOW, dict(inp=inputs(q_stride=2 ** 24))), (ALIGN, dict(out=P + 8)), (OK, dict(cu=(0, 0, 0), total=0)), (OK, dict(cu=(0,), total=0)), (SHAPE, dict(cu=(0,), total=3)),
    (OK, dict(cu=(0, 0), total=0, inp=inputs(q=None, k=None, v=None, g=None), out=0, ws=0)),
])
def test_prefill_refusals(want, kw):
    assert prefill(**kw) == want


def test_prefill_workspace_query():
    lib = ops.load()
    for bad in (dims(Hk=3), dims(dk=96)):
        assert lib.gdn_linattn_prefill_workspace_bytes(ctypes.byref(bad), 1, 64) == 0
    assert lib.gdn_linattn_prefill_workspace_bytes(ctypes.byref(dims()), -1, 64) == 0
    # an upper bound over splits: more sequences or tokens never need less
    size = lambda n, t: lib.gdn_linattn_prefill_workspace_bytes(ctypes.byref(dims()), n, t)  # noqa: E731
    grid = [[size(n, t) for t in (0, 1, 64, 1000, 4096, 40000, 2 ** 20)] for n in (1, 2, 7, 300)]
    assert all(a <= b for row in grid for a, b in zip(row, row[1:]))
    assert all(a <= b for r, s in zip(grid, grid[1:]) for a, b in zip(r, s))


# ---- GPU -----------------------------------------------------------------------

def run_decode(c, B, T, Hk, Hv, dk, dv, head_map, decay, out_dtype, slots=None, **kw):
    """The call on the GPU and the 64-bit recurrence of each sequence."""
    mixed, state = c["mixed"].to(DEV), c["state"].to(DEV)
    q, k, v = views(mixed, Hk, Hv, dk, dv)
    if decay == "token":
        dec = dict(g=c["g"].to(DEV))
    else:
        param = c["rate"] if decay == "rate" else (-c["rate"]).log()
        dec = dict(decay_param=param.to(DEV), decay=ops.DECAY_NEGATIVE_RATE if decay == "rate" else ops.DECAY_LOG_RATE)
    out = ops.linattn_decode_step(q, k, v, state, Hk=Hk, Hv=Hv, dk=dk, dv=dv, head_map=head_map, batch=B,
                                  tokens_per_seq=T, state_slots=slots, out_dtype=out_dtype, **dec, **kw)
    refs = []
    for b in range(B):
        s = b if slots is None else int(slots[b])
        if not 0 <= s < len(state):
            refs.append(None)
            continue
        m = c["mixed"][b * T:(b + 1) * T]
        g = c["g"][b * T:(b + 1) * T] if decay == "token" else c["rate"].expand(T, Hv)
        refs.append(reference(*split_heads(m, Hk, Hv, dk, dv), c["state"][s], g, Hk, head_map,
                              kw.get("scale") or dk ** -0.5))
    return out, state, refs


@pytest.mark.gpu
@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_decode_every_shape_and_dtype(dk, dv, dtype):
    B, T, Hk, Hv = 3, 2, 2, 4
    c = make(B * T, Hk, Hv, dk, dv, dtype, dk + dv, slots=B)
    for out_dtype, decay, head_map in ((torch.float32, "token", ops.MAP_TILED), (dtype, "rate", ops.MAP_GROUPED)):
        out, state, refs = run_decode(c, B, T, Hk, Hv, dk, dv, head_map, decay, out_dtype)
        for b in range(B):
            check(out[b * T:(b + 1) * T], state[b], refs[b], T, dk)


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,Hk,Hv,decay,kw", [
    (1, 1, 1, 1, "rate", {}), (1, 1, 16, 48, "token", {}), (2, 1, 1, 5, "log", {}), (1, 33, 2, 2, "token", {}),
    (65, 1, 4, 8, "rate", dict(stream_state=True)), (5, 8, 2, 6, "log", dict(scale=0.37)),
])
def test_decode_sizes(B, T, Hk, Hv, decay, kw):
    c = make(B * T, Hk, Hv, 128, 128, torch.bfloat16, B + T, pad=12, slots=B + 1)
    out, state, refs = run_decode(c, B, T, Hk, Hv, 128, 128, ops.MAP_TILED, decay, torch.float32, **kw)
    for b in range(B):
        check(out[b * T:(b + 1) * T], state[b], refs[b], T, 128)
    assert torch.equal(state[B].cpu(), c["state"][B])  # a slot nobody named


@pytest.mark.gpu
def test_decode_slots_out_of_range_are_left_alone():
    B, T, Hk, Hv, d = 5, 3, 2, 4, 64
    c = make(B * T, Hk, Hv, d, d, torch.float16, 9, slots=7)
    slots = torch.tensor([6, -1, 0, 7, 3], dtype=torch.int32, device=DEV)
    out = torch.full((B * T, Hv, d), 7.0, device=DEV)
    got, state, refs = run_decode(c, B, T, Hk, Hv, d, d, ops.MAP_GROUPED, "token", torch.float32, slots=slots, out=out)
    assert got is out
    for b in range(B):
        if refs[b] is None:
            assert (out[b * T:(b + 1) * T] == 7.0).all()
        else:
            check(out[b * T:(b + 1) * T], state[int(slots[b])], refs[b], T, d)
    for s in (1, 2, 4, 5):
        assert torch.equal(state[s].cpu(), c["state"][s])


@pytest.mark.gpu
def test_decode_call_and_its_split_agree_bit_for_bit():
    Hk, Hv, d = 2, 4, 128
    c = make(5, Hk, Hv, d, d, torch.bfloat16, 4)
    q, k, v = views(c["mixed"].to(DEV), Hk, Hv, d, d)
    kw = dict(Hk=Hk, Hv=Hv, dk=d, dv=d, head_map=ops.MAP_TILED, batch=1)
    g = c["g"].to(DEV)
    whole = c["state"].to(DEV)
    o = ops.linattn_decode_step(q, k, v, whole, tokens_per_seq=5, g=g, **kw)
    parts = c["state"].to(DEV)
    o1 = ops.linattn_decode_step(q[:3], k[:3], v[:3], parts, tokens_per_seq=3, g=g[:3], **kw)
    o2 = ops.linattn_decode_step(q[3:], k[3:], v[3:], parts, tokens_per_seq=2, g=g[3:], **kw)
    assert torch.equal(whole, parts) and torch.equal(o, torch.cat([o1, o2]))


def run_prefill(c, lens, Hk, Hv, dk, dv, head_map, decay, out_dtype, **kw):
    mixed, state = c["mixed"].to(DEV), c["state"].to(DEV)
    q, k, v = views(mixed, Hk, Hv, dk, dv)
    cu = torch.tensor([0] + list(lens)).cumsum(0)
    dec = dict(g=c["g"].to(DEV)) if decay == "token" else \
        dict(decay_param=c["rate"].to(DEV), decay=ops.DECAY_NEGATIVE_RATE)
    out = ops.linattn_prefill_chunked(q, k, v, state, cu, Hk=Hk, Hv=Hv, dk=dk, dv=dv, head_map=head_map,
                                      out_dtype=out_dtype, **dec, **kw)
    return out, state, cu


def check_prefill(c, lens, Hk, Hv, dk, dv, head_map, decay, out, state, cu, heads=None):
    for i, n in enumerate(lens):
        a, b = int(cu[i]), int(cu[i + 1])
        if n == 0:
            assert torch.equal(state[i].cpu(), c["state"][i])
            continue
        g = c["g"][a:b] if decay == "token" else c["rate"].expand(n, Hv)
        ref = reference(*split_heads(c["mixed"][a:b], Hk, Hv, dk, dv), c["state"][i], g, Hk, head_map, dk ** -0.5)
        check(out[a:b], state[i], ref, n, dk, extra16(out.dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_prefill_every_shape_and_dtype(dk, dv, dtype):
    Hk, Hv, lens = 2, 4, [1, 63, 0, 65, 130, 7]
    c = make(sum(lens), Hk, Hv, dk, dv, dtype, dk + dv, pad=4, slots=len(lens))
    for out_dtype, decay, head_map in ((torch.float32, "rate", ops.MAP_GROUPED), (dtype, "token", ops.MAP_TILED)):
        out, state, cu = run_prefill(c, lens, Hk, Hv, dk, dv, head_map, decay, out_dtype)
        check_prefill(c, lens, Hk, Hv, dk, dv, head_map, decay, out, state, cu)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,Hk,Hv,dtype", [
    ([1], 1, 1, torch.bfloat16), ([64], 1, 3, torch.bfloat16), ([2049], 1, 2, torch.bfloat16),
    ([1500, 700], 2, 2, torch.float16), ([333], 1, 2, torch.float32), ([5] * 40, 1, 2, torch.bfloat16),
    ([900, 0, 1, 0, 31], 2, 4, torch.bfloat16),
])
def test_prefill_lengths(lens, Hk, Hv, dtype):
    c = make(sum(lens), Hk, Hv, 128, 128, dtype, sum(lens), slots=len(lens))
    out, state, cu = run_prefill(c, lens, Hk, Hv, 128, 128, ops.MAP_GROUPED, "token", torch.float32)
    check_prefill(c, lens, Hk, Hv, 128, 128, ops.MAP_GROUPED, "token", out, state, cu)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,Hv", [([257] * 7, 4), ([256, 257, 255, 600, 0, 1025], 2), ([9000], 16), ([3] * 70 + [900] + [0] * 5 + [700], 2),
                                     ([129] * 9, 4), ([129, 128, 127, 193, 320, 321], 2), ([300] * 70, 2), ([12000], 1)])
def test_prefill_segments_keep_to_the_workspace(lens, Hv):
    """Sequences just past and far past one segment, among many short ones: states within the bound, two runs alike bit
    for bit, and no byte outside the workspace that the query asks for."""
    Hk, d, n = 1, 32, sum(lens)
    c = make(n, Hk, Hv, d, d, torch.bfloat16, n, slots=len(lens))
    need = ops.linattn_prefill_workspace_bytes(Hk=Hk, Hv=Hv, dk=d, dv=d, num_seqs=len(lens), total_tokens=n)
    room = torch.full((need + 8192,), 77, dtype=torch.uint8, device=DEV)
    out, state, cu = run_prefill(c, lens, Hk, Hv, d, d, ops.MAP_GROUPED, "token", torch.float32, workspace=room[4096:4096 + need])
    assert (room[:4096] == 77).all() and (room[4096 + need:] == 77).all()
    again, state_again, _ = run_prefill(c, lens, Hk, Hv, d, d, ops.MAP_GROUPED, "token", torch.float32)
    assert torch.equal(out, again) and torch.equal(state, state_again)
    check_prefill(c, lens, Hk, Hv, d, d, ops.MAP_GROUPED, "token", out, state, cu)


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[1] * 5, [8, 3, 0, 5], [9, 8]])
def test_prefill_of_short_sequences(lens):
    Hk, Hv, d = 2, 4, 128
    c = make(sum(lens), Hk, Hv, d, d, torch.float16, 77, slots=len(lens))
    out, state, cu = run_prefill(c, lens, Hk, Hv, d, d, ops.MAP_TILED, "rate", torch.float16)
    check_prefill(c, lens, Hk, Hv, d, d, ops.MAP_TILED, "rate", out, state, cu)


@pytest.mark.gpu
def test_prefill_leaves_the_states_between_segments_as_the_running_sum_left_them():
    # more segments than the card holds at a time, and calls that agree bit for bit
    Hk, Hv, d, n = 4, 8, 128, 20000
    gen = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(n, H * d, generator=gen).to(DEV) * d ** -0.5 for H in (Hk, Hk, Hv))
    g = torch.full((n, Hv), -1e-3, device=DEV)
    cu = torch.tensor([0, n], dtype=torch.int32)
    heads = dict(Hk=Hk, Hv=Hv, dk=d, dv=d)
    need = ops.linattn_prefill_workspace_bytes(num_seqs=1, total_tokens=n, **heads)
    first = None
    for _ in range(4):
        ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
        state = torch.ones(1, Hv, d, d, device=DEV)
        o = ops.linattn_prefill_chunked(q, k, v, state, cu.to(DEV), cu_seqlens_host=cu, g=g, workspace=ws,
                                        head_map=ops.MAP_GROUPED, **heads)
        first = first or (o, state, ws)
        assert torch.equal(o, first[0]) and torch.equal(state, first[1]) and torch.equal(ws, first[2])


@pytest.mark.gpu
def test_growing_states():
    """Log decays above 0 are no decay, but the formula holds for them too."""
    Hk, Hv, d, n = 1, 2, 64, 150
    c = make(n, Hk, Hv, d, d, torch.bfloat16, 8)
    c["g"] = c["g"] + 0.2
    out, state, cu = run_prefill(c, [n], Hk, Hv, d, d, ops.MAP_GROUPED, "token", torch.float32)
    check_prefill(c, [n], Hk, Hv, d, d, ops.MAP_GROUPED, "token", out, state, cu)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_decay_that_is_not_a_number(dtype):
    """It spoils its head's outputs and state from its token on, and nothing else."""
    Hk, Hv, d, n, at = 1, 2, 64, 100, 37
    c = make(n, Hk, Hv, d, d, dtype, 6)
    fine, fine_state, _ = run_prefill(c, [n], Hk, Hv, d, d, ops.MAP_GROUPED, "token", torch.float32)
    c["g"][at, 0] = float("nan")
    out, state, _ = run_prefill(c, [n], Hk, Hv, d, d, ops.MAP_GROUPED, "token", torch.float32)
    assert torch.equal(out[:, 1], fine[:, 1]) and torch.equal(out[:at, 0], fine[:at, 0])
    assert torch.equal(state[0, 1], fine_state[0, 1])
    assert torch.isnan(out[at:, 0]).all() and torch.isnan(state[0, 0]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_forgetting_and_strong_decays(dtype):
    """Log decays of -inf, of -1e5 and of 0 among ordinary ones: exp(g) is 0, 0 and 1."""
    Hk, Hv, d, n = 1, 2, 64, 200
    c = make(n, Hk, Hv, d, d, dtype, 21)
    c["g"][17, 0] = c["g"][64, 1] = c["g"][150, 0] = -float("inf")
    c["g"][40:44] = -1e5
    c["g"][100:130] = 0
    c["g"][:, 1][3] = -80.0
    out, state, cu = run_prefill(c, [n], Hk, Hv, d, d, ops.MAP_GROUPED, "token", torch.float32)
    check_prefill(c, [n], Hk, Hv, d, d, ops.MAP_GROUPED, "token", out, state, cu)
    dec, st, refs = run_decode(c, 1, n, Hk, Hv, d, d, ops.MAP_GROUPED, "token", torch.float32)
    check(dec, st[0], refs[0], n, d)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("what", ["q", "k", "v"])
def test_prefill_what_is_not_finite_stays_behind_its_token(bad, what):
    """A NaN or infinity of one token: earlier tokens, other heads and other sequences keep their values."""
    Hk, Hv, d, lens, at = 2, 2, 64, [150, 70], 75
    c = make(sum(lens), Hk, Hv, d, d, torch.bfloat16, 5, slots=2)
    out0, state0, _ = run_prefill(c, lens, Hk, Hv, d, d, ops.MAP_GROUPED, "token", torch.float32)
    q, k, v = split_heads(c["mixed"], Hk, Hv, d, d)
    dict(q=q, k=k, v=v)[what][at, 1, 3] = bad
    for a, x in zip(views(c["mixed"], Hk, Hv, d, d), (q, k, v)):
        a.copy_(x.reshape(sum(lens), -1))
    out, state, _ = run_prefill(c, lens, Hk, Hv, d, d, ops.MAP_GROUPED, "token", torch.float32)
    # the chunk with the bad value may take another summation order: same bound, not same bits
    check_prefill_part = [(slice(0, at), 1), (slice(0, 150), 0), (slice(150, 220), 0), (slice(150, 220), 1)]
    for rows, h in check_prefill_part:
        torch.testing.assert_close(out[rows, h], out0[rows, h], rtol=2 ** -20, atol=2 ** -20)
    hit = out[at, 1] if what != "v" else out[at, 1, 3:4]
    assert not torch.isfinite(hit).any()
    if what == "q":
        assert torch.equal(state, state0)
    else:
        assert torch.equal(state[1], state0[1]) and torch.equal(state[0, 0], state0[0, 0])
        line = state[0, 1, :, 3] if what == "k" else state[0, 1, 3]
        assert not torch.isfinite(line).any()


@pytest.mark.gpu
def test_prefill_equals_decode_and_leaves_what_is_not_its_own():
    Hk, Hv, d, lens = 2, 4, 128, [70, 3]
    n = sum(lens)
    c = make(n + 9, Hk, Hv, d, d, torch.bfloat16, 31, slots=2)
    mixed, g = c["mixed"].to(DEV), c["g"].to(DEV)
    q, k, v = views(mixed[:n], Hk, Hv, d, d)
    big = torch.full((n + 9, Hv, d), 5.0, device=DEV)
    pool = torch.full((4, Hv, d, d), 3.0, device=DEV)
    pool[1:3] = c["state"].to(DEV)
    need = ops.linattn_prefill_workspace_bytes(Hk=Hk, Hv=Hv, dk=d, dv=d, num_seqs=2, total_tokens=n)
    room = torch.full((max(need, 256) + 512,), 77, dtype=torch.uint8, device=DEV)
    cu = torch.tensor([0, 70, 73], dtype=torch.int32)
    ops.linattn_prefill_chunked(q, k, v, pool[1:3], cu.to(DEV), cu_seqlens_host=cu, Hk=Hk, Hv=Hv, dk=d, dv=d,
                                head_map=ops.MAP_TILED, g=g[:n], out=big[:n], workspace=room[256:256 + max(need, 256)])
    assert (big[n:] == 5.0).all() and (pool[0] == 3.0).all() and (pool[3] == 3.0).all()
    assert (room[:256] == 77).all() and (room[256 + max(need, 256):] == 77).all()
    c2 = dict(c, mixed=c["mixed"][:n], g=c["g"][:n])
    check_prefill(c2, lens, Hk, Hv, d, d, ops.MAP_TILED, "token", big[:n], pool[1:3], cu)
    # the next token of both sequences, on the states that the prefill left
    before = pool[1:3].cpu()
    q1, k1, v1 = views(mixed[n:n + 2], Hk, Hv, d, d)
    o = ops.linattn_decode_step(q1, k1, v1, pool[1:3], Hk=Hk, Hv=Hv, dk=d, dv=d, head_map=ops.MAP_TILED, batch=2,
                                g=g[n:n + 2].contiguous())
    for b in range(2):
        ref = reference(*split_heads(c["mixed"][n + b:n + b + 1], Hk, Hv, d, d), before[b], c["g"][n + b:n + b + 1],
                        Hk, ops.MAP_TILED, d ** -0.5)
        check(o[b:b + 1], pool[1 + b], ref, 1, d)


@pytest.mark.gpu
def test_graphs_streams_and_two_calls_at_once():
    """Prefill and decode captured together and replayed, and the same work on two other streams at once."""
    Hk, Hv, d, lens = 2, 4, 128, [300, 41]
    n = sum(lens)
    kw = dict(Hk=Hk, Hv=Hv, dk=d, dv=d, head_map=ops.MAP_GROUPED)
    sets = []
    for seed in (1, 2):
        c = make(n + 2, Hk, Hv, d, d, torch.bfloat16, seed, slots=2)
        mixed, g = c["mixed"].to(DEV), c["g"].to(DEV)
        cu = torch.tensor([0, 300, 341], dtype=torch.int32)
        s = dict(c=c, state=c["state"].to(DEV), cu=cu, cud=cu.to(DEV), out=torch.empty(n, Hv, d, device=DEV),
                 out1=torch.empty(2, Hv, d, device=DEV), g=g, mixed=mixed,
                 ws=torch.empty(max(256, ops.linattn_prefill_workspace_bytes(Hk=Hk, Hv=Hv, dk=d, dv=d, num_seqs=2,
                                                                            total_tokens=n)), dtype=torch.uint8, device=DEV))
        sets.append(s)

    def both(s, stream):
        q, k, v = views(s["mixed"][:n], Hk, Hv, d, d)
        a = ops.prepare_linattn_prefill_chunked(q, k, v, s["state"], s["cud"], s["cu"], s["out"], s["ws"],
                                                g=s["g"][:n], stream=stream, **kw)
        q, k, v = views(s["mixed"][n:], Hk, Hv, d, d)
        b = ops.prepare_linattn_decode_step(q, k, v, s["state"], s["out1"], batch=2, g=s["g"][n:], stream=stream, **kw)
        return a, b

    want = []
    for s in sets:
        for call in both(s, None):
            call.launch()
        torch.cuda.synchronize()
        want.append([s[x].clone() for x in ("out", "out1", "state")])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in sets:
        s["state"].copy_(s["c"]["state"])
        s["out"].zero_()
        s["out1"].zero_()
    torch.cuda.synchronize()
    calls = [both(s, st) for s, st in zip(sets, streams)]
    for i in range(2):  # interleaved over the two streams
        for pair in calls:
            pair[i].launch()
    torch.cuda.synchronize()
    for s, w in zip(sets, want):
        assert all(torch.equal(s[x], y) for x, y in zip(("out", "out1", "state"), w))
    s, w = sets[0], want[0]
    graph = torch.cuda.CUDAGraph()
    start = s["c"]["state"].to(DEV)
    with torch.cuda.graph(graph):
        for call in both(s, None):
            call.launch()
    for _ in range(3):
        s["state"].copy_(start)
        s["out"].fill_(9)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s[x], y) for x, y in zip(("out", "out1", "state"), w))


@pytest.mark.gpu
def test_binding_refusals():
    Hk, Hv, d = 2, 4, 64
    c = make(4, Hk, Hv, d, d, torch.bfloat16, 3, slots=4)
    q, k, v = views(c["mixed"].to(DEV), Hk, Hv, d, d)
    st, g = c["state"].to(DEV), c["g"].to(DEV)
    kw = dict(Hk=Hk, Hv=Hv, dk=d, dv=d, head_map=ops.MAP_GROUPED, batch=4)
    call = lambda **m: ops.linattn_decode_step(*m.pop("qkv", (q, k, v)), m.pop("state", st),  # noqa: E731
                                               **{**kw, "g": g, **m})
    with pytest.raises(ValueError):
        call(batch=5)                                    # rows that q does not have
    with pytest.raises(ValueError):
        call(g=g[:3])
    with pytest.raises(ValueError):
        call(g=None)
    with pytest.raises(ValueError):
        call(decay_param=c["rate"].to(DEV))              # both
    with pytest.raises(ValueError):
        call(g=c["g"])                                   # on the host
    with pytest.raises(ValueError):
        call(state=st.double())
    with pytest.raises(ValueError):
        call(state_slots=torch.zeros(4, dtype=torch.int64, device=DEV))
    with pytest.raises(ops.GdnError):
        call(dk=32, dv=32, Hk=4, Hv=8, state=torch.zeros(4, 8, 32, 32, device=DEV), g=torch.zeros(4, 8, device=DEV),
             head_map=5)
    out = ops.linattn_decode_step(q[:0], k[:0], v[:0], st, Hk=Hk, Hv=Hv, dk=d, dv=d, head_map=0, batch=0, g=g[:0])
    assert out.shape == (0, Hv, d)
    cu = torch.zeros(5, dtype=torch.int32)
    out = ops.linattn_prefill_chunked(q[:0], k[:0], v[:0], st, cu, Hk=Hk, Hv=Hv, dk=d, dv=d, head_map=0, g=g[:0])
    assert out.shape == (0, Hv, d) and torch.equal(st.cpu(), c["state"])
