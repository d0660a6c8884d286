"""Calls of the linear attention, the norm and the int8 product that their documentation allows and the other tests do not
make: given read-out scales and logarithmic rates in the prefill, separate q, k and v, offsets on the GPU alone, the
streaming hint with every token count, other streams, captured calls that allocate their own workspace, buffers aligned to one
element. Bounds: test_linattn_segments, test_quant_ops."""
import math

import pytest
import torch

from gated_deltanet_linear_step_amd import ops
from test_linattn import DEV, make, split_heads, views
from test_linattn_segments import close, recurrence, weakly_decayed
from test_quant_ops import check_matmul, check_norm, matmul_inputs, norm_inputs

pytestmark = pytest.mark.gpu
B16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("lens", [[5, 3], [70, 9], [640, 30]])  # by the recurrence, in chunks, in segments
@pytest.mark.parametrize("dtype", [torch.float16, F32])
def test_prefill_with_log_rates_a_scale_and_separate_rows(lens, dtype):
    Hk, Hv, d, n, scale = 2, 4, 64, sum(lens), 0.37
    c = weakly_decayed(n, Hk, Hv, d, d, dtype, n, len(lens), 0.1)
    log_rate = torch.tensor([-3.0, -1.0, -5.0, -8.0])
    q, k, v = (x.clone() for x in views(c["mixed"].to(DEV), Hk, Hv, d, d))
    # k's rows apart, v four elements into its buffer
    k = torch.cat([k, torch.full_like(k, float("nan"))], 1)[:, :Hk * d]
    v = torch.cat([torch.full_like(v[:, :4], float("nan")), v], 1)[:, 4:]
    state = c["state"].to(DEV)
    cu = torch.tensor([0] + lens, device=DEV).cumsum(0)  # 64-bit, on the GPU alone
    out = ops.linattn_prefill_chunked(q.view(n, Hk, d), k, v, state, cu, Hk=Hk, Hv=Hv, dk=d, dv=d,
                                      head_map=ops.MAP_GROUPED, decay_param=log_rate.to(DEV), scale=scale)
    at = 0
    for i, m in enumerate(lens):
        # the rate is an f32 exponential, 2 ulp: the reference takes the one that the sequence's tokens share
        g = -log_rate.exp().expand(m, Hv)
        o, S, room_o, room_s, _ = recurrence(c["mixed"][at:at + m], c["state"][i], g, Hk, d, d, ops.MAP_GROUPED)
        # (6 u a token hold an exp of an exact g; 2 ulp of g itself are 4 u |g| more a token, |g| < 0.4: 1.6 u)
        f = scale * math.sqrt(d)
        close(out[at:at + m], o * f, room_o * f * (7.6 / 6))
        close(state[i], S, room_s * (7.6 / 6))
        at += m


@pytest.mark.parametrize("B,T", [(3, 1), (300, 1), (2, 3), (300, 2), (300, 9)])
@pytest.mark.parametrize("dk,dv", [(32, 32), (96, 96), (128, 64), (256, 256)])
def test_the_streaming_hint_changes_no_bit(B, T, dk, dv):
    Hk, Hv = 1, 2
    c = make(B * T, Hk, Hv, dk, dv, B16, B + T, slots=B)
    q, k, v = views(c["mixed"].to(DEV), Hk, Hv, dk, dv)
    got = []
    for hint in (False, True):
        state = c["state"].to(DEV)
        out = ops.linattn_decode_step(q, k, v, state, Hk=Hk, Hv=Hv, dk=dk, dv=dv, head_map=ops.MAP_TILED, batch=B,
                                      tokens_per_seq=T, g=c["g"].to(DEV), stream_state=hint)
        got.append((out, state))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    last = slice((B - 1) * T, B * T)
    o, S, room_o, room_s, _ = recurrence(c["mixed"][last], c["state"][B - 1], c["g"][last], Hk, dk, dv, ops.MAP_TILED)
    close(got[1][0][last], o, room_o)
    close(got[1][1][B - 1], S, room_s)


def chain(x, res, w, wq, ws, state, cu, cud, rate, stream=None):
    """norm -> product -> prefill, each on the given stream, with what they allocate."""
    Hk, Hv, d = 2, 4, 64
    normed = ops.add_rms_norm(x, w, residual=res, quantize=True, stream=stream)
    mixed = ops.quant_matmul(normed["out_q"], normed["out_scale"], wq, ws, stream=stream)
    out = ops.linattn_prefill_chunked(*views(mixed, Hk, Hv, d, d), state, cud, cu_seqlens_host=cu, Hk=Hk, Hv=Hv, dk=d, dv=d,
                                      head_map=ops.MAP_GROUPED, decay_param=rate, decay=ops.DECAY_NEGATIVE_RATE,
                                      out_dtype=B16, stream=stream)
    return dict(normed, mixed=mixed, out=out)


def chain_inputs(seed, lens=(600, 40)):
    Hk, Hv, d, hidden = 2, 4, 64, 256
    C = 2 * Hk * d + Hv * d
    torch.manual_seed(seed)
    x, res = (torch.randn(sum(lens), hidden, device=DEV).to(B16) for _ in range(2))
    wq = torch.randint(-127, 128, (C, hidden), dtype=torch.int8, device=DEV)
    cu = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32)
    return dict(x=x, res=res, w=torch.rand(hidden, device=DEV) + 0.5, wq=wq, ws=torch.full((C,), 2e-4, device=DEV),
                state=torch.randn(2, Hv, d, d, device=DEV), cu=cu, cud=cu.to(DEV), rate=-0.01 * torch.rand(Hv, device=DEV))


def test_other_streams_than_the_current_one():
    """Two chains at once on two streams, beside work on the current one that reuses the memory they free."""
    sets = [chain_inputs(s) for s in (1, 2)]
    starts = [s["state"].clone() for s in sets]
    want = []
    for s in sets:
        got = chain(**s)
        torch.cuda.synchronize()
        want.append({n: t.clone() for n, t in dict(got, state=s["state"]).items()})
        check_norm({n: got[n] for n in ("residual", "out_q", "out_scale")}, s["x"], s["res"], s["w"])
        check_matmul(got["mixed"], got["out_q"], got["out_scale"], s["wq"], s["ws"])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for s, start in zip(sets, starts):
            s["state"].copy_(start)
        torch.cuda.synchronize()
        got = []
        for s, stream in zip(sets, streams):
            got.append(chain(**s, stream=stream))
            torch.full((1 << 20,), float("nan"), device=DEV)
        torch.cuda.synchronize()
        for s, g, w in zip(sets, got, want):
            assert all(torch.equal(t, w[n]) for n, t in dict(g, state=s["state"]).items())


def test_captured_chains_that_allocate_their_own_buffers():
    """Two graphs of whole chains, outputs and workspaces from the graphs' pools, replayed in turn among eager calls."""
    sets = [chain_inputs(s) for s in (3, 4)]
    starts = [s["state"].clone() for s in sets]
    want, graphs = [], []
    for s, start in zip(sets, starts):
        got = chain(**s)
        torch.cuda.synchronize()
        want.append({n: t.clone() for n, t in dict(got, state=s["state"]).items()})
        s["state"].copy_(start)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured = chain(**s)
        graphs.append((graph, captured))
    eager = dict(sets[0], state=starts[0].clone())
    for _ in range(3):
        for s, start in zip(sets, starts):
            s["state"].copy_(start)
        for graph, _ in graphs:
            graph.replay()
        chain(**eager)
        torch.cuda.synchronize()
        for s, (_, captured), w in zip(sets, graphs, want):
            assert all(torch.equal(t, w[n]) for n, t in dict(captured, state=s["state"]).items())


@pytest.mark.parametrize("hidden", [7, 100, 2050, 5003, 17001])
@pytest.mark.parametrize("dtype", [B16, F32])
def test_norm_of_buffers_aligned_to_one_element(hidden, dtype):
    rows = 5
    x, r, w = norm_inputs(rows, hidden + 1, dtype, hidden)
    x, r, w = x[:, 1:], r[:, 1:], w[1:]
    out, res = (torch.full((rows, hidden + 1), 9.0, dtype=dtype, device=DEV) for _ in range(2))
    q = torch.full((rows, hidden + 1), 99, dtype=torch.int8, device=DEV)
    scale = torch.full((rows + 1,), 9.0, device=DEV)
    ops.prepare_add_rms_norm(x, w, residual=r, residual_out=res[:, 1:], out=out[:, 1:], out_q=q[:, 1:],
                             out_scale=scale[1:]).launch()
    check_norm(dict(out=out[:, 1:], residual=res[:, 1:], out_q=q[:, 1:], out_scale=scale[1:]), x, r, w)
    assert (out[:, 0] == 9.0).all() and (res[:, 0] == 9.0).all() and (q[:, 0] == 99).all() and scale[0] == 9.0


@pytest.mark.parametrize("M,N", [(3, 50), (70, 90), (1100, 1100)])
def test_product_of_outputs_and_scales_aligned_to_one_element(M, N):
    a, sa, w, sw = matmul_inputs(M + 1, N + 1, 80, M)
    out = torch.full((M, N + 1), 9.0, dtype=B16, device=DEV)
    ops.prepare_quant_matmul(a[1:], sa[1:], w[1:], sw[1:], out[:, 1:]).launch()
    check_matmul(out[:, 1:], a[1:], sa[1:], w[1:], sw[1:])
    assert (out[:, 0] == 9.0).all()
