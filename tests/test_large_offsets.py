"""Element offsets past 2^31 in states, rows and outputs of the linear attention, the norm and the int8 product: what lies
behind them is compared with 64 bits by the other tests' bounds, and what the call does not own keeps its values."""
import pytest
import torch

from gated_deltanet_linear_step_amd import ops
from test_linattn import check, reference, split_heads, views
from test_linattn_segments import close, recurrence
from test_quant_ops import DEV, check_matmul, check_norm

pytestmark = pytest.mark.gpu
B16 = torch.bfloat16


@pytest.fixture(autouse=True)
def give_memory_back():
    yield
    torch.cuda.empty_cache()


def test_decode_slots_of_a_large_pool():
    Hk, Hv, d, pool = 2, 32, 128, 4300  # 2.25e9 elements
    slots = [pool - 1, 0, pool - 3]
    state = torch.zeros(pool, Hv, d, d, device=DEV)
    gen = torch.Generator().manual_seed(1)
    start = torch.randn(3, Hv, d, d, generator=gen)
    for s, x in zip(slots, start):
        state[s] = x.to(DEV)
    mixed, g = torch.randn(3, 2 * Hk * d + Hv * d, generator=gen).to(B16), -torch.rand(3, Hv, generator=gen)
    out = ops.linattn_decode_step(*views(mixed.to(DEV), Hk, Hv, d, d), state, Hk=Hk, Hv=Hv, dk=d, dv=d,
                                  head_map=ops.MAP_TILED, batch=3, g=g.to(DEV),
                                  state_slots=torch.tensor(slots, dtype=torch.int32, device=DEV))
    for b, s in enumerate(slots):
        ref = reference(*split_heads(mixed[b:b + 1], Hk, Hv, d, d), start[b], g[b:b + 1], Hk, ops.MAP_TILED, d ** -0.5)
        check(out[b:b + 1], state[s], ref, 1, d)
    for s in (1, 2, pool // 2, pool - 4, pool - 2):
        assert (state[s] == 0).all()


def test_prefill_rows_and_outputs():
    Hk, Hv, d, lens = 1, 32, 128, [529900, 100]  # rows of 4352: 2.3e9 elements in, 2.2e9 out
    n, C = sum(lens), 2 * Hk * d + Hv * d
    torch.manual_seed(2)
    mixed = torch.randn(n, C, dtype=B16, device=DEV)
    g = -0.3 * torch.rand(n, Hv, device=DEV) - 0.1
    state = torch.randn(2, Hv, d, d, device=DEV)
    start = state.clone()
    cu = torch.tensor([0, lens[0], n], dtype=torch.int32)
    out = torch.full((n + 1, Hv, d), 5.0, dtype=B16, device=DEV)
    ops.linattn_prefill_chunked(*views(mixed, Hk, Hv, d, d), state, cu.to(DEV), cu_seqlens_host=cu, Hk=Hk, Hv=Hv, dk=d,
                                dv=d, head_map=ops.MAP_GROUPED, g=g, out=out[:n])
    assert (out[n] == 5.0).all()
    heads = [0, 13, 31]
    # the second sequence, and the first one's last tokens: what lies 500 tokens back has decayed by e^-50 at least
    for i, a, b, first, S0 in ((1, lens[0], n, 0, start[1]), (0, lens[0] - 600, lens[0], 500, torch.zeros_like(start[0]))):
        o, S, room_o, room_s, _ = recurrence(mixed[a:b], S0, g[a:b], Hk, d, d, ops.MAP_GROUPED, heads)
        close(out[a + first:b, heads], o[first:], room_o[first:])
        close(state[i, heads], S, room_s)


def test_product_outputs():
    M, N, K = 270000, 8192, 32  # 2.2e9 outputs
    torch.manual_seed(3)
    a = torch.randint(-128, 128, (M, K), dtype=torch.int8, device=DEV)
    w = torch.randint(-128, 128, (N, K), dtype=torch.int8, device=DEV)
    sa, sw = torch.rand(M, device=DEV) + 0.5, torch.rand(N, device=DEV) + 0.5
    out = torch.full((M + 1, N), 9.0, dtype=B16, device=DEV)
    ops.quant_matmul(a, sa, w, sw, out=out[:M])
    assert (out[M] == 9.0).all()
    for rows in (slice(0, 20), slice(M // 2, M // 2 + 20), slice(M - 20, M)):
        check_matmul(out[rows], a[rows], sa[rows], w, sw)


@pytest.mark.parametrize("M,N", [(1100, 40), (40, 1100), (9, 1100)])
def test_product_operands(M, N):
    K, stride = 144, 2 ** 21  # 1100 rows: 2.3e9 bytes
    torch.manual_seed(4)
    a, w = (torch.zeros(n, stride, dtype=torch.int8, device=DEV)[:, :K] for n in (M, N))
    for t in (a, w):
        t.copy_(torch.randint(-128, 128, t.shape, dtype=torch.int8, device=DEV))
    sa, sw = torch.rand(M, device=DEV) + 0.5, torch.rand(N, device=DEV) + 0.5
    check_matmul(ops.quant_matmul(a, sa, w, sw, out_dtype=torch.float32), a, sa, w, sw)


@pytest.mark.parametrize("rows,hidden", [(270000, 8192), (109000, 20000)])  # 2.2e9 elements
def test_norm_rows(rows, hidden):
    torch.manual_seed(5)
    x = torch.randn(rows, hidden, dtype=B16, device=DEV)
    r = torch.randn(rows, hidden, dtype=B16, device=DEV)
    w = 1 + 0.1 * torch.randn(hidden, device=DEV)
    got = ops.add_rms_norm(x, w, residual=r, quantize=True, out_dtype=B16)
    for part in (slice(0, 20), slice(rows // 2, rows // 2 + 20), slice(rows - 20, rows)):
        check_norm({n: t[part] for n, t in got.items()}, x[part], r[part], w)
