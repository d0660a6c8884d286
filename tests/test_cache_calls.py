"""Calls of rope and of the page operators that the header allows: positions below 0, angles of any size, rows far apart, outputs beside one
another; a page twice in a row, pages that are held by no row, tables and pools in which nothing is in use."""
import pytest
import torch

from gated_deltanet_linear_step_amd import ops
from test_pages import Cache
from test_rope import close, mixed, turned

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
B16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("dtype", [B16, F16, F32])
@pytest.mark.parametrize("layout", [ops.ROPE_HALF, ops.ROPE_INTERLEAVED])
@pytest.mark.parametrize("magnitude", [1.0, -0.75])
def test_positions_below_zero(dtype, layout, magnitude):
    q, k, _ = mixed(40, 3, 2, 96, dtype, 1, 0)
    w = ops.rope_frequencies(64, 1e4)[0].to(DEV)
    positions = torch.randint(-2 ** 20, 1, (40,), device=DEV, dtype=torch.int32)
    positions[:3] = torch.tensor([-1, 0, -2 ** 20], device=DEV)
    for x, y in zip((q, k), ops.rope(positions, w, q=q, k=k, layout=layout, magnitude=magnitude)):
        close(y, *turned(x, positions, w, magnitude, layout))
        assert torch.equal(y[..., 64:], x[..., 64:])


@pytest.mark.parametrize("layout", [ops.ROPE_HALF, ops.ROPE_INTERLEAVED])
def test_quarter_turns(layout):
    """Angles of whole quarters of a turn, as near as f64 has them, over all eight octants and both signs. An angle of 2 pi 2^k is a
    rounded product: off by 2^-52 of itself, which is beside the bound's own terms up to 2^20 turns."""
    q, _, _ = mixed(64, 1, 1, 16, F32, 3, 0)
    w = torch.tensor([0.0, 0.125, 0.25, 0.375, 0.5, 1.0, 2.0 ** -20, 0.7], dtype=torch.float64, device=DEV) * (2 * torch.pi)
    positions = torch.arange(-32, 32, device=DEV, dtype=torch.int32)
    got = ops.rope(positions, w, q=q, layout=layout)[0]
    close(got, *turned(q, positions, w, 1.0, layout))


def test_rows_past_32_bits_and_outputs_beside_one_another():
    tokens, far = 20, 1 << 28  # elements from row to row
    buf = torch.zeros(tokens * far, dtype=B16, device=DEV)
    q = buf.as_strided((tokens, 2, 64), (far, 64, 1), 0)
    k = buf.as_strided((tokens, 1, 64), (far, 64, 1), 1024)
    q_out, k_out = (buf.as_strided((tokens, h, 64), (far, 64, 1), at) for h, at in ((2, 4096), (1, 4096 + 128)))
    gen = torch.Generator(DEV).manual_seed(1)
    for x in (q, k):
        x.copy_(torch.randn(x.shape, generator=gen, device=DEV))
    w = ops.rope_frequencies(64)[0].to(DEV)
    positions = torch.arange(tokens, device=DEV, dtype=torch.int32)
    ops.prepare_rope(positions, w, q=q, q_out=q_out, k=k, k_out=k_out).launch()
    for x, y in ((q, q_out), (k, k_out)):
        close(y, *turned(x, positions, w, 1.0, ops.ROPE_HALF))
    # pages whose strides pass 32 bits
    pools = [buf.as_strided((tokens, 1, 16, 64), (far, 1024, 64, 1), at) for at in (8192, 16384)]
    slots = (torch.arange(tokens, device=DEV).flip(0) * 16 + 5).to(torch.int32)
    ops.rope(positions, w, k=k, v=k_out, k_pages=pools[0], v_pages=pools[1], slots=slots)
    assert torch.equal(pools[0][:, :, 5].flip(0), k_out) and torch.equal(pools[1][:, :, 5].flip(0), k_out)


def test_a_page_twice_in_a_row_and_pages_that_no_row_holds():
    """Two references of one row count as two; what is held outside the table (a prefix) is in use and moves too."""
    c = Cache(rows=6, width=5, pages=16, ps=4)
    c.reserve([0, 1], [12, 8])
    page = c.want.table[0][1]
    for row, e in ((0, 3), (2, 0)):
        c.table[row, e] = page
        c.want.table[row][e] = page
        c.refs[page] += 1
        c.want.refs[page] += 1
    c.refs[13] += 2                       # held elsewhere
    c.want.refs[13] += 2
    assert c.fork([0, 2], [3, 4], [16, 3]) == [0, 0]
    c.free([1, 0])
    assert c.reserve([5], [20]) == [0]
    c.compact()
    c.free([2, 3, 4, 5])
    c.compact()
    assert sum(r > 0 for r in c.want.refs) == 1


def test_nothing_in_use():
    c = Cache(rows=3, width=2, pages=9, ps=4)
    c.compact()
    c.free([0, 1, 2])
    assert c.fork([0], [1], [1]) == [2] and c.fork([0], [1], [0]) == [0] and c.reserve([0, 1], [0, 0]) == [0, 0]
    # every page in use
    assert c.reserve([0, 1, 2], [8, 8, 8]) == [0, 0, 0]
    c.refs[6:] = 1
    c.want.refs[6:] = [1] * 3
    c.compact()
    assert c.reserve([0], [8]) == [0] and c.fork([0], [0], [8]) == [2]
