"""The prefill of the decayed linear attention keeps f32 accuracy whatever the types are.

Tolerance. With u = 2^-24 and A, oa as in test_linattn (the recurrence on absolute values): the matrix instructions
take operands of 8-bit parts. Three parts leave nothing of an f32, two nothing of an f16; the first is cut off (what is
left is below 2^-7), the second rounded (2^-16 at most is left), so that the products left out, (1, 2) and (2, 1), are at
most 2^-23 = 2 u each: 4 u of a product. A score has that once, its product with v once more, and its decay three
exponentials and products, 8 u at most: 16 u and one product's rounding in all; a state 4 u, the factor's 4 u and
its product's u. Both are within the 20 u of constant work that test_linattn.check allows beside 6 u a token
and, for an output, dk + 2 roundings of its sum. So a 16-bit output is off by half a unit of its last place beyond
that, and by nothing else: check's `extra` is 0 here.
"""
import pytest
import torch

from gated_deltanet_linear_step_amd import ops
from test_linattn import SHAPES, check, make, reference, run_prefill, split_heads, views

pytestmark = pytest.mark.gpu
B16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def check_rows(c, lens, Hk, dk, out, state, cu):
    for i, n in enumerate(lens):
        a, b = int(cu[i]), int(cu[i + 1])
        if n == 0:
            assert torch.equal(state[i].cpu(), c["state"][i])
            continue
        Hv, dv = out.shape[1:]
        ref = reference(*split_heads(c["mixed"][a:b], Hk, Hv, dk, dv), c["state"][i], c["g"][a:b], Hk, ops.MAP_GROUPED,
                        dk ** -0.5)
        check(out[a:b], state[i], ref, n, dk)


@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("dtype,out_dtype", [(B16, B16), (B16, F16), (F16, F16), (F16, B16), (F32, F16), (F32, B16)])
def test_16_bit_outputs_are_off_by_their_rounding_alone(dk, dv, dtype, out_dtype):
    Hk, Hv, lens = 1, 2, [130, 1, 0, 77]
    c = make(sum(lens), Hk, Hv, dk, dv, dtype, dk + 3 * dv, slots=len(lens))
    out, state, cu = run_prefill(c, lens, Hk, Hv, dk, dv, ops.MAP_GROUPED, "token", out_dtype)
    check_rows(c, lens, Hk, dk, out, state, cu)


def long_mantissas(shape, dtype, gen):
    """Positive numbers around 1 whose bits behind the eighth are all set, or all but the ninth."""
    top = torch.randint(0, 128, shape, generator=gen, dtype=torch.int32)
    power = torch.randint(126, 128, shape, generator=gen, dtype=torch.int32)
    tail = torch.where(torch.rand(shape, generator=gen) < 0.5, 0xFFFF, 0x7FFF).to(torch.int32)
    if dtype == F16:
        tail = tail & 0xE000  # the three bits of an 11-bit number
    return (power * 2 ** 23 + top * 2 ** 16 + tail).view(torch.float32).to(dtype)


@pytest.mark.parametrize("dk,dv", [(64, 64), (96, 96), (128, 128), (256, 256)])
@pytest.mark.parametrize("dtype,out_dtype", [(B16, F16), (B16, F32), (F16, F16), (F16, F32), (F32, F16), (F32, F32)])
@pytest.mark.parametrize("decay", ["token", "none"])
def test_numbers_that_the_parts_cut_worst(dk, dv, dtype, out_dtype, decay):
    """All of one sign, so that what is left out adds up instead of cancelling."""
    Hk, Hv, lens = 1, 2, [97, 9, 1]
    gen = torch.Generator().manual_seed(dk + dv)
    T = sum(lens)
    c = make(T, Hk, Hv, dk, dv, dtype, 5, slots=len(lens))
    c["mixed"] = long_mantissas(tuple(c["mixed"].shape), dtype, gen)
    c["state"] = long_mantissas(tuple(c["state"].shape), F32, gen)
    c["g"] = c["g"] * 0.1 if decay == "token" else torch.zeros_like(c["g"])
    assert all((x.float() > 0.4).all() for x in views(c["mixed"], Hk, Hv, dk, dv))
    out, state, cu = run_prefill(c, lens, Hk, Hv, dk, dv, ops.MAP_GROUPED, "token", out_dtype)
    check_rows(c, lens, Hk, dk, out, state, cu)


@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("dtype", [B16, F16, F32])
def test_16_bit_outputs_are_the_f32_ones_rounded(dk, dv, dtype):
    """Bit for bit, and with the same states: no step of the sums depends on the output's type."""
    Hk, Hv, lens = 2, 4, [600, 33, 9]
    c = make(sum(lens), Hk, Hv, dk, dv, dtype, dk - dv, slots=len(lens))
    wide, state, _ = run_prefill(c, lens, Hk, Hv, dk, dv, ops.MAP_TILED, "rate", F32)
    for out_dtype in (B16, F16):
        out, state16, _ = run_prefill(c, lens, Hk, Hv, dk, dv, ops.MAP_TILED, "rate", out_dtype)
        assert torch.equal(out, wide.to(out_dtype)) and torch.equal(state, state16)


@pytest.mark.parametrize("dtype", [B16, F32])
@pytest.mark.parametrize("power", [127, -100])
def test_values_near_the_ends_of_f32(dtype, power):
    """v and the state up to f32's largest numbers (no part of an operand may overflow), and far below 1."""
    Hk, Hv, d, lens = 1, 2, 64, [130, 20]
    gen = torch.Generator().manual_seed(9)
    c = make(sum(lens), Hk, Hv, d, d, dtype, 9, slots=2)
    q, k, v = (x.float() for x in views(c["mixed"], Hk, Hv, d, d))
    sign = torch.randint(0, 2, v.shape, generator=gen) * 2 - 1
    top = 2.0 ** power * (2 - torch.rand(v.shape, generator=gen) * 2.0 ** -9)  # up to the largest number
    top[torch.rand(v.shape, generator=gen) < 0.2] = 2.0 ** power
    c["mixed"] = torch.cat([q * 2.0 ** -10, k * 2.0 ** -8, sign * torch.clamp(top, max=torch.finfo(dtype).max)], 1).to(dtype)
    assert torch.isfinite(c["mixed"].float()).all()
    c["state"] = c["state"].sign() * 2.0 ** (power - 4) * (1 + torch.rand(c["state"].shape, generator=gen))
    for out_dtype in (F32, B16):
        out, state, cu = run_prefill(c, lens, Hk, Hv, d, d, ops.MAP_GROUPED, "token", out_dtype)
        check_rows(c, lens, Hk, d, out, state, cu)
