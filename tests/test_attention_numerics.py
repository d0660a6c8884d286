"""Attention at the ends of its arithmetic -- values that are not finite in runs of no weight, tiny weights, long sums, huge
scores -- on inputs whose scores f32 holds exactly, against what 64 bits give. Bounds beside each test, with u the type's half step
(attn_reference) and E = 2^-24."""
import math

import pytest
import torch

from attn_reference import E, half_step, near
from gated_deltanet_linear_step_amd import ops

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
B16, F16 = torch.bfloat16, torch.float16
INF = float("inf")


@pytest.mark.parametrize("D,dtype", [(64, B16), (96, F16), (128, B16), (256, F16)])
@pytest.mark.parametrize("bad", [INF, -INF, float("nan")])
@pytest.mark.parametrize("n", [3000, 30000])
def test_what_is_not_finite_reaches_the_row_from_a_run_of_no_weight(D, dtype, bad, n):
    """A value that is seen counts whatever its weight, also where its run of keys is joined with a factor that f32 holds as 0."""
    # the first half's keys have score -1000, the others 0: whole runs have weights of e^-1000
    kp = torch.zeros(-(-n // 64), 1, 64, D, dtype=dtype, device=DEV)
    kp[:n // 128, :, :, 0] = -1000.0
    vp = torch.ones_like(kp)
    vp[0, 0, 5, 3] = bad
    q = torch.zeros(2, 1, D, dtype=dtype, device=DEV)
    q[..., 0] = 1
    k, v = (x.transpose(1, 2).reshape(-1, 1, D)[:n] for x in (kp, vp))
    cu, cu_k = torch.tensor([0, 2], dtype=torch.int32), torch.tensor([0, n], dtype=torch.int32)
    table = torch.arange(len(kp), dtype=torch.int32, device=DEV)[None]
    outs = [ops.attention_prefill(q, k, v, cu, cu_k=cu_k, scale=1.0),
            ops.attention_decode(q, kp, vp, table, torch.tensor([n], dtype=torch.int32, device=DEV), batch=1, tokens_per_seq=2, max_len=n, scale=1.0)]
    for out in outs:
        assert not torch.isfinite(out[:, 0, 3]).any()
        # weights of 1 and values of 1: their sum over their sum, each rounded once
        rest = torch.cat([out[:, 0, :3], out[:, 0, 4:]], 1)
        near(rest, torch.ones_like(rest, dtype=torch.float64), torch.full_like(rest, 2 * half_step(dtype), dtype=torch.float64))


def one_strong_key(D, dtype, Hkv, weak, weak_v, ps):
    """Two pages: the first key of the first has score 0 with a query of one 1 in front, and value 0; the others -weak (scale 1)."""
    kp = torch.zeros(2, Hkv, ps, D, dtype=dtype, device=DEV)
    kp[..., 0] = -weak
    kp[0, :, 0, 0] = 0
    vp = torch.full((2, Hkv, ps, D), weak_v, dtype=dtype, device=DEV)
    vp[0, :, 0] = 0
    return kp, vp


def check_strong(out, lse, n, weak, weak_v, dtype):
    """Scores are exact. A weight is off by exp2's 2 E and its argument's 2 weak E, and by u where it enters the product with V. The
    sum of weights is one of at most 512 at a time, in 32 parts or more: (512 + n / 1024) E and 64 E for joins. An output takes 16 keys at
    a time: n / 16 additions of E. Log and product: 4 E of either's value and 8 E."""
    w = math.exp(-weak)
    total = 1 + (n - 1) * w
    want = (n - 1) * w * weak_v / total
    weights, sums, u = (2 + 2 * weak) * E, (576 + n / 1024) * E, half_step(dtype)
    room = abs(want) * (2 * u + 2 * weights + sums + (n / 16) * E)
    near(out, torch.full_like(out, want, dtype=torch.float64), torch.full_like(out, room, dtype=torch.float64))
    room = weights + sums + 4 * E * abs(math.log(total)) + 8 * E
    near(lse, torch.full_like(lse, math.log(total), dtype=torch.float64), torch.full_like(lse, room, dtype=torch.float64))


@pytest.mark.parametrize("D,dtype,weak,n", [(64, B16, 17.0, 1 << 17), (64, B16, 17.0, 1 << 21), (96, B16, 17.0, 1 << 18), (128, B16, 17.0, 1 << 18),
                                            (256, B16, 17.0, 1 << 18), (64, B16, 12.0, 1 << 20), (128, F16, 0.4, 1 << 18),
                                            (256, F16, 5.0, 1 << 18), (64, F16, 1.3, 1 << 20)])
def test_sums_of_many_weights(D, dtype, weak, n):
    """520 key heads of one query each: no row's keys are split."""
    Hkv = 520
    kp, vp = one_strong_key(D, dtype, Hkv, weak, 1.0, 64)
    weak = -float(kp[1, 0, 0, 0])
    q = torch.zeros(1, Hkv, D, dtype=dtype, device=DEV)
    q[..., 0] = 1
    table = torch.ones(1, n // 64, dtype=torch.int32, device=DEV)
    table[0, 0] = 0
    lse = torch.empty(1, Hkv, device=DEV)
    cu, cu_k = torch.tensor([0, 1], dtype=torch.int32), torch.tensor([0, n], dtype=torch.int32)
    out = ops.attention_prefill(q, kp, vp, cu, cu_k=cu_k, table=table, lse=lse, scale=1.0)
    check_strong(out, lse, n, weak, 1.0, dtype)
