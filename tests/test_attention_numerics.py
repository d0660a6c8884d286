"""Attention at the ends of its arithmetic -- values that are not finite in runs of no weight, tiny weights, long sums, huge
scores -- on inputs whose scores f32 holds exactly, against what 64 bits give. Bounds beside each test, with u the type's half step
(attn_reference) and E = 2^-24."""
import pytest
import torch

from attn_reference import half_step, near
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
