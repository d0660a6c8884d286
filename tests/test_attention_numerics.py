"""Attention at the ends of its arithmetic -- values that are not finite in runs of no weight, tiny weights, long sums, huge
scores -- on inputs whose scores f32 holds exactly, against what 64 bits give. Bounds beside each test, with u the type's half step
(attn_reference) and E = 2^-24."""
import math

import pytest
import torch

from attn_reference import E, attention64, causal, half_step, near
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


def check_strong(out, lse, n, weak, weak_v, dtype, more=0.0):
    """Scores are exact. A weight is off by exp2's 2 E and its argument's 2 weak E, and by u where it enters the product with V. The
    sum of weights is one of at most 512 at a time, in 32 parts or more: (512 + n / 1024) E and 64 E for joins. An output takes 16 keys at
    a time: n / 16 additions of E. Log and product: 4 E of either's value and 8 E."""
    w = math.exp(-weak)
    total = 1 + (n - 1) * w
    want = (n - 1) * w * weak_v / total
    weights, sums, u = (2 + 2 * weak) * E, (576 + n / 1024) * E, half_step(dtype)
    room = abs(want) * (2 * u + 2 * weights + sums + (n / 16) * E) + more
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


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("weak", [17.5, 12.0])
def test_f16_weights_far_below_the_largest_count(D, weak):
    """Weights of e^-17.5 = 2^-25.2 and 2^-17.3 of the largest: off by 2^-32 of that at most where they enter the product."""
    Hkv, n = 520, 1 << 17
    kp, vp = one_strong_key(D, F16, Hkv, weak, 100.0, 64)
    q = torch.zeros(1, Hkv, D, dtype=F16, device=DEV)
    q[..., 0] = 1
    table = torch.ones(1, n // 64, dtype=torch.int32, device=DEV)
    table[0, 0] = 0
    lse = torch.empty(1, Hkv, device=DEV)
    cu, cu_k = torch.tensor([0, 1], dtype=torch.int32), torch.tensor([0, n], dtype=torch.int32)
    out = ops.attention_prefill(q, kp, vp, cu, cu_k=cu_k, table=table, lse=lse, scale=1.0)
    check_strong(out, lse, n, weak, 100.0, F16, n * 100.0 * 2.0 ** -32)


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("weak", [17.5, 12.0])
def test_f16_weights_far_below_the_largest_count_in_steps(D, weak):
    """One run of 1024 keys of a sequence; the same keys as a prefix."""
    n, B = 1024, 600
    kp, vp = one_strong_key(D, F16, 1, weak, 60000.0, 16)
    weak_v = float(vp[1, 0, 0, 0])
    q = torch.zeros(B, 2, D, dtype=F16, device=DEV)
    q[..., 0] = 1
    table = torch.ones(B, n // 16, dtype=torch.int32, device=DEV)
    table[:, 0] = 0
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    lse = torch.empty(B, 2, device=DEV)
    for own, prefix in ((lens, {}), (torch.zeros_like(lens), dict(prefix_table=table[0], prefix_len=n))):
        out = ops.attention_decode(q, kp, vp, table, own, batch=B, max_len=n, lse=lse, scale=1.0, **prefix)
        check_strong(out, lse, n, weak, weak_v, F16, n * weak_v * 2.0 ** -32)


def huge(n, T, Hq, Hkv, D, dtype, seed):
    """Queries and keys of small integers times a power of two: their products' f32 sums are exact, 2^22 (f16) or 2^36 (bf16) times an integer."""
    gen = torch.Generator().manual_seed(seed)
    times = 2.0 ** 11 if dtype == F16 else 2.0 ** 18
    q, k = (torch.randint(-6, 7, (m, h, D), generator=gen).double() * times for m, h in ((T, Hq), (n, Hkv)))
    v = torch.randn(n, Hkv, D, generator=gen)
    return q.to(dtype).to(DEV), k.to(dtype).to(DEV), v.to(dtype).to(DEV)


def check_huge(out, lse, q, k, v, sees, scale):
    """The value of the largest score, the mean where several have it: the next is 2^22 times scale below, of weight 0. Equal scores have
    equal weights, off by u where they enter the product and not in their sum; u of the result, 16 E for the rest. lse is a product and a
    log2, of 8 E and 2^-20."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    for h in range(Hq):
        s = q[:, h].double() @ k[:, h // G].double().T
        assert float(s.abs().max()) < 2.0 ** 24 * float(s[s != 0].abs().min())
        s = torch.where(sees, s, -INF)
        top = s.amax(1, keepdim=True)
        hit = ((s == top) & sees).double()
        some = hit.sum(1, keepdim=True).clamp_min(1)
        want = hit @ v[:, h // G].double() / some
        size = hit @ v[:, h // G].double().abs() / some
        room = size * (16 * E + half_step(q.dtype)) + want.abs() * half_step(q.dtype) + (2.0 ** -25 if q.dtype == F16 else 0)
        near(out[:, h], want, room)
        want = torch.where(sees.any(1), top[:, 0] * scale + some[:, 0].log(), -INF)
        near(lse[:, h], want, torch.where(sees.any(1), want.abs() * 8 * E + 2.0 ** -20, 0.0))


@pytest.mark.parametrize("D,dtype", [(64, B16), (96, F16), (128, B16), (128, F16), (256, B16), (256, F16)])
@pytest.mark.parametrize("T,n", [(200, 200), (300, 3000), (3, 20000)])
def test_huge_scores(D, dtype, T, n):
    Hq, Hkv = 4, 2
    q, k, v = huge(n, T, Hq, Hkv, D, dtype, D + n)
    lse = torch.empty(T, Hq, device=DEV)
    scale = 0.11
    cu, cu_k = torch.tensor([0, T], dtype=torch.int32), torch.tensor([0, n], dtype=torch.int32)
    out = ops.attention_prefill(q, k, v, cu, cu_k=cu_k, lse=lse, scale=scale)
    sees = torch.arange(n, device=DEV)[None] <= torch.arange(T, device=DEV)[:, None] + n - T
    check_huge(out, lse, q, k, v, sees, scale)


@pytest.mark.parametrize("D,dtype", [(64, F16), (96, B16), (128, B16), (256, B16)])
@pytest.mark.parametrize("Hq,n,prefix,T", [(4, 90, 0, 1), (4, 9000, 0, 2), (4, 700, 640, 3), (4, 70000, 0, 1), (40, 300, 160, 2)])
def test_huge_scores_in_steps(D, dtype, Hq, n, prefix, T):
    Hkv, ps = 2, 32
    q, k, v = huge(n + prefix, T, Hq, Hkv, D, dtype, D + n)
    pages = -(-(n + prefix) // ps)
    pad = torch.zeros(pages * ps - n - prefix, Hkv, D, dtype=dtype, device=DEV)
    kp, vp = (torch.cat([x, pad]).view(pages, ps, Hkv, D).transpose(1, 2).contiguous() for x in (k, v))
    table = torch.arange(pages, dtype=torch.int32, device=DEV)
    lse = torch.empty(T, Hq, device=DEV)
    out = ops.attention_decode(q, kp, vp, table[None, prefix // ps:].contiguous(), torch.tensor([n], dtype=torch.int32, device=DEV), batch=1,
                               tokens_per_seq=T, max_len=n, prefix_table=table[:prefix // ps].contiguous() if prefix else None,
                               prefix_len=prefix, lse=lse, scale=0.11)
    sees = torch.arange(n + prefix, device=DEV)[None] <= torch.arange(T, device=DEV)[:, None] + n + prefix - T
    check_huge(out, lse, q, k, v, sees, 0.11)


@pytest.mark.parametrize("D,dtype", [(64, B16), (96, F16), (128, B16), (128, F16), (256, B16)])
@pytest.mark.parametrize("n", [150, 4000])
def test_rows_of_every_size_beside_one_another(D, dtype, n):
    """Scores of 2^-8 to 2^18 in the rows of one wave, prompts and steps."""
    gen = torch.Generator().manual_seed(D + n)
    T, Hq, Hkv = 40, 4, 2
    q = torch.randn(T, Hq, D, generator=gen) * 2.0 ** (torch.arange(T) % 20 - 8.0)[:, None, None]
    k, v = (torch.randn(n, Hkv, D, generator=gen) for _ in range(2))
    q, k, v = (x.to(dtype).to(DEV) for x in (q, k, v))
    lse = torch.empty(T, Hq, device=DEV)
    cu, cu_k = torch.tensor([0, T], dtype=torch.int32), torch.tensor([0, n], dtype=torch.int32)
    sees = causal(T, n, DEV)
    want = attention64(q, k, v, sees, 1.0)
    out = ops.attention_prefill(q, k, v, cu, cu_k=cu_k, lse=lse, scale=1.0)
    near(out, want[0], want[2])
    near(lse, want[1], want[3])
    pages = -(-n // 16)
    kp, vp = (torch.cat([x, x[:pages * 16 - n]]).view(pages, 16, Hkv, D).transpose(1, 2).contiguous() for x in (k, v))
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    for rows in (slice(0, 1), slice(33, 40), slice(0, 40)):
        T = rows.stop - rows.start
        lens = torch.tensor([n - 40 + rows.stop], dtype=torch.int32, device=DEV)
        out = ops.attention_decode(q[rows], kp, vp, table, lens, batch=1, tokens_per_seq=T, max_len=n, scale=1.0)
        near(out, want[0][rows], want[2][rows])


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("n", [70, 3000, 40000])
def test_f16_outputs_of_the_largest_values_are_finite(D, n):
    """Every value is f16's largest, of either sign by element, and so is every average of them, also where the weights were all
    rounded up: one key has score 0, the others -0.6926, and e^-0.6926 = 0.50027 rounds to 0.50049."""
    T, Hq, Hkv = 40, 4, 2
    largest = torch.finfo(F16).max
    k = torch.zeros(n, Hkv, D, dtype=F16, device=DEV)
    k[1:, :, 0] = -1
    v = torch.where(torch.arange(D, device=DEV) % 3 == 0, -largest, largest).to(F16).expand(n, Hkv, D).contiguous()
    q = torch.zeros(T, Hq, D, dtype=F16, device=DEV)
    q[..., 0] = 1
    want = v[:1, 0].double().expand(T, Hq, D)
    pages = -(-n // 16)
    kp, vp = (torch.cat([x, x[:pages * 16 - n]]).view(pages, 16, Hkv, D).transpose(1, 2).contiguous() for x in (k, v))
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    cu, cu_k = torch.tensor([0, T], dtype=torch.int32), torch.tensor([0, n], dtype=torch.int32)
    outs = [ops.attention_prefill(q, k, v, cu, cu_k=cu_k, scale=0.6926)]
    for m in (1, 2, T):
        outs.append(ops.attention_decode(q[T - m:], kp, vp, table, lens, batch=1, tokens_per_seq=m, max_len=n, scale=0.6926))
    # weights and the average are rounded by half a step each, the sums of weights and of outputs by n E
    for out in outs:
        near(out, want[:len(out)], want[:len(out)].abs() * (2 * half_step(F16) + 2 * n * E))
