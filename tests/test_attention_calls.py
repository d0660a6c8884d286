"""Calls of the attention operators that the header allows: keys and values laid out apart, queries that are not finite, rows far apart.
Against 64 bits (attn_reference: its bounds)."""
import pytest
import torch

from attn_reference import attention64, causal, near
from gated_deltanet_linear_step_amd import ops
from test_attention import check_prompts, check_steps, decode_inputs, offsets, on_pages, packed

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
B16, F16 = torch.bfloat16, torch.float16
NAN, INF = float("nan"), float("inf")


def apart(x, pad):
    """x with its first axis pad elements further apart, NaN between."""
    wide = torch.full((x.shape[0], x[0].numel() + pad), NAN, dtype=x.dtype, device=x.device)
    view = wide[:, :x[0].numel()].view(x.shape)
    view.copy_(x)
    return view


@pytest.mark.parametrize("D,dtype", [(64, B16), (96, F16), (128, B16), (256, F16)])
def test_keys_and_values_of_different_strides(D, dtype):
    lens, keys = [5, 200, 1], [300, 200, 4100]
    q, k, v = packed(lens, keys, 6, 2, D, dtype, D)
    kk, vv = apart(k, 8), apart(v, 200)
    assert kk.stride(0) != vv.stride(0)
    lse = torch.empty(sum(lens), 6, device=DEV)
    out = ops.attention_prefill(q, kk, vv, offsets(lens), cu_k=offsets(keys), lse=lse)
    check_prompts(out, lse, q, k, v, lens, keys, D ** -0.5)
    kp, vp, table = on_pages(k, v, keys, 16, 7)
    kp, vp = apart(kp, 40), apart(vp, 8)
    assert kp.stride(0) != vp.stride(0)
    out = ops.attention_prefill(q, kp, vp, offsets(lens), cu_k=offsets(keys), table=table, lse=lse)
    check_prompts(out, lse, q, k, v, lens, keys, D ** -0.5)


@pytest.mark.parametrize("D,dtype", [(64, F16), (96, B16), (128, F16), (256, B16)])
@pytest.mark.parametrize("T", [1, 2, 20])
def test_steps_on_pools_of_different_strides(D, dtype, T):
    lens = [T, 700, 33]
    q, k, v, kp, vp, table, front = decode_inputs(lens, 130, T, 4, 2, D, dtype, 16, T)
    kp, vp = apart(kp, 264), apart(vp, 16)
    lse = torch.empty(len(lens) * T, 4, device=DEV)
    out = ops.attention_decode(q, kp, vp, table, torch.tensor(lens, dtype=torch.int32, device=DEV), batch=len(lens), tokens_per_seq=T, max_len=700,
                               prefix_table=front, prefix_len=130, lse=lse)
    check_steps(out, lse, q, k, v, lens, 130, T, D ** -0.5)


@pytest.mark.parametrize("D,dtype", [(64, B16), (96, F16), (128, F16), (256, B16)])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_queries_that_are_not_finite_keep_it_to_themselves(D, dtype, bad):
    """Rows 3 (one element, of head 1) and 41 (every element) of 70; steps of the same rows behind many keys."""
    T, n, Hq, Hkv = 70, 500, 4, 2
    q, k, v = packed([T], [n], Hq, Hkv, D, dtype, D)
    clean = q.clone()
    q[3, 1, D // 3] = bad
    q[41] = bad
    want = attention64(clean, k, v, causal(T, n, DEV), D ** -0.5)
    mine = torch.zeros(T, Hq, dtype=torch.bool, device=DEV)
    mine[3, 1] = mine[41] = True

    def check(out, lse, rows):
        keep = ~mine[rows][..., None]
        near(torch.where(keep, out.double(), 0), torch.where(keep, want[0][rows], 0), want[2][rows])
        near(torch.where(keep[..., 0], lse.double(), 0), torch.where(keep[..., 0], want[1][rows], 0), want[3][rows])
        # scores of both infinities, of NaN, or of -inf alone (no key): the last's are 0
        got = out[mine[rows]]
        assert (~torch.isfinite(got)).all() if bad != bad else ((~torch.isfinite(got)) | (got == 0)).all()

    lse = torch.empty(T, Hq, device=DEV)
    out = ops.attention_prefill(q, k, v, offsets([T]), cu_k=offsets([n]), lse=lse)
    check(out, lse, slice(0, T))
    kp, vp, table = on_pages(k, v, [n], 16, 3)
    for rows in (slice(40, 44), slice(0, T)):
        m = rows.stop - rows.start
        lse = torch.empty(m, Hq, device=DEV)
        lens = torch.tensor([n - T + rows.stop], dtype=torch.int32, device=DEV)
        out = ops.attention_decode(q[rows], kp, vp, table, lens, batch=1, tokens_per_seq=m, max_len=n, lse=lse)
        check(out, lse, rows)


def test_rows_of_queries_and_outputs_past_32_bits():
    """Rows 2^24 - 8 elements apart: the last ones' offsets pass 2^32 elements."""
    lens, Hq, Hkv, D, far = [290], 2, 1, 64, (1 << 24) - 8
    q, k, v = packed(lens, lens, Hq, Hkv, D, B16, 4)
    buf = torch.empty(lens[0] * far, dtype=B16, device=DEV)
    rows, out = (buf.as_strided((lens[0], Hq, D), (far, D, 1), at) for at in (0, far // 16 * 8))
    rows.copy_(q)
    ops.attention_prefill(rows, k, v, offsets(lens), out=out)
    check_prompts(out, None, q, k, v, lens, lens, D ** -0.5)
    kp, vp, table = on_pages(k, v, lens, 16, 6)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out.zero_()
    ops.attention_decode(rows, kp, vp, table, n, batch=1, tokens_per_seq=lens[0], max_len=lens[0], out=out)
    check_prompts(out, None, q, k, v, lens, lens, D ** -0.5)
    # one query of each of as many sequences, on the same pages
    ops.attention_decode(rows, kp, vp, table.expand(lens[0], -1).contiguous(), n.expand(lens[0]).contiguous(), batch=lens[0], max_len=lens[0], out=out)
    want = attention64(q, k, v, torch.ones(lens[0], lens[0], dtype=torch.bool, device=DEV), D ** -0.5)
    near(out, want[0], want[2])


@pytest.mark.parametrize("D,dtype", [(64, B16), (96, F16), (128, B16), (256, F16)])
@pytest.mark.parametrize("lens,past", [([2048], [10000]), ([150] * 8, [0, 1000, 3000, 500, 12000, 8, 4000, 70]), ([300] * 4, [6000] * 4)],
                         ids=["one", "mixed", "alike"])
def test_blocks_for_every_cu_behind_cached_keys(D, dtype, lens, past):
    """256 to 512 blocks of rows, whose keys are cut where the longest are far longer than the average, and not where they are alike."""
    keys = [a + b for a, b in zip(lens, past)]
    Hq, Hkv = (16, 2) if len(lens) == 1 else (32, 2)
    q, k, v = packed(lens, keys, Hq, Hkv, D, dtype, D)
    lse = torch.empty(sum(lens), Hq, device=DEV)
    kp, vp, table = on_pages(k, v, keys, 64, 5)
    for paged in (False, True):
        out = ops.attention_prefill(q, kp if paged else k, vp if paged else v, offsets(lens), cu_k=offsets(keys), lse=lse,
                                    table=table if paged else None)
        check_prompts(out, lse, q, k, v, lens, keys, D ** -0.5)


@pytest.mark.parametrize("D,dtype", [(64, F16), (128, B16), (256, B16)])
def test_a_prefix_behind_blocks_for_every_cu(D, dtype):
    prefix, B = 7000, 1200
    q, k, v, kp, vp, table, front = decode_inputs([3], prefix, 1, 32, 8, D, dtype, 64, D)
    q = torch.randn(B, 32, D, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
    lse = torch.empty(B, 32, device=DEV)
    out = ops.attention_decode(q, kp, vp, table.expand(B, -1).contiguous(), torch.full((B,), 3, dtype=torch.int32, device=DEV), batch=B, max_len=3,
                               prefix_table=front, prefix_len=prefix, lse=lse)
    want = attention64(q, k, v, torch.ones(B, prefix + 3, dtype=torch.bool, device=DEV), D ** -0.5)
    near(out, want[0], want[2])
    near(lse, want[1], want[3])
