"""Host-only checks of the attention layer's entry points: bad arguments are refused with the documented status before
any HIP call. The pointers are host addresses that the library never dereferences on these paths."""
import ctypes

import pytest
import torch

from gated_deltanet_linear_step_amd import ops

OK, NULL, SHAPE, UNSUPPORTED, OVERFLOW, ALIGN, WORKSPACE = range(7)
_BUF = (ctypes.c_char * 8192)()
A = (ctypes.addressof(_BUF) + 255) // 256 * 256


def vp(x):
    return ctypes.c_void_p(x)


def rope(**kw):
    a = ops.RopeArgs(tokens=3, q_heads=2, kv_heads=1, head_dim=64, rotary_dim=64, layout=0, dtype=ops.BF16, magnitude=1.0,
                     positions=vp(A), inv_freq=vp(A), q=vp(A), q_stride=128, q_out=vp(A), q_out_stride=128, k=vp(A), k_stride=64,
                     k_out=vp(A), k_out_stride=64)
    for n, x in kw.items():
        setattr(a, n, x)
    return ops.load().gdn_rope(ctypes.byref(a), None)


PAGED = dict(k_out=None, v=A, v_stride=64, k_pages=A, v_pages=A, page_stride=16 * 64, num_pages=2, page_size=16, slots=A)


def test_rope_refusals():
    assert ops.load().gdn_rope(None, None) == NULL
    assert rope(tokens=0, q=None, positions=None) == OK
    assert rope(tokens=-1) == SHAPE and rope(magnitude=float("inf")) == SHAPE
    for bad in (dict(dtype=3), dict(layout=2), dict(head_dim=1), dict(head_dim=1025), dict(rotary_dim=0), dict(rotary_dim=66),
                dict(rotary_dim=7)):
        assert rope(**bad) == UNSUPPORTED, bad
    for bad in (dict(positions=None), dict(inv_freq=None), dict(q_out=None), dict(k_out=None), dict(q=None, q_out=None, k=None, k_out=None)):
        assert rope(**bad) == NULL, bad
    for bad in (dict(q_stride=127), dict(q_out_stride=127), dict(k_stride=63), dict(k_out_stride=63), dict(v=A), dict(q_heads=0), dict(kv_heads=0)):
        assert rope(**bad) == SHAPE, bad
    for bad in (dict(positions=A + 2), dict(inv_freq=A + 4), dict(q=A + 1), dict(k=A + 1), dict(q_out=A + 1), dict(k_out=A + 1)):
        assert rope(**bad) == ALIGN, bad
    assert rope(q_heads=1 << 19) == OVERFLOW and rope(tokens=1 << 24) == OVERFLOW
    for bad in (dict(v=None), dict(slots=None), dict(k_pages=None), dict(v_pages=None), dict(k=None)):
        assert rope(**{**PAGED, **bad}) == NULL, bad
    for bad in (dict(page_stride=1023), dict(num_pages=-1), dict(v_stride=63), dict(k_out=A)):
        assert rope(**{**PAGED, **bad}) == SHAPE, bad
    for bad in (0, 8, 24, 2048, -16):
        assert rope(**{**PAGED, **dict(page_size=bad)}) == UNSUPPORTED, bad
    assert rope(**{**PAGED, **dict(num_pages=1 << 27)}) == OVERFLOW
    assert rope(**{**PAGED, **dict(slots=A + 1)}) == ALIGN and rope(**{**PAGED, **dict(v_pages=A + 1)}) == ALIGN


def attention(**kw):
    a = ops.AttentionArgs(q_heads=4, kv_heads=2, head_dim=64, dtype=ops.BF16, scale=0.0, q=vp(A), q_stride=256, out=vp(A),
                          out_stride=256, k=vp(A), v=vp(A), k_stride=128, v_stride=128)
    for n, x in kw.items():
        setattr(a, n, x)
    return a


def cu(*at):
    return (ctypes.c_int32 * len(at))(*at)


def prefill(n=2, cq=(0, 5, 9), ck=None, ws=A, ws_bytes=1 << 40, dev=A, kdev=A, **kw):
    return ops.load().gdn_attention_prefill(ctypes.byref(attention(**kw)), n, cu(*cq) if cq else None, vp(dev), cu(*ck) if ck else None,
                                            vp(kdev) if ck else None, vp(ws), ws_bytes, None)


def test_prefill_refusals():
    assert ops.load().gdn_attention_prefill(None, 1, cu(0, 1), vp(A), None, None, None, 0, None) == NULL
    assert prefill(n=-1) == SHAPE and prefill(cq=None) == NULL and prefill(dev=None) == NULL and prefill(ck=(0, 5, 9), kdev=None) == NULL
    assert prefill(cq=(0, 0, 0)) == OK and prefill(cq=(0, 0, 0), out=None, ws=None) == OK and prefill(n=0, cq=(0,)) == OK
    for bad in ((1, 5, 9), (0, 5, 3), (0, -1, 9)):
        assert prefill(cq=bad) == SHAPE, bad
        assert prefill(ck=bad) == SHAPE, bad
    for bad in (dict(q_heads=3), dict(kv_heads=0), dict(q_heads=0), dict(scale=-1.0), dict(scale=float("nan")), dict(q_stride=255),
                dict(out_stride=255), dict(k_stride=127), dict(v_stride=127), dict(page_size=-16), dict(num_pages=-1)):
        assert prefill(**bad) == SHAPE, bad
    for bad in (dict(head_dim=32), dict(head_dim=65), dict(head_dim=512), dict(dtype=ops.F32), dict(dtype=9), dict(page_size=8),
                dict(page_size=48), dict(page_size=2048)):
        assert prefill(**bad) == UNSUPPORTED, bad
    for bad in (dict(q=None), dict(out=None), dict(k=None), dict(v=None)):
        assert prefill(**bad) == NULL, bad
    for bad in (dict(out=A + 8), dict(k=A + 2), dict(v=A + 8), dict(out_stride=260), dict(k_stride=132), dict(v_stride=130),
                dict(q_stride=257), dict(lse=A + 2), dict(table=A + 1)):
        assert prefill(**bad) == ALIGN, bad
    big = 1 << 24
    for bad in (dict(q_stride=big), dict(out_stride=big), dict(k_stride=big), dict(v_stride=big)):
        assert prefill(**bad) == OVERFLOW, bad
    assert prefill(n=1, cq=(0, 1 << 29)) == OVERFLOW                      # rows times heads
    need = ops.attention_prefill_workspace_bytes(Hq=4, Hkv=2, head_dim=64, num_seqs=2, total_tokens=9)
    assert need > 0
    assert prefill(ws=None) == WORKSPACE and prefill(ws_bytes=need - 1) == WORKSPACE and prefill(ws=A + 16) == ALIGN
    paged = dict(page_size=16, num_pages=3, table=A, table_stride=1, k_stride=2048, v_stride=2048)
    assert prefill(**{**paged, **dict(k_stride=2047)}) == SHAPE
    assert prefill(**{**paged, **dict(table=None)}) == NULL
    assert prefill(**{**paged, **dict(num_pages=0)}) == SHAPE
    assert prefill(ck=(0, 17, 20), **paged) == SHAPE                      # table rows of one page
    assert prefill(ck=(0, 17, 20), **{**paged, **dict(table_stride=-1)}) == SHAPE


def decode(batch=2, T=1, lens=A, max_len=20, prefix=None, prefix_len=0, ws=A, ws_bytes=1 << 40, **kw):
    a = attention(**{**dict(page_size=16, num_pages=3, table=A, table_stride=2, k_stride=2048, v_stride=2048), **kw})
    return ops.load().gdn_attention_decode(ctypes.byref(a), batch, T, vp(lens), max_len, vp(prefix), prefix_len, vp(ws), ws_bytes, None)


def test_decode_refusals():
    assert ops.load().gdn_attention_decode(None, 1, 1, vp(A), 1, None, 0, None, 0, None) == NULL
    assert decode(batch=0, lens=None, ws=None) == OK
    for bad in (dict(batch=-1), dict(T=0), dict(max_len=-1), dict(prefix_len=-1), dict(max_len=33), dict(num_pages=0), dict(q_heads=5),
                dict(prefix=A, prefix_len=5, max_len=0, num_pages=0)):
        assert decode(**bad) == SHAPE, bad
    assert decode(page_size=0) == UNSUPPORTED and decode(dtype=ops.F32) == UNSUPPORTED and decode(head_dim=80) == UNSUPPORTED
    for bad in (dict(lens=None), dict(table=None), dict(prefix_len=3), dict(k=None), dict(v=None), dict(out=None)):
        assert decode(**bad) == NULL, bad
    for bad in (dict(lens=A + 2), dict(prefix=A + 2, prefix_len=3), dict(v=A + 4), dict(ws=A + 128, prefix=A, prefix_len=16)):
        assert decode(**bad) == ALIGN, bad
    assert decode(batch=1 << 16, T=1 << 16) == OVERFLOW and decode(batch=1 << 28, T=4) == OVERFLOW
    need = ops.attention_decode_workspace_bytes(Hq=4, Hkv=2, head_dim=64, batch=2, max_len=20, prefix_len=16)
    assert need > 0
    assert decode(prefix=A, prefix_len=16, ws=None) == WORKSPACE
    assert decode(prefix=A, prefix_len=16, ws_bytes=need - 1) == WORKSPACE


def test_joins_past_a_launch_are_refused():
    """A join takes four rows a workgroup, or with more than 64 runs 32 outputs of one: 2^24 of those are too many threads."""
    few = dict(q_heads=64, q_stride=4096, out_stride=4096, table_stride=128, max_len=2048)
    assert decode(batch=1 << 20, **few) == OVERFLOW
    many = dict(q_heads=64, head_dim=256, q_stride=1 << 14, out_stride=1 << 14, k_stride=8192, v_stride=8192, table_stride=16640,
                max_len=16640 * 16)
    assert decode(batch=1 << 16, **many) == OVERFLOW


def test_workspace_queries_of_bad_counts():
    pre = dict(Hq=4, Hkv=2, head_dim=64, num_seqs=1, total_tokens=5)
    for bad in (dict(Hq=3), dict(Hkv=0), dict(head_dim=48), dict(num_seqs=-1), dict(total_tokens=0)):
        assert ops.attention_prefill_workspace_bytes(**{**pre, **bad}) == 0
    dec = dict(Hq=4, Hkv=2, head_dim=64, batch=1, tokens_per_seq=1, max_len=50000, prefix_len=0)
    assert ops.attention_decode_workspace_bytes(**dec) > 0
    for bad in (dict(Hq=3), dict(head_dim=48), dict(batch=0), dict(tokens_per_seq=0), dict(max_len=-1), dict(prefix_len=-1)):
        assert ops.attention_decode_workspace_bytes(**{**dec, **bad}) == 0
    assert ops.load().gdn_pages_workspace_bytes(-1) == 0 and ops.pages_workspace_bytes(0) > 0


def pages(**kw):
    a = ops.PageArgs(table=vp(A), table_stride=4, rows=2, width=4, refs=vp(A), num_pages=8, page_size=16, data=vp(A), num_planes=2,
                     plane_stride=8 * 64, page_stride=64, page_bytes=64)
    for n, x in kw.items():
        setattr(a, n, x)
    return ctypes.byref(a)


CALLS = {"free": lambda lib, a, n=2, x=A: lib.gdn_pages_free(a, n, vp(x), None, None),
         "reserve": lambda lib, a, n=2, x=A: lib.gdn_pages_reserve(a, n, vp(A), vp(x), vp(A), None),
         "fork": lambda lib, a, n=2, x=A, ws=A, size=1 << 30: lib.gdn_pages_fork(a, n, vp(A), vp(A), vp(A), vp(x), vp(ws), size, None),
         "compact": lambda lib, a, n=2, x=A, ws=A, size=1 << 30: lib.gdn_pages_compact(a, vp(A), vp(x), vp(ws), size, None)}


@pytest.mark.parametrize("name", CALLS)
def test_page_refusals(name):
    lib, call = ops.load(), CALLS[name]
    assert call(lib, None) == NULL
    for bad in (dict(rows=-1), dict(width=-1), dict(num_pages=-1), dict(table_stride=3)):
        assert call(lib, pages(**bad)) == SHAPE, bad
    for bad in (dict(table=None), dict(refs=None)):
        assert call(lib, pages(**bad)) == NULL, bad
    for bad in (dict(table=A + 2), dict(refs=A + 1)):
        assert call(lib, pages(**bad)) == ALIGN, bad
    assert call(lib, pages(), x=None) == NULL and call(lib, pages(), x=A + 2) == ALIGN
    if name != "compact":
        assert call(lib, pages(), n=-1) == SHAPE and call(lib, pages(), n=1025) == OVERFLOW and call(lib, pages(), n=0) == OK
    if name in ("reserve", "fork"):
        assert call(lib, pages(page_size=0)) == SHAPE
    if name in ("fork", "compact"):
        for bad in (dict(num_planes=-1), dict(page_bytes=-16), dict(page_stride=48), dict(plane_stride=-16)):
            assert call(lib, pages(**bad)) == SHAPE, bad
        for bad in (dict(data=A + 8), dict(page_bytes=56), dict(page_stride=72), dict(plane_stride=520)):
            assert call(lib, pages(**bad)) == ALIGN, bad
        assert call(lib, pages(data=None)) == NULL and call(lib, pages(page_bytes=1 << 31, page_stride=1 << 31)) == OVERFLOW
        assert call(lib, pages(), ws=None) == WORKSPACE and call(lib, pages(), ws=A + 64) == ALIGN
        assert call(lib, pages(), size=ops.pages_workspace_bytes(8) - 1) == WORKSPACE


def test_the_binding_refuses_what_it_cannot_marshal():
    cpu = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        ops.prepare_attention_prefill(cpu, cpu, cpu, cpu, cpu, cpu, None)
    with pytest.raises(ValueError, match="GPU"):
        ops.prepare_rope(torch.zeros(4, dtype=torch.int32), torch.zeros(2, dtype=torch.float64), q=cpu, q_out=cpu)
    with pytest.raises(ValueError, match="GPU"):
        ops.prepare_pages_free(torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


def test_sequences_of_more_than_2_30_keys_are_refused():
    far = (1 << 30) + 1
    paged = dict(page_size=1024, num_pages=3, table=A, table_stride=1 << 22, k_stride=1 << 20, v_stride=1 << 20)
    assert prefill(n=1, cq=(0, 5), ck=(0, far), **paged) == OVERFLOW
    assert decode(max_len=far, **paged) == OVERFLOW
    assert decode(max_len=5, prefix=A, prefix_len=far, **paged) == OVERFLOW


@pytest.mark.parametrize("name", CALLS)
def test_page_counts_past_their_walks_are_refused(name):
    """Pages and entries are walked with 32-bit indices: more than 2^30 pages, or entries in all rows, are refused."""
    most = 1 << 30
    call, lib = CALLS[name], ops.load()
    assert call(lib, pages(num_pages=most + 1)) == OVERFLOW
    assert call(lib, pages(rows=1 << 15, width=(1 << 15) + 1, table_stride=1 << 16)) == OVERFLOW
    assert call(lib, pages(rows=1, width=most + 1, table_stride=most + 1)) == OVERFLOW


def test_runs_of_more_keys_than_their_sums_resolve_are_refused():
    """2^21 keys of a prompt's sequence and of a prefix; a step's own keys are split, whatever their number."""
    most = 1 << 21
    paged = dict(page_size=1024, num_pages=3, table=A, table_stride=1 << 22, k_stride=1 << 20, v_stride=1 << 20, ws=None)
    assert prefill(n=1, cq=(0, 5), ck=(0, most), **paged) == WORKSPACE
    assert prefill(n=1, cq=(0, 5), ck=(0, most + 1), **paged) == OVERFLOW
    assert decode(max_len=5, prefix=A, prefix_len=most, **paged) == WORKSPACE
    assert decode(max_len=5, prefix=A, prefix_len=most + 1, **paged) == OVERFLOW
    assert decode(max_len=1 << 30, **paged) == WORKSPACE and decode(T=70, max_len=1 << 30, **paged) == WORKSPACE
