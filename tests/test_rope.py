"""Rotary positions against 64 bits. An output a c - b s is off by the f32 roundings of c and s and of what turns them: the
angle's rest of at most 1/8 turn is rounded once (2^-28 turn, pi 2^-27 rad), cosine and sine are a library's, 2 ulp (2^-22
of a value below 1), magnitude and the products add 2^-23 each; so (|a| + |b|) m (2^-21), and half a step of the type.
Frequencies: double precision against the same formula, 2^-46 of a value (pow and log, a few units each)."""
import math

import pytest
import torch

from gated_deltanet_linear_step_amd import ops

DEV = torch.device("cuda:0")
B16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAN = float("nan")


def turned(x, positions, w, m, layout):
    """(outputs, room) in 64 bits of x [tokens][heads][D]."""
    half = len(w)
    a, b = (x[..., :half], x[..., half:2 * half]) if layout == ops.ROPE_HALF else (x[..., :2 * half:2], x[..., 1:2 * half:2])
    a, b = a.double(), b.double()
    angle = positions.double()[:, None, None] * w
    c, s = m * angle.cos(), m * angle.sin()
    want, room = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    first, second = (slice(0, half), slice(half, 2 * half)) if layout == ops.ROPE_HALF else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    want[..., first], want[..., second] = a * c - b * s, b * c + a * s
    size = (a.abs() + b.abs()) * abs(m) * 2.0 ** -21
    u = torch.finfo(x.dtype).eps / 2
    for part in (first, second):
        room[..., part] = size + u * want[..., part].abs() + (2.0 ** -25 if x.dtype == F16 else 0)
    return want, room


def close(got, want, room):
    assert ((got.double() - want).abs() <= room).all(), ((got.double() - want).abs() - room).max().item()


def mixed(tokens, Hq, Hkv, D, dtype, seed, pad):
    gen = torch.Generator(DEV).manual_seed(seed)
    x = torch.randn(tokens, (Hq + 2 * Hkv) * D + pad, generator=gen, device=DEV).to(dtype)
    q, k, v = x[:, pad:].split([Hq * D, Hkv * D, Hkv * D], 1)
    return tuple(y.unflatten(1, (-1, D)) for y in (q, k, v))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [B16, F16, F32])
@pytest.mark.parametrize("layout", [ops.ROPE_HALF, ops.ROPE_INTERLEAVED])
@pytest.mark.parametrize("D,rot,pad", [(64, 64, 0), (128, 32, 0), (128, 128, 1), (96, 48, 8), (256, 64, 3), (80, 18, 0), (7, 2, 0), (7, 6, 5), (1024, 1024, 0)])
def test_turns(D, rot, pad, layout, dtype):
    tokens, Hq, Hkv = 37, 3, 2
    q, k, _ = mixed(tokens, Hq, Hkv, D, dtype, D + rot, pad)
    w, _ = ops.rope_frequencies(rot, 1e6)
    w = w.to(DEV)
    positions = torch.randint(0, 2 ** 20, (tokens,), device=DEV, dtype=torch.int32)
    positions[:6] = torch.tensor([0, 1, 2, 2 ** 31 - 1, 2 ** 30 + 1, 12345], device=DEV)
    # angles of 2^31 rad are exact to 2^-22 in 64 bits: beside the bound's own terms
    far = (positions > 2 ** 24)[:, None, None] * 2.0 ** -21
    got = ops.rope(positions, w, q=q, k=k, layout=layout, magnitude=1.25)
    for x, y in zip((q, k), got):
        want, room = turned(x, positions, w, 1.25, layout)
        close(y, want, room + far * 1.25 * x.double().abs().amax(-1, keepdim=True))
        assert torch.equal(y[..., rot:], x[..., rot:])
    # the same in place, one of the two alone
    qq, kk = q.clone(), k.clone()
    ops.prepare_rope(positions, w, q=qq, q_out=qq, layout=layout, magnitude=1.25).launch()
    ops.prepare_rope(positions, w, k=kk, k_out=kk, layout=layout, magnitude=1.25).launch()
    assert torch.equal(qq, got[0]) and torch.equal(kk, got[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [B16, F16, F32])
@pytest.mark.parametrize("layout", [ops.ROPE_HALF, ops.ROPE_INTERLEAVED])
@pytest.mark.parametrize("D,rot,ps,tokens", [(128, 128, 16, 300), (256, 64, 64, 65), (96, 96, 1024, 9), (50, 10, 16, 40), (64, 64, 32, 1)])
def test_keys_and_values_go_to_their_slots(D, rot, ps, tokens, layout, dtype):
    Hq, Hkv, pages = 4, 2, 30
    q, k, v = mixed(tokens, Hq, Hkv, D, dtype, ps, 0)
    w = ops.rope_frequencies(rot)[0].to(DEV)
    positions = torch.arange(tokens, device=DEV, dtype=torch.int32) * 7
    slots = torch.randperm(pages * ps, device=DEV)[:tokens].to(torch.int32)
    slots[tokens // 2] = [-1, pages * ps, 2 ** 31 - 1][tokens % 3] if tokens > 1 else slots[0]
    kp, vp = (torch.full((pages, Hkv, ps, D), 7.0, dtype=dtype, device=DEV) for _ in range(2))
    wide = torch.full((pages, Hkv * ps * D + 40), 7.0, dtype=dtype, device=DEV)
    spaced = wide[:, :Hkv * ps * D].view(pages, Hkv, ps, D)
    got = ops.rope(positions, w, q=q, k=k, v=v, k_pages=kp, v_pages=vp, slots=slots, layout=layout)
    rows = ops.rope(positions, w, q=q, k=k, layout=layout)
    assert torch.equal(got, rows[0])
    want_k, want_v = torch.full_like(kp, 7.0), torch.full_like(vp, 7.0)
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pages * ps:
            want_k[s // ps, :, s % ps], want_v[s // ps, :, s % ps] = rows[1][t], v[t]
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)
    # pages further apart, keys and values beside each other
    ops.rope(positions, w, k=k, v=v, k_pages=spaced, v_pages=torch.full_like(wide, 7.0)[:, :Hkv * ps * D].view(pages, Hkv, ps, D),
             slots=slots, layout=layout)
    assert torch.equal(spaced, want_k) and (wide[:, Hkv * ps * D:] == 7.0).all()


@pytest.mark.gpu
def test_copied_elements_keep_their_bits():
    """NaN with payloads, infinities and subnormals in what is not turned, and in values."""
    bits = torch.randint(-2 ** 15, 2 ** 15, (5, 1, 128), dtype=torch.int16, device=DEV)
    x = bits.view(B16)
    w = ops.rope_frequencies(32)[0].to(DEV)
    pos = torch.arange(5, device=DEV, dtype=torch.int32)
    q, k = ops.rope(pos, w, q=x, k=x)
    assert torch.equal(q.view(torch.int16)[..., 32:], bits[..., 32:])
    kp, vp = (torch.zeros(1, 1, 16, 128, dtype=B16, device=DEV) for _ in range(2))
    ops.rope(pos, w, k=x, v=x, k_pages=kp, v_pages=vp, slots=pos)
    assert torch.equal(vp.view(torch.int16)[0, 0, :5], bits[:, 0])
    assert torch.equal(kp.view(torch.int16)[0, 0, :5, 32:], bits[:, 0, 32:])


@pytest.mark.gpu
def test_no_tokens_and_captured_calls():
    w = ops.rope_frequencies(64)[0].to(DEV)
    empty = torch.zeros(0, 2, 64, device=DEV)
    assert ops.rope(torch.zeros(0, dtype=torch.int32, device=DEV), w, q=empty)[0].shape == (0, 2, 64)
    q, k, v = mixed(20, 4, 2, 64, B16, 1, 0)
    pos, slots = torch.arange(20, device=DEV, dtype=torch.int32), torch.arange(20, device=DEV, dtype=torch.int32)
    kp, vp = (torch.zeros(2, 2, 16, 64, dtype=B16, device=DEV) for _ in range(2))
    want = ops.rope(pos, w, q=q, k=k, v=v, k_pages=kp, v_pages=vp, slots=slots)
    want_k, want_v = kp.clone(), vp.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ops.rope(pos, w, q=q, k=k, v=v, k_pages=kp, v_pages=vp, slots=slots)
    for _ in range(3):
        kp.zero_(), vp.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(kp, want_k) and torch.equal(vp, want_v)


# ---- frequencies (host) -------------------------------------------------------------------------------

def check_w(got, want):
    assert len(got) == len(want) and all(abs(a - b) <= 2.0 ** -46 * b for a, b in zip(got.tolist(), want))


@pytest.mark.parametrize("r,theta", [(2, 10000.0), (64, 10000.0), (128, 1e6), (6, 2.5)])
def test_frequencies(r, theta):
    plain = [theta ** (-2 * i / r) for i in range(r // 2)]
    w, m = ops.rope_frequencies(r, theta)
    check_w(w, plain)
    assert m == 1.0
    w, m = ops.rope_frequencies(r, theta, scaling=ops.ROPE_LINEAR, factor=4.0)
    check_w(w, [x / 4 for x in plain])
    assert m == 1.0
    if r > 2:
        w, m = ops.rope_frequencies(r, theta, scaling=ops.ROPE_BASE, factor=8.0)
        check_w(w, [(theta * 8 ** (r / (r - 2))) ** (-2 * i / r) for i in range(r // 2)])
        assert m == 1.0 and abs(w[-1].item() * 8 / plain[-1] - 1) < 1e-12 and w[0] == 1
    for fast, slow, length in ((32.0, 1.0, 4096.0), (4.0, 4.0, 8192.0), (1e9, 1e-9, 100.0)):
        w, m = ops.rope_frequencies(r, theta, scaling=ops.ROPE_BANDS, factor=16.0, original_length=length, beta_fast=fast, beta_slow=slow)
        index = lambda n: r * math.log(length / (n * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        low, high = (min(max(x, 0), r - 1) for x in (math.floor(index(fast)), math.ceil(index(slow))))
        share = [min(max((i - low) / (high - low), 0), 1) if high > low else float(i > low) for i in range(r // 2)]
        check_w(w, [x * (1 - s) + x / 16 * s for x, s in zip(plain, share)])
        assert abs(m - (0.1 * math.log(16) + 1)) < 1e-6


@pytest.mark.parametrize("kw,status", [(dict(rotary_dim=0), 3), (dict(rotary_dim=7), 3), (dict(rotary_dim=1026), 3), (dict(scaling=4), 3),
                                       (dict(scaling=-1), 3), (dict(theta=1.0), 2), (dict(theta=NAN), 2), (dict(scaling=1, factor=0.5), 2),
                                       (dict(rotary_dim=2, scaling=2, factor=2.0), 3), (dict(scaling=3, factor=2.0), 2),
                                       (dict(scaling=3, factor=2.0, original_length=100.0, beta_fast=1.0, beta_slow=2.0), 2),
                                       (dict(scaling=3, factor=2.0, original_length=100.0, beta_slow=0.0), 2)])
def test_frequencies_refused(kw, status):
    with pytest.raises(ops.GdnError) as e:
        ops.rope_frequencies(**{**dict(rotary_dim=64), **kw})
    assert e.value.status == status
