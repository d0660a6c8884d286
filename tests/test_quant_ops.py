"""The residual RMS norm with 8-bit output (gdn_add_rms_norm) and the int8 product with row scales
(gdn_quant_matmul): refusals on the CPU, values on the GPU against 64 bits, and a layer made of them.

Tolerances, u = 2^-24. The norm's sum of n squares is formed in f32 from h (one rounding, u |h| at most;
relative 2 u of a square) in lanes, a tree and at most ceil(n / 64) terms in a row per lane: its relative
error is below (n / 64 + 12) u, half of that in its root; 1 / sqrt, the products with h and the weight add
8 u. So y is off by at most e = (n / 128 + 16) u relative, plus (where x and residual cancel) u (|x| + |r|)
times |y / h|. An 8-bit value is off by at most half a step, and half a step more where y 127 / max |y| lies
within 254 e of a half: so |q s - y| <= s (1/2 + 254 e), and q equals the nearest integer away from halves.
The product's integer sums are exact: three f32 roundings (the sum's conversion, two products), 3 u, then the
output's own.
"""
import ctypes

import pytest
import torch

from gated_deltanet_linear_step_amd import ops

U = 2.0 ** -24
DEV = "cuda:0"
OK, NULL, SHAPE, UNSUPPORTED, OVERFLOW, ALIGN = 0, 1, 2, 3, 4, 5
_BUF = (ctypes.c_float * 4096)()
P = (ctypes.addressof(_BUF) + 255) // 256 * 256  # never dereferenced: validation fails first


def vp(x):
    return ctypes.c_void_p(x) if x else None


# ---- refusals (CPU) ------------------------------------------------------------

def norm(**kw):
    given = dict(rows=2, hidden=64, dtype=ops.BF16, x=vp(P), x_stride=64, residual=vp(P), residual_stride=64,
                 residual_out=vp(P), residual_out_stride=64, weight=vp(P), eps=0.0, out_dtype=ops.BF16, out=vp(P),
                 out_stride=64, out_q=vp(P), out_q_stride=64, out_scale=vp(P))
    given.update(kw)
    args = ops.NormArgs(**given)
    return ops.load().gdn_add_rms_norm(ctypes.byref(args), None)


@pytest.mark.parametrize("want,kw", [
    (SHAPE, dict(rows=-1)), (SHAPE, dict(hidden=0)), (SHAPE, dict(x_stride=63)), (SHAPE, dict(residual_stride=3)),
    (SHAPE, dict(residual_out_stride=3)), (SHAPE, dict(out_stride=3)), (SHAPE, dict(out_q_stride=63)),
    (SHAPE, dict(eps=-1.0)), (SHAPE, dict(eps=float("nan"))), (UNSUPPORTED, dict(dtype=3)),
    (UNSUPPORTED, dict(out_dtype=-1)), (NULL, dict(x=None)), (NULL, dict(weight=None)),
    (NULL, dict(out=None, out_q=None, out_scale=None)), (NULL, dict(out_scale=None)), (NULL, dict(out_q=None)),
    (ALIGN, dict(x=vp(P + 1))), (ALIGN, dict(residual=vp(P + 1))), (ALIGN, dict(weight=vp(P + 2))),
    (ALIGN, dict(out=vp(P + 1))), (ALIGN, dict(out_scale=vp(P + 2))), (ALIGN, dict(dtype=ops.F32, x=vp(P + 2))),
    (OVERFLOW, dict(hidden=2 ** 24 + 1)), (OVERFLOW, dict(hidden=2 ** 31 - 1, rows=0)),
    (OK, dict(rows=0)), (OK, dict(rows=0, x=None, weight=None)),
])
def test_norm_refusals(want, kw):
    assert norm(**kw) == want


def test_norm_null_args():
    assert ops.load().gdn_add_rms_norm(None, None) == NULL


def matmul(M=4, N=4, K=64, a=P, a_stride=64, a_scale=P, w=P, w_stride=64, w_scale=P, out_dtype=ops.BF16, out=P, out_stride=4):
    return ops.load().gdn_quant_matmul(M, N, K, vp(a), a_stride, vp(a_scale), vp(w), w_stride, vp(w_scale), out_dtype,
                                       vp(out), out_stride, None)


@pytest.mark.parametrize("want,kw", [
    (SHAPE, dict(M=-1)), (SHAPE, dict(N=-1)), (SHAPE, dict(K=0)), (UNSUPPORTED, dict(K=40)), (UNSUPPORTED, dict(out_dtype=3)),
    (OVERFLOW, dict(K=131072, a_stride=131072, w_stride=131072)), (OVERFLOW, dict(M=2 ** 31 - 1, N=2 ** 31 - 1, out_stride=2 ** 31)),
    (OVERFLOW, dict(M=2 ** 31 - 1)), (OVERFLOW, dict(N=2 ** 31 - 1, out_stride=2 ** 31)),
    (OVERFLOW, dict(M=2 ** 31 - 256, N=257, out_stride=257)), (OVERFLOW, dict(M=2 ** 20, N=2 ** 20, out_stride=2 ** 20)),
    (NULL, dict(M=2 ** 31 - 256, N=256, out_stride=256, out=0)), (NULL, dict(M=1, N=2 ** 31 - 256, out_stride=2 ** 31, out=0)),
    (OVERFLOW, dict(a_stride=2 ** 23)), (OVERFLOW, dict(w_stride=2 ** 23)),
    (NULL, dict(a=0)), (NULL, dict(w=0)), (NULL, dict(out=0)), (NULL, dict(a_scale=0)), (NULL, dict(w_scale=0)),
    (SHAPE, dict(a_stride=48)), (SHAPE, dict(w_stride=48)), (SHAPE, dict(out_stride=3)),
    (ALIGN, dict(a=P + 8)), (ALIGN, dict(w=P + 4)), (ALIGN, dict(a_stride=72)), (ALIGN, dict(w_stride=88)),
    (ALIGN, dict(a_scale=P + 2)), (ALIGN, dict(w_scale=P + 1)), (ALIGN, dict(out=P + 1)),
    (OK, dict(M=0)), (OK, dict(N=0, w=0, out=0, out_stride=0)),
])
def test_matmul_refusals(want, kw):
    assert matmul(**kw) == want


# ---- the norm ------------------------------------------------------------------

def norm_reference(x, r, w, eps):
    x = x.cpu().double()
    h = x + (r.cpu().double() if r is not None else 0)
    y = h / (h.square().mean(1, keepdim=True) + eps).sqrt() * w.cpu().double()
    cancel = U * (x.abs() + (r.cpu().double().abs() if r is not None else 0))
    return h, y, cancel


def check_norm(got, x, r, w, eps=1e-6):
    h, y, cancel = norm_reference(x, r, w, eps)
    n = x.shape[1]
    e = (n / 128 + 16) * U
    slope = (w.cpu().double() / (h.square().mean(1, keepdim=True) + eps).sqrt()).abs()
    room = e * y.abs() + (cancel + U * h.abs()) * slope
    half = lambda t: torch.finfo(t.dtype).eps / 2  # noqa: E731
    tiny = lambda t: torch.finfo(t.dtype).smallest_normal * torch.finfo(t.dtype).eps  # noqa: E731
    if "out" in got:
        o = got["out"]
        assert ((o.cpu().double() - y).abs() <= room + half(o) * (y.abs() + room) + tiny(o)).all()
    if "residual" in got:
        o = got["residual"]
        assert ((o.cpu().double() - h).abs() <= cancel + half(o) * (h.abs() + cancel) + tiny(o)).all()
    if "out_q" in got:
        top = y.abs().amax(1)
        s = got["out_scale"].cpu().double()
        assert ((s - top / 127).abs() <= top / 127 * (e + 2 * U) + (cancel * slope).amax(1) / 127).all()
        q = got["out_q"].cpu().double()
        assert q.abs().max() <= 127
        exact = y * 127 / top[:, None]
        near = 254 * (e + 4 * U) + ((cancel + U * h.abs()) * slope).amax(1, keepdim=True) * 254 / top[:, None]
        assert ((q - exact).abs() <= 0.5 + near).all()


def norm_inputs(rows, hidden, dtype, seed, stride=None):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, stride or hidden, generator=gen).to(dtype).to(DEV)[:, :hidden]
    r = torch.randn(rows, stride or hidden, generator=gen).to(dtype).to(DEV)[:, :hidden]
    w = (1 + 0.2 * torch.randn(hidden, generator=gen)).to(DEV)
    return x, r, w


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,hidden", [(1, 1), (3, 7), (2, 64), (5, 513), (4, 1000), (2, 1024), (3, 2048), (2, 2056),
                                         (1300, 5), (600, 16400), (4200, 1000),
                                         (3000, 1500), (7, 4096), (2, 5003), (2, 8192), (2, 8200), (1, 16384), (2, 20001), (1, 40008)])
def test_norm_sizes(rows, hidden, dtype):
    x, r, w = norm_inputs(rows, hidden, dtype, rows + hidden)
    check_norm(ops.add_rms_norm(x, w, residual=r, quantize=True, out_dtype=dtype), x, r, w)
    check_norm(ops.add_rms_norm(x, w, quantize=True), x, None, w)
    check_norm(ops.add_rms_norm(x, w, residual=r), x, r, w)


@pytest.mark.gpu
@pytest.mark.parametrize("hidden,stride", [(256, 257), (250, 256), (2048, 2060), (2048, 2049)])
@pytest.mark.parametrize("dtype,out_dtype", [(torch.bfloat16, torch.float32), (torch.float32, torch.float16),
                                             (torch.float16, torch.bfloat16)])
def test_norm_strides_and_out_dtypes(hidden, stride, dtype, out_dtype):
    x, r, w = norm_inputs(6, hidden, dtype, hidden, stride)
    out = torch.full((7, stride), 9.0, dtype=out_dtype, device=DEV)
    q = torch.full((7, stride), 99, dtype=torch.int8, device=DEV)
    res = torch.full((7, stride), 9.0, dtype=dtype, device=DEV)
    scale = torch.full((8,), 9.0, device=DEV)
    ops.prepare_add_rms_norm(x, w, residual=r, residual_out=res[:6, :hidden], out=out[:6, :hidden], out_q=q[:6, :hidden],
                             out_scale=scale[:6], eps=1e-3).launch()
    check_norm(dict(out=out[:6, :hidden], residual=res[:6, :hidden], out_q=q[:6, :hidden], out_scale=scale[:6]), x, r, w, 1e-3)
    # the row ends and the rows behind the last one keep what they held
    for t, mark in ((out, 9.0), (q, 99), (res, 9.0)):
        assert (t[6] == mark).all() and (t[:, hidden:] == mark).all()
    assert (scale[6:] == 9.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("hidden", [96, 2048, 5003])
def test_norm_in_place(hidden):
    x, r, w = norm_inputs(9, hidden, torch.bfloat16, 3)
    x0, r0 = x.clone(), r.clone()
    got = ops.add_rms_norm(x, w, residual=r, residual_out=r, out=x, quantize=True)
    assert got["out"] is x and got["residual"] is r
    check_norm(got, x0, r0, w)
    x = x0.clone()
    got = ops.add_rms_norm(x, w, residual=r0, residual_out=x, quantize=True)
    check_norm(got, x0, r0, w)


@pytest.mark.gpu
@pytest.mark.parametrize("hidden", [40, 2048, 9001])
def test_norm_rows_of_zeros_and_rows_that_are_not_finite(hidden):
    x, r, w = norm_inputs(6, hidden, torch.float32, 8)
    r.zero_()
    x[0] = 0
    x[1, hidden // 2] = float("nan")
    x[2, hidden - 1] = float("inf")
    x[3] *= 1e-30  # y = x / sqrt(eps): far below 2^-100 only after the square root's 1e3
    x[4] *= 1e-36
    got = ops.add_rms_norm(x, w, residual=r, quantize=True, out_dtype=torch.float32)
    s, q = got["out_scale"].cpu(), got["out_q"].cpu()
    assert s[0] == 0 and (q[0] == 0).all() and (got["out"][0] == 0).all()
    assert torch.isnan(s[1]) and torch.isnan(s[2]) and (q[1:3] == 0).all()
    assert torch.isnan(got["out"][1]).any() and torch.isnan(got["out"][2]).any()
    assert s[4] == 0 and (q[4] == 0).all()
    keep = [3, 5]
    check_norm({n: t[keep] for n, t in got.items()}, x[keep], r[keep], w)


@pytest.mark.gpu
def test_norm_in_place_of_the_largest_numbers():
    # the squares' sum is infinite, so y is 0 -- also where a thread reads the row's last elements only after
    # their owner has stored h over the residual: x + h is infinite
    for hidden in (528, 2056, 2600):
        x = torch.full((700, hidden), 2e38, device=DEV)
        r = torch.zeros_like(x)
        got = ops.add_rms_norm(x, torch.ones(hidden, device=DEV), residual=r, residual_out=r, quantize=True,
                               out_dtype=torch.float32)
        assert (got["out"] == 0).all() and (got["out_q"] == 0).all() and (got["out_scale"] == 0).all()
        assert torch.equal(r, x)


# ---- the product ---------------------------------------------------------------

def matmul_inputs(M, N, K, seed, pad=0):
    gen = torch.Generator().manual_seed(seed)
    draw = lambda n: torch.randint(-128, 128, (n, K + pad), generator=gen, dtype=torch.int8).to(DEV)[:, :K]  # noqa: E731
    sa, sw = (torch.rand(n, generator=gen).add(0.5).mul(1e-2).to(DEV) for n in (M, N))
    return draw(M), sa, draw(N), sw


def check_matmul(out, a, sa, w, sw):
    exact = (a.cpu().double() @ w.cpu().double().t()) * sa.cpu().double()[:, None] * sw.cpu().double()
    fin = torch.finfo(out.dtype)
    room = 3.01 * U * exact.abs()
    off = (out.cpu().double() - exact).abs() - room - fin.eps / 2 * (exact.abs() + room) - fin.smallest_normal * fin.eps
    assert (off <= 0).all(), f"over the bound by {off.max():.3e}"


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 16), (1, 17, 48), (2, 64, 64), (15, 33, 80), (16, 16, 128), (17, 100, 2048), (31, 130, 272), (32, 256, 1040),
    (33, 48, 512), (64, 512, 2048), (65, 64, 96), (100, 2050, 160), (128, 128, 4112), (130, 257, 1024), (255, 300, 64),
    (256, 256, 256), (257, 513, 400), (300, 1000, 2064), (700, 129, 144), (1025, 520, 128),
])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_matmul_sizes(M, N, K, out_dtype):
    a, sa, w, sw = matmul_inputs(M, N, K, M + N + K)
    check_matmul(ops.quant_matmul(a, sa, w, sw, out_dtype=out_dtype), a, sa, w, sw)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(3, 40, 64), (60, 200, 320), (300, 384, 512)])
def test_matmul_strides_leave_the_rest_alone(M, N, K):
    a, sa, w, sw = matmul_inputs(M, N, K, 7, pad=32)
    out = torch.full((M + 1, N + 3), 9.0, dtype=torch.float16, device=DEV)
    ops.prepare_quant_matmul(a, sa, w, sw, out[:M, :N]).launch()
    check_matmul(out[:M, :N], a, sa, w, sw)
    assert (out[M] == 9.0).all() and (out[:, N:] == 9.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 40, 300])
def test_matmul_extremes(M):
    """Sums at the ends of the range, zero and NaN scales."""
    N, K = 70, 8192
    a = torch.full((M, K), -128, dtype=torch.int8, device=DEV)
    w = torch.full((N, K), -128, dtype=torch.int8, device=DEV)
    w[1::2] = 127
    sa, sw = torch.ones(M, device=DEV), torch.ones(N, device=DEV)
    out = ops.quant_matmul(a, sa, w, sw, out_dtype=torch.float32)
    assert (out[:, 0::2] == 2.0 ** 27).all() and (out[:, 1::2] == -128.0 * 127 * K).all()
    sa[M - 1], sw[3], sw[4] = 0.0, float("nan"), 0.0
    out = ops.quant_matmul(a, sa, w, sw, out_dtype=torch.float32)
    assert torch.isnan(out[:, 3]).all() and (out[:, 4] == 0).all()
    keep = [n for n in range(N) if n != 3]
    assert torch.isfinite(out[:, keep]).all() and (out[M - 1, keep] == 0).all()


@pytest.mark.gpu
def test_matmul_binding_refusals():
    a, sa, w, sw = matmul_inputs(4, 8, 64, 1)
    with pytest.raises(ValueError):
        ops.quant_matmul(a[:, :48], sa, w, sw)
    with pytest.raises(ValueError):
        ops.quant_matmul(a, sa[:3], w, sw)
    with pytest.raises(ValueError):
        ops.quant_matmul(a, sa.cpu(), w, sw)
    with pytest.raises(TypeError):
        ops.quant_matmul(a.float(), sa, w, sw)
    with pytest.raises(ops.GdnError):
        ops.quant_matmul(a[:, 8:56], sa, w[:, 8:56], sw)  # not 16-byte aligned
    assert ops.quant_matmul(a[:0], sa[:0], w, sw).shape == (0, 8)
    x = torch.zeros(0, 64, device=DEV)
    assert ops.add_rms_norm(x, torch.ones(64, device=DEV), quantize=True)["out_q"].shape == (0, 64)
    with pytest.raises(ValueError):
        ops.add_rms_norm(x, torch.ones(63, device=DEV))
    # counts past 32 bits are not cut off
    many = x.new_zeros(1, 64).expand(2 ** 32 + 5, 64)
    with pytest.raises(ValueError, match="32 bits"):
        ops.prepare_add_rms_norm(many, torch.ones(64, device=DEV), out=many)
    with pytest.raises(ValueError, match="32 bits"):
        ops.prepare_quant_matmul(a[:1].expand(2 ** 32 + 5, 64), sa, w, sw, torch.empty(4, 8, device=DEV))


# ---- a layer of them -----------------------------------------------------------

def quantized_weight(n, k, gen):
    w = torch.randn(n, k, generator=gen) * k ** -0.5
    s = w.abs().amax(1) / 127
    return (w / s[:, None]).round().to(torch.int8).to(DEV), s.to(DEV)


@pytest.mark.gpu
@pytest.mark.parametrize("rule", ["decay", "delta"])
def test_layer_of_them(rule):
    """norm -> int8 projection -> conv -> linear attention (or the gated delta layer) -> norm -> int8 projection ->
    residual norm, for a packed prompt and then one decode step, eagerly and as a replayed graph. Each
    product is checked against 64 bits on its own inputs; the graph against the eager run, bit for bit."""
    Hk, Hv, d, hidden, lens = 2, 4, 64, 320, [70, 9]
    C, n, B = 2 * Hk * d + Hv * d, 79, 2
    gen = torch.Generator().manual_seed(12)
    rand = lambda *s: torch.randn(*s, generator=gen).to(DEV)  # noqa: E731
    w1, w2 = (1 + 0.1 * rand(hidden)), (1 + 0.1 * rand(Hv * d))
    win, win_s = quantized_weight(C, hidden, gen)
    wout, wout_s = quantized_weight(hidden, Hv * d, gen)
    conv_w = (rand(C, 4) * 0.5).bfloat16()
    rate = torch.linspace(-1, -0.05, Hv, device=DEV)
    heads = dict(Hk=Hk, Hv=Hv, dk=d, dv=d, head_map=ops.MAP_GROUPED)
    cu = torch.tensor([0, 70, 79], dtype=torch.int32)
    cud = cu.to(DEV)

    def layer(x, res, conv_state, state, batch):
        normed = ops.add_rms_norm(x, w1, residual=res, quantize=True)
        mixed = ops.quant_matmul(normed["out_q"], normed["out_scale"], win, win_s, out_dtype=torch.bfloat16)
        y = ops.conv_update(mixed, conv_w, conv_state, cu_seqlens=None if batch else cud, num_seqs=B,
                            y_dtype=torch.bfloat16)
        q, k, v = y[:, :Hk * d], y[:, Hk * d:2 * Hk * d], y[:, 2 * Hk * d:]
        T = len(x)
        if rule == "delta":
            g = dict(g=rate.expand(T, Hv).contiguous(), beta=torch.full((T, Hv), 0.5, device=DEV))
            o = ops.decode_step(q, k, v, state, batch=B, out_dtype=torch.bfloat16, **g, **heads) if batch else \
                ops.prefill_chunked(q, k, v, state, cud, cu_seqlens_host=cu, out_dtype=torch.bfloat16, **g, **heads)
        else:
            g = dict(decay_param=rate, decay=ops.DECAY_NEGATIVE_RATE)
            o = ops.linattn_decode_step(q, k, v, state, batch=B, out_dtype=torch.bfloat16, **g, **heads) if batch else \
                ops.linattn_prefill_chunked(q, k, v, state, cud, cu_seqlens_host=cu, out_dtype=torch.bfloat16, **g, **heads)
        inner = ops.add_rms_norm(o.view(T, Hv * d), w2, quantize=True)
        back = ops.quant_matmul(inner["out_q"], inner["out_scale"], wout, wout_s, out_dtype=torch.bfloat16)
        check = ((normed, x, res, w1), (inner, o.view(T, Hv * d), None, w2)), \
            ((mixed, normed, win, win_s), (back, inner, wout, wout_s))
        return back, normed["residual"], check

    x, res = rand(n, hidden).bfloat16(), rand(n, hidden).bfloat16()
    x1, res1 = rand(B, hidden).bfloat16(), rand(B, hidden).bfloat16()
    conv_state, state = torch.zeros(B, C, 3, dtype=torch.bfloat16, device=DEV), torch.zeros(B, Hv, d, d, device=DEV)
    for args, batch in (((x, res), 0), ((x1, res1), B)):
        back, h, (norms, products) = layer(*args, conv_state, state, batch)
        for got, a, b, w in norms:
            check_norm(got, a, b, w)
        for out, q8, w, s in products:
            check_matmul(out, q8["out_q"], q8["out_scale"], w, s)
        last = back
    if rule == "delta":
        return
    # the decode step as a graph: three replays, each against an eager run from the same states
    c0, s0 = conv_state.clone(), state.clone()
    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):
        layer(x1, res1, conv_state, state, B)
    torch.cuda.synchronize()
    conv_state.copy_(c0)
    state.copy_(s0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured, captured_h, _ = layer(x1, res1, conv_state, state, B)
    ce, se = c0.clone(), s0.clone()
    conv_state.copy_(c0)
    state.copy_(s0)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        eager, eager_h, _ = layer(x1, res1, ce, se, B)
        torch.cuda.synchronize()
        assert torch.equal(captured, eager) and torch.equal(captured_h, eager_h)
        assert torch.equal(state, se) and torch.equal(conv_state, ce)
    assert torch.isfinite(last.float()).all()
