"""Every kernel that gdn_quant_matmul and gdn_add_rms_norm choose between, at sizes that leave a remainder in every
direction: values against 64 bits with test_quant_ops' bounds, strides, the ends of the range, NaN scales, and rows past
one round of the norm's grid."""
import ctypes

import pytest
import torch

from gated_deltanet_linear_step_amd import ops
from test_quant_ops import DEV, check_matmul, check_norm, matmul_inputs, norm_inputs

OK, NULL, SHAPE, UNSUPPORTED, OVERFLOW = 0, 1, 2, 3, 4

# kernel (outputs a workgroup, its threads) and a size that the choice sends to it
KERNELS = {(16, 16, 512): (13, 1037), (16, 32, 512): (5, 8200), (32, 32, 256): (65, 129), (64, 32, 256): (100, 2050),
           (64, 64, 256): (1025, 520), (64, 128, 256): (1100, 1100), (128, 128, 256): (1601, 1500),
           (256, 256, 512): (3001, 3003)}
SIZES = pytest.mark.parametrize("M,N", KERNELS.values(), ids=["x".join(map(str, k[:2])) for k in KERNELS])


@pytest.mark.parametrize("kernel", KERNELS, ids=lambda k: "x".join(map(str, k[:2])))
def test_each_size_takes_the_kernel_it_is_here_for(kernel):
    (rows, cols, threads), (M, N) = kernel, KERNELS[kernel]
    info = ops.quant_matmul_launch_info(M, N, 400)
    assert (info["workgroups"], info["threads"]) == (-(-M // rows) * -(-N // cols), threads)


def test_launch_info_refuses_what_the_product_refuses():
    lib, info = ops.load(), ops.LaunchInfo()
    call = lambda *c: lib.gdn_quant_matmul_launch_info(*c, ctypes.byref(info))  # noqa: E731
    assert lib.gdn_quant_matmul_launch_info(4, 4, 64, None) == NULL
    assert call(-1, 4, 64) == call(4, -1, 64) == call(4, 4, 0) == SHAPE
    assert call(4, 4, 40) == UNSUPPORTED
    assert call(4, 4, 131072) == call(2 ** 31 - 1, 4, 64) == call(2 ** 20, 2 ** 20, 64) == OVERFLOW
    assert call(0, 4, 64) == OK and info.workgroups == 0
    # no launch of 2^32 threads, whatever the shape
    for M, N in ((1, 2 ** 31 - 256), (16, 2 ** 27 - 15), (2 ** 31 - 256, 256), (17, 2 ** 31 - 256), (300000, 1700000)):
        assert call(M, N, 64) == OK and info.workgroups * info.threads < 2 ** 32


@pytest.mark.gpu
@SIZES
@pytest.mark.parametrize("K", [16, 128, 272, 400, 656])
def test_product(M, N, K):
    """K of one to six stages, even and odd counts of them, with and without a last one that is not whole."""
    a, sa, w, sw = matmul_inputs(M, N, K, M + K)
    for out_dtype in (torch.bfloat16, torch.float16, torch.float32):
        check_matmul(ops.quant_matmul(a, sa, w, sw, out_dtype=out_dtype), a, sa, w, sw)


@pytest.mark.gpu
@SIZES
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_product_of_strided_rows_leaves_the_rest_alone(M, N, out_dtype):
    a, sa, w, sw = matmul_inputs(M, N, 208, 7, pad=48)
    out = torch.full((M + 1, N + 3), 9.0, dtype=out_dtype, device=DEV)
    ops.prepare_quant_matmul(a, sa, w, sw, out[:M, :N]).launch()
    check_matmul(out[:M, :N], a, sa, w, sw)
    assert (out[M] == 9.0).all() and (out[:, N:] == 9.0).all()


@pytest.mark.gpu
@SIZES
def test_product_at_the_ends_of_the_range(M, N):
    """The largest sums, and scales of zero and NaN in the first and the last row and column."""
    K = 8192
    a = torch.full((M, K), -128, dtype=torch.int8, device=DEV)
    w = torch.full((N, K), -128, dtype=torch.int8, device=DEV)
    w[1::2] = 127
    sa, sw = torch.ones(M, device=DEV), torch.ones(N, device=DEV)
    out = ops.quant_matmul(a, sa, w, sw, out_dtype=torch.float32)
    assert (out[:, 0::2] == 2.0 ** 27).all() and (out[:, 1::2] == -128.0 * 127 * K).all()
    sa[M - 1], sw[0], sw[N - 1], sw[4] = 0.0, float("nan"), float("nan"), 0.0
    out = ops.quant_matmul(a, sa, w, sw, out_dtype=torch.float32)
    assert torch.isnan(out[:, 0]).all() and torch.isnan(out[:, N - 1]).all() and (out[:, 4] == 0).all()
    assert torch.isfinite(out[:, 1:N - 1]).all() and (out[M - 1, 1:N - 1] == 0).all()
    assert (out[:M - 1, 1:4:2] == -128.0 * 127 * K).all()
    sa[0] = float("nan")
    out = ops.quant_matmul(a, sa, w, sw, out_dtype=torch.float32)
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1:, 1:N - 1]).all()


# ---- the norm: more rows than its grid has workgroups (at most 2048 threads a CU, 64 at least a workgroup) ------------

@pytest.mark.gpu
@pytest.mark.parametrize("rows,hidden", [(8200, 100), (8200, 500), (8200, 519), (4200, 1001), (2600, 2049), (2600, 2570),
                                         (2600, 4000), (1100, 5003), (1100, 8000), (520, 9001), (520, 16000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_rows_past_the_grid(rows, hidden, dtype):
    x, r, w = norm_inputs(rows, hidden, dtype, rows + hidden)
    got = ops.add_rms_norm(x, w, residual=r, quantize=True, out_dtype=dtype)
    check_norm(got, x, r, w)
    # in place, bit for bit the same
    x1, r1 = x.clone(), r.clone()
    placed = ops.add_rms_norm(x1, w, residual=r1, residual_out=r1, out=x1, quantize=True)
    assert placed["out"] is x1 and placed["residual"] is r1
    assert all(torch.equal(placed[n], got[n]) for n in got)
