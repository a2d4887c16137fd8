"""Edges of the serving operators: many tiles per cluster, scales and magnitudes far apart, ranges of rows that
overlap, calls at once from several threads, and calls without rows."""

import numpy as np
import pytest
import torch

from mxfp4_w4a4_post_block_b200 import batq as BQ
import serving_ref as R
from test_gpu_serving import BF, F32, ok, w4a16_case, w4a16_check, w4a16_run

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ W4A16

@pytest.mark.parametrize("S,N,M,out_dtype,fmt", [
    (16, 512, 37888, F32, "mxfp4"), (16, 1024, 37888, BF, "mxfp4"), (16, 2304, 24576, F32, "nvfp4"),
    (16, 2560, 24576, F32, "mxfp4"), (4, 2560, 37888, BF, "mxfp4"), (4, 4096, 24576, BF, "mxfp4"),
    (16, 4096, 24576, F32, "nvfp4")])
def test_w4a16_many_tiles_per_cluster(S, N, M, out_dtype, fmt):
    """Clusters of two to eight CTAs that exchange the sums of four tiles and more: two buffers in turn, whose sums
    must not be replaced before all of a CTA has read them.  (The values, and bit for bit at every repeat.)"""
    x, A, B, codes, lin, _ = w4a16_case(S, N, M, fmt, BF, False, S + N)
    first = w4a16_run(x, A, B, codes, lin, fmt, out_dtype)
    w4a16_check(first, x, A, B, codes, lin, fmt)
    w, s, xd = R.cuda(codes), R.cuda(R.tile_scales(lin)), x.cuda()
    out = torch.empty_like(first)
    wf = BQ.BATQ_W4_MXFP4 if fmt == "mxfp4" else BQ.BATQ_W4_NVFP4
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(100):
        out.fill_(7.0)
        BQ.batq_linear_w4a16(xd, None, None, w, s, M, out, w_format=wf)
        differ += (out != first).sum()
    assert int(differ) == 0
    ok()


@pytest.mark.parametrize("S", [1, 3])
@pytest.mark.parametrize("out_dtype", [F32, BF])
def test_w4a16_nvfp4_values_on_their_bound(S, out_dtype):
    """The block Hadamard transform of a block whose 32 terms all add up, on a power of two: 32 x 0.70710683 / (2 sqrt 8)
    rounds to 4, and its bound's fp32 products to just below 4, so that the value's exponent is the larger one."""
    N, M, rng = 128, 48, np.random.default_rng(31)
    H2 = np.array([[1, 1], [1, -1]])
    H4, H8 = np.kron(H2, H2), np.kron(np.kron(H2, H2), H2)
    A = (H8 / np.sqrt(8)).astype(np.float32)
    B = np.repeat((H4 / 2).astype(np.float32)[None], N // 32, 0)
    codes, lin = R.random_weights(rng, M, N, "nvfp4")
    x = (rng.standard_normal((S, N)) * 0.01).astype(np.float32)
    x[:, 32:64] = np.kron(H4[:, 1], H8[:, 7]) * np.float32(0.70710683)  # the signs of one column of the block's P
    x = torch.from_numpy(x)
    w4a16_check(w4a16_run(x, A, B, codes, lin, "nvfp4", out_dtype), x, A, B, codes, lin, "nvfp4")


@pytest.mark.parametrize("x_mag,a_mag,b_mag", [(1e30, 1e-30, 1e-20), (1e-20, 1e-10, 1e35), (1e10, 1e30, 1e-30)])
def test_w4a16_nvfp4_transforms_of_far_magnitudes(x_mag, a_mag, b_mag):
    """x, A and B whose product is ordinary, while A times B is not in fp32's range.  (x times B has to be: the
    transform's own sums hold it.)"""
    x, A, B, codes, lin, _ = w4a16_case(3, 256, 32, "nvfp4", F32, True, 32)
    x, A, B = x * x_mag, (A * np.float32(a_mag)).astype(np.float32), (B * np.float32(b_mag)).astype(np.float32)
    w4a16_check(w4a16_run(x, A, B, codes, lin, "nvfp4", F32), x, A, B, codes, lin, "nvfp4")
