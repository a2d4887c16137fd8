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
