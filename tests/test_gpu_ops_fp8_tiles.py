"""8-bit products large enough that a CTA takes several tiles: sums, barrier
phases, scale rings and output staging carried from one tile to the next.
References and bounds are those of the small products' tests."""
import numpy as np
import pytest
import torch

from tests import ops_ref as R
from tests.test_gpu_ops_fp8 import _check, _np, _rows_ref, _x, ops  # noqa: F401

pytestmark = pytest.mark.gpu


def _weights_ref(b):
    return R.values(_np(b.codes).astype(np.float64), _np(b.scales), 128)


# The last column tile has 64 (bf16) or 32 and 96 (fp32) columns, so that a half of
# it is written in an odd number of 128-byte passes, and a pair's next tile follows
# at once: one K block is the shortest main loop there is.
@pytest.mark.parametrize("form", ["weights", "rows"])
@pytest.mark.parametrize("N,out", [(1600, "bf16"), (1600, "fp32"), (1568, "fp32"), (1632, "fp32"), (1696, "bf16")])
def test_tiles_of_an_odd_number_of_passes(ops, N, out, form):  # noqa: F811
    M, K = 8192, 128
    a = ops.quantize_fp8(_x(M, K, seed=N))
    w = _x(N, K, seed=N + 1, std=0.1)
    b = ops.quantize_fp8(w) if form == "rows" else ops.quantize_fp8_weight(w)
    first = ops.gemm_fp8(a, b, out_dtype=out)
    _check(first, _rows_ref(a), _rows_ref(b) if form == "rows" else _weights_ref(b), 1)
    for _ in range(5):
        assert torch.equal(ops.gemm_fp8(a, b, out_dtype=out), first)
    for r in range(0, M, 1024):            # no more tiles than pairs: each takes one
        part = ops.Fp8(a.codes[r:r + 1024], a.scales[:, r:r + 1024])
        assert torch.equal(ops.gemm_fp8(part, b, out_dtype=out), first[r:r + 1024])
