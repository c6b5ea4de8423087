"""The operators' torch calls at the edges of what their documentation allows."""
import pytest
import torch

from tests.test_gpu_ops_fp8 import _x, ops  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", ["fp32", "bf16"])
def test_weight_gradient_of_no_rows(ops, out):  # noqa: F811
    """dW = dy^T x of an empty batch: zeros, also into a given view, which keeps
    what lies around it, and captured."""
    t = lambda n: ops.quantize_fp8(_x(0, n), transpose=True)
    dw = ops.gemm_fp8(t(130), t(264), out_dtype=out)
    assert dw.shape == (130, 264) and not dw.any()
    big = torch.full((132, 300), 7.0, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = ops.gemm_fp8(t(130), t(264), out=big[1:131, 5:269])
    big.fill_(7.0)
    g.replay()
    assert got.data_ptr() == big[1:, 5:].data_ptr() and not big[1:131, 5:269].any()
    assert float(big.sum()) == 7.0 * (132 * 300 - 130 * 264)
