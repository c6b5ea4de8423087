"""The norm gradient with more rows a block than its ring of bulk copies has
stages (and, where rows are too long for a ring, several rows a block): stages
filled again, phases turned over, column sums of many rows, rows written in place
of the gradients they came from.  References and bounds are the small tests'."""
import pytest
import torch

from tests.test_gpu_ops_norm import (EPS, _backward, _check_backward, _check_forward, _forward,  # noqa: F401
                                     _inputs, ops)

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32

# blocks x stages on 148 SMs: 444 x 4 (2056 bf16; 3 stages with a full gate), 148 x 3
# (8192 bf16; 2 with a full gate), 444 x 4 (1032 fp32), 1184 x 4 (256); without a
# ring: 8192 and 2056 with a full gate in fp32, 16384 in bf16
CASES = [(3000, 2056, BF16, "none"), (3000, 2056, BF16, "channel"), (3000, 2056, BF16, "token"),
         (3000, 2056, BF16, "full"), (3000, 2056, FP32, "full"), (1000, 8192, BF16, "channel"),
         (1000, 8192, BF16, "full"), (700, 8192, FP32, "token"), (3000, 1032, FP32, "full"),
         (3000, 1032, FP32, "channel"), (6000, 256, BF16, "none"), (6000, 256, FP32, "full"),
         (500, 16384, BF16, "channel")]


@pytest.mark.parametrize("T,D,dtype,gate", CASES)
def test_both_norms(ops, T, D, dtype, gate):  # noqa: F811
    v = _inputs(T, D, dtype, gate, True, True, seed=T + D)
    f = _forward(ops, v, 0.5)
    _check_forward(v, 0.5, f, dtype)
    b = _backward(ops, v, 0.5, f)
    _check_backward(v, 0.5, f, b, dtype, T, v["dr"])
    again = _backward(ops, v, 0.5, f)
    assert all(torch.equal(x, y) for x, y in zip(b, again) if x is not None)


# a stage holds y, [r, dh], [dr], [gate]: each may be absent.  16384 without the
# second norm is the ring of four vectors a thread
@pytest.mark.parametrize("T,D,dtype", [(3000, 1032, BF16), (3000, 2056, FP32), (500, 16384, BF16)])
@pytest.mark.parametrize("post,pre,dr,gate", [(True, True, False, "full"), (True, True, False, "channel"),
                                              (False, True, True, "token"), (True, False, True, "full"),
                                              (True, False, True, "none"), (False, False, True, "channel")])
def test_absent_arrays(ops, T, D, dtype, post, pre, dr, gate):  # noqa: F811
    v = _inputs(T, D, dtype, gate, post, pre, seed=T)
    f = _forward(ops, v, 1.0)
    b = _backward(ops, v, 1.0, f, dr="dr" if dr else None)
    _check_backward(v, 1.0, f, b, dtype, T, v["dr"] if dr else None)


@pytest.mark.parametrize("T,D", [(3000, 2056), (1000, 8192), (500, 16384)])
def test_in_place(ops, T, D):  # noqa: F811
    """dx over dr, dy over dh: a row's gradients are written while later rows of
    the same arrays are on their way in."""
    from latentmoe_expert_routing_b200 import binding as B
    v = _inputs(T, D, BF16, "channel", True, True)
    f = _forward(ops, v, 0.5)
    want = _backward(ops, v, 0.5, f)
    dr, dh = v["dr"].clone(), v["dh"].clone()
    s = [torch.empty(D, device="cuda") for _ in range(3)]
    n = B.moe_norm_residual_workspace(T, D)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    a = B.moe_norm_args(T=T, D=D, dtype=B.MOE_BF16, gate_kind=B.MOE_GATE_CHANNEL, residual_scale=0.5, eps=EPS,
                        y=v["y"].data_ptr(), ldy=D, post_weight=v["post"].data_ptr(), pre_weight=v["pre"].data_ptr(),
                        gate=v["gate"].data_ptr(), r=f.r.data_ptr(), ldr=D, rstd_y=f.rstd_y.data_ptr(),
                        rstd_r=f.rstd_r.data_ptr(), dr=dr.data_ptr(), lddr=D, dh=dh.data_ptr(), lddh=D,
                        dx=dr.data_ptr(), lddx=D, dy=dh.data_ptr(), lddy=D, dpost_weight=s[0].data_ptr(),
                        dpre_weight=s[1].data_ptr(), dgate=s[2].data_ptr())
    B.moe_norm_residual_backward(a, ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    for got, t in zip([dr, dh] + s, want):
        assert torch.equal(got, t)
