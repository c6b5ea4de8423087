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


def test_several_threads_at_once(ops):  # noqa: F811
    """Every operator from four host threads at once, each on a stream of its own,
    the first calls of their shapes included: the bits of one thread's calls."""
    import threading
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g).cuda()
    T, E, k, D = 300, 64, 4, 1032
    l, x, y, dr, w3 = n(T, E), n(T, D), n(T, D), n(T, D), n(E, 136, D)
    wn, gate = n(D), n(T, D)

    def run():
        idx, w = ops.route_topk(l, k)
        counts, offsets, perm, pos = ops.route_group(idx, E)
        dl = ops.route_topk_backward(l, idx, w, w)
        f = ops.norm_residual(x, y, post_weight=wn, gate=gate, pre_weight=wn, stats=True)
        b = ops.norm_residual_backward(dr, dr, y, f, post_weight=wn, gate=gate, pre_weight=wn)
        p = ops.gemm_fp8(ops.quantize_fp8(x, perm=perm, k=k), ops.quantize_fp8_weight(w3), offsets=offsets)
        q = ops.gemm_fp8(ops.quantize_fp8(y, transpose=True), ops.quantize_fp8(x, transpose=True))
        return [idx, w, offsets, perm, pos, dl, f.r, f.h, *b, p, q]

    torch.cuda.synchronize()
    got, errors, start = [None] * 4, [], threading.Barrier(4)

    def work(i):
        try:
            start.wait(60)
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    got[i] = run()
            torch.cuda.current_stream().synchronize()
        except Exception as e:                    # reported below: a thread's own is lost
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    want = run()
    for o in got:
        assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_what_is_no_tensor_raises_value_error(ops):  # noqa: F811
    """As the module says of wrong arguments, whichever argument it is."""
    l, x = torch.randn(4, 16).cuda(), torch.randn(4, 64).cuda()
    idx, w = ops.route_topk(l, 3)
    f, q, m = ops.norm_residual(x, x, stats=True), ops.quantize_fp8(x), ops.quantize_fp8_weight(x)
    m3 = ops.Fp8(m.codes[None], m.scales[None])
    bad = dict(
        logits=lambda: ops.route_topk([[0.0]], 1), k=lambda: ops.route_topk(l, -1),
        bias=lambda: ops.route_topk(l, 3, bias=[0.0] * 16), score=lambda: ops.route_topk(l, 3, score="relu"),
        idx=lambda: ops.route_topk_backward(l, None, w, w), w=lambda: ops.route_topk_backward(l, idx, 1.0, w),
        dw=lambda: ops.route_topk_backward(l, idx, w, None), group=lambda: ops.route_group(None, 4),
        n_experts=lambda: ops.route_group(idx, -1), x=lambda: ops.norm_residual(None, x),
        y=lambda: ops.norm_residual(x, None), post=lambda: ops.norm_residual(x, x, post_weight=1.0),
        gate=lambda: ops.norm_residual(x, x, gate=0.5), dr=lambda: ops.norm_residual_backward(3, None, x, f),
        y_backward=lambda: ops.norm_residual_backward(x, None, None, f),
        gate_backward=lambda: ops.norm_residual_backward(x, None, x, f, gate=0.5),
        forward=lambda: ops.norm_residual_backward(x, None, x, None),
        parts=lambda: ops.norm_residual_backward(x, None, x, (x, None)),
        rows=lambda: ops.quantize_fp8(None), perm=lambda: ops.quantize_fp8(x, perm=[0, 1]),
        weight=lambda: ops.quantize_fp8_weight(2.0), a=lambda: ops.gemm_fp8(None, m), b=lambda: ops.gemm_fp8(q, x),
        a_codes=lambda: ops.gemm_fp8(ops.Fp8(None, q.scales), m), b_codes=lambda: ops.gemm_fp8(q, ops.Fp8(None, m.scales)),
        a_scales=lambda: ops.gemm_fp8(ops.Fp8(q.codes, None), m), b_scales=lambda: ops.gemm_fp8(q, ops.Fp8(m.codes, None)),
        offsets=lambda: ops.gemm_fp8(q, m3, offsets=[0, 4]), out=lambda: ops.gemm_fp8(q, m, out=3))
    for name, call in bad.items():
        with pytest.raises(ValueError):
            call()
            pytest.fail(name)


def test_sync_reports_what_a_kernel_found(ops):  # noqa: F811
    from latentmoe_expert_routing_b200 import binding as B
    ops.sync()
    idx = torch.tensor([[0, 9], [1, 2]], dtype=torch.int32, device="cuda")
    with torch.cuda.stream(torch.cuda.Stream()):
        assert ops.route_group(idx, 4)[0].tolist() == [1, 1, 1, 0]
        with pytest.raises(B.MoeError) as e:
            ops.sync()
    assert e.value.status == B.MOE_ERR_DEVICE_CHECK
    for device in (None, 0, "cuda", "cuda:0", torch.device("cuda", 0)):
        ops.sync(device)                                      # cleared


def test_weight_gradients_do_not_hold_the_workspace(ops):  # noqa: F811
    """What a program keeps of a norm's gradient is the column sums, not megabytes
    of partial ones behind them (nor are they saved with them)."""
    T, D = 600, 1032
    n = lambda *s: torch.randn(*s).cuda()
    x, wn, g = n(T, D), n(D), n(D)
    f = ops.norm_residual(x, x, post_weight=wn, gate=g, pre_weight=wn, stats=True)
    b = ops.norm_residual_backward(x, x, x, f, post_weight=wn, gate=g, pre_weight=wn)
    for t in (b.dpost_weight, b.dpre_weight, b.dgate):
        assert t.untyped_storage().nbytes() <= 3 * D * 4
