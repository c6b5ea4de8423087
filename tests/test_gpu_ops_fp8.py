"""8-bit quantisation and products on the GPU against 64-bit forms.

Codes and scales are defined by single fp32 operations and a rounding: equal.
Products of the same codes: the tensor core adds 128 products of a block (each
exact in fp32) with at most 4 x 33 roundings or truncations of 2^-23 of the
running magnitude, the scale product is one rounding, and adding up the blocks
is one rounding for each: (132 * 2 + KB + 4) 2^-24 of the sum of magnitudes;
a bf16 result adds half a step, 2^-8 of its value."""
import numpy as np
import pytest
import torch

from tests import ops_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from latentmoe_expert_routing_b200 import build
    build.build()
    from latentmoe_expert_routing_b200 import ops
    return ops


def _x(R_, K, dtype=torch.bfloat16, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(R_, K, generator=g) * std).to(dtype).cuda()


def _np(t):
    return t.detach().float().cpu().numpy()


def _same_codes(q, codes, scales):
    assert np.array_equal(_np(q.codes), codes.astype(np.float32))
    assert np.array_equal(_np(q.scales).view(np.int32), scales.astype(np.float32).view(np.int32))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 128), (3, 127), (17, 129), (64, 8192), (33, 7688), (130, 520), (16, 1000)])
def test_quantize_rows(ops, M, K, dtype):
    x = _x(M, K, dtype, seed=K)
    q = ops.quantize_fp8(x)
    c, s = R.quantize(x)
    _same_codes(q, c, s.T)
    t = ops.quantize_fp8(x, transpose=True)
    c, s = R.quantize(x.t())
    _same_codes(t, c, s.T)
    _same_codes(ops.quantize_fp8(x, relu2=True), *(lambda r: (r[0], r[1].T))(
        R.quantize(x.float().clamp_min(0).square())))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("N,K", [(1, 1), (128, 128), (129, 127), (300, 520), (40, 1000), (256, 384)])
def test_quantize_weight(ops, N, K, dtype):
    w = _x(3 * N, K, dtype, seed=N).view(3, N, K)
    q, t = ops.quantize_fp8_weight(w, transposed=True)
    for m in range(3):
        c, s = R.quantize(w[m], 128)
        _same_codes(ops.Fp8(q.codes[m], q.scales[m]), c, s)
        _same_codes(ops.Fp8(t.codes[m], t.scales[m]), c.T, s.T)
    _same_codes(ops.quantize_fp8_weight(w[1]), *R.quantize(w[1], 128))


def test_quantize_range_of_values(ops):
    """Subnormal and huge blocks, zeros, every kind of rounding step, NaN, inf."""
    x = _x(8, 512, torch.float32, seed=2)
    x[0] = 0
    x[1] *= 1e-36
    x[2] *= 1e37
    x[3, :128] = 2.0 ** -110
    x[4, :256] = torch.linspace(-448, 448, 256, device="cuda")
    x[5, 128:256] = torch.tensor(np.resize(R.e4m3_grid(), 128), dtype=torch.float32, device="cuda")
    x[5, 128] = 448
    c, s = R.quantize(x)
    _same_codes(ops.quantize_fp8(x), c, s.T)
    x[6, 130], x[7, 3] = float("nan"), float("inf")
    q = ops.quantize_fp8(x)
    v = _np(q.codes) * np.repeat(_np(q.scales).T, 128, 1)
    assert np.isnan(v[6, 130]) and np.isfinite(np.delete(v[6], 130)).all()
    assert np.isnan(v[7, :128]).all() and np.isfinite(v[7, 128:]).all()


def test_quantize_gathers_rows(ops):
    x = _x(10, 264, seed=4)
    perm = torch.tensor([29, 0, 1, 14, 14, -1, 30, 7, 2 ** 31 - 1, 3], dtype=torch.int32, device="cuda")
    q = ops.quantize_fp8(x, perm=perm, k=3)                     # rows 9 0 0 4 4 - - 2 - 1
    want = torch.zeros(10, 264, device="cuda", dtype=x.dtype)
    for i, r in enumerate([9, 0, 0, 4, 4, None, None, 2, None, 1]):
        if r is not None:
            want[i] = x[r]
    c, s = R.quantize(want)
    _same_codes(q, c, s.T)


def test_quantize_strided_and_guarded(ops):
    """Views; and through the C call nothing past a row's codes is written."""
    from latentmoe_expert_routing_b200 import binding as B
    big = _x(40, 600, seed=5)
    for v in (big[:, 5:300], big[::2, 8:264], big.t()[:100]):
        a, b = ops.quantize_fp8(v), ops.quantize_fp8(v.contiguous())
        assert torch.equal(a.codes.view(torch.uint8), b.codes.view(torch.uint8)) and torch.equal(a.scales, b.scales)
        a, b = ops.quantize_fp8(v, transpose=True), ops.quantize_fp8(v.contiguous(), transpose=True)
        assert torch.equal(a.codes.view(torch.uint8), b.codes.view(torch.uint8)) and torch.equal(a.scales, b.scales)
    st = torch.cuda.current_stream().cuda_stream
    codes = torch.full((42, 320), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((5, 48), -1.0, device="cuda")
    B.moe_quantize_fp8(big.data_ptr(), B.MOE_BF16, 40, 300, 600, None, 40, 1, 0, codes.data_ptr(), 320,
                       scales.data_ptr(), 48, st)
    assert (codes[:40, 300:] == 0xAB).all() and (codes[40:] == 0xAB).all()
    assert (scales[:3, 40:] == -1).all() and (scales[3:] == -1).all() and (scales[:3, :40] > 0).all()


def _rows_ref(q):
    return R.values(_np(q.codes).astype(np.float64), _np(q.scales).T)


def _check(out, a, b, KB):
    ref, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    tol = (264 + KB + 4) * 2.0 ** -24 * mag + (2.0 ** -8 * np.abs(ref) if out.dtype == torch.bfloat16 else 0.0)
    err = np.abs(out.detach().cpu().double().numpy() - ref)
    assert (err <= tol).all(), (float((err - tol).max()), float(err.max()))
    return float(np.linalg.norm(err) / max(np.linalg.norm(ref), 1e-300))


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 128, 128), (1, 10240, 2048), (16, 256, 7688), (17, 130, 129), (32, 64, 1000), (33, 520, 384),
    (64, 300, 2048), (65, 128, 128), (100, 1000, 640), (128, 384, 512), (129, 257, 130), (200, 8, 4096),
    (300, 512, 256), (777, 1032, 520), (1500, 2500, 400)])
def test_gemm(ops, M, N, K, out):
    a = ops.quantize_fp8(_x(M, K, seed=M))
    b = ops.quantize_fp8_weight(_x(N, K, seed=N + 1, std=0.1))
    got = ops.gemm_fp8(a, b, out_dtype=out)
    _check(got, _rows_ref(a), R.values(_np(b.codes).astype(np.float64), _np(b.scales), 128), -(-K // 128))


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (130, 70, 1), (64, 256, 100), (300, 520, 1000), (257, 300, 129), (512, 1000, 2048)])
def test_gemm_of_two_row_operands(ops, M, N, K):
    a, b = ops.quantize_fp8(_x(M, K, seed=M)), ops.quantize_fp8(_x(N, K, seed=N + 1))
    _check(ops.gemm_fp8(a, b, out_dtype="fp32"), _rows_ref(a), _rows_ref(b), -(-K // 128))


def test_training_step_of_a_linear_layer(ops):
    """y, dx and dw of y = x w^T from one set of bf16 tensors."""
    M, K, N = 200, 520, 300
    x, w, dy = _x(M, K, seed=1), _x(N, K, seed=2, std=0.05), _x(M, N, seed=3, std=0.01)
    q, t = ops.quantize_fp8_weight(w, transposed=True)
    wv = R.values(*R.quantize(w, 128), 128)
    xr, dr = R.values(*R.quantize(x)), R.values(*R.quantize(dy))
    xt, dt = R.values(*R.quantize(x.t())), R.values(*R.quantize(dy.t()))
    _check(ops.gemm_fp8(ops.quantize_fp8(x), q), xr, wv, 5)
    _check(ops.gemm_fp8(ops.quantize_fp8(dy), t), dr, wv.T, 3)
    dw = ops.gemm_fp8(ops.quantize_fp8(dy, transpose=True), ops.quantize_fp8(x, transpose=True), out_dtype="fp32")
    _check(dw, dt, xt, 2)
    # the whole chain against the unquantised gradient: E4M3 is off by half a step, 2^-4, per
    # factor, independent from element to element
    ref = dy.double().t() @ x.double()
    assert float((dw.double() - ref).norm() / ref.norm()) < 2 * 2.0 ** -4


def _grouped(ops, sizes, N, K, out, lead=0, tail=0, seed=0):
    E = len(sizes)
    P = lead + sum(sizes) + tail
    off = torch.tensor([lead] + list(lead + np.cumsum(sizes)), dtype=torch.int32, device="cuda")
    a = ops.quantize_fp8(_x(P, K, seed=seed))
    b = ops.quantize_fp8_weight(_x(E * N, K, seed=seed + 1, std=0.1).view(E, N, K))
    o = torch.full((P, N), 7.0, dtype=torch.bfloat16 if out == "bf16" else torch.float32, device="cuda")
    ops.gemm_fp8(a, b, offsets=off, out=o)
    av = _rows_ref(a)
    assert (o[:lead] == 7.0).all() and (o[P - tail:] == 7.0).all()
    for e in range(E):
        r0, r1 = int(off[e]), int(off[e + 1])
        if r1 > r0:
            bv = R.values(_np(b.codes[e]).astype(np.float64), _np(b.scales[e]), 128)
            _check(o[r0:r1], av[r0:r1], bv, -(-K // 128))


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("sizes,N,K,lead,tail", [
    ([1], 128, 128, 0, 0), ([0, 0, 3, 0], 130, 200, 0, 5), ([5, 0, 40, 16, 17, 1, 2, 100], 260, 520, 3, 4),
    ([0] * 31 + [9] + [0] * 40, 64, 128, 0, 0), ([300, 0, 129, 128, 1, 511], 300, 384, 7, 130),
    ([200, 150, 400], 520, 1000, 0, 0), ([1] * 70, 136, 256, 0, 1), ([0, 0], 64, 64, 6, 0), ([64] * 5, 128, 640, 0, 0)])
def test_gemm_grouped(ops, sizes, N, K, lead, tail, out):
    _grouped(ops, sizes, N, K, out, lead, tail, seed=len(sizes))


def test_gemm_grouped_offsets_out_of_order(ops):
    """Wrong offsets are clamped: rows and weights stay inside, rows that the
    clamped ranges name are those groups' products, others are untouched."""
    a = ops.quantize_fp8(_x(50, 128, seed=1))
    b = ops.quantize_fp8_weight(_x(4 * 128, 128, seed=2).view(4, 128, 128))
    off = torch.tensor([-5, 20, 10, 99, 30], dtype=torch.int32, device="cuda")   # 0 20 20 50 50
    o = torch.full((50, 128), 7.0, device="cuda")
    ops.gemm_fp8(a, b, offsets=off, out=o)
    av = _rows_ref(a)
    for e, r0, r1 in ((0, 0, 20), (2, 20, 50)):
        _check(o[r0:r1], av[r0:r1], R.values(_np(b.codes[e]).astype(np.float64), _np(b.scales[e]), 128), 1)


def test_gemm_strided_codes_and_output(ops):
    a, b = ops.quantize_fp8(_x(70, 200, seed=1)), ops.quantize_fp8_weight(_x(90, 200, seed=2))
    want = ops.gemm_fp8(a, b)
    wide = torch.zeros(70, 416, dtype=torch.uint8, device="cuda")
    for off in (16, 5):
        wide[:, off:off + 200] = a.codes.view(torch.uint8)
        got = ops.gemm_fp8(ops.Fp8(wide[:, off:off + 200], a.scales), b)
        assert torch.equal(got, want)
    sc = torch.zeros(2, 99, device="cuda")
    sc[:, 3:73] = a.scales
    assert torch.equal(ops.gemm_fp8(ops.Fp8(a.codes, sc[:, 3:73]), b), want)
    for M in (70, 700):
        a = ops.quantize_fp8(_x(M, 200, seed=3))
        o = torch.full((M + 1, 120), 7.0, dtype=torch.bfloat16, device="cuda")
        for off in (0, 8, 3):
            o.fill_(7.0)
            ops.gemm_fp8(a, b, out=o[:M, off:off + 90])
            assert torch.equal(o[:M, off:off + 90], ops.gemm_fp8(a, b))
            assert (o[M] == 7).all() and (o[:, :off] == 7).all() and (o[:, off + 90:] == 7).all()


def test_gemm_nan_stays_in_its_row(ops):
    x = _x(40, 300, seed=6)
    x[3, 5], x[17, 299] = float("nan"), float("inf")
    for M in (40, 300):
        y = torch.cat([x] * (M // 40 + 1))[:M]
        o = ops.gemm_fp8(ops.quantize_fp8(y), ops.quantize_fp8_weight(_x(64, 300, seed=7)))
        bad = o.isnan().all(1)
        assert bad.nonzero().flatten().tolist() == [i for i in range(M) if i % 40 in (3, 17)]
        assert o[~bad].isfinite().all()


def test_gemm_empty_and_refusals(ops):
    b = ops.quantize_fp8_weight(_x(64, 256))
    e = ops.quantize_fp8(_x(0, 256))
    assert ops.gemm_fp8(e, b).shape == (0, 64)
    a = ops.quantize_fp8(_x(5, 256))
    for bad in (lambda: ops.gemm_fp8(a, ops.Fp8(b.codes[:, :128], b.scales)),
                lambda: ops.gemm_fp8(a, ops.Fp8(b.codes, b.scales.t().contiguous()[:1])),
                lambda: ops.gemm_fp8(ops.Fp8(a.codes, a.scales.t()), b),
                lambda: ops.gemm_fp8(a, b, offsets=torch.zeros(2, dtype=torch.int32, device="cuda")),
                lambda: ops.gemm_fp8(a, b, out=torch.zeros(5, 63, device="cuda")),
                lambda: ops.gemm_fp8(a, b, out_dtype="fp16"),
                lambda: ops.gemm_fp8(ops.Fp8(a.codes.float(), a.scales), b),
                lambda: ops.quantize_fp8(_x(4, 8), relu2=True, transpose=True),
                lambda: ops.quantize_fp8(_x(4, 8).half())):
        with pytest.raises(ValueError):
            bad()


def test_captured_and_on_two_streams(ops):
    """Quantise and multiply captured as a graph (split K, plain and grouped),
    replayed on new inputs; then from two streams at once.  Bits are equal: there
    is one order of sums."""
    x = _x(48, 2048, seed=1)
    w = ops.quantize_fp8_weight(_x(640, 2048, seed=2))
    we = ops.quantize_fp8_weight(_x(4 * 256, 2048, seed=3).view(4, 256, 2048))
    off = torch.tensor([0, 10, 10, 40, 48], dtype=torch.int32, device="cuda")

    def run(t):
        q = ops.quantize_fp8(t)
        return ops.gemm_fp8(q, w), ops.gemm_fp8(q, we, offsets=off)

    run(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run(x)
    new = _x(48, 2048, seed=9)
    x.copy_(new)
    g.replay()
    want = run(new)
    assert all(torch.equal(p, q) for p, q in zip(out, want))
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(run(new))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for o in got for p, q in zip(o, want))
    from latentmoe_expert_routing_b200 import binding as B
    B.moe_sync(None, torch.cuda.current_stream().cuda_stream)            # no wait ran out
