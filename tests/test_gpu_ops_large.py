"""Sizes whose element numbers pass 2^31, and first calls inside a capture.  Rows,
experts and columns are independent of each other: what lies behind the border is
compared bit for bit with the same call on a slice of it."""
import os
import subprocess
import sys

import pytest
import torch

from tests.test_gpu_ops_fp8 import ops  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _room():
    if torch.cuda.is_available() and torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 50 GB")
    yield
    torch.cuda.empty_cache()                          # the library allocates beside torch


def _randn(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, device="cuda", dtype=dtype).normal_()


def _same(a, b):
    return all(torch.equal(x.view(torch.uint8) if x.element_size() == 1 else x,
                           y.view(torch.uint8) if y.element_size() == 1 else y) for x, y in zip(a, b))


def test_rows_of_more_than_2_31_elements(ops):  # noqa: F811
    M, K, n = 2200000, 1024, 1100                      # x, codes and the product
    x, w = _randn(M, K), ops.quantize_fp8_weight(_randn(K, K))
    q = ops.quantize_fp8(x)
    y = ops.gemm_fp8(q, w)
    part = ops.quantize_fp8(x[-n:])
    assert _same((q.codes[-n:], q.scales[:, -n:]), part)
    assert torch.equal(y[-n:], ops.gemm_fp8(part, w))
    del y, q
    t, last = ops.quantize_fp8(x, transpose=True), M - M % 128     # blocks start at multiples of 128 rows
    p = ops.quantize_fp8(x[last - 1280:], transpose=True)
    assert _same((t.codes[:, last - 1280:], t.scales[-p.scales.shape[0]:]), p)


def test_experts_of_more_than_2_31_codes(ops):  # noqa: F811
    E, F, L, rows = 220, 5120, 2048, 4
    w = _randn(E, F, L)
    q, t = ops.quantize_fp8_weight(w, transposed=True)
    a, d = ops.quantize_fp8(_randn(E * rows, L)), ops.quantize_fp8(_randn(E * rows, F))
    off = (torch.arange(E + 1, device="cuda") * rows).int()
    y, dx = ops.gemm_fp8(a, q, offsets=off), ops.gemm_fp8(d, t, offsets=off)
    for e in (0, 204, 205, E - 1):                     # 2^31 codes end in expert 204
        qe, te = ops.quantize_fp8_weight(w[e:e + 1], transposed=True)
        assert _same((q.codes[e], q.scales[e], t.codes[e], t.scales[e]),
                     (qe.codes[0], qe.scales[0], te.codes[0], te.scales[0]))
        s = slice(e * rows, (e + 1) * rows)
        assert torch.equal(y[s], ops.gemm_fp8(ops.Fp8(a.codes[s], a.scales[:, s]), qe, offsets=off[:2]))
        assert torch.equal(dx[s], ops.gemm_fp8(ops.Fp8(d.codes[s], d.scales[:, s]), te, offsets=off[:2]))


def test_norms_of_more_than_2_31_elements(ops):  # noqa: F811
    T, D, n = 140000, 16384, 400
    x, y, dr, wn = _randn(T, D), _randn(T, D), _randn(T, D), 1 + 0.1 * _randn(D)
    f = ops.norm_residual(x, y, post_weight=wn, gate=wn, pre_weight=wn, stats=True)
    b = ops.norm_residual_backward(dr, dr, y, f, post_weight=wn, gate=wn, pre_weight=wn)
    s = slice(T - n, T)
    fs = ops.norm_residual(x[s], y[s], post_weight=wn, gate=wn, pre_weight=wn, stats=True)
    bs = ops.norm_residual_backward(dr[s], dr[s], y[s], fs, post_weight=wn, gate=wn, pre_weight=wn)
    assert _same((f.r[s], f.h[s], f.rstd_y[s], f.rstd_r[s], b.dx[s], b.dy[s]), (*fs, bs.dx, bs.dy))


def test_logits_of_more_than_2_31_elements(ops):  # noqa: F811
    T, E, k, n = 4300000, 512, 8, 3000
    l = _randn(T, E)
    idx, w = ops.route_topk(l, k, score="softmax")
    dl = ops.route_topk_backward(l, idx, w, w, score="softmax")
    i2, w2 = ops.route_topk(l[-n:], k, score="softmax")
    assert _same((idx[-n:], w[-n:], dl[-n:]), (i2, w2, ops.route_topk_backward(l[-n:], i2, w2, w2, score="softmax")))
    counts, offsets, perm, pos = ops.route_group(idx, E)
    assert int(offsets[-1]) == T * k and torch.equal(counts.long(), torch.bincount(idx.view(-1), minlength=E))
    assert torch.equal(pos[perm.long()], torch.arange(T * k, device="cuda", dtype=torch.int32))
    e = idx.view(-1)[perm.long()]
    assert bool(((e[1:] > e[:-1]) | ((e[1:] == e[:-1]) & (perm[1:] > perm[:-1]))).all())


CAPTURED_FIRST = """
import torch
from latentmoe_expert_routing_b200 import ops
n = lambda *s: torch.empty(*s, device="cuda", dtype=torch.bfloat16).normal_()
T, E, k, D, F = 200, 16, 4, 520, 264
l, x, y, dr, w3, wn = n(T, E), n(T, D), n(T, D), n(T, D), n(E, F, D), n(D)
big, rows = n(700, D), n(T, F)

def run():
    idx, w = ops.route_topk(l, k)
    counts, offsets, perm, pos = ops.route_group(idx, E)
    out = [idx, w, counts, offsets, perm, pos, ops.route_topk_backward(l, idx, w, w)]
    f = ops.norm_residual(x, y, post_weight=wn, gate=wn, pre_weight=wn, stats=True)
    b = ops.norm_residual_backward(dr, dr, y, f, post_weight=wn, gate=wn, pre_weight=wn)
    q, t = ops.quantize_fp8_weight(w3, transposed=True)
    h = ops.gemm_fp8(ops.quantize_fp8(x, perm=perm, k=k), q, offsets=offsets)
    one = ops.Fp8(q.codes[0], q.scales[0])
    wide = ops.gemm_fp8(ops.quantize_fp8(big), one)
    dw = ops.gemm_fp8(ops.quantize_fp8(rows, transpose=True), ops.quantize_fp8(x, transpose=True), out_dtype="fp32")
    few = ops.gemm_fp8(ops.quantize_fp8(x[:9], relu2=True), one, out_dtype="fp32")
    return out + [f.r, f.h, *b, h, wide, dw, few]

torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = run()
g.replay()
ops.sync()
assert all(torch.equal(a, b) for a, b in zip(out, run()))
"""


def test_first_calls_captured():
    """No operator needs a call before the one that is captured."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CAPTURED_FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-1500:]
