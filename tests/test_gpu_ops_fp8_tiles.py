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


# One to five K blocks, odd and even, with a partial last one.  Two to four tiles
# a pair (74 pairs; wide) or a CTA (296; tall); from 2049 rows on the wide form's
# tiles run in more than one band of eight row tiles.
@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(5000, 2600, 128), (4200, 3100, 300), (2100, 8000, 520), (8192, 2048, 256)])
def test_wide_products_of_several_tiles(ops, M, N, K, out):  # noqa: F811
    a, b = ops.quantize_fp8(_x(M, K, seed=M)), ops.quantize_fp8_weight(_x(N, K, seed=N, std=0.1))
    got = ops.gemm_fp8(a, b, out_dtype=out)
    _check(got, _rows_ref(a), _weights_ref(b), -(-K // 128))
    assert torch.equal(ops.gemm_fp8(a, b, out_dtype=out), got)


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(5000, 2600, 128), (4200, 3100, 300), (2100, 8000, 520)])
def test_row_operands_of_several_tiles(ops, M, N, K, out):  # noqa: F811
    a, b = ops.quantize_fp8(_x(M, K, seed=M)), ops.quantize_fp8(_x(N, K, seed=N, std=0.1))
    got = ops.gemm_fp8(a, b, out_dtype=out)
    _check(got, _rows_ref(a), _rows_ref(b), -(-K // 128))
    assert torch.equal(ops.gemm_fp8(a, b, out_dtype=out), got)


@pytest.mark.parametrize("M,N,K,out", [(9, 100000, 128, "bf16"), (16, 150000, 300, "fp32"), (30, 90000, 520, "bf16"),
                                       (50, 80000, 300, "bf16"), (64, 120008, 256, "fp32")])
def test_tall_products_of_several_tiles(ops, M, N, K, out):  # noqa: F811
    a, b = ops.quantize_fp8(_x(M, K, seed=M)), ops.quantize_fp8_weight(_x(N, K, seed=N, std=0.1))
    got = ops.gemm_fp8(a, b, out_dtype=out)
    _check(got, _rows_ref(a), _weights_ref(b), -(-K // 128))
    assert torch.equal(ops.gemm_fp8(a, b, out_dtype=out), got)


# groups of uneven sizes, empty ones and one that has most of the rows; the mean
# (9, 25, 50: tall of 16, 32 and 64 rows; 130: wide) chooses the form
@pytest.mark.parametrize("E,mean,N,K,out", [(64, 9, 1800, 300, "bf16"), (64, 25, 1800, 128, "fp32"),
                                            (64, 50, 1400, 520, "bf16"), (40, 130, 1800, 300, "bf16"),
                                            (40, 130, 1416, 128, "fp32"), (24, 210, 2600, 384, "bf16")])
@pytest.mark.parametrize("skew", [False, True])
def test_grouped_products_of_several_tiles(ops, E, mean, N, K, out, skew):  # noqa: F811
    rng = np.random.default_rng(E + mean)
    share = rng.exponential(size=E)
    share[rng.permutation(E)[: E // 2 if skew else 4]] = 0
    if skew:
        share[E // 3] = 9 * share.sum()
    sizes = np.floor(share / share.sum() * E * mean).astype(int)
    off = torch.tensor(np.concatenate([[5], 5 + np.cumsum(sizes)]), dtype=torch.int32, device="cuda")
    P = E * mean + 10
    assert int(off[-1]) <= P - 5
    a = ops.quantize_fp8(_x(P, K, seed=E))
    b = ops.quantize_fp8_weight(_x(E * N, K, seed=mean, std=0.1).view(E, N, K))
    o = torch.full((P, N), 7.0, dtype=torch.bfloat16 if out == "bf16" else torch.float32, device="cuda")
    ops.gemm_fp8(a, b, offsets=off, out=o)
    assert (o[:5] == 7).all() and (o[int(off[-1]):] == 7).all()
    av = _rows_ref(a)
    for e in range(E):
        r0, r1 = int(off[e]), int(off[e + 1])
        if r1 > r0:
            _check(o[r0:r1], av[r0:r1], _weights_ref(ops.Fp8(b.codes[e], b.scales[e])), -(-K // 128))
    again = torch.full_like(o, 7.0)
    assert torch.equal(ops.gemm_fp8(a, b, offsets=off, out=again), o)


def test_gradient_of_grouped_rows(ops):  # noqa: F811
    """The rows' gradient of a grouped product: the experts' transposed weights."""
    E, F, L, sizes = 6, 300, 520, [40, 0, 3, 129, 64, 1]
    off = torch.tensor([0] + list(np.cumsum(sizes)), dtype=torch.int32, device="cuda")
    w, dy = _x(E * F, L, seed=3, std=0.1).view(E, F, L), _x(sum(sizes), F, seed=4)
    _, t = ops.quantize_fp8_weight(w, transposed=True)
    d = ops.quantize_fp8(dy)
    dx = ops.gemm_fp8(d, t, offsets=off, out_dtype="fp32")
    dv = _rows_ref(d)
    for e in range(E):
        r0, r1 = int(off[e]), int(off[e + 1])
        wv = R.values(*R.quantize(w[e], 128), 128)
        if r1 > r0:
            _check(dx[r0:r1], dv[r0:r1], wv.T, -(-F // 128))
