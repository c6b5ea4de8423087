"""Stand-alone routing on the GPU against plain 64-bit forms.

Indices and groups are whole numbers and have to be equal.  Weights: s is one
rounding of a 64-bit value (2^-24), the sum of k of them k - 1 more, then an
addition, a quotient and a product: (k + 4) 2^-24 relative.  Gradients in fp32:
expf and its argument (|l - m| <= 24 here) are good to 2 + 24 units, the softmax
sum, the slot sums and the products add fewer than 2 k + 16: 2^-24 (64 + 2 k)
relative to the row's largest |u| (every term is at most that in size); a bf16
gradient adds half a step, 2^-8 of its value."""
import numpy as np
import pytest
import torch

from tests import ops_ref as R

pytestmark = pytest.mark.gpu
NEG = -float("inf")


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from latentmoe_expert_routing_b200 import build
    build.build()
    from latentmoe_expert_routing_b200 import ops
    return ops


def _logits(T, E, dtype=torch.float32, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * std).to(dtype).cuda()


def _check(ops, l, k, **kw):
    idx, w = ops.route_topk(l, k, **kw)
    ri, rw, chosen = R.route(l, k, **kw)
    assert np.array_equal(idx.cpu().numpy(), ri)
    err = np.abs(w.cpu().double().numpy() - rw)
    assert (err <= (k + 4) * 2.0 ** -24 * np.abs(rw) + 1e-38).all()
    return idx, w, chosen


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 512, 22), (5, 33, 33), (64, 512, 22), (37, 128, 8), (9, 1000, 64),
                                   (130, 31, 3), (3, 1024, 64), (17, 96, 32), (33, 257, 24), (8, 64, 64)])
def test_topk(ops, T, E, k, score):
    l = _logits(T, E, seed=T)
    b = torch.randn(E, generator=torch.Generator().manual_seed(E)).mul(0.1).cuda()
    _check(ops, l, k, bias=b, score=score, scale=2.5)
    _check(ops, l.bfloat16(), k, score=score, renorm=False)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k,G,keep", [(256, 8, 8, 4), (64, 6, 32, 3), (40, 10, 4, 1), (512, 22, 64, 9), (128, 64, 2, 1)])
def test_groups(ops, E, k, G, keep, score):
    l = _logits(50, E, seed=E)
    b = torch.randn(E, generator=torch.Generator().manual_seed(1)).mul(0.1).cuda()
    _check(ops, l, k, bias=b, score=score, n_group=G, topk_group=keep, scale=5.0)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k", [(48, 8), (512, 22), (700, 40)])
def test_ties_go_to_the_lower_expert(ops, E, k, score):
    l = torch.round(_logits(40, E, seed=3) * 2) / 2            # few distinct values
    l[0] = 0.0
    l[1] = 40.0                                                 # saturated scores
    idx, _, _ = _check(ops, l, k, score=score)
    assert idx[0].tolist() == list(range(k))
    _check(ops, l, k, score=score, bias=torch.zeros(E, device="cuda"))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups", [(1, 1), (4, 2)])
@pytest.mark.parametrize("E", [64, 512])
def test_masked_logits(ops, score, groups, E):
    """Rows with nothing left, with fewer experts than slots, NaN, the types'
    lowest values; the weight of a slot without an expert is 0."""
    k = 10
    l = _logits(12, E, seed=5)
    l[0] = NEG
    l[1] = float("nan")
    l[2] = NEG
    l[2, [7, E - 1, 20]] = torch.tensor([0.5, -1.0, 2.0], device="cuda")
    l[3, ::2] = NEG
    l[4, :E - 1] = torch.finfo(torch.float32).min
    l[5, ::3] = float("nan")
    l[6] = torch.finfo(torch.float32).min
    l[8] = -95.0 - 0.01 * torch.arange(E, device="cuda")       # scores below fp32's normal range
    b = torch.linspace(-0.2, 0.3, E, device="cuda")
    for bias in (None, b):
        for renorm in (True, False):
            idx, w, chosen = _check(ops, l, k, score=score, bias=bias, renorm=renorm, n_group=groups[0],
                                    topk_group=groups[1])
            i, w = idx.cpu().numpy(), w.cpu().numpy()
            assert all(len(set(r)) == k and r.min() >= 0 and r.max() < E for r in i)
            assert i[0].tolist() == list(range(k)) and not w[:2].any()
            assert np.isfinite(w).all() and not w[~chosen].any()


def test_infinite_logits_and_biases(ops):
    l = _logits(4, 64, seed=6)
    l[0, [3, 9]] = float("inf")
    idx, w, _ = _check(ops, l, 4, score="softmax", renorm=False)
    assert idx[0, :2].tolist() == [3, 9] and w[0, :2].tolist() == [0.5, 0.5]
    b = torch.zeros(64, device="cuda")
    b[5], b[6], b[7] = NEG, float("nan"), float("inf")
    idx, w, _ = _check(ops, l, 64, bias=b)
    assert (idx[:, 0] == 7).all() and set(idx[0, -2:].tolist()) == {5, 6} and (w[:, -2:] == 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_wide_scores(ops, dtype):
    """Peaked softmax rows: most scores lie many orders below the largest."""
    l = _logits(20, 300, dtype, seed=8, std=12.0)
    _check(ops, l, 24, score="softmax")
    _check(ops, l, 24, score="sigmoid")


def test_strided_logits_and_empty(ops):
    big = _logits(40, 200, seed=9)
    for view in (big[:, 3:99], big[::3, :64], big.t()[:50]):
        a = ops.route_topk(view, 5)
        c = ops.route_topk(view.contiguous(), 5)
        assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
    idx, w = ops.route_topk(big[:0], 5)
    assert idx.shape == (0, 5) and w.shape == (0, 5)
    assert ops.route_topk_backward(big[:0], idx, w, w).shape == (0, 200)


def test_matches_the_layer(ops):
    """On an fp32 layer's own logits: the layer's routing, bit for bit."""
    from latentmoe_expert_routing_b200 import inputs as I, layer as LY
    for cfg in (I.CONFIGS["tiny_fp32"], I.CONFIGS["tiny_fp32"].replace(E=64, k=6, n_group=8, topk_group=3)):
        W = LY.weights_for(cfg)
        lay = LY.layer_for(cfg, W)
        _, idx, w = lay(I.hidden(cfg, "cuda"))
        i2, w2 = ops.route_topk(lay.router_logits(cfg.T), cfg.k, bias=W["gate_bias"], n_group=cfg.n_group,
                                topk_group=cfg.topk_group, scale=cfg.rsf)
        c, o, p, q = ops.route_group(i2, cfg.E)
        assert torch.equal(idx, i2) and torch.equal(w.view(torch.int32), w2.view(torch.int32))
        for a, b in zip(lay.routing(cfg.T), (c, o, p, q)):
            assert torch.equal(a, b)
        lay.close()


@pytest.mark.parametrize("T,E,k", [(1, 4, 1), (7, 16, 4), (300, 512, 22), (1024, 128, 8), (33, 1024, 64), (5, 3, 3)])
def test_group(ops, T, E, k):
    idx = torch.rand(T, E, generator=torch.Generator().manual_seed(T)).argsort(1)[:, :k].int().cuda()
    for got, want in zip(ops.route_group(idx, E), R.group(idx.cpu().numpy(), E)):
        assert np.array_equal(got.cpu().numpy(), want)


def test_group_repeated_missing_and_wrong_experts(ops):
    from latentmoe_expert_routing_b200 import binding as B
    st = torch.cuda.current_stream().cuda_stream
    B.moe_sync(None, st)
    idx = torch.tensor([[5, 5, 5], [0, 5, 0], [1, 1, 2]] * 500, dtype=torch.int32, device="cuda")
    for got, want in zip(ops.route_group(idx, 8), R.group(idx.cpu().numpy(), 8)):
        assert np.array_equal(got.cpu().numpy(), want)
    B.moe_sync(None, st)
    idx[3, 1], idx[700, 0], idx[1499, 2] = -1, 8, 2 ** 31 - 1
    got = ops.route_group(idx, 8)
    for g, want in zip(got, R.group(idx.cpu().numpy(), 8)):
        assert np.array_equal(g.cpu().numpy(), want)
    assert got[2][-3:].tolist() == [-1, -1, -1]
    with pytest.raises(B.MoeError) as e:
        B.moe_sync(None, st)
    assert e.value.status == B.MOE_ERR_DEVICE_CHECK
    B.moe_sync(None, st)                                        # cleared
    c, o, p, q = ops.route_group(idx[:0], 8)
    assert not c.any() and not o.any() and o.numel() == 9 and p.numel() == 0


def _grad_tol(u, k, ref, dtype):
    t = 2.0 ** -24 * (64 + 2 * k) * np.abs(u).max(1, keepdims=True)
    return t + (2.0 ** -8 * np.abs(ref) if dtype == torch.bfloat16 else 0.0)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,dtype", [(1, 2, 1, torch.float32), (40, 512, 22, torch.float32),
                                         (33, 128, 8, torch.bfloat16), (3, 1000, 64, torch.float32),
                                         (9, 31, 31, torch.bfloat16)])
def test_gradient(ops, T, E, k, dtype, renorm, score):
    l = _logits(T, E, dtype, seed=T + E)
    if E > 8 and T > 2:
        l[0] = NEG
        l[1, ::2] = NEG
        l[2, 3] = float("nan")
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(k)).cuda()
    idx, w, chosen = _check(ops, l, k, score=score, renorm=renorm, scale=2.0)
    dl = ops.route_topk_backward(l, idx, w, dw, score=score, renorm=renorm, scale=2.0)
    ref = R.route_backward(l, idx, chosen, dw, score, renorm, 2.0)
    err = np.abs(dl.cpu().double().numpy() - ref)
    assert dl.dtype == dtype and (err <= _grad_tol(2.0 * dw.cpu().double().numpy(), k, ref, dtype)).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(ops, renorm, score):
    """Central differences of the 64-bit weights at fixed indices: truncation
    h^2 / 6 times a third derivative below 8 |u|, rounding 2^-52 / h."""
    T, E, k, h = 3, 24, 5, 1e-4
    l = _logits(T, E, seed=1)
    idx, w, chosen = _check(ops, l, k, score=score, renorm=renorm, scale=1.5)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(2)).cuda()
    dl = ops.route_topk_backward(l, idx, w, dw, score=score, renorm=renorm, scale=1.5).cpu().double()
    l64, d64, i, c = l.cpu().double(), dw.cpu().double(), idx.cpu(), torch.from_numpy(chosen)
    f = lambda x: (R.route_weights(x, i, c, score, renorm, 1.5) * d64).sum(1)
    for e in range(E):
        step = torch.zeros_like(l64)
        step[:, e] = h
        diff = (f(l64 + step) - f(l64 - step)) / (2 * h)
        u = 1.5 * d64.abs().sum(1)
        assert ((dl[:, e] - diff).abs() <= u * (8 * h * h / 6 + 2 ** -52 / h + 2.0 ** -24 * (64 + 2 * k))).all()


def test_gradient_skips_wrong_indices(ops):
    l = _logits(6, 40, seed=4)
    idx, w = ops.route_topk(l, 4, renorm=False)
    dw = torch.ones_like(w)
    want = ops.route_topk_backward(l, idx, w, dw, renorm=False)
    want[2, idx[2, 1].long()] = 0.0
    idx[2, 1] = 40
    assert torch.equal(ops.route_topk_backward(l, idx, w, dw, renorm=False), want)
    idx[2, 1] = -7
    assert torch.equal(ops.route_topk_backward(l, idx, w, dw, renorm=False), want)


def test_captured_and_on_another_stream(ops):
    """Routing, grouping and gradient captured as one graph, replayed on new
    logits in place; and the same calls on two streams at once."""
    l = _logits(300, 256, seed=11)
    dw = torch.randn(300, 8, generator=torch.Generator().manual_seed(3)).cuda()

    def run(x):
        idx, w = ops.route_topk(x, 8, score="softmax")
        return (idx, w) + ops.route_group(idx, 256) + (ops.route_topk_backward(x, idx, w, dw, score="softmax"),)

    run(l)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run(l)
    for seed in (12, 13):
        new = _logits(300, 256, seed=seed)
        l.copy_(new)
        g.replay()
        want = run(new)
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    xs = [_logits(2000, 256, seed=20 + i) for i in range(2)]
    dw = torch.randn(2000, 8, generator=torch.Generator().manual_seed(4)).cuda()
    want = [run(x) for x in xs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in xs], []
    for _ in range(3):
        for s, x in zip(streams, xs):
            with torch.cuda.stream(s):
                got.append(run(x))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(o, want[i % 2]))
