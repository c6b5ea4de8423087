"""The stand-alone operators together, as a program uses them: routed experts in
8 bits from router logits to the next block's input, and the layer between two
norms of a residual stream."""
import numpy as np
import pytest
import torch

from latentmoe_expert_routing_b200 import inputs as I
from tests import ops_ref as R
from tests.gpu_common import np32, np64, oracle_rows

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from latentmoe_expert_routing_b200 import build
    build.build()
    from latentmoe_expert_routing_b200 import ops
    return ops


def _numbers(g, *shape, zeros=0.5):
    """-1, 0 and 1, `zeros` of them 0: every sum of products below is a small whole
    number, which bf16 holds, so no rounding depends on the order of a sum."""
    v = torch.randint(0, 2, shape, generator=g) * 2 - 1
    return (v * (torch.rand(*shape, generator=g) >= zeros)).float()


@pytest.mark.parametrize("T,E,k,L,F", [(1, 4, 2, 128, 136), (37, 16, 4, 200, 264), (600, 8, 3, 128, 256)])
def test_routed_experts_in_8_bits(ops, T, E, k, L, F):
    """route, group, gather and quantise, up, squared ReLU and quantise, down,
    weighted sum, norm and residual.  The up products are whole numbers below 256
    (at most 25 non-zero terms of 0.9 zeros are expected; checked), so H is exact
    in bf16 and its codes are the reference's; the down products then differ by
    the products' own bound, and r by what norm_residual adds."""
    g = torch.Generator().manual_seed(T)
    x, logits = _numbers(g, T, L), torch.randn(T, E, generator=g)
    x[:, 0] = 1.0                                               # no empty block
    up, down = _numbers(g, E, F, L, zeros=0.9), _numbers(g, E, L, F, zeros=0.5)
    stream, wn = torch.randn(T, L, generator=g), 1 + 0.1 * torch.randn(L, generator=g)
    c = lambda t: t.bfloat16().cuda()

    idx, w = ops.route_topk(logits.cuda(), k, scale=2.5)
    counts, offsets, perm, pos = ops.route_group(idx, E)
    z = ops.quantize_fp8(c(x), perm=perm, k=k)
    wu, wd = ops.quantize_fp8_weight(c(up)), ops.quantize_fp8_weight(c(down))
    h = ops.gemm_fp8(z, wu, offsets=offsets, out_dtype="bf16")
    y = ops.gemm_fp8(ops.quantize_fp8(h, relu2=True), wd, offsets=offsets, out_dtype="fp32")
    combined = (y[pos.long().view(T, k)] * w[:, :, None]).sum(1)
    f = ops.norm_residual(c(stream), c(combined.cpu()), post_weight=c(wn), pre_weight=c(wn), residual_scale=0.5)

    ri, rw, _ = R.route(logits, k, scale=2.5)
    assert np.array_equal(idx.cpu().numpy(), ri)
    tok = perm.cpu().numpy() // k
    exp = ri.reshape(-1)[perm.cpu().numpy()]
    hid = np.einsum("pl,pfl->pf", x.numpy()[tok].astype(np.float64), up.numpy()[exp].astype(np.float64))
    assert np.abs(hid).max() < 256
    # A block's sum is a whole number n_b times 448^2, its scale product 448^-2 within three
    # roundings, and adding a block is one more: h before its own rounding is within
    # (KB + 4) 2^-24 sum |n_b| of the whole number, far less than half a bf16 step from it
    # where that is not 0, so it is rounded to it; where the blocks cancel (n, then -n), what
    # is left is that error itself, whose square rounds to code 0 or, in a block without
    # another number, stands for itself.
    KL = -(-L // 128)
    slack = (KL + 4) * U * np.einsum("pl,pfl->pf", np.abs(x.numpy()[tok]), np.abs(up.numpy()[exp]))
    hv = np64(h)
    assert np.array_equal(hv[hid != 0], hid[hid != 0]) and (np.abs(hv) <= slack)[hid == 0].all()
    codes, scales = R.quantize(torch.from_numpy(np.maximum(hid, 0) ** 2).float())
    act = R.values(codes, scales)
    ref = np.einsum("pf,plf->pl", act, down.numpy()[exp].astype(np.float64))
    mag = np.einsum("pf,plf->pl", np.abs(act), np.abs(down.numpy()[exp]).astype(np.float64))
    KB = -(-F // 128)
    # the products' bound, and two roundings of the weights' scales (1 / 448 times 448)
    # those squares, rounded up to a code: at most F of (6 x 2^-24 x 200)^2 = 5e-9, 2e-6 in all,
    # which is less than what the products' bound gives to a single whole number
    left = F * (1.07 * slack.max()) ** 2
    assert left < 264 * U and (np.abs(np64(y) - ref) <= (264 + KB + 8) * U * mag + left).all()
    r = R.norm_r(c(stream), c(combined.cpu()), c(wn), None, 0.5, 1e-5)
    err = (f.r.cpu().double() - r).abs()
    big = (0.5 * c(stream).cpu().double()).abs() + (r - 0.5 * c(stream).cpu().double()).abs()
    assert bool((err <= 32 * U * big + 2.0 ** -8 * r.abs()).all())
    hn = R.norm_h(f.r, c(wn), 1e-5)
    assert bool(((f.h.cpu().double() - hn).abs() <= (32 * U + 2.0 ** -8) * hn.abs()).all())


def test_chain_captured(ops):
    """The whole chain as one graph, replayed on new inputs in place."""
    T, E, k, L, F = 64, 8, 2, 256, 384
    g = torch.Generator().manual_seed(3)
    make = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()
    x, logits, s, wn = make(T, L), make(T, E), make(T, L), make(L)
    wu, wd = ops.quantize_fp8_weight(make(E, F, L)), ops.quantize_fp8_weight(make(E, L, F))

    def run():
        idx, w = ops.route_topk(logits, k, score="softmax")
        _, offsets, perm, pos = ops.route_group(idx, E)
        h = ops.gemm_fp8(ops.quantize_fp8(x, perm=perm, k=k), wu, offsets=offsets)
        y = ops.gemm_fp8(ops.quantize_fp8(h, relu2=True), wd, offsets=offsets)
        o = (y[pos.long().view(T, k)].float() * w[:, :, None]).sum(1).bfloat16()
        f = ops.norm_residual(s, o, post_weight=wn, gate=wn, pre_weight=wn)
        return idx, w, y, f.r, f.h

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for _ in range(2):
        x.copy_(make(T, L))
        logits.copy_(make(T, E))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, run()))


def test_layer_between_two_norms(ops):
    """LatentMoE.block_step: the layer's own output through norm_residual."""
    from latentmoe_expert_routing_b200 import layer as LY
    cfg = I.CONFIGS["tiny_fp32"]
    W = LY.weights_for(cfg)
    lay = LY.layer_for(cfg, W)
    h, x, gw = I.hidden(cfg, "cuda"), torch.flip(I.hidden(cfg, "cuda"), [0]), I.norm_weight(cfg, "cuda")
    r, nh, idx, w = lay.block_step(h, x, post_weight=gw, gate=gw, residual_scale=0.5, next_weight=gw)
    lay.sync()
    ref = oracle_rows(cfg, W, h)
    assert np.array_equal(idx.cpu().numpy(), ref["topk_idx"])
    out, _, _ = lay(h)
    lay.sync()
    want = R.norm_r(x, out, gw, gw, 0.5, 1e-5)
    big = (0.5 * x.cpu().double()).abs() + (want - 0.5 * x.cpu().double()).abs()
    assert bool(((r.cpu().double() - want).abs() <= 33 * U * big).all())
    hn = R.norm_h(r, gw, 1e-5)
    assert bool(((nh.cpu().double() - hn).abs() <= 33 * U * hn.abs()).all())
    with pytest.raises(ValueError):
        LY.LatentMoE.block_step(type("L", (), dict(out_dtype="fp32", dtype="bf16"))(), h, x)
    lay.close()
