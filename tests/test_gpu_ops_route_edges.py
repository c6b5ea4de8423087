"""Routing where it can go wrong besides the small ordinary cases: infinite biases
in groups, peaked rows, many rows and blocks.  References are 64-bit forms."""
import numpy as np
import pytest
import torch

from tests import ops_ref as R
from tests.test_gpu_ops_route import ops  # noqa: F401

pytestmark = pytest.mark.gpu
NEG = -float("inf")


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G", [(32, 4), (512, 64)])
def test_group_of_an_infinite_bias_and_nothing_else(ops, E, G, score):  # noqa: F811
    """Such a group scores -inf like any group without two eligible experts: it is
    not eligible beside topk_group better ones, so the rows choose as if all of it
    were masked (the renormalised weights, too: its scores have no part in them;
    k + 4 roundings, and one of each score on the reference's side)."""
    size, k, keep = E // G, 6, 2
    l = torch.randn(20, E, generator=torch.Generator().manual_seed(1))
    l[:, size:2 * size - 1] = NEG
    masked = l.clone()
    masked[:, 2 * size - 1] = NEG
    b = torch.zeros(E)
    b[2 * size - 1] = float("inf")
    idx, w = ops.route_topk(l.cuda(), k, bias=b.cuda(), score=score, n_group=G, topk_group=keep)
    ri, rw, _ = R.route(masked, k, score=score, n_group=G, topk_group=keep)
    assert np.array_equal(idx.cpu().numpy(), ri)
    assert (np.abs(w.cpu().double().numpy() - rw) <= (k + 6) * 2.0 ** -24 * rw).all()


def _gradient_by_pairs(l, idx, dw, score, renorm):
    """(dlogits, the size of what each is made of) in 64 bits.  Every difference
    u_e - C is the sum over experts i of share_i (u_e - u_i), so that nothing
    cancels which the gradient's own terms do not; with u* of the largest weight
    its terms are |u_e - u*|, |u*| times what the weights lack to 1, and the sum
    of share_i |u_i - u*|."""
    s, _ = R.scores64(l, score)
    T, E = s.shape
    out, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        at = idx[t].cpu().numpy()
        u, chosen = np.zeros(E), np.zeros(E, bool)
        u[at], chosen[at] = dw[t].double().numpy(), True
        p = np.where(chosen, s[t], 0.0)
        if score == "sigmoid" and not renorm:
            out[t] = p * u * (1 - p)
            size[t] = np.abs(out[t])
            continue
        S = p.sum() + 1e-20
        share, rest = (p / S, 1e-20 / S) if renorm else (p, s[t][~chosen].sum())
        star = u[share.argmax()]
        d = (share * (u[:, None] - u)).sum(1) + rest * u                 # u_e - C
        terms = np.abs(u - star) + np.abs(star) * rest + (share * np.abs(u - star)).sum()
        if score == "sigmoid":
            out[t], size[t] = share * d * (1 - s[t]), share * terms * (1 - s[t])
        elif renorm:
            out[t] = share * d - s[t] * (share * u).sum() * rest
            size[t] = share * terms + s[t] * (np.abs(star) + (share * np.abs(u - star)).sum()) * rest
        else:
            out[t], size[t] = s[t] * d, s[t] * terms
    return out, size


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k", [(8, 1), (8, 2), (40, 5), (512, 22), (128, 64)])
def test_gradient_of_peaked_rows(ops, E, k, renorm, score):  # noqa: F811
    """One expert has nearly all of the weight (up to 1 - 1e-7): the gradient is as
    exact as its own terms.  A score is off by 2 + 24 units of 2^-24 (expf and its
    argument, at most 24) and 16 + 6 of its sum and quotient, a weight's sum and
    quotient add k, a product of three such factors and the sums over the slots 24."""
    T = 12
    g = torch.Generator().manual_seed(E)
    l = torch.randn(T, E, generator=g)
    l[torch.arange(T), torch.randint(E, (T,), generator=g)] += torch.linspace(4, 16, T)
    dw = torch.randn(T, k, generator=g)
    idx, w = ops.route_topk(l.cuda(), k, score=score, renorm=renorm)
    dl = ops.route_topk_backward(l.cuda(), idx, w, dw.cuda(), score=score, renorm=renorm)
    ref, size = _gradient_by_pairs(l, idx, dw, score, renorm)
    err = np.abs(dl.cpu().double().numpy() - ref)
    assert (err <= (128 + 2 * k) * 2.0 ** -24 * size + 1e-37).all(), float((err / (size + 1e-37)).max() * 2 ** 24)


def test_gradient_of_the_most_rows(ops):  # noqa: F811
    """2^31 - 1 rows: the last block's warps stand for rows up to 2^31.  One expert,
    logit 0, weights not renormalised: s (1 - s) dw = 1/4 everywhere."""
    from latentmoe_expert_routing_b200 import binding as B
    T = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 26 GB")
    l = torch.zeros(T, dtype=torch.bfloat16, device="cuda")
    idx = torch.zeros(T, dtype=torch.int32, device="cuda")
    one = torch.ones(T, device="cuda")
    dl = torch.zeros(T + 8, dtype=torch.bfloat16, device="cuda")
    B.moe_route_topk_backward(l.data_ptr(), B.MOE_BF16, 1, idx.data_ptr(), one.data_ptr(), one.data_ptr(), T, 1, 1,
                              B.MOE_SCORE_SIGMOID, 0, 1.0, dl.data_ptr(), 1, torch.cuda.current_stream().cuda_stream)
    assert (dl[T:] == 0).all()
    for part in dl[:T].split(1 << 28):
        assert bool((part == 0.25).all())
    del l, idx, one, dl, part
    torch.cuda.empty_cache()                          # the library allocates beside torch


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,G,keep,dtype", [
    (2100, 64, 6, 1, 1, torch.float32), (2500, 160, 8, 8, 3, torch.float32), (2100, 512, 22, 1, 1, torch.bfloat16),
    (700, 512, 22, 64, 9, torch.float32), (9500, 24, 3, 1, 1, torch.bfloat16)])
def test_many_rows(ops, T, E, k, G, keep, dtype, score):  # noqa: F811
    """Four and eight rows a block, several rows a warp (more than 9472 rows), and
    lanes that no eligible expert falls to."""
    g = torch.Generator().manual_seed(T)
    l = torch.randn(T, E, generator=g).to(dtype).cuda()
    l[::7, ::4] = NEG
    b = torch.randn(E, generator=g).mul(0.1).cuda()
    kw = dict(bias=b, score=score, n_group=G, topk_group=keep, scale=2.5)
    idx, w = ops.route_topk(l, k, **kw)
    ri, rw, _ = R.route(l, k, **kw)
    assert np.array_equal(idx.cpu().numpy(), ri)
    assert (np.abs(w.cpu().double().numpy() - rw) <= (k + 4) * 2.0 ** -24 * np.abs(rw) + 1e-38).all()


@pytest.mark.parametrize("T,E,k", [(9000, 64, 4), (20000, 9, 3), (5000, 512, 22), (3300, 1024, 20)])
def test_group_of_many_blocks(ops, T, E, k):  # noqa: F811
    """More than 32 blocks of 1024 pairs: the scan over the blocks takes several
    steps.  Uneven experts, some without a pair."""
    g = torch.Generator().manual_seed(T)
    idx = (torch.rand(T, k, generator=g).pow(3) * (E - 1)).int().cuda()
    for got, want in zip(ops.route_group(idx, E), R.group(idx.cpu().numpy(), E)):
        assert np.array_equal(got.cpu().numpy(), want)
