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
